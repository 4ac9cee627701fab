// evict.cu -- eviction from a paged cache by accumulated attention weight
// (attn_evict_paged).
//
// For each (sequence, KV head): of its n keys the c = min(n, keep) of the
// highest rank stay.  A key's rank is its weight, +inf for a protected key
// (born among the first `sink` or the last `recent` tokens) and -inf for a
// NaN; ties go to the lowest place.  Attention does not depend on the order
// of its keys, so a kept key below c stays where it is, and the i-th kept key
// at or above c moves into the i-th evicted place below c: no more rows move
// than have to, and no moved row's source is another's destination, so the
// moves need no order among themselves.
//
// A unit (sequence, head) is one cluster of thread blocks, each with a slice
// of the keys:
//   1. ranks as order-preserving 32-bit integers, kept in shared memory where
//      the slice fits (else read again, from L2);
//   2. the c-th largest by radix selection, 8 bits at a time: a histogram of
//      the digit over the keys that match the prefix so far, in copies to
//      spread the collisions of alike weights, summed over the cluster's
//      blocks through distributed shared memory.  It ends early once all keys
//      of the digit stay, or all of them are alike (keys that were never
//      looked at tie at zero);
//   3. one bit per key, kept or not, and the counts of evicted places below c
//      and of kept keys above, prefix-summed;
//   4. the moves: pair i finds its place and its key by binary search in
//      those counts, and 16 bytes a thread go from row to row.
// Small cuts take the latency of those steps, one wave of blocks after the other
// (8 heads of 1044 keys cut to 1024: 48 sequences 10.8 us, 55, the last that three
// blocks an SM hold at once, 11.3, 64 13.4, 72 16.9; 8 heads of 32768 keys to
// 2048: 18.8, 64 blocks in all), large ones the bandwidth of the moved rows (64
// x 8 heads of up to 8192 keys to 1024: 78 to 82 us, 79 to 83% of the measured
// HBM bandwidth).
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "plan.h"

namespace cg = cooperative_groups;

namespace vgqa {

namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 3;           // 80 registers a thread: with 4 some would spill (ragged prompts 89.6 us, 80.5 with 3)
constexpr int kWarps = kThreads / 32;
constexpr int kCopies = 2;                // histogram copies (64 units of 1044 keys x 8: 17.4 us, 4 take 17.8, 8 take 18.9)
constexpr int kBatch = 8;                 // loads of a thread in flight
constexpr int kMaxCluster = 8;
constexpr int kCoarse = 4;                // words (of 32 keys) per entry of the prefix counts

struct Evict {
    const float *w;
    const int32_t *born, *seen, *keep;
    float *w_out;
    int32_t *born_out;
    __nv_bfloat16 *k_cache, *v_cache;
    int32_t *cu_out;
    long long ld;
    int sink, recent;
    int slice_words;           // words of 32 keys a block takes of the longest sequence
    int cached;                // keys of a slice that fit in shared memory (all or none: see smem)
};

// rank as an unsigned integer of the same order: NaN counts as -inf, -0 as +0
__device__ __forceinline__ uint32_t order_of(float w, bool fixed) {
    if (fixed) w = INFINITY;
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// this block's sequence lengths: only cu_k counts
__device__ __forceinline__ bool key_length(const Params &p, int b, bool report, int &Lk) {
    const int k0 = p.cu_k[b], k1 = p.cu_k[b + 1];
    Lk = k1 - k0;
    const uint32_t bad = (k0 < 0 || Lk < 0) ? ATTN_DEV_ERR_OFFSETS : Lk > p.s_max ? ATTN_DEV_ERR_K_TOO_LONG : 0u;
    if (bad && report) atomicOr(p.err, bad);
    return bad == 0;
}

// inclusive sum over the block's threads; `scratch` [kWarps]
__device__ __forceinline__ int block_scan(int v, int *scratch, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = v;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        const int x = scratch[i];
        if (i < warp) before += x;
        all += x;
    }
    total = all;
    return v + before;
}

// the new lengths' prefix sums
__device__ void write_offsets(const Params &p, const Evict &e, int *scratch) {
    int carry = 0;
    for (int b0 = 0; b0 < p.B_max; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        int c = 0, Lk;
        if (b < p.B_max && key_length(p, b, true, Lk)) c = min(Lk, max(0, e.keep[b]));
        int total;
        const int s = block_scan(c, scratch, total);
        if (b < p.B_max) e.cu_out[b + 1] = carry + s;
        carry += total;
    }
    if (threadIdx.x == 0) e.cu_out[0] = 0;
}

// the place of the i-th set bit (from 0) of w, by halves
__device__ __forceinline__ int nth_bit(uint32_t w, int i) {
    int at = 0;
#pragma unroll
    for (int h = 16; h; h >>= 1) {
        const int n = __popc(w & ((1u << h) - 1u));
        if (i >= n) {
            i -= n;
            at += h;
            w >>= h;
        }
    }
    return at;
}

// the place of the i-th set bit (from 0) of the kCoarse words from entry a on
__device__ __forceinline__ int pick(const uint32_t *bits, int a, int i, int words) {
    uint32_t x[kCoarse];
#pragma unroll
    for (int k = 0; k < kCoarse; ++k) x[k] = a * kCoarse + k < words ? bits[a * kCoarse + k] : 0u;
    int at = a * kCoarse * 32;
    uint32_t w = x[0];
    bool past = true;
#pragma unroll
    for (int k = 0; k + 1 < kCoarse; ++k) {
        const int n = __popc(x[k]);
        past = past && i >= n;
        if (past) {
            i -= n;
            at += 32;
            w = x[k + 1];
        }
    }
    return at + nth_bit(w, i);
}

// Shared memory: this, then either the slice's ranks (steps 1 and 2) or, from
// step 3 on and behind them, the whole unit's bits and prefix counts.
struct Head {
    uint32_t hist[2][256 * kCopies];
    uint32_t count[4][256];               // each pass's digit counts of this block (read by the cluster)
    uint32_t total[256];                  // and of the cluster
    int found[3];                         // the digit, the keys above it, the keys of it
    uint32_t alike[4][2];                 // and, or of the ranks that a pass counted in this block
    uint32_t all, any;                    // and of the cluster
    int scratch[kWarps];
};

__global__ void __launch_bounds__(kThreads, kBlocksPerSm) evict_kernel(const Params p, const Evict e) {
    extern __shared__ uint4 smem_raw[];
    Head &sh = *reinterpret_cast<Head *>(smem_raw);
    uint32_t *body = reinterpret_cast<uint32_t *>(&sh + 1);
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int unit = blockIdx.x / CS, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    dependent_start(false);
    if (unit == p.B_max * p.Hkv) {        // the extra cluster
        if (rank == 0) write_offsets(p, e, sh.scratch);
        return;
    }
    const int b = unit / p.Hkv, hk = unit % p.Hkv;
    const int keep = e.keep[b], seen = e.seen[b];   // on their way with the length
    int n;
    if (!key_length(p, b, false, n)) return;
    const int c = min(n, max(0, keep));
    if (c == 0) return;
    const float *w = e.w + (long long)unit * e.ld;
    const int32_t *born = e.born + (long long)unit * e.ld;
    float *w_out = e.w_out + (long long)unit * e.ld;
    int32_t *born_out = e.born_out + (long long)unit * e.ld;
    const bool copy_w = w_out != w, copy_born = born_out != born;
    // this block's slice, in whole words
    const int words = (n + 31) / 32, per = (words + CS - 1) / CS;
    const int w0 = min(words, rank * per), w1 = min(words, w0 + per);
    const int lo = w0 * 32, hi = min(n, w1 * 32);
    if (c == n) {                         // nothing to evict
        for (int j = lo + tid; j < hi; j += kThreads) {
            if (copy_w) w_out[j] = w[j];
            if (copy_born) born_out[j] = born[j];
        }
        return;
    }
    const int last = seen - e.recent;
    const bool cached = e.cached >= per * 32;
    for (int i = tid; i < 256 * kCopies; i += kThreads) sh.hist[0][i] = 0;
    if (tid < 8) sh.alike[tid >> 1][tid & 1] = tid & 1 ? 0u : ~0u;
    // one pass over the ledger: ranks into shared memory, entries below c to
    // the result (those of evicted keys are written again by the moves)
    if (cached || copy_w || copy_born)
        for (int j0 = lo + tid; j0 < hi; j0 += kBatch * kThreads) {
            float x[kBatch];
            int a[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int j = j0 + i * kThreads;
                x[i] = j < hi ? __ldcg(w + j) : 0.f;
                a[i] = j < hi ? __ldcg(born + j) : 0;
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int j = j0 + i * kThreads;
                if (j < hi && cached) body[j - lo] = order_of(x[i], a[i] < e.sink || a[i] >= last);
                if (j < min(hi, c)) {
                    if (copy_w) w_out[j] = x[i];
                    if (copy_born) born_out[j] = a[i];
                }
            }
        }
    // the ranks of kBatch keys of a thread, kThreads apart; past the slice's
    // end `none`
    auto read_ranks = [&](int j0, uint32_t none, uint32_t (&u)[kBatch]) {
        if (cached) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) u[i] = j0 + i * kThreads < hi ? body[j0 + i * kThreads - lo] : none;
        } else {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int j = j0 + i * kThreads;
                const int a = j < hi ? __ldcg(born + j) : 0;
                const float x = j < hi ? __ldcg(w + j) : 0.f;
                u[i] = j < hi ? order_of(x, a < e.sink || a >= last) : none;
            }
        }
    };
    __syncthreads();

    // ---- the c-th largest rank: after the passes, the ranks above it are those
    // with rank >> shift above `prefix`, and `need` of the `ties` equal to it stay
    uint32_t prefix = 0;
    int need = c, ties = n, shift = 32;
    const uint32_t *tie_count = nullptr;                // this block's count of the last digit chosen
    for (int pass = 0; pass < 4 && ties != need; ++pass) {
        shift -= 8;
        uint32_t all = ~0u, any = 0u;
        uint32_t *hist = sh.hist[pass & 1];
        for (int j0 = lo + tid; j0 < hi; j0 += kBatch * kThreads) {
            uint32_t u[kBatch];
            read_ranks(j0, 0u, u);
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (j0 + i * kThreads < hi && (pass == 0 || (u[i] >> (shift + 8)) == prefix)) {
                    atomicAdd(&hist[((u[i] >> shift) & 255u) * kCopies + (lane % kCopies)], 1u);
                    all &= u[i];
                    any |= u[i];
                }
        }
        all = __reduce_and_sync(0xffffffffu, all);
        any = __reduce_or_sync(0xffffffffu, any);
        if (lane == 0) {
            atomicAnd(&sh.alike[pass][0], all);
            atomicOr(&sh.alike[pass][1], any);
        }
        __syncthreads();
        uint32_t mine = 0;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) mine += hist[tid * kCopies + ((i + lane) % kCopies)];
        for (int i = tid; i < 256 * kCopies; i += kThreads) sh.hist[(pass + 1) & 1][i] = 0;
        sh.count[pass][tid] = mine;
        if (CS > 1) {
            // four digits a thread and, in another warp, a block's ranks a lane
            cluster.sync();
            if (tid < 64) {
                uint4 sum = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r)
                    if (r < CS) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(cluster.map_shared_rank(&sh.count[pass][4 * tid], r));
                        sum = make_uint4(sum.x + x.x, sum.y + x.y, sum.z + x.z, sum.w + x.w);
                    }
                *reinterpret_cast<uint4 *>(&sh.total[4 * tid]) = sum;
            } else if (warp == 2) {
                const uint32_t *theirs = cluster.map_shared_rank(&sh.alike[pass][0], min(lane, CS - 1));
                all = __reduce_and_sync(0xffffffffu, theirs[0]);
                any = __reduce_or_sync(0xffffffffu, theirs[1]);
                if (lane == 0) {
                    sh.all = all;
                    sh.any = any;
                }
            }
        } else {
            sh.total[tid] = mine;
            if (tid == 0) {
                sh.all = sh.alike[pass][0];
                sh.any = sh.alike[pass][1];
            }
        }
        __syncthreads();
        if (pass > 0 && sh.all == sh.any) {             // the same in all threads
            prefix = sh.all;
            shift = 0;
            break;
        }
        if (warp == 0) {
            // lane l: digits 255 - 8 l down to 248 - 8 l
            uint32_t d[8];
            *reinterpret_cast<uint4 *>(d) = *reinterpret_cast<const uint4 *>(sh.total + 248 - 8 * lane);
            *reinterpret_cast<uint4 *>(d + 4) = *reinterpret_cast<const uint4 *>(sh.total + 252 - 8 * lane);
            int sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += (int)d[i];
            int upto = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += x;
            }
            int above = upto - sum;
            if (above < need && upto >= need) {         // one lane holds the digit
                bool open = true;
#pragma unroll
                for (int i = 7; i >= 0; --i)
                    if (open) {
                        if (above + (int)d[i] >= need) {
                            sh.found[0] = 248 - 8 * lane + i;
                            sh.found[1] = above;
                            sh.found[2] = (int)d[i];
                            open = false;
                        } else {
                            above += (int)d[i];
                        }
                    }
            }
        }
        __syncthreads();
        prefix = (prefix << 8) | (uint32_t)sh.found[0];
        need -= sh.found[1];
        ties = sh.found[2];
        tie_count = &sh.count[pass][prefix & 255u];
    }

    // ---- bits: kept if above the threshold, or one of its first `need` ties.
    // A bit says evicted below c and kept from c on: the ones below c are the
    // places to fill, the ones above the keys that fill them.  They go behind
    // the ranks, which other warps still read.
    uint32_t *bits = body + (cached ? e.cached : 0);
    uint32_t *pre = bits + e.slice_words * CS;          // [slice_words CS / kCoarse + 2] prefix counts
    const bool all_ties = ties == need;
    uint32_t *tie_bits = pre + (e.slice_words * CS / kCoarse + 2);   // [slice_words]
    for (int j0 = lo + tid; j0 - lane < hi; j0 += kBatch * kThreads) {
        uint32_t u[kBatch];
        read_ranks(j0, 0u, u);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int j = j0 + i * kThreads, first = j - lane;          // the word's first key
            if (first < hi) {
                const uint32_t r = u[i] >> shift;
                const uint32_t above = __ballot_sync(0xffffffffu, j < hi && r > prefix);
                const uint32_t tie = __ballot_sync(0xffffffffu, j < hi && r == prefix);
                const uint32_t below = c - first >= 32 ? 0xffffffffu : c > first ? (1u << (c - first)) - 1u : 0u;
                if (lane == 0) {
                    bits[first / 32] = (all_ties ? above | tie : above) ^ below;
                    if (!all_ties) tie_bits[first / 32 - w0] = tie;
                }
            }
        }
    }
    if (!all_ties) {
        // the first `need` ties in order: those of the blocks before this one
        // count first, then a thread settles a word
        int before = 0;
        for (int r = 0; r < rank; ++r) before += (int)*cluster.map_shared_rank(tie_count, r);
        __syncthreads();
        for (int i0 = w0; i0 < w1; i0 += kThreads) {
            const int wd = i0 + tid;
            const uint32_t tie = wd < w1 ? tie_bits[wd - w0] : 0u;
            const int k = __popc(tie);
            int total;
            const int stay = need - before - (block_scan(k, sh.scratch, total) - k);     // of this word's ties
            if (wd < w1 && stay > 0) bits[wd] ^= stay >= k ? tie : tie & ((1u << nth_bit(tie, stay)) - 1u);
            before += total;
        }
    }
    // ---- every block gets the whole unit's bits
    if (CS > 1) {
        cluster.sync();
        for (int i0 = tid; i0 < words; i0 += 4 * kThreads) {
            uint32_t x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + k * kThreads;
                x[k] = i < words ? cluster.map_shared_rank(bits, i / per)[i] : 0u;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = i0 + k * kThreads;
                if (i < words && (i < w0 || i >= w1)) bits[i] = x[k];
            }
        }
        cluster.sync();                                 // also: nobody leaves while others read its memory
    } else {
        __syncthreads();
    }
    // prefix counts of the interesting bits at every kCoarse words: evicted
    // places first, then, from the word of c on, kept keys.  The word that
    // holds c has both; its low bits belong to the places.
    const int coarse = (words + kCoarse - 1) / kCoarse;
    int carry = 0;
    for (int i0 = 0; i0 < coarse; i0 += kThreads) {
        const int i = i0 + tid;
        int s = 0;
        if (i < coarse)
            for (int k = 0; k < kCoarse; ++k)
                if (i * kCoarse + k < words) s += __popc(bits[i * kCoarse + k]);
        int total;
        const int inc = block_scan(s, sh.scratch, total);
        if (i < coarse) pre[i] = carry + inc - s;
        carry += total;
    }
    __syncthreads();
    // the bits in order: the m evicted places below c, then the m kept keys that
    // take them
    const int m = carry / 2;
    // the places of the i-th and the k-th bit, searched for side by side
    auto locate = [&](int i, int k, int &pi, int &pk) {
        int ai = 0, zi = coarse, ak = 0, zk = coarse;   // pre[a] <= i < pre[z]
        while (zi - ai > 1 || zk - ak > 1) {
            const int mi = (ai + zi) >> 1, mk = (ak + zk) >> 1;
            const bool li = (int)pre[mi] <= i, lk = (int)pre[mk] <= k;
            if (zi - ai > 1) (li ? ai : zi) = mi;
            if (zk - ak > 1) (lk ? ak : zk) = mk;
        }
        pi = pick(bits, ai, i - (int)pre[ai], words);
        pk = pick(bits, ak, k - (int)pre[ak], words);
    };

    // ---- moves, an equal share of the pairs for each block and, in runs of up
    // to 32, for each warp: a lane locates one pair, then the warp copies them
    // one row of K and one of V after the other, kBatch pieces a lane in flight
    const int m0 = (int)((long long)m * rank / CS), m1 = (int)((long long)m * (rank + 1) / CS);
    const int lpp = p.D / 4;                            // lanes a pair: 16-byte pieces of a K and a V row
    const int pp = 32 / lpp, sub = lane / lpp, piece = lane % lpp;
    const int slot_mask = (1 << p.page_shift) - 1;
    __nv_bfloat16 *cache = piece < lpp / 2 ? e.k_cache : e.v_cache;
    cache += (long long)hk * p.D + (piece % (lpp / 2)) * 8;
    const int run = min(32, (m1 - m0 + kWarps - 1) / kWarps);
    for (int i0 = m0 + warp * run; i0 < m1; i0 += kWarps * run) {
        const int np = min(run, m1 - i0);
        long long to_at = -1, from_at = 0;              // elements from the cache's start
        if (lane < np) {
            int to, from;
            locate(i0 + lane, m + i0 + lane, to, from);
            const int et = page_entry(p, b, to), ef = page_entry(p, b, from);
            const float x = __ldcg(w + from);
            const int a = __ldcg(born + from);
            w_out[to] = x;
            born_out[to] = a;
            const int pt = page_checked(p, et), pf = page_checked(p, ef);
            if (pt < p.num_pages && pf < p.num_pages) {
                to_at = pt * p.page_stride + (to & slot_mask) * p.k_stride;
                from_at = pf * p.page_stride + (from & slot_mask) * p.k_stride;
            }
        }
        for (int q = 0; q < np; q += kBatch * pp) {
            uint4 val[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int i = q + u * pp + sub;
                const long long from = __shfl_sync(0xffffffffu, from_at, i & 31);
                const long long to = __shfl_sync(0xffffffffu, to_at, i & 31);
                if (i < np && to >= 0) val[u] = __ldcg(reinterpret_cast<const uint4 *>(cache + from));
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int i = q + u * pp + sub;
                const long long to = __shfl_sync(0xffffffffu, to_at, i & 31);
                if (i < np && to >= 0) *reinterpret_cast<uint4 *>(cache + to) = val[u];
            }
        }
    }
}

constexpr int kMaxSmem = 200 * 1024;
constexpr int kMaxKeys = 1 << 19;         // bits, counts and ties of 2^19 keys take 144 KB

// words of a slice, and shared memory of the bits, for clusters of `cs` blocks
int slice_words(int s_max, int cs) { return ((s_max + 31) / 32 + cs - 1) / cs; }
size_t bits_bytes(int s_max, int cs) {
    const size_t words = (size_t)slice_words(s_max, cs) * cs;
    return words * 4 + (words / kCoarse + 2) * 4 + (size_t)slice_words(s_max, cs) * 4;
}

}  // namespace

cudaError_t evict_prepare() {
    return cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
}

namespace {

cudaError_t launch_evict(const Params &p, Evict e, int sms, cudaStream_t stream) {
    // A cluster per unit: as many blocks as fill the device, but no slice
    // under 1024 keys (8 units of 32768 keys: 8 blocks each 18.9 us; 4 took 29.4 where 8 took 19.9)
    const long long units = (long long)p.B_max * p.Hkv;
    int cs = 1;
    while (cs < kMaxCluster && units * cs * 2 <= sms * kBlocksPerSm && p.s_max >= 2048 * cs) cs *= 2;
    e.slice_words = slice_words(p.s_max, cs);
    const size_t fixed = sizeof(Head) + bits_bytes(p.s_max, cs), ranks = (size_t)e.slice_words * 32 * 4;
    e.cached = fixed + ranks <= (size_t)kMaxSmem ? e.slice_words * 32 : 0;
    return launch_dependent(evict_kernel, dim3((unsigned)((p.B_max * p.Hkv + 1) * cs)), dim3(kThreads),
                            fixed + (e.cached ? ranks : 0), stream, cs > 1 ? cs : 0, p, e);
}

bool overlap(const void *a, const void *b, size_t na, size_t nb) {
    const char *x = static_cast<const char *>(a), *y = static_cast<const char *>(b);
    return x < y + nb && y < x + na;
}

}  // namespace

}  // namespace vgqa

using namespace vgqa;

ATTN_EXPORT int attn_evict_paged(attn_plan_t plan, const float *weight, const int32_t *born, const int32_t *seen,
                                 const int32_t *keep, int sink, int recent, float *weight_out, int32_t *born_out,
                                 int64_t ld, void *k_cache, void *v_cache, int64_t page_stride, int64_t token_stride,
                                 int page_size, int num_pages, const int32_t *block_table, int bt_stride,
                                 const int32_t *cu_k, int32_t *cu_k_out, void *stream) {
    if (!plan || !live(plan)) return ATTN_E_BAD_PLAN;
    if (!weight || !born || !seen || !keep || !weight_out || !born_out || !k_cache || !v_cache || !cu_k || !cu_k_out)
        return ATTN_E_NULL;
    const int rc = check_paging(plan, page_stride, token_stride, page_size, num_pages, block_table, bt_stride);
    if (rc != ATTN_OK) return rc;
    const attn_plan_desc &d = plan->d;
    if (d.s_max > kMaxKeys) return ATTN_E_UNSUPPORTED;
    if (sink < 0 || recent < 0 || ld < d.s_max || ld > (1ll << 38)) return ATTN_E_INVALID_ARG;
    if ((long long)d.B_max * d.Hkv >= (1ll << 27)) return ATTN_E_UNSUPPORTED;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return ATTN_E_ALIGNMENT;
    for (const void *ptr : {(const void *)weight, (const void *)born, (const void *)seen, (const void *)keep,
                            (const void *)weight_out, (const void *)born_out, (const void *)cu_k,
                            (const void *)cu_k_out})
        if (!aligned(ptr, 4)) return ATTN_E_ALIGNMENT;
    // in place, or apart
    const size_t led = (size_t)d.B_max * d.Hkv * ld * 4, cu = ((size_t)d.B_max + 1) * 4;
    if ((weight_out != weight && overlap(weight, weight_out, led, led)) ||
        (born_out != born && overlap(born, born_out, led, led)) || overlap(weight_out, born_out, led, led) ||
        overlap(weight_out, born, led, led) || overlap(born_out, weight, led, led) ||
        overlap(cu_k, cu_k_out, cu, cu) || overlap(keep, cu_k_out, cu - 4, cu) || overlap(seen, cu_k_out, cu - 4, cu))
        return ATTN_E_INVALID_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_E_CUDA;
    if (dev != plan->device) return ATTN_E_DEVICE;
    Params p{};
    p.cu_k = cu_k;
    p.err = plan->err;
    p.B_max = d.B_max;
    p.s_max = d.s_max;
    p.Hkv = d.Hkv;
    p.D = d.D;
    p.k_stride = token_stride;
    p.block_table = block_table;
    p.bt_stride = bt_stride;
    p.page_shift = log2_exact(page_size);
    p.num_pages = num_pages;
    p.page_stride = page_stride;
    Evict e{};
    e.w = weight;
    e.born = born;
    e.seen = seen;
    e.keep = keep;
    e.w_out = weight_out;
    e.born_out = born_out;
    e.k_cache = static_cast<__nv_bfloat16 *>(k_cache);
    e.v_cache = static_cast<__nv_bfloat16 *>(v_cache);
    e.cu_out = cu_k_out;
    e.ld = ld;
    e.sink = sink;
    e.recent = recent;
    return launch_evict(p, e, d.num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTN_OK : ATTN_E_CUDA;
}
