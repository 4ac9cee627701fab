// key_weights_tc.cu -- accumulated attention weights on the fifth-generation
// tensor cores: key j of KV head hk gathers
//     w_j = sum over visible rows r = (qi, g) of e^(s_{r,j} - lse_r).
//
// The product is taken transposed, S^T [128 keys x N rows] = K Q^T
// (tcgen05.mma, fp32 in tensor memory): a tensor-memory lane, and so a
// thread, then owns one key and sums over its columns alone -- no exchange
// between threads, no atomics, a fixed order.  What a key that does not
// belong to the sequence, or is not finite, brings into its lane stays there.
//
// Work.  An item is 256 keys (two sub-tiles of 128) of one (sequence, KV
// head); it meets the row tiles of qtile = min(max_q, 128 / G) query tokens
// (N >= G qtile columns), counted from the sequence's end, whose last token
// sees its first key.  The items' row tiles, in order, are the positions of
// one line; each of C persistent blocks (about one per SM) takes an equal
// stretch of it, computed on the device from cu_seqlens.  K is loaded once
// per item (once per part, where a stretch ends inside an item); a cut item's
// parts, 256 sums each, are added in block order by whichever block finishes
// last.  Decode has one row tile per item: no cuts, K streams through.
//
// Measured: 64 ragged sequences of a decode step (8 KV heads, 554 MB) 87 to 96
// us, 88 to 97% of the measured HBM bandwidth (from 64-key pages 111 us for 97,
// from 8-key pages 222); 2 x 1025..2048 tokens over 24k..32k keys, 64 heads, 1.65
// to 2.0 ms by their lengths and the power cap, half of the measured tensor rate:
// the exponentials need 1.2 ms of the special-function unit (79% busy).
//
// Warps: 0-15 epilogue (warp w: sub-tile w / 4 mod 2, lanes 32 (w mod 4), and
// of the columns, where there are 64 or more, half w / 8: four warps a
// scheduler hide one another's latencies; at the end of an item the first
// half adds the second's sums).  16 issues the MMAs, one row tile ahead of the
// epilogue (two buffers of S); 17 loads K and Q by TMA (128-byte swizzle,
// mbarrier rings); 18 stages -lse log2 e of each row tile.  Every wait is
// bounded, as in the attention kernels.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "key_weights.h"
#include "tc.cuh"

namespace vgqa {

namespace {

constexpr int kSubKeys = 128;             // keys per sub-tile (MMA M)
constexpr int kItemKeys = 256;
constexpr int kHalfWarps = 8;             // epilogue warps of a half of the columns
constexpr int kMmaWarp = 16, kLoadWarp = 17, kLseWarp = 18;
constexpr int kThreads = 608;
constexpr int kSumSlots = 4;              // sums on their way from half to half (at most 3 are)
constexpr int kMaxStages = 8;
constexpr size_t kMinSmem = 120 * 1024;   // one block per SM: tensor memory is never waited for

template <int D, int N>
struct Layout {
    static constexpr int kHalves = D / 64;
    static constexpr int kSub = kSubKeys * D * 2;             // one sub-tile of K
    static constexpr int kQ = N * D * 2;                      // one row tile of Q
    static constexpr int kColHalves = N >= 64 ? 2 : 1;          // halves of the columns
    // ring depths: 200 KB in all, K in what Q leaves (with the largest tiles two
    // row tiles and two items of K; three and one and a half took as long)
    static constexpr int kQStages = kQ == 32768 ? 2 : 4;
    static constexpr int kKStages = (200 * 1024 - kQStages * kQ) / kSub < kMaxStages
                                        ? (200 * 1024 - kQStages * kQ) / kSub
                                        : kMaxStages;
    static constexpr uint32_t kTmemCols = 4 * N < 32 ? 32 : 4 * N;
};

// ------------------------------------------------------------ schedule

struct SeqInfo {
    int q0, Lq, k0, Lk;
    int nkt, nrt, ksat;       // items, row tiles, items that meet all row tiles
    long long tot;            // positions of one KV head
};

// quotients of numbers that are nearly always small (a 64-bit division takes
// some hundred cycles, in every block and role before its first load)
__device__ __forceinline__ long long quotient(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// row tiles that see key tile kt
__device__ __forceinline__ int row_tiles(const SeqInfo &s, int kt, int qtile) {
    return min(s.nrt, (s.Lk - 1 - kt * kItemKeys) / qtile + 1);
}

__device__ __forceinline__ SeqInfo seq_info(const Params &p, int b, bool report) {
    SeqInfo s;
    s.nkt = s.nrt = s.ksat = 0;
    s.tot = 0;
    if (!load_lengths(p, b, report, s.q0, s.Lq, s.k0, s.Lk) || s.Lk == 0) return s;
    s.nkt = (s.Lk + kItemKeys - 1) / kItemKeys;
    s.nrt = (s.Lq + p.qtile - 1) / p.qtile;
    if (s.nrt <= 1) {                     // decode; or no query: its items only pass on what they had
        s.ksat = s.nkt;
        s.tot = s.nkt;
        return s;
    }
    const int all = s.Lk - 1 - (s.nrt - 1) * p.qtile;
    s.ksat = all < 0 ? 0 : min(s.nkt, all / kItemKeys + 1);
    s.tot = (long long)s.ksat * s.nrt;
    for (int kt = s.ksat; kt < s.nkt; ++kt) s.tot += row_tiles(s, kt, p.qtile);
    return s;
}

// a block's stretch [lo, hi) of the T positions
struct Share {
    long long lo, hi, T, pb;  // pb: first position of sequence b
    int C, b;
};

__device__ __forceinline__ int block_of(long long pos, const Share &sh) { return (int)(((pos + 1) * sh.C - 1) / sh.T); }

// All threads: thread t sums a run of sequences, a block scan places them, and
// the thread whose run holds the stretch's first position finds its sequence.
__device__ bool block_share(const Params &p, int tid, long long *scan, long long *found, Share &sh) {
    const int per = (p.B_max + kThreads - 1) / kThreads;
    const int b0 = min(p.B_max, tid * per), b1 = min(p.B_max, b0 + per);
    long long mine = 0, one = 0;          // positions of the run, and of its last sequence
    for (int b = b0; b < b1; ++b) {
        one = seq_info(p, b, blockIdx.x == 0).tot * p.Hkv;
        mine += one;
    }
    long long inc = mine;
    const int lane = tid & 31, warp = tid >> 5;
#pragma unroll 1
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    // (short code: what runs once is paid for in instruction fetches)
    long long T = lane < kThreads / 32 ? scan[lane] : 0, below = lane < warp ? T : 0;
#pragma unroll 1
    for (int d = 16; d; d >>= 1) {
        T += __shfl_xor_sync(0xffffffffu, T, d);
        below += __shfl_xor_sync(0xffffffffu, below, d);
    }
    inc += below;
    sh.T = T;
    sh.C = (int)min((long long)gridDim.x, T);
    if ((int)blockIdx.x >= sh.C) return false;
    // T c / C, rounded down, for c and c + 1
    const long long q = quotient(T, sh.C);
    const uint32_t r = (uint32_t)(T - q * sh.C), c = blockIdx.x;
    sh.lo = q * c + r * c / (uint32_t)sh.C;
    sh.hi = q * (c + 1) + r * (c + 1) / (uint32_t)sh.C;
    long long at = inc - mine;
    if (sh.lo >= at && sh.lo < inc) {
        for (int b = b0; b < b1; ++b) {
            const long long n = per == 1 ? one : seq_info(p, b, false).tot * p.Hkv;
            if (sh.lo < at + n) {
                found[0] = at;
                found[1] = b;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    sh.pb = found[0];
    sh.b = (int)found[1];
    return true;
}

// Walks a stretch item by item; every role runs its own.
struct Walker {
    SeqInfo s;
    int b, hk, kt, R, w;      // R row tiles, w = max(R, 1) positions
    int r0, r1;               // this stretch's part of them
    long long g, hi, P;       // next position, end, the item's first position

    __device__ void set(const Params &p) {
        R = s.Lq > 0 ? row_tiles(s, kt, p.qtile) : 0;
        w = max(R, 1);
        r0 = (int)(g - P);
        r1 = (int)min((long long)w, hi - P);
    }
    __device__ void init(const Params &p, const Share &sh) {
        b = sh.b;
        g = sh.lo;
        hi = sh.hi;
        s = seq_info(p, b, false);
        long long rem = g - sh.pb;
        hk = (int)quotient(rem, s.tot);
        rem -= hk * s.tot;
        P = g - rem;
        const int full = max(s.nrt, 1);
        if (rem < (long long)s.ksat * full) {
            kt = (int)quotient(rem, full);
            P += (long long)kt * full;
        } else {
            kt = s.ksat;
            P += (long long)kt * full;
            rem -= (long long)kt * full;
            for (int n; rem >= (n = row_tiles(s, kt, p.qtile)); ++kt) {
                rem -= n;
                P += n;
            }
        }
        set(p);
    }
    __device__ bool next(const Params &p) {
        g = P + r1;
        if (g >= hi) return false;
        P += w;               // r1 == w here
        if (++kt == s.nkt) {
            kt = 0;
            if (++hk == p.Hkv) {
                hk = 0;
                do s = seq_info(p, ++b, false);
                while (s.tot == 0);
            }
        }
        set(p);
        return true;
    }
    // first key of sub-tile u, or -1 if the sequence ends before it
    __device__ int sub_key(int u) const {
        const int j = kt * kItemKeys + u * kSubKeys;
        return j < s.Lk ? j : -1;
    }
    // first token of row tile r's box of queries: the box ends with the tile, or
    // starts with the buffer (then it ends behind the tile)
    __device__ int first_token(int r, int qtile) const { return max(s.Lq - (r + 1) * qtile, -s.q0); }
    // where the box of packed K starts, in keys from the sequence's first (maybe
    // before it): moved back to end with the sequence, but not before row 0
    __device__ int packed_start(int j0) const { return max(min(j0, s.Lk - kSubKeys), -s.k0); }
};

// ------------------------------------------------------------ kernel

// sum over 16 columns of 2^(s scale + nl); MASKED: only those in `vis`.  Taking
// some of the exponentials on the FMA pipe (a polynomial) was measured and
// lost, since four warps a scheduler wait on each other's latencies before
// they exhaust the special-function unit: 1 of 16 columns 1.68 ms where none
// takes 1.67, 3 of 16 1.79.
template <bool MASKED>
__device__ __forceinline__ void add_columns(const uint32_t (&v)[16], const float *nl, float2 scale, uint32_t vis,
                                            float2 (&acc)[2]) {
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        const float4 l = *reinterpret_cast<const float4 *>(nl + i);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = i + 2 * h;
            const float2 t = ffma2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), scale,
                                   h ? make_float2(l.z, l.w) : make_float2(l.x, l.y));
            float2 e = make_float2(ex2(t.x), ex2(t.y));
            if (MASKED) {                     // a row with lse = -inf (nl = inf) counts for nothing, whatever its score
                if (!(vis >> c & 1u) || (h ? l.z : l.x) == INFINITY) e.x = 0.f;
                if (!(vis >> (c + 1) & 1u) || (h ? l.w : l.y) == INFINITY) e.y = 0.f;
            }
            acc[h] = fadd2(acc[h], e);
        }
    }
}

template <int D, int N, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1) key_weights_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                                                                     const __grid_constant__ CUtensorMap tm_k,
                                                                     const Params p, const KeyWeights kw) {
    using L = Layout<D, N>;
    constexpr int KS = L::kKStages, QS = L::kQStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *ring_k = smem, *ring_q = ring_k + KS * L::kSub;
    float *nl = reinterpret_cast<float *>(ring_q + QS * L::kQ);            // [2][N]
    float *sums = nl + 2 * N;                                              // [kSumSlots][kItemKeys]
    uint64_t *k_full = reinterpret_cast<uint64_t *>(sums + kSumSlots * kItemKeys), *k_empty = k_full + KS;
    uint64_t *q_full = k_empty + KS, *q_empty = q_full + QS;
    // [buffer]: scores and normalisers there; scores read; normalisers read
    uint64_t *s_full = q_empty + QS, *s_free = s_full + 2, *l_empty = s_free + 2;
    uint64_t *x_full = l_empty + 2, *drain = x_full + kSumSlots;
    long long *scan = reinterpret_cast<long long *>(drain + 1);            // [kThreads / 32]
    long long *found = scan + kThreads / 32;                               // [2]
    volatile int *stop = reinterpret_cast<volatile int *>(found + 2);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(found + 2) + 1;
    int2 *tiles = reinterpret_cast<int2 *>(found + 3);                     // [2] a row tile's first token, and its columns
                                                                           // (negated: rows with lse = -inf among them)

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < KS; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < QS; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 2);     // the MMA issuer's commit and the normalisers' warp
            mbar_init(&s_free[i], L::kColHalves * kHalfWarps);
            mbar_init(&l_empty[i], L::kColHalves * kHalfWarps);
        }
        for (int i = 0; i < kSumSlots; ++i) mbar_init(&x_full[i], kHalfWarps);
        mbar_init(drain, 1);
        *stop = 0;
        fence_barrier_init();
    }
    if (tid == kLoadWarp * 32) {
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_k);
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(smem_u32(tmem_slot), L::kTmemCols);
        tc::tmem_relinquish();
    }
    dependent_start();
    Share sh;
    const bool has_work = block_share(p, tid, scan, found, sh);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int G = p.G, QT = p.qtile, ncols = G * QT;

    if (has_work && warp == kLoadWarp) {

        // ------------------------------------------------------ loads
        const uint64_t pol_k = l2_evict_first(), pol_q = l2_evict_normal();
        const uint32_t q_bytes = (uint32_t)(L::kHalves * ncols * 128);
        int ks = 0, qs = 0, nk = 0, nq = 0;
        uint32_t kph = 0, qph = 0;
        bool ok = true;
        auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, wait_bar(bar, parity, stop, p));
        };
        Walker it;
        it.init(p, sh);
        do {
            if (it.R == 0) continue;
#pragma unroll 1
            for (int u = 0; u < 2 && ok; ++u) {
                const int j0 = it.sub_key(u);
                if (j0 < 0) break;
                uint8_t *dst = ring_k + ks * L::kSub;
                if constexpr (PAGED) {
                    // lane: box lane / halves of page_box keys, D-half lane mod
                    // halves; the table is read while the slot is waited for
                    const int nbox = kSubKeys / p.page_box, bi = lane / L::kHalves, hf = lane % L::kHalves;
                    const bool box = bi < nbox;
                    const int key = j0 + bi * p.page_box;
                    const bool in = box && key < it.s.Lk;
                    const int entry = in ? page_entry(p, it.b, key) : 0;
                    if (nk >= KS && !(ok = wait_all(&k_empty[ks], kph ^ 1))) break;
                    if (lane == 0) mbar_arrive_expect_tx(&k_full[ks], L::kSub);
                    __syncwarp();
                    if (box) {
                        const int page = in ? page_checked(p, entry) : p.num_pages;
                        const int slot = key & ((1 << p.page_shift) - 1);
                        uint8_t *to = dst + hf * (kSubKeys * 128) + bi * p.page_box * 128;
                        if (p.page_rows)
                            tma_load_3d(to, &tm_k, &k_full[ks], hf * 64, it.hk, page * p.page_rows + slot, pol_k);
                        else
                            tma_load_4d(to, &tm_k, &k_full[ks], hf * 64, it.hk, slot, page, pol_k);
                    }
                } else {
                    if (nk >= KS && !(ok = wait_all(&k_empty[ks], kph ^ 1))) break;
                    if (lane == 0) mbar_arrive_expect_tx(&k_full[ks], L::kSub);
                    __syncwarp();
                    if (lane < L::kHalves)
                        tma_load_3d(dst + lane * (kSubKeys * 128), &tm_k, &k_full[ks], lane * 64, it.hk,
                                    it.s.k0 + it.packed_start(j0), pol_k);
                }
                ++nk;
                if (++ks == KS) {
                    ks = 0;
                    kph ^= 1;
                }
            }
#pragma unroll 1
            for (int r = it.r0; r < it.r1 && ok; ++r) {
                if (nq >= QS && !(ok = wait_all(&q_empty[qs], qph ^ 1))) break;
                if (lane == 0) mbar_arrive_expect_tx(&q_full[qs], q_bytes);
                __syncwarp();
                if (lane < L::kHalves)
                    tma_load_3d(ring_q + qs * L::kQ + lane * (N * 128), &tm_q, &q_full[qs], lane * 64, it.hk * G,
                                it.s.q0 + it.first_token(r, QT), pol_q);
                ++nq;
                if (++qs == QS) {
                    qs = 0;
                    qph ^= 1;
                }
            }
        } while (ok && it.next(p));
        if (!ok) *stop = 1;
        // loads in flight land before the block can leave
        for (int i = 0; i < min(nk, KS); ++i) {
            if (--ks < 0) {
                ks = KS - 1;
                kph ^= 1;
            }
            mbar_wait(&k_full[ks], kph);
        }
        for (int i = 0; i < min(nq, QS); ++i) {
            if (--qs < 0) {
                qs = QS - 1;
                qph ^= 1;
            }
            mbar_wait(&q_full[qs], qph);
        }
    } else if (has_work && warp == kMmaWarp) {

        // ------------------------------------------------------ MMA issue
        // the whole warp goes along, with values that are the same in all of
        // its lanes, and one elected lane issues
        constexpr uint32_t kId = tc::idesc_bf16_f32(kSubKeys, N, false);
        auto uniform = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
        auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, wait_bar(bar, parity, stop, p));
        };
        const uint32_t tm = uniform(tmem);
        const uint64_t k_desc = tc::smem_desc_sw128(uniform(smem_u32(ring_k)), 16, 1024);
        const uint64_t q_desc = tc::smem_desc_sw128(uniform(smem_u32(ring_q)), 16, 1024);
        uint32_t ks = 0, qs = 0, j = 0, kph = 0, qph = 0;
        bool ok = true, ready = false;       // ready: the next row tile's barriers were seen complete
        Walker it;
        it.init(p, sh);
        do {
            if (it.R == 0) continue;
            const uint32_t nsub = uniform(it.sub_key(1) >= 0 ? 2 : 1), n = uniform(it.r1 - it.r0);
            const uint32_t slot0 = ks, slot1 = ks + 1 == KS ? 0 : ks + 1;
            for (uint32_t u = 0; u < nsub && ok; ++u) {
                ok = wait_all(&k_full[ks], kph);
                if (++ks == KS) {
                    ks = 0;
                    kph ^= 1;
                }
            }
            const uint64_t a0 = k_desc + (slot0 * L::kSub >> 4), a1 = k_desc + (slot1 * L::kSub >> 4);
            for (uint32_t r = 0; r < n && ok; ++r, ++j) {
                const uint32_t buf = j & 1;
                if (!ready) {
                    if (!(ok = wait_all(&q_full[qs], qph))) break;
                    if (j >= 2 && !(ok = wait_all(&s_free[buf], ((j >> 1) - 1) & 1))) break;
                }
                tc::fence_after_sync();
                const uint64_t bd = q_desc + (qs * L::kQ >> 4);
                const uint32_t d = tm + buf * 2 * N, qe = smem_u32(&q_empty[qs]), sf = smem_u32(&s_full[buf]);
                if (++qs == QS) {
                    qs = 0;
                    qph ^= 1;
                }
                // the two sub-tiles' products take turns, so that no product
                // waits for the one before it
                auto issue = [&](int k_from, int k_to) {
#pragma unroll
                    for (int kk = k_from; kk < k_to; ++kk) {
                        const uint32_t ao = ((kk >> 2) * kSubKeys * 128 + (kk & 3) * 32) >> 4;
                        const uint32_t bo = ((kk >> 2) * N * 128 + (kk & 3) * 32) >> 4;
                        tc::mma_bf16_ss_elected(d, a0 + ao, bd + bo, kId, kk > 0);
                        if (nsub == 2) tc::mma_bf16_ss_elected(d + N, a1 + ao, bd + bo, kId, kk > 0);
                    }
                };
                if (tc::elect_one()) issue(0, D / 32);
                __syncwarp();
                // what the next row tile needs is looked at while these run
                ready = __all_sync(0xffffffffu, mbar_test_wait(&q_full[qs], qph) &&
                                                    (j == 0 || mbar_test_wait(&s_free[buf ^ 1], (((j + 1) >> 1) - 1) & 1)));
                if (tc::elect_one()) {
                    issue(D / 32, D / 16);
                    tc::commit(sf);
                    tc::commit(qe);
                }
                __syncwarp();
            }
            if (ok && tc::elect_one()) {
                tc::commit(smem_u32(&k_empty[slot0]));
                if (nsub == 2) tc::commit(smem_u32(&k_empty[slot1]));
            }
            __syncwarp();
        } while (ok && it.next(p));
        if (!ok) *stop = 1;
        // nothing that was issued may still run when the memory is freed
        if (tc::elect_one()) tc::commit(smem_u32(drain));
        __syncwarp();
        mbar_wait(drain, 0);
        __syncwarp();
    } else if (has_work && warp == kLseWarp) {

        // ------------------------------------------------------ normalisers
        int j = 0;
        bool ok = true;
        constexpr int kPer = (N + 31) / 32;
        int tok[kPer], off[kPer];            // column lane + 32 i: its token in the tile, its offset in lse
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = lane + 32 * i;
            tok[i] = c < ncols ? c / G : -1;
            off[i] = tok[i] * p.Hq + c % G;
        }
        Walker it;
        it.init(p, sh);
        do {
            if (it.R == 0) continue;
            for (int r = it.r0; r < it.r1 && ok; ++r, ++j) {
                const int t0 = it.first_token(r, QT);                      // may be negative: another sequence's rows
                const int lo = max(0, it.s.Lq - (r + 1) * QT), hi = it.s.Lq - r * QT;   // the tile's tokens
                const float *src = p.lse + ((long long)it.s.q0 + t0) * p.Hq + it.hk * G;
                float v[kPer];
                bool skip = false;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const bool row = tok[i] >= 0 && t0 + tok[i] >= lo && t0 + tok[i] < hi;
                    v[i] = row ? src[off[i]] : -INFINITY;
                    skip |= row && v[i] == -INFINITY;
                }
                skip = __any_sync(0xffffffffu, skip);
                const int buf = j & 1;
                if (j >= 2 &&
                    !(ok = __all_sync(0xffffffffu, wait_bar(&l_empty[buf], ((j >> 1) - 1) & 1, stop, p))))
                    break;
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (lane + 32 * i < N) nl[buf * N + lane + 32 * i] = -v[i] * kLog2e;
                if (lane == 0) tiles[buf] = make_int2(t0, skip ? (t0 - hi) * G : (hi - t0) * G);
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_full[buf]);
            }
        } while (ok && it.next(p));
        if (!ok) *stop = 1;
    } else if (has_work && warp < L::kColHalves * kHalfWarps) {

        // ------------------------------------------------------ exponentials and sums
        constexpr int kCols = N / L::kColHalves;                   // this warp's columns
        const int half = warp / kHalfWarps, wi = warp % kHalfWarps;
        const int u = wi >> 2, lane_key = (wi & 3) * 32 + lane, x = u * kSubKeys + lane_key;
        const int col0 = half * kCols;
        const uint32_t ts = tmem + ((uint32_t)((wi & 3) * 32) << 16) + u * N + col0;
        const float2 scale = make_float2(p.scale_log2, p.scale_log2);
        const bool writes = half == 0;
        auto wwait = [&](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, wait_bar(bar, parity, stop, p));
        };
        int j = 0, joined = 0;                                   // row tiles and items so far
        bool ok = true, ready = false;                           // ready: the next row tile's scores were seen
        Walker it;
        it.init(p, sh);
        do {
            const int n = it.R > 0 ? it.r1 - it.r0 : 0;
            if (n == 0 && !writes) continue;
            const int j0 = it.sub_key(u);
            const bool live = j0 >= 0;
            const int key = (PAGED ? j0 : it.packed_start(j0)) + lane_key;
            const bool mine = writes && live && key >= j0 && key < it.s.Lk;
            const int old = it.s.Lk - it.s.Lq;                   // keys below it were there before
            const long long at = ((long long)it.b * p.Hkv + it.hk) * kw.ld + key;
            // what the key had gathered, on its way while the products run
            float before = 0.f;
            if (mine && kw.w_in && kw.decay != 0.f && key < old) before = __ldcg(kw.w_in + at);
            float total = 0.f, carry = 0.f;
            for (int i = 0; i < n; ++i, ++j) {
                const int buf = j & 1;
                if (!__all_sync(0xffffffffu, ready) && !(ok = wwait(&s_full[buf], (j >> 1) & 1))) break;
                tc::fence_after_sync();
                const int2 tile = tiles[buf];
                const int t0 = tile.x, cols = abs(tile.y);
                const bool skip = tile.y < 0;
                // every column from `all_from` on sees all of the sub-tile's keys, none
                // before `any_from` sees any of them
                const int any_from = max(0, max(-t0, j0 - old - t0)) * G;
                const int all_from = max(0, max(-t0, j0 + kSubKeys - 1 - old - t0)) * G;
                const uint32_t tb = ts + buf * 2 * N;
                const float *n0 = nl + buf * N + col0;
                float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int ch = 0; ch < kCols / 16; ++ch) {
                    const int c0 = col0 + ch * 16;
                    const bool some = live && c0 + 16 > any_from && c0 < cols;
                    uint32_t v[16];
                    if (some) {
                        tc::ld_32x32b_x16(tb + ch * 16, v);
                        tc::wait_ld();
                    }
                    if (ch + 1 == kCols / 16) {
                        // everything read: the buffer is free, and the next one
                        // may be there already
                        tc::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s_free[buf]);
                        ready = mbar_test_wait(&s_full[buf ^ 1], ((j + 1) >> 1) & 1);
                    }
                    if (some) {
                        if (c0 >= all_from && c0 + 16 <= cols && !skip) {
                            add_columns<false>(v, n0 + ch * 16, scale, 0, acc);
                        } else {
                            // columns [first, cols) see this key
                            const int first = max(0, max(-t0, key - old - t0)) * G;
                            const int lo = min(16, max(0, first - c0)), hi = min(16, cols - c0);
                            add_columns<true>(v, n0 + ch * 16, scale, (1u << hi) - (1u << min(lo, hi)), acc);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&l_empty[buf]);
                const float2 s2 = fadd2(acc[0], acc[1]);
                add_compensated(total, carry, s2.x + s2.y);
            }
            if (!ok) break;
            if (L::kColHalves == 2 && n > 0) {
                const int slot = joined % kSumSlots;
                float *xs = sums + slot * kItemKeys + x;
                if (!writes) {
                    *xs = total;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&x_full[slot]);
                } else {
                    if (!(ok = wwait(&x_full[slot], (joined / kSumSlots) & 1))) break;
                    total += *xs;
                }
                ++joined;
            }
            if (!writes) continue;
            bool all = true;
            if (live && (it.r0 > 0 || it.r1 < it.w)) {
                // a part of the item's sums; of the item's blocks, the one whose
                // warp is the last to finish adds them all up in block order (the
                // first part of an item is its block's last: slot 2 c + 1, every
                // other part slot 2 c).  Each warp counts for its own 32 keys, so
                // no barrier joins warps of which one may have given up.
                const int c0 = block_of(it.P, sh), c1 = block_of(it.P + it.w - 1, sh), c = (int)blockIdx.x;
                uint32_t *ticket = kw.ticket + c0 * kHalfWarps + wi;
                __stcg(kw.part + (long long)(2 * c + (c == c0)) * kItemKeys + x, total);
                __threadfence();
                __syncwarp();
                uint32_t done = 0;
                if (lane == 0) done = atomicAdd(ticket, 1u);
                all = __shfl_sync(0xffffffffu, done, 0) == (uint32_t)(c1 - c0);
                if (all) {
                    __threadfence();
                    total = 0.f;
                    for (int i = c0; i <= c1; ++i) total += __ldcg(kw.part + (long long)(2 * i + (i == c0)) * kItemKeys + x);
                    if (lane == 0) *ticket = 0u;
                }
            }
            if (all && mine) {
                kw.w_out[at] = kw.decay * before + total;
                if (kw.born && key >= old) kw.born[at] = kw.seen[it.b] - (it.s.Lk - key);
            }
        } while (it.next(p));
        if (!ok) *stop = 1;
    }

    // free the tensor memory once every role is done with it
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, L::kTmemCols);
    }
}

template <int D, int N>
constexpr size_t smem_need() {
    using L = Layout<D, N>;
    // alignment slack, rings, normalisers, sums, barriers, scan, found, flags and row tiles
    const size_t need = 1024 + (size_t)L::kKStages * L::kSub + (size_t)L::kQStages * L::kQ + 2 * N * 4 +
                        kSumSlots * kItemKeys * 4 + (2 * L::kKStages + 2 * L::kQStages + kSumSlots + 7) * 8 + (kThreads / 32 + 2) * 8 + 24;
    return need > kMinSmem ? need : kMinSmem;
}

using Kernel = void (*)(CUtensorMap, CUtensorMap, Params, KeyWeights);

template <int D, int N>
void pick(bool paged, Kernel &fn, size_t &smem) {
    fn = paged ? (Kernel)key_weights_tc_kernel<D, N, true> : (Kernel)key_weights_tc_kernel<D, N, false>;
    smem = smem_need<D, N>();
}

void pick(int D, int n, bool paged, Kernel &fn, size_t &smem) {
    if (D == 64) {
        n == 16 ? pick<64, 16>(paged, fn, smem) : n == 32 ? pick<64, 32>(paged, fn, smem)
            : n == 64 ? pick<64, 64>(paged, fn, smem) : pick<64, 128>(paged, fn, smem);
    } else {
        n == 16 ? pick<128, 16>(paged, fn, smem) : n == 32 ? pick<128, 32>(paged, fn, smem)
            : n == 64 ? pick<128, 64>(paged, fn, smem) : pick<128, 128>(paged, fn, smem);
    }
}

}  // namespace

int key_weights_columns(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

int key_weights_part_floats() { return 2 * kItemKeys; }
int key_weights_tickets() { return kHalfWarps; }

cudaError_t key_weights_tc_prepare(int D, int columns) {
    for (bool paged : {false, true}) {
        Kernel fn;
        size_t smem;
        pick(D, columns, paged, fn, smem);
        const cudaError_t e = cudaFuncSetAttribute((const void *)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_key_weights_tc(const Params &p, const KeyWeights &kw, const CUtensorMap &tm_q,
                                  const CUtensorMap &tm_k, int columns, int ctas, cudaStream_t stream) {
    Kernel fn;
    size_t smem;
    pick(p.D, columns, p.block_table != nullptr, fn, smem);
    return launch_dependent(fn, dim3(ctas), dim3(kThreads), smem, stream, 0, tm_q, tm_k, p, kw);
}

}  // namespace vgqa
