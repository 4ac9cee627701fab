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
// Warps: 0-7 epilogue (warp w: sub-tile w / 4, lanes 32 (w mod 4)); 8 issues
// the MMAs; 9 loads K and Q by TMA (128-byte swizzle, mbarrier rings); 10
// stages -lse log2 e of each row tile.  Every wait is bounded, as in the
// attention kernels.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "key_weights.h"
#include "tc.cuh"

namespace vgqa {

namespace {

constexpr int kSubKeys = 128;             // keys per sub-tile (MMA M)
constexpr int kItemKeys = 256;
constexpr int kEpiWarps = 8;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kLseWarp = 10;
constexpr int kThreads = 352;
constexpr int kLseStages = 4;
constexpr int kMaxStages = 8;
constexpr size_t kMinSmem = 120 * 1024;   // one block per SM: tensor memory is never waited for

template <int D, int N>
struct Layout {
    static constexpr int kHalves = D / 64;
    static constexpr int kSub = kSubKeys * D * 2;             // one sub-tile of K
    static constexpr int kQ = N * D * 2;                      // one row tile of Q
    // ring depths: 200 KB in all; K first where N is small (decode streams
    // K), at least two items' worth of K otherwise
    static constexpr int kQStages = N == 128 ? 2 : 4;
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
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += seq_info(p, b, blockIdx.x == 0).tot * p.Hkv;
    long long inc = mine;
    const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    long long T = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) inc += scan[i];
        T += scan[i];
    }
    sh.T = T;
    sh.C = (int)min((long long)gridDim.x, T);
    if ((int)blockIdx.x >= sh.C) return false;
    sh.lo = T * blockIdx.x / sh.C;
    sh.hi = T * (blockIdx.x + 1) / sh.C;
    long long at = inc - mine;
    if (sh.lo >= at && sh.lo < inc) {
        for (int b = b0; b < b1; ++b) {
            const long long n = seq_info(p, b, false).tot * p.Hkv;
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
        hk = (int)(rem / s.tot);
        rem -= hk * s.tot;
        P = g - rem;
        const int full = max(s.nrt, 1);
        if (rem < (long long)s.ksat * full) {
            kt = (int)(rem / full);
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
    // first key of sub-tile u, or -1 if the sequence ends before it; where its
    // box starts (packed K: moved back to end with the sequence, so that no
    // load passes the last key of a buffer)
    __device__ int sub_key(int u) const {
        const int j = kt * kItemKeys + u * kSubKeys;
        return j < s.Lk ? j : -1;
    }
};

// ------------------------------------------------------------ kernel

// sum over 32 (or 16) columns of 2^(s scale + nl); MASKED: only those in `vis`
template <int W, bool MASKED>
__device__ __forceinline__ void add_columns(const uint32_t (&v)[W], const float *nl, float scale, uint32_t vis,
                                            float2 (&acc)[4]) {
    const float2 sc = make_float2(scale, scale);
#pragma unroll
    for (int i = 0; i < W; i += 4) {
        const float4 l = *reinterpret_cast<const float4 *>(nl + i);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = i + 2 * h;
            const float2 t = ffma2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), sc,
                                   h ? make_float2(l.z, l.w) : make_float2(l.x, l.y));
            float2 e = make_float2(ex2(t.x), ex2(t.y));
            if (MASKED) {
                if (!(vis >> c & 1u)) e.x = 0.f;
                if (!(vis >> (c + 1) & 1u)) e.y = 0.f;
            }
            acc[(c >> 1) & 3] = fadd2(acc[(c >> 1) & 3], e);
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
    float *nl = reinterpret_cast<float *>(ring_q + QS * L::kQ);            // [kLseStages][N]
    uint64_t *k_full = reinterpret_cast<uint64_t *>(nl + kLseStages * N), *k_empty = k_full + KS;
    uint64_t *q_full = k_empty + KS, *q_empty = q_full + QS;
    uint64_t *l_full = q_empty + QS, *l_empty = l_full + kLseStages;
    uint64_t *s_full = l_empty + kLseStages, *s_free = s_full + 2, *drain = s_free + 2;
    long long *scan = reinterpret_cast<long long *>(drain + 1);            // [kThreads / 32]
    long long *found = scan + kThreads / 32;                               // [2]
    volatile int *stop = reinterpret_cast<volatile int *>(found + 2);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(found + 2) + 1;

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
        for (int i = 0; i < kLseStages; ++i) {
            mbar_init(&l_full[i], 1);
            mbar_init(&l_empty[i], kEpiWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_free[i], kEpiWarps);
        }
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
                                    it.s.k0 + min(j0, it.s.Lk - kSubKeys), pol_k);
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
                // the box ends with the row tile's last token
                if (lane < L::kHalves)
                    tma_load_3d(ring_q + qs * L::kQ + lane * (N * 128), &tm_q, &q_full[qs], lane * 64, it.hk * G,
                                it.s.q0 + it.s.Lq - (r + 1) * QT, pol_q);
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
        if (lane == 0) {
            constexpr uint32_t kId = tc::idesc_bf16_f32(kSubKeys, N, false);
            const uint32_t k0 = smem_u32(ring_k), q0 = smem_u32(ring_q);
            int ks = 0, qs = 0, j = 0;
            uint32_t kph = 0, qph = 0;
            bool ok = true;
            Walker it;
            it.init(p, sh);
            do {
                if (it.R == 0) continue;
                const int nsub = it.sub_key(1) >= 0 ? 2 : 1;
                int slot[2];
                for (int u = 0; u < nsub && ok; ++u) {
                    slot[u] = ks;
                    ok = wait_bar(&k_full[ks], kph, stop, p);
                    if (++ks == KS) {
                        ks = 0;
                        kph ^= 1;
                    }
                }
                for (int r = it.r0; r < it.r1 && ok; ++r, ++j) {
                    const int buf = j & 1;
                    if (!(ok = wait_bar(&q_full[qs], qph, stop, p))) break;
                    if (j >= 2 && !(ok = wait_bar(&s_free[buf], ((j >> 1) - 1) & 1, stop, p))) break;
                    tc::fence_after_sync();
                    const uint64_t bd = tc::smem_desc_sw128(q0 + qs * L::kQ, 16, 1024);
                    for (int u = 0; u < nsub; ++u) {
                        const uint64_t ad = tc::smem_desc_sw128(k0 + slot[u] * L::kSub, 16, 1024);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const int hf = kk >> 2, cc = (kk & 3) * 32;
                            tc::mma_bf16_ss(tmem + (buf * 2 + u) * N, ad + ((hf * kSubKeys * 128 + cc) >> 4),
                                            bd + ((hf * N * 128 + cc) >> 4), kId, kk > 0);
                        }
                    }
                    tc::commit(smem_u32(&q_empty[qs]));
                    tc::commit(smem_u32(&s_full[buf]));
                    if (++qs == QS) {
                        qs = 0;
                        qph ^= 1;
                    }
                }
                if (ok)
                    for (int u = 0; u < nsub; ++u) tc::commit(smem_u32(&k_empty[slot[u]]));
            } while (ok && it.next(p));
            if (!ok) *stop = 1;
            // nothing this thread issued may still run when the memory is freed
            tc::commit(smem_u32(drain));
            mbar_wait(drain, 0);
        }
        __syncwarp();
    } else if (has_work && warp == kLseWarp) {

        // ------------------------------------------------------ normalisers
        int ls = 0, j = 0;
        uint32_t lph = 0;
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
                const int t0 = it.s.Lq - (r + 1) * QT;                     // may be negative: those rows do not exist
                const float *src = p.lse + ((long long)it.s.q0 + t0) * p.Hq + it.hk * G;
                float v[kPer];
#pragma unroll
                for (int i = 0; i < kPer; ++i) v[i] = tok[i] >= 0 && t0 + tok[i] >= 0 ? __ldg(src + off[i]) : -INFINITY;
                if (j >= kLseStages &&
                    !(ok = __all_sync(0xffffffffu, wait_bar(&l_empty[ls], lph ^ 1, stop, p))))
                    break;
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (lane + 32 * i < N)   // a row that saw nothing (lse = -inf) weighs nothing
                        nl[ls * N + lane + 32 * i] = v[i] == -INFINITY ? -INFINITY : -v[i] * kLog2e;
                __syncwarp();
                if (lane == 0) mbar_arrive(&l_full[ls]);
                if (++ls == kLseStages) {
                    ls = 0;
                    lph ^= 1;
                }
            }
        } while (ok && it.next(p));
        if (!ok) *stop = 1;
    } else if (has_work && warp < kEpiWarps) {

        // ------------------------------------------------------ exponentials and sums
        const int u = warp >> 2, lane_key = (warp & 3) * 32 + lane;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const float scale = p.scale_log2;
        auto wwait = [&](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, wait_bar(bar, parity, stop, p));
        };
        int ls = 0, j = 0;
        uint32_t lph = 0;
        bool ok = true;
        Walker it;
        it.init(p, sh);
        do {
            const int j0 = it.sub_key(u);
            const bool live = j0 >= 0;
            const int key = (PAGED ? j0 : min(j0, it.s.Lk - kSubKeys)) + lane_key;
            const bool mine = live && key >= j0 && key < it.s.Lk;
            const int old = it.s.Lk - it.s.Lq;                   // keys below it were there before
            const long long at = ((long long)it.b * p.Hkv + it.hk) * kw.ld + key;
            const bool whole = it.r0 == 0 && it.r1 == it.w;
            // what the key had gathered, on its way while the products run
            float before = 0.f;
            if (mine && kw.w_in && kw.decay != 0.f && key < old) before = __ldcg(kw.w_in + at);
            float total = 0.f, carry = 0.f;
            if (it.R > 0) {
                for (int r = it.r0; r < it.r1; ++r, ++j) {
                    const int buf = j & 1;
                    if (!(ok = wwait(&l_full[ls], lph)) || !(ok = wwait(&s_full[buf], (j >> 1) & 1))) break;
                    tc::fence_after_sync();
                    if (live) {
                        const int t0 = it.s.Lq - (r + 1) * QT;
                        // columns [first, ncols) see this key; all of them see every
                        // key of the sub-tile where `clear`
                        const int first = max(0, max(-t0, key - old - t0)) * G;
                        const bool clear = t0 >= 0 && j0 + kSubKeys - 1 - old - t0 <= 0 && ncols == N;
                        const uint32_t ts = tmem + lane_base + (buf * 2 + u) * N;
                        const float *n0 = nl + ls * N;
                        float2 acc[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[i] = make_float2(0.f, 0.f);
                        if constexpr (N == 16) {
                            uint32_t v[16];
                            tc::ld_32x32b_x16(ts, v);
                            tc::wait_ld();
                            const uint32_t vis = first >= 16 ? 0u : (0xffffffffu << first) & ((1u << ncols) - 1u);
                            if (clear) add_columns<16, false>(v, n0, scale, 0, acc);
                            else add_columns<16, true>(v, n0, scale, vis, acc);
                        } else {
                            uint32_t v[2][32];
                            tc::ld_32x32b_x32(ts, v[0]);
#pragma unroll
                            for (int ch = 0; ch < N / 32; ++ch) {
                                tc::wait_ld();
                                if (ch + 1 < N / 32) tc::ld_32x32b_x32(ts + (ch + 1) * 32, v[(ch + 1) & 1]);
                                if (clear) {
                                    add_columns<32, false>(v[ch & 1], n0 + ch * 32, scale, 0, acc);
                                } else {
                                    const int lo = min(32, max(0, first - ch * 32)), hi = min(32, max(0, ncols - ch * 32));
                                    const uint32_t vis = (uint32_t)((1ull << hi) - 1ull) & (uint32_t)~((1ull << lo) - 1ull);
                                    add_columns<32, true>(v[ch & 1], n0 + ch * 32, scale, vis, acc);
                                }
                            }
                        }
                        const float2 s2 = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
                        // compensated: many row tiles may add up
                        const float y = (s2.x + s2.y) - carry, t = total + y;
                        carry = (t - total) - y;
                        total = t;
                    }
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&s_free[buf]);
                        mbar_arrive(&l_empty[ls]);
                    }
                    if (++ls == kLseStages) {
                        ls = 0;
                        lph ^= 1;
                    }
                }
                if (!ok) break;
            }
            bool write = true;
            if (!whole && live) {
                // this part's sums; of the item's blocks, the one whose warp is
                // the last to finish adds them all up in block order (the first
                // part of an item is its block's last: slot 2 c + 1, every other
                // part slot 2 c).  Each warp counts for its own 32 keys, so no
                // barrier joins warps of which one may have given up.
                const int c0 = block_of(it.P, sh), c1 = block_of(it.P + it.w - 1, sh), c = (int)blockIdx.x;
                const int x = u * kSubKeys + lane_key;
                uint32_t *ticket = kw.ticket + c0 * kEpiWarps + warp;
                __stcg(kw.part + (long long)(2 * c + (c == c0)) * kItemKeys + x, total);
                __threadfence();
                __syncwarp();
                uint32_t done = 0;
                if (lane == 0) done = atomicAdd(ticket, 1u);
                write = __shfl_sync(0xffffffffu, done, 0) == (uint32_t)(c1 - c0);
                if (write) {
                    __threadfence();
                    total = 0.f;
                    for (int i = c0; i <= c1; ++i) total += __ldcg(kw.part + (long long)(2 * i + (i == c0)) * kItemKeys + x);
                    if (lane == 0) *ticket = 0u;
                }
            }
            if (write && mine) {
                kw.w_out[at] = kw.decay * before + total;
                if (kw.born && key >= old) kw.born[at] = __ldg(kw.seen + it.b) - (it.s.Lk - key);
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
    // alignment slack, rings, normalisers, barriers, scan, found, flags
    const size_t need = 1024 + (size_t)L::kKStages * L::kSub + (size_t)L::kQStages * L::kQ + kLseStages * N * 4 +
                        (2 * L::kKStages + 2 * L::kQStages + 2 * kLseStages + 5) * 8 + (kThreads / 32 + 2) * 8 + 16;
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
int key_weights_tickets() { return kEpiWarps; }

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
    fn<<<ctas, kThreads, smem, stream>>>(tm_q, tm_k, p, kw);
    return cudaGetLastError();
}

}  // namespace vgqa
