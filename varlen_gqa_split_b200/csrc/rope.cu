// rope.cu -- rotary positions with several axes over packed tokens
// (attn_rope_apply), and the append of new keys and values to a paged cache
// with the rotation of queries and keys in the same pass
// (attn_append_paged).  The mathematics is in rope.cuh.
//
// Both are bound by memory: each element is read once and written once.  A
// block takes a few whole tokens; it computes the cosines and sines of their
// pairs once into shared memory (64-bit integer angle and sincospif, about 40
// instructions a pair) and every head of those tokens reuses them.  A thread
// then moves V pairs at a time, two 16-byte loads and two 16-byte stores,
// several heads in flight at once.
#include <algorithm>
#include <cmath>
#include <new>

#include "common.cuh"
#include "kernels.h"
#include "plan.h"
#include "rope.cuh"

struct attn_rope_s {
    vgqa::RopeTable tab;
    int D, n_axes, layout;
};

namespace vgqa {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;                // rows (token, head) of a thread in flight
constexpr int kMaxFactors = 2048;         // (cos, sin) pairs of a block's tokens: 16 KB

template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeTable tab, const T *x,
                                                        long long xs, long long n_tok, int H, int D,
                                                        const int32_t *__restrict__ pos, long long ps, float sign,
                                                        T *out, long long os, int tpb, int groups) {
    extern __shared__ float2 cs[];            // [tpb][n]
    const int n = tab.n;
    const long long t0 = (long long)blockIdx.x * tpb;
    const int nt = (int)min((long long)tpb, n_tok - t0);
    for (int i = threadIdx.x; i < nt * n; i += kThreads) {
        const int t = i / n, pr = i % n;
        cs[i] = rope_cos_sin(tab, pr, __ldg(pos + tab.axis[pr] * ps + t0 + t), sign);
    }
    __syncthreads();
    // thread = (group, row lane); rows = the tokens' heads
    const int lanes = kThreads / groups;
    const int g = threadIdx.x % groups, r0 = threadIdx.x / groups;
    if (r0 >= lanes) return;
    int a, b;
    rope_offsets<V, HALF>(g, n, D, a, b);
    const bool turn = g * V < n;
    const int rows = nt * H;
    using W = Vec<T, V>;
    for (int r = r0; r < rows; r += kUnroll * lanes) {
        W u[kUnroll], w[kUnroll];
        int tok[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int ri = r + i * lanes;
            if (ri < rows) {
                tok[i] = ri / H;
                const T *src = x + (t0 + tok[i]) * xs + (long long)(ri - tok[i] * H) * D;
                u[i] = *reinterpret_cast<const W *>(src + a);
                if (b >= 0) w[i] = *reinterpret_cast<const W *>(src + b);
            }
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int ri = r + i * lanes;
            if (ri < rows) {
                if (turn) rope_rotate<T, V, HALF>(u[i], w[i], cs + tok[i] * n + g * V);
                T *dst = out + (t0 + tok[i]) * os + (long long)(ri - tok[i] * H) * D;
                *reinterpret_cast<W *>(dst + a) = u[i];
                if (b >= 0) *reinterpret_cast<W *>(dst + b) = w[i];
            }
        }
    }
}

// Everything an append needs besides the plan's Params (q, k, v of Params
// are the new tokens' rows here, k_stride the cache's token stride).
struct Append {
    __nv_bfloat16 *q_out;                     // [T_q, Hq, D]
    __nv_bfloat16 *k_cache, *v_cache;
    const int32_t *pos;
    long long pos_stride, qs, ks, vs;         // axis stride; token strides of q, k, v
    long long n_tok;
    int tpb, groups;
};

template <int V, bool HALF>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ RopeTable tab, const Params p,
                                                          const Append ap) {
    using T = __nv_bfloat16;
    using W = Vec<T, V>;
    extern __shared__ float2 cs[];            // [tpb][n], then [tpb] cache offsets, [tpb] sequences
    const int n = tab.n, tpb = ap.tpb, tid = threadIdx.x;
    long long *slot = reinterpret_cast<long long *>(cs + tpb * n);
    int *seq = reinterpret_cast<int *>(slot + tpb);
    const long long t0 = (long long)blockIdx.x * tpb;
    const int nt = (int)min((long long)tpb, ap.n_tok - t0);

    // the sequence of each token: the one whose range covers it
    for (int i = tid; i < tpb; i += kThreads) seq[i] = -1;
    __syncthreads();
    for (int b = tid; b < p.B_max; b += kThreads) {
        const long long lo = max((long long)__ldg(p.cu_q + b), t0), hi = min((long long)__ldg(p.cu_q + b + 1), t0 + nt);
        for (long long t = lo; t < hi; ++t) seq[t - t0] = b;
    }
    for (int i = tid; i < nt * n; i += kThreads) {
        const int t = i / n, pr = i % n;
        cs[i] = rope_cos_sin(tab, pr, __ldg(ap.pos + tab.axis[pr] * ap.pos_stride + t0 + t), 1.f);
    }
    __syncthreads();
    // where its key goes: -1 not at all (no sequence, or a rejected one), -2
    // rotated but not stored (a bad table entry, or more queries than keys)
    for (int i = tid; i < nt; i += kThreads) {
        long long at = -1;
        int q0, Lq, k0, Lk;
        if (seq[i] >= 0 && load_lengths(p, seq[i], true, q0, Lq, k0, Lk)) {
            const int j = Lk - Lq + (int)(t0 + i - q0);
            at = -2;
            if (j >= 0) {
                const int page = page_of(p, seq[i], j);
                if (page < p.num_pages)
                    at = page * p.page_stride + (long long)(j & ((1 << p.page_shift) - 1)) * p.k_stride;
            }
        }
        slot[i] = at;
    }
    // a sequence that has to be reported but owns no token of any block
    if (blockIdx.x == 0)
        for (int b = tid; b < p.B_max; b += kThreads) {
            int q0, Lq, k0, Lk;
            load_lengths(p, b, true, q0, Lq, k0, Lk);
        }
    __syncthreads();

    const int lanes = kThreads / ap.groups;
    const int g = tid % ap.groups, r0 = tid / ap.groups;
    if (r0 >= lanes) return;
    int a, b;
    rope_offsets<V, HALF>(g, n, p.D, a, b);
    const bool turn = g * V < n;
    const int nq = ap.q_out ? p.Hq : 0, heads = nq + 2 * p.Hkv, rows = nt * heads;
    for (int r = r0; r < rows; r += kUnroll * lanes) {
        W u[kUnroll], w[kUnroll];
        T *dst[kUnroll];
        int tok[kUnroll];
        bool rot[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int ri = r + i * lanes;
            dst[i] = nullptr;
            if (ri < rows) {
                tok[i] = ri / heads;
                const int h = ri - tok[i] * heads, hk = h - nq;
                const long long t = t0 + tok[i], at = slot[tok[i]];
                const T *src;
                rot[i] = turn && hk < p.Hkv;
                if (hk < 0) {
                    src = p.q + t * ap.qs + h * p.D;
                    if (at != -1) dst[i] = ap.q_out + (t * p.Hq + h) * p.D;
                } else if (hk < p.Hkv) {
                    src = p.k + t * ap.ks + hk * p.D;
                    if (at >= 0) dst[i] = ap.k_cache + at + hk * p.D;
                } else {
                    src = p.v + t * ap.vs + (hk - p.Hkv) * p.D;
                    if (at >= 0) dst[i] = ap.v_cache + at + (hk - p.Hkv) * p.D;
                }
                if (dst[i]) {
                    u[i] = *reinterpret_cast<const W *>(src + a);
                    if (b >= 0) w[i] = *reinterpret_cast<const W *>(src + b);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            if (dst[i]) {
                if (rot[i]) rope_rotate<T, V, HALF>(u[i], w[i], cs + tok[i] * n + g * V);
                *reinterpret_cast<W *>(dst[i] + a) = u[i];
                if (b >= 0) *reinterpret_cast<W *>(dst[i] + b) = w[i];
            }
        }
    }
}

// Tokens per block: enough (token, head, group) items for every thread to
// have kUnroll of them in flight at least once, fewer where the blocks would
// not cover the SMs, and no more factors than shared memory is set aside for.
int tokens_per_block(long long n_tok, int heads, int groups, int n) {
    const long long want = std::max(1, 2 * kUnroll * kThreads / (heads * groups));
    const long long cover = std::max(1ll, n_tok / (2 * 148));
    return (int)std::max(1ll, std::min({want, cover, (long long)(kMaxFactors / std::max(1, n))}));
}

// The widest access, in elements, that divides the pairs and the copied rest
// and that every pointer and stride keeps aligned: 16 bytes where they allow,
// else 8, else one element.
int access_width(int size, int n, int D, uintptr_t bits) {
    for (int bytes : {16, 8}) {
        const int v = bytes / size;
        if (n % v == 0 && D % v == 0 && bits % bytes == 0) return v;
    }
    return 1;
}

template <typename T, int V>
cudaError_t launch_rope(const attn_rope_s &r, const void *x, long long xs, long long n_tok, int H, const int32_t *pos,
                        long long ps, bool grad, void *out, long long os, cudaStream_t s) {
    const int n = r.tab.n, groups = rope_groups(n, r.D, V), tpb = tokens_per_block(n_tok, H, groups, n);
    const long long blocks = (n_tok + tpb - 1) / tpb;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    const size_t smem = (size_t)tpb * n * sizeof(float2);
    auto *xi = static_cast<const T *>(x);
    auto *oi = static_cast<T *>(out);
    const float sign = grad ? -1.f : 1.f;
    if (r.layout == ATTN_ROPE_HALF)
        rope_kernel<T, V, true><<<(unsigned)blocks, kThreads, smem, s>>>(r.tab, xi, xs, n_tok, H, r.D, pos, ps, sign,
                                                                          oi, os, tpb, groups);
    else
        rope_kernel<T, V, false><<<(unsigned)blocks, kThreads, smem, s>>>(r.tab, xi, xs, n_tok, H, r.D, pos, ps, sign,
                                                                           oi, os, tpb, groups);
    return cudaGetLastError();
}

template <int V>
cudaError_t launch_append(const RopeTable &tab, bool half, const Params &p, Append ap, cudaStream_t s) {
    const int heads = (ap.q_out ? p.Hq : 0) + 2 * p.Hkv;
    ap.groups = rope_groups(tab.n, p.D, V);
    ap.tpb = tokens_per_block(ap.n_tok, heads, ap.groups, std::max(tab.n, 64));
    const long long blocks = (ap.n_tok + ap.tpb - 1) / ap.tpb;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    const size_t smem = (size_t)ap.tpb * (tab.n * sizeof(float2) + sizeof(long long) + sizeof(int));
    if (half)
        append_kernel<V, true><<<(unsigned)blocks, kThreads, smem, s>>>(tab, p, ap);
    else
        append_kernel<V, false><<<(unsigned)blocks, kThreads, smem, s>>>(tab, p, ap);
    return cudaGetLastError();
}

}  // namespace

}  // namespace vgqa

using namespace vgqa;

ATTN_EXPORT int attn_rope_create(attn_rope_t *out, int D, int n_pairs, int n_axes, const double *freq,
                                 const int32_t *axis, int layout, float scale) {
    if (!out) return ATTN_E_NULL;
    *out = nullptr;
    if (!freq || !axis) return ATTN_E_NULL;
    if (D < 2 || D > 2 * kRopeMaxPairs || n_pairs < 1 || 2 * n_pairs > D || n_axes < 1 || n_axes > kRopeMaxAxes ||
        (layout != ATTN_ROPE_HALF && layout != ATTN_ROPE_INTERLEAVED) || !std::isfinite(scale))
        return ATTN_E_INVALID_ARG;
    for (int i = 0; i < n_pairs; ++i)
        if (!std::isfinite(freq[i]) || axis[i] < 0 || axis[i] >= n_axes) return ATTN_E_INVALID_ARG;
    attn_rope_s *r = new (std::nothrow) attn_rope_s{};
    if (!r) return ATTN_E_NOMEM;
    r->D = D;
    r->n_axes = n_axes;
    r->layout = layout;
    r->tab.n = n_pairs;
    r->tab.scale = scale;
    for (int i = 0; i < n_pairs; ++i) {
        // fraction of a turn per unit position in units of 2^-64 (long double
        // carries 64 bits; whole turns drop out)
        long double t = (long double)freq[i] / 6.283185307179586476925286766559005768L;
        t -= floorl(t);
        const long double f = floorl(ldexpl(t, 64) + 0.5L);
        r->tab.turn[i] = f >= 18446744073709551616.0L ? 0ull : (unsigned long long)f;
        r->tab.axis[i] = (uint8_t)axis[i];
    }
    *out = r;
    return ATTN_OK;
}

ATTN_EXPORT void attn_rope_destroy(attn_rope_t rope) { delete rope; }

ATTN_EXPORT int attn_rope_apply(attn_rope_t rope, int dtype, const void *x, int64_t x_token_stride, int64_t T, int H,
                                const int32_t *pos, int64_t pos_stride, int grad, void *out, int64_t out_token_stride,
                                void *stream) {
    if (!rope || !x || !pos || !out) return ATTN_E_NULL;
    const int size = dtype == ATTN_DTYPE_F32 ? 4 : 2;
    if (dtype != ATTN_DTYPE_BF16 && dtype != ATTN_DTYPE_F16 && dtype != ATTN_DTYPE_F32) return ATTN_E_UNSUPPORTED;
    if (T < 0 || T >= (1ll << 31) || H < 1 || H > 65536) return ATTN_E_INVALID_ARG;
    const long long row = (long long)H * rope->D;
    if (x_token_stride < row || out_token_stride < row || x_token_stride > (1ll << 38) ||
        out_token_stride > (1ll << 38) || (rope->n_axes > 1 && pos_stride < T))
        return ATTN_E_INVALID_ARG;
    if (!aligned(x, size) || !aligned(out, size) || !aligned(pos, 4)) return ATTN_E_ALIGNMENT;
    if (T == 0) return ATTN_OK;
    // in place element for element, or not overlapping at all: a shifted
    // overlap would read what another thread wrote
    const char *xb = static_cast<const char *>(x), *ob = static_cast<const char *>(out);
    const bool same = xb == ob && x_token_stride == out_token_stride;
    if (!same && xb < ob + ((T - 1) * out_token_stride + row) * size &&
        ob < xb + ((T - 1) * x_token_stride + row) * size) {
        // two sets of heads of one buffer: same stride, disjoint within it
        const long long gap = std::llabs(xb - ob) % (x_token_stride * size);
        if (x_token_stride != out_token_stride || gap < row * size || x_token_stride * size - gap < row * size)
            return ATTN_E_INVALID_ARG;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const uintptr_t bits = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out) |
                           (uintptr_t)(x_token_stride * size) | (uintptr_t)(out_token_stride * size);
    const int v = access_width(size, rope->tab.n, rope->D, bits);
    cudaError_t e = cudaErrorInvalidValue;
#define VGQA_ROPE(T_, V_) e = launch_rope<T_, V_>(*rope, x, x_token_stride, T, H, pos, pos_stride, grad != 0, out, out_token_stride, s)
    if (dtype == ATTN_DTYPE_F32) {
        if (v == 4) VGQA_ROPE(float, 4);
        else if (v == 2) VGQA_ROPE(float, 2);
        else VGQA_ROPE(float, 1);
    } else if (dtype == ATTN_DTYPE_F16) {
        if (v == 8) VGQA_ROPE(__half, 8);
        else if (v == 4) VGQA_ROPE(__half, 4);
        else VGQA_ROPE(__half, 1);
    } else {
        if (v == 8) VGQA_ROPE(__nv_bfloat16, 8);
        else if (v == 4) VGQA_ROPE(__nv_bfloat16, 4);
        else VGQA_ROPE(__nv_bfloat16, 1);
    }
#undef VGQA_ROPE
    return e == cudaSuccess ? ATTN_OK : ATTN_E_CUDA;
}

ATTN_EXPORT int attn_append_paged(attn_plan_t plan, attn_rope_t rope, const void *q, int64_t q_token_stride,
                                  const void *k, int64_t k_token_stride, const void *v, int64_t v_token_stride,
                                  int64_t T_q, const int32_t *pos, int64_t pos_stride, void *q_out, void *k_cache,
                                  void *v_cache, int64_t page_stride, int64_t token_stride, int page_size,
                                  int num_pages, const int32_t *block_table, int bt_stride, const int32_t *cu_q,
                                  const int32_t *cu_k, void *stream) {
    if (!plan || !live(plan)) return ATTN_E_BAD_PLAN;
    if (!k || !v || !k_cache || !v_cache || !cu_q || !cu_k || (rope && !pos) || !q != !q_out) return ATTN_E_NULL;
    int rc = check_paging(plan, page_stride, token_stride, page_size, num_pages, block_table, bt_stride);
    if (rc != ATTN_OK) return rc;
    const attn_plan_desc &d = plan->d;
    if (T_q < 0 || T_q >= (1ll << 31) || (rope && rope->n_axes > 1 && pos_stride < T_q)) return ATTN_E_INVALID_ARG;
    if (rope && rope->D != d.D) return ATTN_E_INVALID_ARG;
    const long long qrow = (long long)d.Hq * d.D, krow = (long long)d.Hkv * d.D;
    for (long long st : {(long long)k_token_stride, (long long)v_token_stride, q ? (long long)q_token_stride : krow})
        if (st < krow || st % 8 != 0 || st > (1ll << 38)) return ATTN_E_INVALID_ARG;
    if (q && q_token_stride < qrow) return ATTN_E_INVALID_ARG;
    for (const void *ptr : {q, k, v, (const void *)q_out, (const void *)k_cache, (const void *)v_cache})
        if (!aligned(ptr, 16)) return ATTN_E_ALIGNMENT;
    if (!aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(pos, 4)) return ATTN_E_ALIGNMENT;
    // q_out is q itself (packed) or apart from it
    if (q && q_out != q && T_q > 0) {
        const char *a = static_cast<const char *>(q), *b = static_cast<const char *>(q_out);
        if (a < b + T_q * qrow * 2 && b < a + ((T_q - 1) * q_token_stride + qrow) * 2) return ATTN_E_INVALID_ARG;
    } else if (q && q_token_stride != qrow) {
        return ATTN_E_INVALID_ARG;
    }
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_E_CUDA;
    if (dev != plan->device) return ATTN_E_DEVICE;
    if (T_q == 0) return ATTN_OK;

    Params p{};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.cu_q = cu_q;
    p.cu_k = cu_k;
    p.err = plan->err;
    p.B_max = d.B_max;
    p.s_max = d.s_max;
    p.Hq = d.Hq;
    p.Hkv = d.Hkv;
    p.D = d.D;
    p.max_q = d.max_q;
    p.k_stride = token_stride;
    p.block_table = block_table;
    p.bt_stride = bt_stride;
    p.page_shift = log2_exact(page_size);
    p.num_pages = num_pages;
    p.page_stride = page_stride;
    Append ap{};
    ap.q_out = static_cast<__nv_bfloat16 *>(q_out);
    ap.k_cache = static_cast<__nv_bfloat16 *>(k_cache);
    ap.v_cache = static_cast<__nv_bfloat16 *>(v_cache);
    ap.pos = pos;
    ap.pos_stride = pos_stride;
    ap.qs = q_token_stride;
    ap.ks = k_token_stride;
    ap.vs = v_token_stride;
    ap.n_tok = T_q;
    RopeTable none{};
    const RopeTable &tab = rope ? rope->tab : none;      // no pairs: everything is copied
    const bool half = !rope || rope->layout == ATTN_ROPE_HALF;
    // strides and pointers are 16-byte ones here; only the pair count may be odd
    const int w = access_width(2, tab.n, d.D, 0);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = w == 8   ? launch_append<8>(tab, half, p, ap, s)
                          : w == 4 ? launch_append<4>(tab, half, p, ap, s)
                                   : launch_append<1>(tab, half, p, ap, s);
    return e == cudaSuccess ? ATTN_OK : ATTN_E_CUDA;
}
