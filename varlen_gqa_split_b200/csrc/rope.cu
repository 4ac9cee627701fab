// rope.cu -- rotary positions with several axes over packed tokens
// (attn_rope_apply), and the append of new keys and values to a paged cache
// with the rotation of queries and keys in the same pass
// (attn_append_paged).  The mathematics is in rope.cuh.
//
// Both are bound by memory: each element is read once and written once.  A
// block takes a few tokens at a time; it computes the cosines and sines of
// their pairs once into shared memory (64-bit integer angle and sincospif,
// about 40 instructions a pair), and a thread keeps those of its token and its
// V pairs in registers while it goes through some of the token's heads: two
// 16-byte loads and two 16-byte stores a head, several heads in flight.
// Measured: 8192 tokens x 72 heads of 128, bf16, 48.3 us, 96% of the measured
// HBM bandwidth (8 heads a thread, two in flight: 55.9; 16: 62); 64 tokens x
// 40 heads 2.9 us; four chunks of 512 to 2048 tokens of 2048 rows each appended
// 24.5 to 25.8 us, 62 to 66% (a block whose rows lie behind the last sequence
// finds that out only after its factors: with all 8192 rows live 33.2, 77%).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>
#include <new>
#include <unordered_set>

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

constexpr int kThreads = 256;             // at most; a block has what its tokens need
constexpr int kBlocksPerSm = 4;
constexpr int kUnroll = 3;                // heads of a thread in flight at once
constexpr int kMaxHeads = 3;              // heads a thread goes through, unless there are too many
constexpr int kAppendUnroll = 2;          // and in an append, whose registers also hold addresses
constexpr int kAppendHeads = 5;
constexpr int kMaxFactors = 2048;         // (cos, sin) pairs of a block's tokens: 16 KB

// How threads are laid out: `groups` neighbours share a head, `lanes` heads
// are worked on side by side, `tokens` tokens in a block.
struct Shape {
    int groups, lanes, tokens, threads;
    long long blocks;
};

// Heads per thread: enough work to keep the factors' cost small, but a thread
// per head while the whole call would not fill the device twice over.
Shape shape_of(long long n_tok, int heads, int groups, int n, int most, int sms) {
    Shape s;
    s.groups = groups;
    const long long fill = 2ll * sms * kThreads * kBlocksPerSm;
    const int each = (int)std::max(1ll, std::min<long long>(most, n_tok * heads * groups / fill));
    s.lanes = std::min((heads + each - 1) / each, kThreads / groups);
    s.tokens = std::max(1, std::min(kThreads / (groups * s.lanes), kMaxFactors / std::max(n, 1)));
    s.tokens = (int)std::min<long long>(s.tokens, n_tok);
    s.threads = (s.tokens * groups * s.lanes + 31) / 32 * 32;
    s.blocks = (n_tok + s.tokens - 1) / s.tokens;
    return s;
}

// SMs of the current device (asked once per device)
int current_sms() {
    static std::atomic<int> known[64];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    std::atomic<int> *at = dev < 64 ? &known[dev] : nullptr;
    if (at && (sms = at->load(std::memory_order_relaxed)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 1;
    if (at) at->store(sms, std::memory_order_relaxed);
    return sms;
}

// the cosines and sines of tokens [t0, t0 + nt): cs[token][pair]
__device__ __forceinline__ void fill_factors(const RopeTable &tab, float2 *cs, const int32_t *pos,
                                             long long ps, long long t0, int nt, float sign) {
    for (int i = threadIdx.x; i < nt * tab.n; i += blockDim.x) {
        const int t = i / tab.n, pr = i - t * tab.n;
        cs[i] = rope_cos_sin(tab, pr, pos[tab.axis[pr] * ps + t0 + t], sign);
    }
}

template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    rope_kernel(const __grid_constant__ RopeTable tab, const T *x, long long xs, long long n_tok, int H, int D,
                const int32_t *pos, long long ps, float sign, T *out, long long os, int groups, int lanes,
                int tokens) {
    extern __shared__ float2 cs[];
    dependent_start();
    const int n = tab.n;
    const long long t0 = (long long)blockIdx.x * tokens;
    const int nt = (int)min((long long)tokens, n_tok - t0);
    const int g = threadIdx.x % groups, y = threadIdx.x / groups, lane = y % lanes, tok = y / lanes;
    int a, b;
    rope_offsets<V, HALF>(g, n, D, a, b);
    const bool turn = g * V < n, live = tok < nt;
    using W = Vec<T, V>;
    const T *src = x + (t0 + tok) * xs + a;
    T *dst = out + (t0 + tok) * os + a;
    const int d = b - a;                      // from the first access to the second
    W u[kUnroll], w[kUnroll];
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            if (live && h + i * lanes < H) {
                u[i] = *reinterpret_cast<const W *>(src + (h + i * lanes) * D);
                if (b >= 0) w[i] = *reinterpret_cast<const W *>(src + (h + i * lanes) * D + d);
            }
    };
    load(lane);                               // on its way while the factors are computed
    fill_factors(tab, cs, pos, ps, t0, nt, sign);
    __syncthreads();
    if (!live) return;
    float2 f[V];
    if (turn)
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = cs[tok * n + g * V + i];
    for (int h = lane; h < H; h += kUnroll * lanes) {
        if (h != lane) load(h);
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            if (h + i * lanes < H) {
                if (turn) rope_rotate<T, V, HALF>(u[i], w[i], f);
                *reinterpret_cast<W *>(dst + (h + i * lanes) * D) = u[i];
                if (b >= 0) *reinterpret_cast<W *>(dst + (h + i * lanes) * D + d) = w[i];
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
    int groups, lanes, tokens;
};

template <int V, bool HALF>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    append_kernel(const __grid_constant__ RopeTable tab, const Params p, const Append ap) {
    using T = __nv_bfloat16;
    using W = Vec<T, V>;
    extern __shared__ float2 cs[];            // [tokens][n], then [tokens] cache offsets, [tokens] (sequence, key)
    dependent_start();
    const int n = tab.n, tokens = ap.tokens, tid = threadIdx.x, D = p.D;
    long long *slot = reinterpret_cast<long long *>(cs + tokens * n);
    int2 *owner = reinterpret_cast<int2 *>(slot + tokens);
    const long long t0 = (long long)blockIdx.x * tokens;
    const int nt = (int)min((long long)tokens, ap.n_tok - t0);
    const int lanes = ap.lanes;
    const int g = tid % ap.groups, y = tid / ap.groups, lane = y % lanes, tok = y / lanes;
    int a, b;
    rope_offsets<V, HALF>(g, n, D, a, b);
    const bool turn = g * V < n, live = tok < nt;
    const int nq = ap.q_out ? p.Hq : 0, nkv = 2 * p.Hkv, d = b - a;
    const long long t = t0 + tok;
    W u[kAppendUnroll], w[kAppendUnroll];
    // heads h0, h0 + lanes, ... below `heads` from `from(h)`
    auto load = [&](int h0, int heads, auto from) {
#pragma unroll
        for (int i = 0; i < kAppendUnroll; ++i)
            if (h0 + i * lanes < heads) {
                const T *src = from(h0 + i * lanes) + a;
                u[i] = *reinterpret_cast<const W *>(src);
                if (b >= 0) w[i] = *reinterpret_cast<const W *>(src + d);
            }
    };
    auto q_at = [&](int h) { return p.q + t * ap.qs + h * D; };
    auto kv_at = [&](int h) { return h < p.Hkv ? p.k + t * ap.ks + h * D : p.v + t * ap.vs + (h - p.Hkv) * D; };
    if (live) load(lane, nq, q_at);           // on its way while the places are looked up

    // the sequence of each token, the one whose range covers it, and its key
    for (int i = tid; i < tokens; i += blockDim.x) owner[i] = make_int2(-1, 0);
    __syncthreads();
    for (int s = tid; s < p.B_max; s += blockDim.x) {
        int q0, Lq, k0, Lk;
        if (!load_lengths(p, s, blockIdx.x == 0, q0, Lq, k0, Lk)) continue;
        const int lo = (int)max(0ll, q0 - t0), hi = (int)min((long long)nt, q0 + Lq - t0);
        for (int i = lo; i < hi; ++i) owner[i] = make_int2(s, (int)(Lk - Lq + (t0 + i - q0)));
    }
    fill_factors(tab, cs, ap.pos, ap.pos_stride, t0, nt, 1.f);
    __syncthreads();
    // each token's page is looked up while the queries go through
    int entry = 0;
    const int2 mine = tid < nt ? owner[tid] : make_int2(-1, 0);
    if (mine.x >= 0 && mine.y >= 0) entry = page_entry(p, mine.x, mine.y);
    float2 f[V];
    if (live && turn)
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = cs[tok * n + g * V + i];
    const bool owned = live && owner[tok].x >= 0;
    for (int h0 = lane; owned && h0 < nq; h0 += kAppendUnroll * lanes) {
        if (h0 != lane) load(h0, nq, q_at);
#pragma unroll
        for (int i = 0; i < kAppendUnroll; ++i)
            if (h0 + i * lanes < nq) {
                T *dst = ap.q_out + (t * p.Hq + h0 + i * lanes) * D + a;
                if (turn) rope_rotate<T, V, HALF>(u[i], w[i], f);
                *reinterpret_cast<W *>(dst) = u[i];
                if (b >= 0) *reinterpret_cast<W *>(dst + d) = w[i];
            }
    }
    if (owned) load(lane, nkv, kv_at);
    // where the key goes, or -1: no sequence, a bad table entry, or a query
    // before the first key
    if (tid < nt) {
        long long at = -1;
        if (mine.x >= 0 && mine.y >= 0) {
            const int page = page_checked(p, entry);
            if (page < p.num_pages)
                at = page * p.page_stride + (long long)(mine.y & ((1 << p.page_shift) - 1)) * p.k_stride;
        }
        slot[tid] = at;
    }
    __syncthreads();
    if (!owned) return;
    const long long at = slot[tok];
    if (at < 0) return;
    for (int h0 = lane; h0 < nkv; h0 += kAppendUnroll * lanes) {
        if (h0 != lane) load(h0, nkv, kv_at);
#pragma unroll
        for (int i = 0; i < kAppendUnroll; ++i) {
            const int h = h0 + i * lanes;
            if (h < nkv) {
                T *dst = (h < p.Hkv ? ap.k_cache + h * D : ap.v_cache + (h - p.Hkv) * D) + at + a;
                if (turn && h < p.Hkv) rope_rotate<T, V, HALF>(u[i], w[i], f);
                *reinterpret_cast<W *>(dst) = u[i];
                if (b >= 0) *reinterpret_cast<W *>(dst + d) = w[i];
            }
        }
    }
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
    const Shape sh = shape_of(n_tok, H, rope_groups(r.tab.n, r.D, V), r.tab.n, kMaxHeads, current_sms());
    if (sh.blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    const size_t smem = (size_t)sh.tokens * r.tab.n * sizeof(float2);
    auto *fn = r.layout == ATTN_ROPE_HALF ? rope_kernel<T, V, true> : rope_kernel<T, V, false>;
    return launch_dependent(fn, dim3((unsigned)sh.blocks), dim3(sh.threads), smem, s, 0, r.tab,
                            static_cast<const T *>(x), xs, n_tok, H, r.D, pos, ps, grad ? -1.f : 1.f,
                            static_cast<T *>(out), os, sh.groups, sh.lanes, sh.tokens);
}

template <int V>
cudaError_t launch_append(const RopeTable &tab, bool half, const Params &p, Append ap, int sms, cudaStream_t s) {
    const Shape sh = shape_of(ap.n_tok, (ap.q_out ? p.Hq : 0) + 2 * p.Hkv, rope_groups(tab.n, p.D, V), tab.n,
                              kAppendHeads, sms);
    if (sh.blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    ap.groups = sh.groups;
    ap.lanes = sh.lanes;
    ap.tokens = sh.tokens;
    const size_t smem = (size_t)sh.tokens * (tab.n * sizeof(float2) + sizeof(long long) + sizeof(int2));
    auto *fn = half ? append_kernel<V, true> : append_kernel<V, false>;
    return launch_dependent(fn, dim3((unsigned)sh.blocks), dim3(sh.threads), smem, s, 0, tab, p, ap);
}

}  // namespace

}  // namespace vgqa

using namespace vgqa;

namespace {

std::mutex g_mu;
std::unordered_set<attn_rope_s *> g_ropes;

// The fraction of a turn per unit position in units of 2^-64, rounded.  Whole
// turns are dropped by the C library's long double sine and cosine, which
// reduce an argument of any size exactly: the angle comes back from them in
// [-pi, pi], good to its 64 bits, where the quotient freq / 2 pi would keep 64
// bits of the whole turns too and lose as many of the fraction.
unsigned long long turn_of(double freq) {
    const long double turns = atan2l(sinl(freq), cosl(freq)) / 6.283185307179586476925286766559005768L;
    const long double f = roundl(ldexpl(turns, 64));                 // in [-2^63, 2^63]
    return f >= 9223372036854775808.0L ? 1ull << 63 : (unsigned long long)(long long)f;
}

bool known(attn_rope_s *r) {
    std::lock_guard<std::mutex> lk(g_mu);
    return g_ropes.count(r) != 0;
}

}  // namespace

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
        r->tab.turn[i] = turn_of(freq[i]);
        r->tab.axis[i] = (uint8_t)axis[i];
    }
    try {
        std::lock_guard<std::mutex> lk(g_mu);
        g_ropes.insert(r);
    } catch (...) {
        delete r;
        return ATTN_E_NOMEM;
    }
    *out = r;
    return ATTN_OK;
}

ATTN_EXPORT void attn_rope_destroy(attn_rope_t rope) {
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (!g_ropes.erase(rope)) return;
    }
    delete rope;
}

ATTN_EXPORT int attn_rope_apply(attn_rope_t rope, int dtype, const void *x, int64_t x_token_stride, int64_t T, int H,
                                const int32_t *pos, int64_t pos_stride, int grad, void *out, int64_t out_token_stride,
                                void *stream) {
    if (!rope || !x || !pos || !out) return ATTN_E_NULL;
    if (!known(rope)) return ATTN_E_BAD_PLAN;
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
    // the positions are read while rows are written
    const char *pb = reinterpret_cast<const char *>(pos);
    if (pb < ob + ((T - 1) * out_token_stride + row) * size &&
        ob < pb + ((rope->n_axes - 1) * (rope->n_axes > 1 ? pos_stride : 0) + T) * 4)
        return ATTN_E_INVALID_ARG;
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
    if (rope && !known(rope)) return ATTN_E_BAD_PLAN;
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
    // q_out is q itself (packed) or apart from all that is read
    if (q && T_q > 0) {
        auto overlaps = [&](const void *in, long long stride, long long row) {
            const char *a = static_cast<const char *>(in), *b = static_cast<const char *>(q_out);
            return a < b + T_q * qrow * 2 && b < a + ((T_q - 1) * stride + row) * 2;
        };
        if (q_out == q ? q_token_stride != qrow : overlaps(q, q_token_stride, qrow)) return ATTN_E_INVALID_ARG;
        if (overlaps(k, k_token_stride, krow) || overlaps(v, v_token_stride, krow)) return ATTN_E_INVALID_ARG;
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
    p.rows_q = (int)T_q;
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
    const cudaError_t e = w == 8   ? launch_append<8>(tab, half, p, ap, d.num_sms, s)
                          : w == 4 ? launch_append<4>(tab, half, p, ap, d.num_sms, s)
                                   : launch_append<1>(tab, half, p, ap, d.num_sms, s);
    return e == cudaSuccess ? ATTN_OK : ATTN_E_CUDA;
}
