// key_weights_simt.cu -- accumulated attention weights on the CUDA cores.
//
// With s the scaled score and lse the row's normaliser (attn_run's), key j of
// KV head hk gathers
//     w_j = sum over query tokens qi and heads h of hk, j visible to qi, of
//           e^(s_{qi,h,j} - lse_{qi,h}),
// the column sums of the attention matrix.  One thread owns one key: its row
// of K stays in registers, the query rows come through shared memory 16 at a
// time (as fp32, broadcast reads), and the sum never leaves the thread, so no
// result depends on an order of arrival.
#include "common.cuh"
#include "kernels.h"
#include "key_weights.h"

namespace vgqa {

namespace {

constexpr int kKeys = 128;                // keys (threads) per block
constexpr int kRowsStep = 16;             // query rows staged at once

template <int D>
__global__ void __launch_bounds__(kKeys) key_weights_simt_kernel(const Params p, const KeyWeights kw) {
    __shared__ float4 qs[kRowsStep][D / 4];
    __shared__ float nl[kRowsStep];       // -lse in base 2
    const int b = blockIdx.z, hk = blockIdx.y, tid = threadIdx.x;
    int q0, Lq, k0, Lk;
    if (!load_lengths(p, b, blockIdx.x == 0 && hk == 0 && tid == 0, q0, Lq, k0, Lk)) return;
    const int j0 = blockIdx.x * kKeys, j = j0 + tid;
    if (j0 >= Lk) return;
    const int old = Lk - Lq;              // keys below it were there before this call's tokens
    const bool mine = j < Lk;
    uint4 kv[D / 8];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) kv[i] = make_uint4(0, 0, 0, 0);
    if (mine) {
        long long off = -1;
        if (p.block_table) {
            const int page = page_of(p, b, j);
            if (page < p.num_pages)
                off = page * p.page_stride + (long long)(j & ((1 << p.page_shift) - 1)) * p.k_stride;
        } else {
            off = ((long long)k0 + j) * p.k_stride;
        }
        if (off >= 0) {
            const uint4 *src = reinterpret_cast<const uint4 *>(p.k + off + hk * D);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) kv[i] = __ldg(src + i);
        }
    }
    const int G = p.G;
    const int qi_first = max(0, j0 - old);              // the first query that sees any key of the block
    const long long r_begin = (long long)qi_first * G, r_end = (long long)Lq * G;
    // first row that sees this key
    const long long mine_from = (long long)max(0, j - old) * G;
    float total = 0.f, carry = 0.f;
    for (long long r = r_begin; r < r_end; r += kRowsStep) {
        const int nr = (int)min((long long)kRowsStep, r_end - r);
        __syncthreads();
        for (int i = tid; i < nr * (D / 8); i += kKeys) {
            const int row = i / (D / 8), c = i % (D / 8);
            const long long tok = q0 + (r + row) / G;
            const int h = hk * G + (int)((r + row) % G);
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p.q + (tok * p.Hq + h) * D) + c);
            qs[row][2 * c] = make_float4(bf16lo(x.x), bf16hi(x.x), bf16lo(x.y), bf16hi(x.y));
            qs[row][2 * c + 1] = make_float4(bf16lo(x.z), bf16hi(x.z), bf16lo(x.w), bf16hi(x.w));
        }
        if (tid < nr) {
            const long long tok = q0 + (r + tid) / G;
            const float l = __ldg(p.lse + tok * p.Hq + hk * G + (int)((r + tid) % G));
            nl[tid] = -l * kLog2e;
        }
        __syncthreads();
        float part = 0.f;
        for (int row = 0; row < nr; ++row) {
            float acc = 0.f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const float4 x = qs[row][2 * i], y = qs[row][2 * i + 1];
                acc = fmaf(bf16lo(kv[i].x), x.x, acc);
                acc = fmaf(bf16hi(kv[i].x), x.y, acc);
                acc = fmaf(bf16lo(kv[i].y), x.z, acc);
                acc = fmaf(bf16hi(kv[i].y), x.w, acc);
                acc = fmaf(bf16lo(kv[i].z), y.x, acc);
                acc = fmaf(bf16hi(kv[i].z), y.y, acc);
                acc = fmaf(bf16lo(kv[i].w), y.z, acc);
                acc = fmaf(bf16hi(kv[i].w), y.w, acc);
            }
            // (a row that saw nothing, lse = -inf, weighs nothing)
            if (mine && r + row >= mine_from && nl[row] != INFINITY) part += ex2(fmaf(acc, p.scale_log2, nl[row]));
        }
        add_compensated(total, carry, part);
    }
    if (!mine) return;
    const long long at = ((long long)b * p.Hkv + hk) * kw.ld + j;
    const float before = kw.w_in && kw.decay != 0.f && j < old ? kw.decay * kw.w_in[at] : 0.f;
    kw.w_out[at] = before + total;
    if (kw.born && j >= old) kw.born[at] = __ldg(kw.seen + b) - (Lk - j);
}

}  // namespace

cudaError_t launch_key_weights_simt(const Params &p, const KeyWeights &kw, cudaStream_t stream) {
    const dim3 grid((p.s_max + kKeys - 1) / kKeys, p.Hkv, p.B_max);
    if (p.D == 64)
        key_weights_simt_kernel<64><<<grid, kKeys, 0, stream>>>(p, kw);
    else
        key_weights_simt_kernel<128><<<grid, kKeys, 0, stream>>>(p, kw);
    return cudaGetLastError();
}

}  // namespace vgqa
