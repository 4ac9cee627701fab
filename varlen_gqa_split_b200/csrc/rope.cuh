// rope.cuh -- rotary positions with several axes: the table, the angle and
// the rotation of one group of pairs (device code and host struct, internal).
//
// Pair i of a head turns by theta = pos[axis_i] * f_i:
//     (u, w) -> scale (u cos theta - w sin theta, u sin theta + w cos theta).
// The angle is kept in turns as a 64-bit fixed-point fraction: with
// F_i = f_i / 2 pi * 2^64 mod 2^64, the product pos * F_i mod 2^64 is the exact
// fraction of a turn for this F_i, since whole turns wrap away by themselves.
// F_i is off by at most 2 units whatever the size of f_i (half a unit of
// rounding; three long double results of 64 bits before it), so the product by
// at most 2^-63 |pos| turns: 2^-32 turns (1.5e-9 rad) at the farthest
// positions.  An angle in 32-bit floating point would be off by 0.06 rad at
// position 2^20.  Its quarter turns are split off; of the rest,
// in [-1/8, 1/8] turn, rounded to 33 bits, 24 bits go to sincospif and what they leave,
// b <= 2^-25 rad, comes in by sin(a + b) = sin a + b cos a.  Cosine and sine are
// then within 1.6 * 2^-24: one unit of sincospif, half a one of the last sum,
// and the 34th bit.  (The fraction as one float would cost up to 9.4e-8 rad.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace vgqa {

constexpr int kRopeMaxPairs = 128;        // head sizes up to 256
constexpr int kRopeMaxAxes = 8;

// passed to the kernels by value (1.2 KB of parameters): a rotation needs no
// device memory of its own and serves any device
struct RopeTable {
    unsigned long long turn[kRopeMaxPairs];   // F_i
    uint8_t axis[kRopeMaxPairs];
    int n;                                    // pairs; elements [2 n, D) are copied
    float scale;
};

// (scale cos, scale sin) of pair i at `pos` positions; sign -1 turns backwards
__device__ __forceinline__ float2 rope_cos_sin(const RopeTable &tab, int i, int pos, float sign) {
    const unsigned long long t = (unsigned long long)(long long)pos * tab.turn[i];
    const uint32_t quarter = (uint32_t)((t + (1ull << 61)) >> 62);
    // 2^-33 turns, rounded, in [-2^30, 2^30]
    const int rest = (int)((long long)(t - ((unsigned long long)quarter << 62) + (1ull << 30)) >> 31);
    const float a = (float)rest;
    const float b = (float)(rest - (int)a) * 7.314590e-10f;   // rad: 2 pi 2^-33
    float s, c;
    sincospif(a * 2.3283064365386963e-10f, &s, &c);           // half turns: 2^-32
    const float sb = fmaf(b, c, s), cb = fmaf(-b, s, c);
    const float x = quarter & 1 ? sb : cb, y = quarter & 1 ? cb : sb;
    // cosine: c, -s, -c, s; sine: s, c, -s, -c
    const float cosine = (quarter + 1) & 2 ? -x : x, sine = quarter & 2 ? -y : y;
    return make_float2(cosine * tab.scale, sine * tab.scale * sign);
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// V elements moved by one access
template <typename T, int V> struct alignas(sizeof(T) * V) Vec { T e[V]; };

// The elements of group g of a head: 2 V of them in two accesses of V.  The
// first n / V groups hold V pairs each ("half": elements g V .. and n + g V
// ..; "interleaved": 2 g V .. and the next V), the others the D - 2 n copied
// elements, of which the last group may hold V only.
template <int V, bool HALF>
__device__ __forceinline__ void rope_offsets(int g, int n, int D, int &a, int &b) {
    if (g * V < n) {
        a = HALF ? g * V : 2 * g * V;
        b = HALF ? n + g * V : a + V;
    } else {
        a = 2 * n + (g - n / V) * 2 * V;
        b = a + V < D ? a + V : -1;
    }
}
__host__ __device__ __forceinline__ int rope_groups(int n, int D, int V) {
    return n / V + (D - 2 * n + 2 * V - 1) / (2 * V);
}

// two 16-bit elements of a word
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t w);
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float x, float y);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// one pair turned by c = (cos, sin)
__device__ __forceinline__ float2 turn_pair(float u, float w, float2 c) {
    return make_float2(u * c.x - w * c.y, u * c.y + w * c.x);
}

// rotate the V pairs held in (x, y) by the factors cs[0 .. V)
template <typename T, int V, bool HALF>
__device__ __forceinline__ void rope_rotate(Vec<T, V> &x, Vec<T, V> &y, const float2 *cs) {
    if constexpr (sizeof(T) == 2 && V > 1) {
        uint32_t *xw = reinterpret_cast<uint32_t *>(&x), *yw = reinterpret_cast<uint32_t *>(&y);
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
            const float2 a = unpack2<T>(xw[k]), b = unpack2<T>(yw[k]);
            if constexpr (HALF) {             // words of two firsts and of two seconds
                const float2 p = turn_pair(a.x, b.x, cs[2 * k]), q = turn_pair(a.y, b.y, cs[2 * k + 1]);
                xw[k] = pack2<T>(p.x, q.x);
                yw[k] = pack2<T>(p.y, q.y);
            } else {                          // words of one pair
                const float2 p = turn_pair(a.x, a.y, cs[k]), q = turn_pair(b.x, b.y, cs[V / 2 + k]);
                xw[k] = pack2<T>(p.x, p.y);
                yw[k] = pack2<T>(q.x, q.y);
            }
        }
    } else {
        T *p[2] = {x.e, y.e};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            // the pair's two elements: i of x and i of y, or 2 i and 2 i + 1 of x then y
            T &u = HALF ? p[0][i] : p[(2 * i) / V][(2 * i) % V];
            T &w = HALF ? p[1][i] : p[(2 * i + 1) / V][(2 * i + 1) % V];
            const float2 r = turn_pair(to_f32(u), to_f32(w), cs[i]);
            u = from_f32<T>(r.x);
            w = from_f32<T>(r.y);
        }
    }
}

}  // namespace vgqa
