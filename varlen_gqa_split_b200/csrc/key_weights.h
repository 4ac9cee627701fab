// key_weights.h -- what the accumulated-attention-weight kernels share
// (internal).
#pragma once

#include "params.h"

namespace vgqa {

// Besides the plan's Params (lse is an input here and out unused):
struct KeyWeights {
    const float *w_in;         // [B_max, Hkv, ld], or NULL: start from zero
    float *w_out;              // [B_max, Hkv, ld]
    const int32_t *seen;       // [B_max] or NULL
    int32_t *born;             // [B_max, Hkv, ld] or NULL
    long long ld;
    float decay;
    float *part;               // tensor-core path: two parts of 256 sums per block, for items cut
                               // between blocks (NULL where one row tile holds all rows: no cuts)
    uint32_t *ticket;          // and counts of finished parts, eight per block (one a warp)
};

// total += part, compensated by `carry`: many thousand rows may add up.  An
// infinite total is kept as it is (its compensation would be inf - inf).
__device__ __forceinline__ void add_compensated(float &total, float &carry, float part) {
    const float y = part - carry, t = total + y;
    carry = fabsf(t) < INFINITY ? (t - total) - y : 0.f;
    total = t;
}

}  // namespace vgqa
