// plan.h -- the plan object behind attn_plan_t and the host helpers that the
// entry points share (internal).
#pragma once

#include <cudaTypedefs.h>
#include <stdint.h>

#include "../../include/varlen_gqa.h"
#include "params.h"

#define ATTN_EXPORT extern "C" __attribute__((visibility("default")))

struct attn_plan_s {
    attn_plan_desc d;
    int device;
    int NT;                    // tensor-core path: row fragments of 8
    float scale_log2;
    void *scratch;             // one allocation: error word, partials
    uint32_t *err;
    uint32_t *ticket;          // fused-merge arrival counters
    size_t ticket_bytes;
    int merge_bytes;           // tensor-core path: shared bytes of the merge area
    int qtile;                 // tensor-core path: query tokens per row tile
    int max_rt;                // tensor-core path: row tiles per sequence at most
    int direct;                // warp-MMA path: one block per unit, no merge
    float *o_part;
    float2 *ml_part;
    int kw_columns;            // attn_key_weights: columns of a row tile; 0: CUDA cores (G > 128)
    int kw_qtile;              // its query tokens per row tile
    int kw_ctas;               // its blocks
    float *kw_part;            // its scratch for items cut between blocks
    uint32_t *kw_ticket;
    unsigned long long wait_ns; // limit of one bounded wait in the kernels
};

namespace vgqa {

// where the keys live when the cache is paged (attn_run_paged)
struct Paging {
    const int32_t *block_table;
    int bt_stride, page_size, num_pages;
    long long page_stride;
};

// whether `p` is a plan that has been made and not destroyed
bool live(attn_plan_s *p);

inline bool aligned(const void *ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }

// the exponent of a power of two, or -1
int log2_exact(long long x);

// the paged-cache arguments' contract (attn_run_paged); an ATTN_* code
int check_paging(const attn_plan_s *plan, int64_t page_stride, int64_t token_stride, int page_size, int num_pages,
                 const int32_t *block_table, int bt_stride);

// tensor maps (api.cpp)
int encode_kv_map(CUtensorMap *map, const void *base, int Hkv, int D, int block_n, long long token_stride,
                  long long rows = 0x7fffffff);
int encode_paged_map(CUtensorMap *map, const void *base, int Hkv, int D, int page_size, int num_pages,
                     long long token_stride, long long page_stride);
int encode_q_map(CUtensorMap *map, const void *base, int Hq, int D, int G, int qtile, long long rows = 0x7fffffff);

}  // namespace vgqa
