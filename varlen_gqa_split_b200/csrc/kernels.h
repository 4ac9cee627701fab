// kernels.h -- host-side launchers of libvgqa's kernels (internal).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>

namespace vgqa {

struct Params;

// A launch as a programmatic dependent of the work before it in the stream,
// in clusters of `cluster` blocks where it is not zero.  EVERY kernel launched
// with it calls dependent_start() before its first read of global memory, and
// reads what the kernel before it may have written by plain loads (a read-only
// load may be moved ahead of the wait).  The wait covers the grid just before
// it in the stream alone, so every grid of the library that lets its successor
// start early waits for its own predecessor before it completes.  Takes 0.5 to 1 us off a small call
// that follows another (64 tokens rotated 3.45 -> 2.9 us).
template <typename... A>
cudaError_t launch_dependent(void (*fn)(A...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, int cluster,
                             const A &...args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

// CUDA-core split kernel (any row count), 16 query rows per block
size_t simt_smem_bytes(int D);
size_t simt_merge_capacity(int D);
cudaError_t simt_prepare(int D);
cudaError_t launch_split_simt(const Params &p, dim3 grid, cudaStream_t stream);
constexpr int kSimtRowsPerBlock = 16;
constexpr int kSimtBlockN = 64;

// Persistent TMA-fed tensor-core split kernel, NT = ceil(G * max_q / 8) in
// {1, 2}, `ctas` blocks sharing the flattened tile space
size_t mma_stage_bytes(int D);
size_t mma_merge_bytes(int D, int NT, int ctas);
size_t mma_smem_bytes(int D, int NT, int stages, int ctas);
int mma_block_n();
int mma_threads();
cudaError_t mma_prepare(int D, int NT, int stages, int ctas);
cudaError_t launch_split_mma(const Params &p, const CUtensorMap &tm_k, const CUtensorMap &tm_v, int NT,
                             int stages, int ctas, cudaStream_t stream);

// Persistent TMA-fed tcgen05 split kernel (accumulators in tensor memory),
// up to tc_rows() query rows per KV head
size_t tc_stage_bytes(int D);
size_t tc_smem_need(int D, int stages);    // bytes the layout uses
size_t tc_smem_bytes(int D, int stages);   // bytes requested at launch (>= half an SM)
int tc_rows();
int tc_parts_per_block();
int tc_unit_cost();                        // fixed cost of a unit, in tiles, for the shares
cudaError_t tc_prepare(int D, int stages, int ctas);
cudaError_t launch_split_tc(const Params &p, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                            const CUtensorMap &tm_v, int stages, int ctas, cudaStream_t stream);

// log-sum-exp merge of the persistent kernels' partial slots (2 * ctas
// blocks, launched as a programmatic dependent of the split kernel)
size_t combine_slots_smem(int ctas);
int combine_slots_split(int rows, int D);   // blocks per partial slot (S)
cudaError_t combine_slots_prepare(int D, int ctas);
cudaError_t launch_combine_slots(const Params &p, int ctas, cudaStream_t stream);

// log-sum-exp merge of the CUDA-core kernel's dense [.., nsplit] partials
int combine_blocks(const Params &p);
cudaError_t launch_combine(const Params &p, cudaStream_t stream);

// accumulated attention weights on the CUDA cores (any row count)
struct KeyWeights;
cudaError_t launch_key_weights_simt(const Params &p, const KeyWeights &kw, cudaStream_t stream);

// ... and on the tensor cores: rows (G heads x query tokens) in tiles of up
// to 128, `columns` wide
int key_weights_columns(int rows);
int key_weights_part_floats();             // per block, for cut items: floats of scratch
int key_weights_tickets();                 // and counters
cudaError_t key_weights_tc_prepare(int D, int columns);
cudaError_t launch_key_weights_tc(const Params &p, const KeyWeights &kw, const CUtensorMap &tm_q,
                                  const CUtensorMap &tm_k, int columns, int ctas, cudaStream_t stream);

// eviction: opt in to its shared memory (once per plan, outside capture)
cudaError_t evict_prepare();

}  // namespace vgqa
