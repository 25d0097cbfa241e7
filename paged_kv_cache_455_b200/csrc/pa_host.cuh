// pa_host.cuh -- host-side services of pa.cu that the other translation units
// with C entry points use: the launch count, the tensor maps of the pools and
// the test hooks' settings.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "pa.h"

namespace pa {

// Counts one kernel launch (pa_launch_count).
void count_launch();

// Settings of the hooks in include/pa_testing.h: the wait limit in
// nanoseconds (0: the default) and the withheld CTA (-1: none).
unsigned long long test_wait_ns();
int test_withhold_cta();

// A tag for the arrival counters of one call that splits its work: never 0,
// distinct for consecutive calls of this process.
uint32_t next_epoch();

// Tensor map over a pool [nb, bs, Hkv, d] for boxes of `tr` token rows of one
// head that land in shared memory as [8-row group][128-byte column][row][128
// bytes], 128-byte swizzled (tr a multiple of 8).  False if it cannot be
// encoded.
bool pool_map_grouped(CUtensorMap *out, const void *base, int64_t nb, int bs, int hkv, int d,
                      pa_dtype dt, int tr);

// Tensor map over bf16 query rows [total_q, Hq, d] for boxes of 64 elements,
// `group` heads, `tokens` tokens, 128-byte swizzled.
bool query_map(CUtensorMap *out, const void *query, int total_q, int hq, int d, int group,
               int tokens);

// The argument checks of pa_decode_attention; *group and *bs_log2 receive
// Hq / Hkv and log2(block_size).
pa_status check_attention(const void *out, const void *query, const void *k_pool,
                          const void *v_pool, const int32_t *block_tables, int max_blocks,
                          const int32_t *context_lens, int num_seqs, int max_context_len,
                          int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                          int64_t num_blocks, pa_dtype dtype, int *group, int *bs_log2);

// True if the GPU can read and write `ptr` at that same address.
bool device_addressable(const void *ptr);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Launches `kernel` as a programmatic dependent of the kernel ahead on the
// stream; the kernel must execute griddepcontrol.wait in every CTA.
// With `cluster` > 1 that many consecutive CTAs form a cluster.
template <typename... KArgs, typename... Args>
inline pa_status launch_clusters(void (*kernel)(KArgs...), unsigned cluster, unsigned grid,
                                 unsigned threads, size_t smem, void *stream, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    count_launch();
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <typename... KArgs, typename... Args>
inline pa_status launch_dependent(void (*kernel)(KArgs...), unsigned grid, unsigned threads,
                                  size_t smem, void *stream, Args... args)
{
    return launch_clusters(kernel, 1, grid, threads, smem, stream, args...);
}

}  // namespace pa
