// pa_q8_decode.cu -- pa_decode_attention_q8: checks, work split, launches.
#include <algorithm>
#include <cstring>

#include "pa.h"
#include "pa_host.cuh"
#include "pa_launch.cuh"
#include "pa_q8_decode.cuh"

namespace {

struct Launch {
    pa::Q8DecodeParams p;
    CUtensorMap tk, tv;
    int grid;
    int chunks;              // 32-sequence chunks the prefix has room for
    void *stream;
};

// With `launch` false, L.grid receives the most CTAs the kernel runs at once.
template <int D, int G>
pa_status run(Launch &L, bool launch)
{
    auto fn = &pa::q8_decode_kernel<D, G>;
    const int smem = pa::Q8Smem<D, G>::bytes + 8 * (L.chunks + 1);
    int cap = 0;
    const pa_status st = pa::grid_capacity(reinterpret_cast<const void *>(fn), pa::Q8Smem<D, G>::kThreads,
                                           smem, &cap);
    if (st != PA_OK)
        return st;
    if (!launch) {
        L.grid = std::min(cap, pa::kQ8MaxCtas);
        return PA_OK;
    }
    return pa::launch_dependent(fn, (unsigned)L.grid, pa::Q8Smem<D, G>::kThreads, smem, L.stream, L.tk, L.tv,
                                L.p);
}

template <int D>
pa_status run_group(Launch &L, int group, bool launch)
{
    switch (group) {
    case 1: return run<D, 1>(L, launch);
    case 2: return run<D, 2>(L, launch);
    case 4: return run<D, 4>(L, launch);
    case 8: return run<D, 8>(L, launch);
    default: return PA_ERR_UNSUPPORTED;
    }
}

pa_status run_any(Launch &L, int head_dim, int group, bool launch)
{
    return head_dim == 128 ? run_group<128>(L, group, launch) : run_group<256>(L, group, launch);
}

}  // namespace

extern "C" pa_status pa_decode_attention_q8(void *out, const void *query, const void *k_pool,
                                            const void *v_pool, const float *k_scales,
                                            const float *v_scales, const int32_t *block_tables,
                                            int max_blocks_per_seq, const int32_t *context_lens,
                                            int num_seqs, int max_context_len, int num_q_heads,
                                            int num_kv_heads, int head_dim, int block_size,
                                            int64_t num_blocks, float scale, void *workspace,
                                            size_t workspace_bytes, int32_t *dev_status,
                                            void *stream)
{
    return pa_decode_attention_q8_strided(out, query, k_pool, v_pool, k_scales, v_scales,
                                          block_tables, max_blocks_per_seq, context_lens, 1,
                                          num_seqs, max_context_len, num_q_heads, num_kv_heads,
                                          head_dim, block_size, num_blocks, scale, workspace,
                                          workspace_bytes, dev_status, stream);
}

extern "C" pa_status pa_decode_attention_q8_strided(
    void *out, const void *query, const void *k_pool, const void *v_pool, const float *k_scales,
    const float *v_scales, const int32_t *block_tables, int max_blocks_per_seq,
    const int32_t *context_lens, int64_t context_lens_stride, int num_seqs, int max_context_len,
    int num_q_heads, int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
    float scale, void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream)
{
    if ((head_dim != 128 && head_dim != 256) || (block_size != 16 && block_size != 32) ||
        num_seqs > pa::kQ8MaxSeqs)
        return PA_ERR_UNSUPPORTED;
    int group = 0, bs_log2 = 0;
    pa_status st = pa::check_attention(out, query, k_pool, v_pool, block_tables,
                                       max_blocks_per_seq, context_lens, num_seqs,
                                       max_context_len, num_q_heads, num_kv_heads, head_dim,
                                       block_size, num_blocks, PA_DTYPE_BF16, &group, &bs_log2);
    if (st != PA_OK)
        return st;
    if (num_seqs == 0)
        return PA_OK;
    if (!k_scales || !v_scales || context_lens_stride < 0)
        return PA_ERR_INVALID_ARG;
    Launch L;
    std::memset(&L.p, 0, sizeof(L.p));
    pa::Q8DecodeParams &p = L.p;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.q = static_cast<const __nv_bfloat16 *>(query);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.len_stride = context_lens_stride;
    p.dev_status = dev_status;
    p.num_blocks = num_blocks;
    p.num_seqs = num_seqs;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.max_blocks = max_blocks_per_seq;
    p.block_size = block_size;
    p.bs_log2 = bs_log2;
    p.ctx_cap = max_blocks_per_seq * block_size;
    p.hpc_log2 = num_kv_heads % 4 == 0 ? 2 : (num_kv_heads % 2 == 0 ? 1 : 0);
    p.hpc = 1 << p.hpc_log2;
    p.tt_log2 = 7 - p.hpc_log2;
    p.box_log2 = block_size == 32 ? 5 : 4;
    p.head_groups = num_kv_heads / p.hpc;
    p.scale_log2 = scale * pa::kLog2e;
    // a segment's end takes ~2 us, a tile's bytes 1.5 us (d 256) or 0.75 us
    p.end_tiles = head_dim == 256 ? 1 : 3;
    const unsigned long long wait_ns = pa::test_wait_ns();
    p.wait_ns = wait_ns ? wait_ns : pa::kWaitLimitNs;
    p.withhold_cta = pa::test_withhold_cta();
    L.stream = stream;
    // (rounded up, so that few sizes occur)
    for (L.chunks = 1; 32 * L.chunks < num_seqs;)
        L.chunks *= 2;
    if (!pa::pool_map_grouped(&L.tk, k_pool, num_blocks, block_size, num_kv_heads, head_dim,
                              PA_DTYPE_FP8_E4M3, block_size) ||
        !pa::pool_map_grouped(&L.tv, v_pool, num_blocks, block_size, num_kv_heads, head_dim,
                              PA_DTYPE_FP8_E4M3, block_size))
        return PA_ERR_CUDA;
    st = run_any(L, head_dim, group, false);
    if (st != PA_OK)
        return st;
    const int64_t seg_tiles = (std::max(max_context_len, 1) + (1 << p.tt_log2) - 1) >> p.tt_log2;
    L.grid = (int)std::min<int64_t>(L.grid, num_seqs * (int64_t)p.head_groups * seg_tiles);
    // Segments of one tile need no cutting, and a workspace that is missing or
    // too small allows none: then every CTA takes whole segments.
    const int rows = p.hpc * group;
    p.slot_floats = (rows * head_dim + 2 * rows + 1 + 3) / 4 * 4;
    const size_t counters_off = ((size_t)L.grid * 2 * p.slot_floats * 4 + 127) / 128 * 128;
    const bool split = seg_tiles > 1 && L.grid > 1 && workspace != nullptr &&
                       pa::aligned16(workspace) &&
                       workspace_bytes >= counters_off + (size_t)L.grid * 128;
    p.mode = split ? 0 : 1;
    if (split) {
        p.pieces = static_cast<float *>(workspace);
        p.counters = reinterpret_cast<unsigned long long *>(static_cast<uint8_t *>(workspace) +
                                                            counters_off);
        p.epoch = pa::next_epoch();
        // Pieces of a segment, when all are as long as the longest: from six on
        // a kernel of its own joins them (8K contexts of 4 KV heads of 256: 4 of
        // them, 37 pieces, 27.0 us with it and 28.8 us without; 8, 33.4 and 34.8;
        // 24, 6 pieces, 70.0 and 70.3; 32, 4 to 5 pieces, 89.1 and 88.4; 64
        // contexts of up to 4K, about 3, 53.2 and 49.2).
        const int64_t segments = num_seqs * (int64_t)p.head_groups;
        p.merge_later = num_seqs <= 32 && L.grid >= 6 * segments;
    }
    st = run_any(L, head_dim, group, true);
    if (st != PA_OK || !p.merge_later)
        return st;
    return pa::launch_dependent(pa::q8_merge_kernel,
                                (unsigned)(num_seqs * p.head_groups * p.hpc * group * head_dim / 128),
                                pa::kQ8MergeThreads, 0, stream, p, L.grid, group, head_dim);
}
