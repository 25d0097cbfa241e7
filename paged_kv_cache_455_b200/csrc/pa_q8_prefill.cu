// pa_q8_prefill.cu -- pa_prefill_attention_q8: checks and launch.
#include <algorithm>

#include "pa.h"
#include "pa_host.cuh"
#include "pa_launch.cuh"
#include "pa_q8_prefill.cuh"

namespace {

template <int D, int G>
pa_status run(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
              const pa::Q8PrefillParams &p, unsigned grid, void *stream)
{
    auto fn = &pa::q8_prefill_kernel<D, G>;
    constexpr int smem = pa::Q8PrefillSmem<D>::bytes;
    int cap = 0;   // (sets the kernel's shared-memory limit, once per device)
    const pa_status st = pa::grid_capacity(reinterpret_cast<const void *>(fn), pa::kQpThreads,
                                           smem, &cap);
    if (st != PA_OK)
        return st;
    return pa::launch_clusters(fn, (unsigned)p.split, grid, pa::kQpThreads, smem, stream, tq, tk, tv,
                               p);
}

template <int D>
pa_status run_group(int group, const CUtensorMap &tq, const CUtensorMap &tk,
                    const CUtensorMap &tv, const pa::Q8PrefillParams &p, unsigned grid,
                    void *stream)
{
    switch (group) {
    case 1: return run<D, 1>(tq, tk, tv, p, grid, stream);
    case 2: return run<D, 2>(tq, tk, tv, p, grid, stream);
    case 4: return run<D, 4>(tq, tk, tv, p, grid, stream);
    case 8: return run<D, 8>(tq, tk, tv, p, grid, stream);
    default: return PA_ERR_UNSUPPORTED;
    }
}

}  // namespace

extern "C" pa_status pa_prefill_attention_q8(void *out, const void *query,
                                             const int32_t *cu_q_lens, int total_q, int max_q_len,
                                             const void *k_pool, const void *v_pool,
                                             const float *k_scales, const float *v_scales,
                                             const int32_t *block_tables, int max_blocks_per_seq,
                                             const int32_t *context_lens, int num_seqs,
                                             int max_context_len, int num_q_heads,
                                             int num_kv_heads, int head_dim, int block_size,
                                             int64_t num_blocks, float scale, int32_t *dev_status,
                                             void *stream)
{
    return pa_prefill_attention_q8_strided(
        out, query, cu_q_lens, total_q, max_q_len, k_pool, v_pool, k_scales, v_scales,
        block_tables, max_blocks_per_seq, context_lens, 1, num_seqs, max_context_len, num_q_heads,
        num_kv_heads, head_dim, block_size, num_blocks, scale, dev_status, stream);
}

extern "C" pa_status pa_prefill_attention_q8_strided(
    void *out, const void *query, const int32_t *cu_q_lens, int total_q, int max_q_len,
    const void *k_pool, const void *v_pool, const float *k_scales, const float *v_scales,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
    int64_t context_lens_stride, int num_seqs, int max_context_len, int num_q_heads,
    int num_kv_heads, int head_dim, int block_size, int64_t num_blocks, float scale,
    int32_t *dev_status, void *stream)
{
    if (total_q < 0 || max_q_len < 0)
        return PA_ERR_INVALID_ARG;
    if ((head_dim != 128 && head_dim != 256) || (block_size != 16 && block_size != 32))
        return PA_ERR_UNSUPPORTED;
    const bool nothing = num_seqs == 0 || total_q == 0 || max_q_len == 0;
    int group = 0, bs_log2 = 0;
    pa_status st = pa::check_attention(out, query, k_pool, v_pool, block_tables,
                                       max_blocks_per_seq, context_lens, nothing ? 0 : num_seqs,
                                       max_context_len, num_q_heads, num_kv_heads, head_dim,
                                       block_size, num_blocks, PA_DTYPE_BF16, &group, &bs_log2);
    if (st != PA_OK)
        return st;
    if (num_seqs < 0 || max_q_len > max_context_len)
        return PA_ERR_INVALID_ARG;
    if (nothing)
        return PA_OK;
    if (!cu_q_lens || !k_scales || !v_scales || context_lens_stride < 0)
        return PA_ERR_INVALID_ARG;
    pa::Q8PrefillParams p;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.cu_q_lens = cu_q_lens;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.len_stride = context_lens_stride;
    p.dev_status = dev_status;
    p.num_blocks = num_blocks;
    p.total_q = total_q;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.block_size = block_size;
    p.bs_log2 = bs_log2;
    p.ctx_cap = max_blocks_per_seq * block_size;
    const int tq_tokens = pa::kQpRows / group;
    p.qblocks = (max_q_len + tq_tokens - 1) / tq_tokens;
    p.scale_log2 = scale * pa::kLog2e;
    const int64_t blocks = (int64_t)num_seqs * num_kv_heads * p.qblocks;
    // Clusters of up to eight CTAs per row block, as long as that leaves each
    // at least four tiles: what one wave of one CTA per SM holds, and two CTAs
    // for up to 148 row blocks (their lengths differ, and the second wave fills
    // what the short ones leave).  A CTA costs ~8 us besides its tiles, so more
    // waves of smaller parts lose: 8 sequences of 5 tokens over 500-4000, 4
    // heads of 256, 28 us in clusters of 4 and 52 us in clusters of 8; 32 such
    // sequences 67 us in single CTAs, 58 us in pairs, 89 us in fours.
    p.split = 1;
    while (p.split < 8 && blocks * (p.split == 1 ? 1 : 2 * p.split) <= 148 &&
           max_context_len / pa::kQpTile >= 4 * 2 * p.split)
        p.split *= 2;
    const int64_t grid = blocks * p.split;
    if (grid > INT32_MAX)
        return PA_ERR_INVALID_ARG;
    alignas(64) CUtensorMap tq, tk, tv;
    if (!pa::query_map(&tq, query, total_q, num_q_heads, head_dim, group, tq_tokens) ||
        !pa::pool_map_grouped(&tk, k_pool, num_blocks, block_size, num_kv_heads, head_dim,
                              PA_DTYPE_FP8_E4M3, 16) ||
        !pa::pool_map_grouped(&tv, v_pool, num_blocks, block_size, num_kv_heads, head_dim,
                              PA_DTYPE_FP8_E4M3, 16))
        return PA_ERR_CUDA;
    return head_dim == 128 ? run_group<128>(group, tq, tk, tv, p, (unsigned)grid, stream)
                           : run_group<256>(group, tq, tk, tv, p, (unsigned)grid, stream);
}
