// pa_q8_prefill.cuh -- chunked-prefill attention over a block-scaled E4M3
// cache on the 5th-generation tensor cores (tcgen05.mma kind::f8f6f4).  Same
// contract as prefill_tc_kernel, with K and V the codes times their block's
// scales, and the same structure: one CTA per (sequence, KV head, 128 query
// rows), row r being (token r / G, query head r % G of the group).
//
// The codes are the B operands as the TMA brings them; nothing is converted.
// A query row is scaled by a power of two and split into two E4M3 parts, hi
// and lo, in tensor memory:  S = hi K^T + lo K^T.  The softmax multiplies the
// logits of each 16-token box by its block's K scale, and the weights by its
// block's V scale before they are split: with m a running reference of
// s + log2 vs,
//     x = vs 2^(s - m) = hi + lo,
// hi the E4M3 part (4 bits, down to 2^-6, subnormal to 2^-9), lo the rest as
// E5M2 (3 bits, down to 2^-14, subnormal to 2^-16):  O += hi V + lo V.  A row's
// largest weight lies between 2^5 (where a new m puts it) and 2^8.75 (past
// which m moves).  So a weight x is off by at most 2^-7 x + min(2^-13, 2^-3 x +
// 2^-17), that is by 2^-18 of the row's largest beside 2^-7 of itself, and only
// those below 2^-22 of the largest vanish; row sums take the fp32 weights.  The
// two products at twice bf16's rate cost as much tensor time as one bf16 product
// would.
//
//   warps 0-11  softmax: three sets of four warps take tiles in turn, one query
//               row per thread.  A set settles the rows' reference for its tile
//               and passes it on to the next set before it goes on to the
//               exponentials, so the loads, maxima and waits of two tiles pass
//               behind the exponentials of a third
//   warp 12     MMA issue of S_{j+2} once S_j has been read
//   warp 15     MMA issue of P_j V_j (with one warp for both, the tensor cores
//               idled between its waits)
//   warp 13     TMA of K
//   warp 14     TMA of V, block scales
// Tensor memory columns: S buffers of 64 at 0 and 64, two buffers of weights (hi
// and lo, 16 columns each, four values per column), O [192, 192 + d), Q hi
// (d / 4).  Q lo stays in shared memory, where the bf16 queries were: of all
// operands it costs least there.  Cycles of the products alone, per tile at
// d = 256: all in tensor memory 1025 (no room for it; d = 128 has some, unused),
// Q lo in shared memory 1126, the weights in shared memory 1347.
//
// What bounds it: the tensor cores' 1126 cycles a tile, and around them the
// softmax warps (528 cycles a tile of exponentials on each scheduler, as much of
// conversions beside them) and the rescales, for which the product of the
// tile waits for that of the tile before.  Measured: 16 sequences' chunks of 512
// tokens over 1-4K, 16 query and 4 KV heads of 256, 340 us (1.09 PFLOP/s counted
// once, 2.2 of 8-bit products); a bf16 kernel at cuBLAS's rate would take 226 us.
// 32 query and 8 KV heads of 128: 600 us, floor 243.  The code of a tile should
// stay small: with a second set of exponentials behind a branch that no tile took
// the first case took 384 us.
// A CTA's start and end (Q converted, the first tiles, the last products, the
// output) take ~8 us besides, hidden by nothing: one CTA fills an SM's tensor
// memory.
//
// Few query rows (drafted tokens, single chunks) over long contexts leave most
// SMs idle, and there is no workspace to split into: then a cluster of SPLIT
// CTAs shares a row block, each taking a part of the tiles, and joins the parts
// through distributed shared memory.
#pragma once

#include "pa_prefill.cuh"
#include "pa_ptx8.cuh"

namespace pa {

struct Q8PrefillParams {
    __nv_bfloat16 *out;
    const float *k_scales, *v_scales;
    const int32_t *cu_q_lens, *block_tables, *context_lens;
    int64_t len_stride;      // elements between context_lens
    int32_t *dev_status;
    int64_t num_blocks;
    int total_q, num_q_heads, num_kv_heads;
    int num_seqs, max_blocks, block_size, bs_log2;
    int ctx_cap;
    int qblocks;             // row blocks per (sequence, KV head)
    int split;               // CTAs (a cluster) per row block
    float scale_log2;
};

constexpr int kQpRows = 128;             // query rows per CTA
constexpr int kQpTile = 64;              // tokens per stage
constexpr int kQpBoxes = kQpTile / 16;
constexpr int kQpSets = 3;              // softmax sets of four warps, on tiles in turn
constexpr int kQpThreads = 128 * kQpSets + 128;
constexpr int kQpWarpS = 4 * kQpSets, kQpWarpK = kQpWarpS + 1, kQpWarpV = kQpWarpS + 2,
              kQpWarpPV = kQpWarpS + 3;
// log2 of a row's largest weight when the row gets a reference, and of the
// largest one for which it gets no new one (E4M3 ends at 448 = 2^8.8).  The
// lower, the rarer the moves, and the fewer bits small weights keep: with 0 and
// 8 a tail of 2^-17 beside a weight of 1 loses a tenth of itself.  5 drafted
// tokens of 32 sequences of 500-4000, 4 heads of 256: 55.9 us, 54.0 with 0 and
// 8, 56.1 with 5 and 8; 8 prompts of 1024, 132.8 us, 127.5 and 134.3.
constexpr float kQpLift = 5.f, kQpGrow = 8.75f;

template <int D>
struct Q8PrefillSmem {
    static constexpr int kGroup = 8 * D;                 // bytes between 8-token groups
    static constexpr int kBox = 16 * D;
    static constexpr int kStage = kQpTile * D;           // K or V of a tile
    // (V is read about three tiles after K)
    static constexpr int kK = D == 256 ? 4 : 7, kV = D == 256 ? 6 : 9;
    static constexpr int q_bytes = kQpRows * D * 2;      // Q as it comes (bf16)
    static constexpr int k_off = q_bytes;
    static constexpr int v_off = k_off + kK * kStage;
    static constexpr int scale_off = v_off + kV * kStage;   // [stage][ks 4, vs 4]
    static constexpr int row_off = scale_off + kV * 2 * kQpBoxes * 4;   // [set][rows] floats
    static constexpr int bar_off = row_off + 2 * kQpRows * 4;
    // kfull, kempty [kK], vfull, vempty [kV], pready [sets], pvdone [2 sets], sfull [sets],
    // sfree[2], qfull, qready, drain[2], settled[2][4].  (Who waits on a barrier has seen the
    // phase before, or knows that it is over: so a parity names one phase.)
    static constexpr int kBars = 2 * (kK + kV) + 4 * kQpSets + 14;
    static constexpr int flag_off = bar_off + 8 * kBars;
    static constexpr int bytes = 1024 + flag_off + 16;
    static_assert(bytes <= kSmemBudget, "shared memory per CTA");
    // a split's accumulator, [row][D] fp32, goes where the stages were
    static_assert(kQpRows * D * 4 <= (kK + kV) * kStage, "room for an accumulator");
    static constexpr uint32_t tmem_cols = 512;
    static_assert(192 + D + D / 4 <= 512, "tensor memory columns");
};

template <int D, int G>
__global__ void __launch_bounds__(kQpThreads, 1)
    q8_prefill_kernel(const __grid_constant__ CUtensorMap tmap_q,
                      const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v, const Q8PrefillParams p)
{
    using L = Q8PrefillSmem<D>;
    constexpr int TQ = kQpRows / G;
    constexpr int SK = L::kK, SV = L::kV;
    constexpr int NCH = D / 128;                 // 128-byte columns of a token
    constexpr uint32_t IDESC_S = ptx::umma_idesc_f8(128, kQpTile, false, false, false, false);
    constexpr uint32_t IDESC_HI = ptx::umma_idesc_f8(128, D, false, false, false, true);
    constexpr uint32_t IDESC_LO = ptx::umma_idesc_f8(128, D, true, false, false, true);

    extern __shared__ uint8_t smem_raw[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gen = smem_raw + (base - raw);
    float *scales = reinterpret_cast<float *>(gen + L::scale_off);
    float *rows_s = reinterpret_cast<float *>(gen + L::row_off);
    const uint32_t bars = base + L::bar_off;
    const uint32_t kfull = bars, kempty = kfull + 8 * SK, vfull = kempty + 8 * SK,
                   vempty = vfull + 8 * SV, pready = vempty + 8 * SV, pvdone = pready + 8 * kQpSets,
                   sfull = pvdone + 16 * kQpSets, sfree = sfull + 8 * kQpSets, qfull = sfree + 16,
                   qready = qfull + 8, drain = qready + 8, settled = drain + 16;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gen + L::flag_off);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(gen + L::flag_off + 4);
    volatile int *tall_flag = reinterpret_cast<volatile int *>(gen + L::flag_off + 8);

    const int rank = blockIdx.x % p.split;               // within the cluster
    const int qb = p.qblocks - 1 - (int)(blockIdx.x / p.split % p.qblocks);
    const int rest = blockIdx.x / p.split / p.qblocks;
    const int h = rest % p.num_kv_heads;
    int b = rest / p.num_kv_heads;

    if (tid == 0) {
        ptx::prefetch_tensormap(&tmap_q);
        ptx::mbar_init(qfull, 1);
    } else if (tid >= 32 && tid < 32 + L::kBars) {
        const uint32_t bar = bars + 8 * (tid - 32);
        if (bar != qfull)
            ptx::mbar_init(bar, bar >= pready && bar < pvdone ? 4
                                : bar >= sfree && bar < qfull ? 4
                                : bar == qready               ? 4 * kQpSets
                                                              : 1);
    } else if (tid == 32 * kQpWarpPV) {
        *abort_flag = 0;
        *tall_flag = 0;
    }
    ptx::fence_mbar_init();
    ptx::grid_wait_prerequisites();
    if (p.num_seqs <= 32) {
        // The longest contexts first: sequence b is the one with b longer
        // ones (ties by index).
        const int len = lane < p.num_seqs ? p.context_lens[lane * p.len_stride] : INT_MIN;
        int longer = 0;
        for (int i = 0; i < p.num_seqs; ++i) {
            const int other = __shfl_sync(kFull, len, i);
            longer += other > len || (other == len && i < lane);
        }
        b = __ffs(__ballot_sync(kFull, lane < p.num_seqs && longer == b)) - 1;
    }
    const int q0 = p.cu_q_lens[b];
    const int n = p.cu_q_lens[b + 1] - q0;
    const int ctx = p.context_lens[b * p.len_stride];
    const int tok0 = qb * TQ;
    const bool rows_ok = n >= 0 && q0 >= 0 && (int64_t)q0 + n <= p.total_q;
    auto zero_rows = [&](int count) {
        for (int idx = tid; idx < count * G * D; idx += kQpThreads) {
            const int tok = idx / (G * D), r = idx - tok * G * D;
            p.out[((int64_t)(q0 + tok0 + tok) * p.num_q_heads + h * G) * D + r] =
                __float2bfloat16_rn(0.f);
        }
    };
    if (!rows_ok || n > ctx || ctx > p.ctx_cap) {
        if (tid == 0 && qb == 0 && h == 0 && rank == 0)
            report(p.dev_status, PA_DEV_BAD_CONTEXT);
        if (rows_ok && tok0 < n && rank == 0)
            zero_rows(min(TQ, n - tok0));
        return;
    }
    if (tok0 >= n)
        return;
    const int ntok = min(TQ, n - tok0);
    const int pos0 = ctx - n + tok0;
    const int all_tiles = (pos0 + ntok - 1) / kQpTile + 1;
    const int last_tok = min(all_tiles * kQpTile, ctx);  // tokens the tiles hold
    const int nblk = (last_tok - 1) / p.block_size + 1;
    // this CTA's tiles: first, first + 1, ...
    const int first = (int)((int64_t)all_tiles * rank / p.split);
    const int ntiles = (int)((int64_t)all_tiles * (rank + 1) / p.split) - first;
    auto boxes = [&](int i) { return min(kQpBoxes, (last_tok - (first + i) * kQpTile + 15) >> 4); };

    // Q, before the block ids are known good
    if (tid == 0 && ntiles > 0) {
        ptx::mbar_arrive_expect_tx(qfull, (uint32_t)L::q_bytes);
        for (int c = 0; c < D / 64; ++c)
            ptx::tma_load_3d_nohint(base + (uint32_t)(c * kQpRows * 128), &tmap_q, c * 64, h * G,
                                    q0 + tok0, qfull);
    }
    if (warp == kQpWarpPV) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_holder), L::tmem_cols);
        ptx::tmem_relinquish();
    }
    bool bad = false;
    const int32_t *trow = p.block_tables + (int64_t)b * p.max_blocks;
    for (int i = tid; i < nblk; i += kQpThreads) {
        const int id = trow[i];
        bad |= id < 0 || (int64_t)id >= p.num_blocks;
    }
    ptx::tc_fence_before();
    bad = __syncthreads_or(bad);
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const uint32_t s_tm = tmem, p_tm = tmem + 128, o_tm = tmem + 192;
    const uint32_t qh_tm = o_tm + D;

    if (bad) {
        if (tid == 0) {
            report(p.dev_status, PA_DEV_BAD_BLOCK);
            if (ntiles > 0)                              // no copy may land after the CTA is gone
                ptx::mbar_wait_bounded(qfull, 0, kWaitLimitNs);
        }
        __syncwarp();
    } else if (ntiles == 0) {
        // (a split of more CTAs than tiles)
    } else if (warp == kQpWarpK || warp == kQpWarpV) {
        // ================================================== TMA producers
        // lane x < 4 issues box x (tokens 16 x ..) of each tile
        const bool is_k = warp == kQpWarpK;
        const uint32_t full = is_k ? kfull : vfull, empty = is_k ? kempty : vempty;
        const void *tmap = is_k ? static_cast<const void *>(&tmap_k)
                                : static_cast<const void *>(&tmap_v);
        const int S = is_k ? SK : SV;
        bool ok = true;
        if (lane == 0) {
            ptx::prefetch_tensormap(tmap);
        }
        // block ids come 32 at a time, one batch ahead
        auto batch_ids = [&](int bt) {
            const int i = bt * 32 + lane;
            return i < nblk ? __ldg(trow + i) : -1;
        };
        int cur_batch = (first * kQpTile) >> (p.bs_log2 + 5);
        int ids_cur = batch_ids(cur_batch), ids_next = batch_ids(cur_batch + 1);
        // this lane's box of tile i: its block, or -1 past the context
        auto box_id = [&](int i) {
            const int blk = ((first + i) * kQpTile + (lane & 3) * 16) >> p.bs_log2;
            const int from_cur = __shfl_sync(kFull, ids_cur, blk & 31);
            const int from_next = __shfl_sync(kFull, ids_next, blk & 31);
            const int id = (blk >> 5) == cur_batch ? from_cur : from_next;
            return blk < nblk ? id : -1;
        };
        auto load_scale = [&](const float *s, int id) {
            return id < 0 ? 0.f : __ldcg(s + (int64_t)id * p.num_kv_heads + h);
        };
        int id = box_id(0);
        float ks = 0.f, vs = 0.f;
        if (!is_k) {
            ks = load_scale(p.k_scales, id);
            vs = load_scale(p.v_scales, id);
        }
        int issued = 0;
        for (int i = 0; i < ntiles; ++i) {
            if (__any_sync(kFull, *abort_flag != 0))
                break;
            // the next tile's block and scales, a tile ahead of their use
            const int bt = ((first + i) * kQpTile) >> (p.bs_log2 + 5);
            if (bt != cur_batch) {
                cur_batch = bt;
                ids_cur = ids_next;
                ids_next = batch_ids(bt + 1);
            }
            const int id_n = i + 1 < ntiles ? box_id(i + 1) : -1;
            float ks_n = 0.f, vs_n = 0.f;
            if (!is_k) {
                ks_n = load_scale(p.k_scales, id_n);
                vs_n = load_scale(p.v_scales, id_n);
            }
            const int s = i % S, nbox = boxes(i);
            if (i >= S && !__all_sync(kFull, ptx::mbar_wait_bounded(
                                                 empty + 8u * s, (uint32_t)((i / S - 1) & 1),
                                                 kWaitLimitNs))) {
                ok = false;
                break;
            }
            const uint32_t dst = base + (uint32_t)((is_k ? L::k_off : L::v_off) + s * L::kStage);
            if (lane == 0)
                ptx::mbar_expect_tx(full + 8u * s, (uint32_t)(nbox * L::kBox));
            __syncwarp();
            if (lane < nbox) {
                const int row = id * p.block_size +
                                (((first + i) * kQpTile + lane * 16) & (p.block_size - 1));
                ptx::tma_load_5d(dst + (uint32_t)(lane * L::kBox), tmap, 0, 0, 0, row >> 3, h,
                                 full + 8u * s, ptx::policy_evict_normal());
            }
            if (!is_k && lane < kQpBoxes) {
                scales[s * 2 * kQpBoxes + lane] = ks;
                scales[s * 2 * kQpBoxes + kQpBoxes + lane] = vs;
                if (vs > 0x1p32f)
                    *tall_flag = 1;
            }
            __syncwarp();
            if (lane == 0)
                ptx::mbar_arrive(full + 8u * s);     // (also releases the scales)
            issued = i + 1;
            id = id_n;
            ks = ks_n;
            vs = vs_n;
        }
        if (lane == 0) {
            if (!ok) {
                report(p.dev_status, PA_DEV_WAIT_TIMEOUT);
                *abort_flag = 1;
            }
            // no copy may land after the CTA is gone
            if (is_k)
                ptx::mbar_wait_bounded(qfull, 0, kWaitLimitNs);
            for (int i = max(0, issued - S); i < issued; ++i)
                ptx::mbar_wait_bounded(full + 8u * (i % S), (uint32_t)((i / S) & 1), kWaitLimitNs);
        }
        __syncwarp();
    } else if (warp == kQpWarpS || warp == kQpWarpPV) {
        // ====================================================== MMA issue
        auto ready = [&](uint32_t b1, uint32_t p1, uint32_t b2, uint32_t p2) -> bool {
            if (__all_sync(kFull, ptx::mbar_test_wait(b1, p1) && ptx::mbar_test_wait(b2, p2)))
                return true;
            if (__any_sync(kFull, *abort_flag != 0))
                return false;
            return __all_sync(kFull, ptx::mbar_wait_bounded(b1, p1, kWaitLimitNs)) &&
                   __all_sync(kFull, ptx::mbar_wait_bounded(b2, p2, kWaitLimitNs));
        };
        auto issue_s = [&](int j) {
            ptx::tc_fence_after();
            const uint32_t d = s_tm + (uint32_t)((j & 1) * 64);
            const uint64_t kd = ptx::umma_desc_sw128(
                base + (uint32_t)(L::k_off + (j % SK) * L::kStage), 16, L::kGroup);
            if (ptx::elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk) {
                    const uint64_t at =
                        kd + (uint64_t)(((kk >> 2) * 1024 + (kk & 3) * 32) >> 4);
                    ptx::umma_f8_ts(d, qh_tm + (uint32_t)(kk * 8), at, IDESC_S, kk > 0);
                    ptx::umma_f8_ss(d,
                                    ptx::umma_desc_sw128(base + (uint32_t)((kk >> 2) * kQpRows * 128 +
                                                                           (kk & 3) * 32),
                                                         16, 1024),
                                    at, IDESC_S, true);
                }
                ptx::umma_commit(sfull + 8u * (j % kQpSets));
                ptx::umma_commit(kempty + 8u * (j % SK));
            }
            __syncwarp();
        };
        auto issue_pv = [&](int j) -> bool {
            const int s = j % kQpSets, vsn = j % SV;
            if (!ready(pready + 8u * s, (uint32_t)((j / kQpSets) & 1), vfull + 8u * vsn,
                       (uint32_t)((j / SV) & 1)))
                return false;
            ptx::tc_fence_after();
            const int steps = (boxes(j) + 1) >> 1;       // 32 tokens each
            const uint64_t vd = ptx::umma_desc_sw128(
                base + (uint32_t)(L::v_off + vsn * L::kStage), 1024, L::kGroup);
            if (ptx::elect_one()) {
                for (int t = 0; t < steps; ++t) {
                    const uint64_t at = vd + (uint64_t)((t * 2 * L::kBox) >> 4);
                    const uint32_t pa = p_tm + (uint32_t)((j & 1) * 32 + t * 8);
                    ptx::umma_f8_ts(o_tm, pa, at, IDESC_HI, j > 0 || t > 0);
                    ptx::umma_f8_ts(o_tm, pa + 16, at, IDESC_LO, true);
                }
                ptx::umma_commit(pvdone + 8u * (j % (2 * kQpSets)));
                ptx::umma_commit(vempty + 8u * vsn);
            }
            __syncwarp();
            return true;
        };
        bool ok = true;
        if (warp == kQpWarpS) {
            ok = ready(qready, 0, kfull, 0);
            for (int j = 0; ok && j < ntiles; ++j) {
                if (j > 0 && !(ok = j < 2 ? ready(kfull + 8u * (j % SK), 0, qready, 0)
                                          : ready(kfull + 8u * (j % SK), (uint32_t)((j / SK) & 1),
                                                  sfree + 8u * (j & 1),
                                                  (uint32_t)(((j - 2) >> 1) & 1))))
                    break;
                issue_s(j);
            }
        } else {
            for (int j = 0; ok && j < ntiles; ++j)
                ok = issue_pv(j);
        }
        if (!ok) {
            if (lane == 0) {
                report(p.dev_status, PA_DEV_WAIT_TIMEOUT);
                *abort_flag = 1;
            }
            // products already issued finish before the memory goes
            const uint32_t mine = drain + (warp == kQpWarpS ? 0u : 8u);
            if (ptx::elect_one())
                ptx::umma_commit(mine);
            __syncwarp();
            ptx::mbar_wait_bounded(mine, 0, kWaitLimitNs);
        }
        __syncwarp();
    } else {
        // =================================================== softmax warps
        const int w4 = warp & 3, set = warp >> 2;        // tiles set, set + kQpSets, ...
        const int r = w4 * 32 + lane;                    // query row = TMEM lane
        const int pos = min(pos0 + r / G, ctx - 1);
        const uint32_t lane_tm = (uint32_t)(w4 * 32) << 16;
        float m_ref = -INFINITY, l = 0.f, fac = 0.f;     // l relative to m_ref
        bool fail = false;
        auto give_up = [&]() {
            fail = true;
            if (lane == 0) {
                report(p.dev_status, PA_DEV_WAIT_TIMEOUT);
                *abort_flag = 1;
            }
            __syncwarp();
        };
        auto wait = [&](uint32_t bar, uint32_t parity) {
            if (fail || __all_sync(kFull, ptx::mbar_test_wait(bar, parity)))
                return;
            if (__any_sync(kFull, *abort_flag != 0) ||
                !__all_sync(kFull, ptx::mbar_wait_bounded(bar, parity, kWaitLimitNs)))
                give_up();
        };
        wait(qfull, 0);
        if (!fail) {
            // this set's part of the row of Q from its swizzled copy (64-element
            // columns of 16384 bytes), 32 elements at a time
            constexpr int NQ = (D / 32 + kQpSets - 1) / kQpSets;
            uint32_t w[NQ][16];
            uint32_t top2 = 0;                           // largest of the even, the odd elements
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                const int c = set + x * kQpSets;
                if (c >= D / 32)
                    break;
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[x][4 * u]), "=r"(w[x][4 * u + 1]), "=r"(w[x][4 * u + 2]),
                                   "=r"(w[x][4 * u + 3])
                                 : "r"(base + (uint32_t)((c >> 1) * kQpRows * 128 + r * 128) +
                                       ((uint32_t)((4 * (c & 1) + u) ^ (r & 7)) << 4)));
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    top2 = ptx::max_u16x2(top2, w[x][k] & 0x7fff7fffu);
            }
            // the row's largest exponent; behind the barrier the row has been
            // read, and its low parts may take its place
            uint8_t *exps = reinterpret_cast<uint8_t *>(rows_s);
            exps[set * kQpRows + r] = (uint8_t)(max(top2 << 16, top2) >> 23);
            ptx::barrier_or(1 + w4, 32 * kQpSets, false);
            int ef = exps[r];
#pragma unroll
            for (int k = 1; k < kQpSets; ++k)
                ef = max(ef, (int)exps[k * kQpRows + r]);
            // (the sign of the softmax scale goes into Q, so that logit
            // factors are not negative)
            const float sig = __uint_as_float((uint32_t)min(254, 261 - ef) << 23);
            const float sigma = p.scale_log2 < 0.f ? -sig : sig;
            fac = ef < 255 ? p.scale_log2 / sigma : __int_as_float(0x7fc00000);
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                const int c = set + x * kQpSets;
                if (c >= D / 32)
                    break;
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    uint32_t h2[2], l2[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // (8 bits of a value below 256: exact in f16 but
                        // far below E4M3's quantum, and so is what is left)
                        const uint32_t y =
                            ptx::pack_f16x2(ptx::bf16lo_to_f32(w[x][2 * k + e]) * sigma,
                                            ptx::bf16hi_to_f32(w[x][2 * k + e]) * sigma);
                        h2[e] = f16x2_to_e4m3x2(y);
                        l2[e] = f16x2_to_e4m3x2(ptx::sub_f16x2(y, e4m3x2_to_f16x2(h2[e])));
                    }
                    hi[k] = h2[0] | (h2[1] << 16);
                    lo[k] = l2[0] | (l2[1] << 16);
                }
                ptx::tmem_st8(qh_tm + lane_tm + (uint32_t)(c * 8), hi);
                // (128-element columns of 16384 bytes, swizzled)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     base + (uint32_t)((c >> 2) * kQpRows * 128 + r * 128) +
                                     ((uint32_t)((2 * (c & 3) + u) ^ (r & 7)) << 4)),
                                 "r"(lo[4 * u]), "r"(lo[4 * u + 1]), "r"(lo[4 * u + 2]),
                                 "r"(lo[4 * u + 3])
                                 : "memory");
            }
            ptx::fence_proxy_async_smem();
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0)
                ptx::mbar_arrive(qready);
        } else {
            ptx::barrier_or(1 + w4, 32 * kQpSets, false);    // (the others' barrier)
        }
        // Product j.  Its barrier's phase before was product j - 6's: a set has
        // seen that end before it passed on the reference of tile j - 1, and
        // whoever waits here has taken it (or a later one).
        auto wait_pv = [&](int j) {
            wait(pvdone + 8u * (j % (2 * kQpSets)), (uint32_t)((j / (2 * kQpSets)) & 1));
        };
        // the reference that another set's warp of these rows left with tile i
        // (and with it this warp's sum in the same terms)
        auto take_reference = [&](int i) {
            wait(settled + 8u * (4 * (i & 1) + w4), (uint32_t)((i >> 1) & 1));
            const float m = rows_s[r];
            if (m != m_ref && m_ref != -INFINITY)
                l = ptx::times_2_to(l, m_ref - m);
            m_ref = m;
        };
        for (int i = set; i < ntiles && !fail; i += kQpSets) {
            const int pb = i % kQpSets, vsn = i % SV;
            wait(sfull + 8u * pb, (uint32_t)((i / kQpSets) & 1));
            // V is in: so are the tile's block scales
            wait(vfull + 8u * vsn, (uint32_t)((i / SV) & 1));
            if (fail)
                break;
            ptx::tc_fence_after();
            const int tstart = (first + i) * kQpTile;
            const uint32_t sa = s_tm + lane_tm + (uint32_t)((i & 1) * 64);
            float sv[kQpTile], kf[kQpBoxes], lv[kQpBoxes], cand = -INFINITY;
            // Once a V scale above 2^32 has been met, x = 2^(s - m + lv) of a small
            // one may be no normal number, while its row sum x / vs still counts:
            // then x is carried 2^96 times as large until the sum has been taken.
            const float bias = *tall_flag == 0 ? 0.f : 96.f;
            {
                uint32_t u0[16], u1[16], u2[16], u3[16];
                ptx::tmem_ld16(sa, u0);
                ptx::tmem_ld16(sa + 16, u1);
                ptx::tmem_ld16(sa + 32, u2);
                ptx::tmem_ld16(sa + 48, u3);
#pragma unroll
                for (int x = 0; x < kQpBoxes; ++x) {
                    const float f = fac * scales[vsn * 2 * kQpBoxes + x];
                    const float vw = scales[vsn * 2 * kQpBoxes + kQpBoxes + x];
                    kf[x] = f == 0.f ? 1.2e-38f : f;     // (a masked -inf stays one)
                    lv[x] = fmaxf(ptx::lg2(vw), -64.f);
                }
                ptx::tmem_wait_ld();
                // S may be overwritten
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    ptx::mbar_arrive(sfree + 8u * (i & 1));
                ptx::tmem_hold16(u0);
                ptx::tmem_hold16(u1);
                ptx::tmem_hold16(u2);
                ptx::tmem_hold16(u3);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    sv[e] = __uint_as_float(u0[e]);
                    sv[16 + e] = __uint_as_float(u1[e]);
                    sv[32 + e] = __uint_as_float(u2[e]);
                    sv[48 + e] = __uint_as_float(u3[e]);
                }
            }
            if (tstart + kQpTile - 1 > pos0) {
#pragma unroll
                for (int c = 0; c < kQpTile; ++c)
                    sv[c] = tstart + c <= pos ? sv[c] : -INFINITY;
            }
#pragma unroll
            for (int x = 0; x < kQpBoxes; ++x) {
                float a = ptx::max3(sv[16 * x], sv[16 * x + 1], sv[16 * x + 2]);
                float c = ptx::max3(sv[16 * x + 3], sv[16 * x + 4], sv[16 * x + 5]);
#pragma unroll
                for (int e = 6; e < 14; e += 4) {
                    a = ptx::max3(a, sv[16 * x + e], sv[16 * x + e + 1]);
                    c = ptx::max3(c, sv[16 * x + e + 2], sv[16 * x + e + 3]);
                }
                a = ptx::max3(a, sv[16 * x + 14], sv[16 * x + 15]);
                cand = fmaxf(cand, fmaf(fmaxf(a, c), kf[x], lv[x]));
            }
            if (i > 0)
                take_reference(i - 1);
            if (fail)
                break;
            // one row of the warp that has to move takes along all that may: O is
            // rescaled once, and they need not move by themselves soon after
            const bool move = __any_sync(kFull, cand > m_ref + kQpGrow);
            float alpha = 1.f;
            if (move && cand - kQpLift > m_ref) {
                const float by = m_ref - (cand - kQpLift);
                if (m_ref != -INFINITY) {                // (else nothing to rescale)
                    const float root = ptx::ex2(0.5f * by);   // (l may take less than 2^-126)
                    l = l * root * root;
                    alpha = root * root;
                }
                m_ref = cand - kQpLift;
            }
            rows_s[r] = m_ref;
            __syncwarp();
            if (lane == 0)
                ptx::mbar_arrive(settled + 8u * (4 * (i & 1) + w4));
            const float nref = m_ref == -INFINITY ? 0.f : -m_ref;
            uint32_t hi[16], lo[16];                     // weights, four tokens each
            // x = 2^(s - m + log2 vs); the row sum takes x / vs, box by box
#pragma unroll
            for (int x = 0; x < kQpBoxes; ++x) {         // 16 tokens at a time
                float *v = sv + 16 * x;
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                const float2 k2 = make_float2(kf[x], kf[x]);
                const float n = nref + (lv[x] + bias);
                const float2 n2 = make_float2(n, n);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float2 y = ptx::fma2(make_float2(v[e], v[e + 1]), k2, n2);
                    v[e] = ptx::ex2(y.x);
                    v[e + 1] = ptx::ex2(y.y);
                    sum[e >> 1 & 1] = ptx::add2(sum[e >> 1 & 1], make_float2(v[e], v[e + 1]));
                }
                // (in two half steps: the factor may be below the normal numbers)
                const float root = ptx::ex2(-0.5f * (lv[x] + bias));
                l = fmaf(((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) * root, root, l);
                if (bias != 0.f) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        v[e] *= 0x1p-96f;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t h2[2], r2[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // (11 bits and 2^-24: far below what hi + lo keep)
                        const uint32_t y =
                            ptx::pack_f16x2(v[4 * k + 2 * e], v[4 * k + 2 * e + 1]);
                        h2[e] = f16x2_to_e4m3x2(y);
                        // the rest as E5M2, the upper byte of an f16: rounded
                        // (half away from zero) by an add below it
                        r2[e] = ptx::sub_f16x2(y, e4m3x2_to_f16x2(h2[e])) + 0x00800080u;
                    }
                    hi[4 * x + k] = h2[0] | (h2[1] << 16);
                    lo[4 * x + k] = ptx::prmt(r2[0], r2[1], 0x7531u);
                }
            }
            // the buffer's weights of two tiles ago have been used
            if (i >= 2)
                wait_pv(i - 2);
            if (fail)
                break;
            ptx::tc_fence_after();
            ptx::tmem_st16(p_tm + lane_tm + (uint32_t)((i & 1) * 32), hi);
            ptx::tmem_st16(p_tm + lane_tm + (uint32_t)((i & 1) * 32 + 16), lo);
            const int from = last_tok - tstart;          // tokens of this tile
            if (from < kQpTile && (from & 31) != 0) {
                // V rows of the last 32-token step past the context: their
                // weight is 0, but 0 * NaN is NaN
                const int to = (from + 31) & ~31;
                const uint32_t vst = base + (uint32_t)(L::v_off + vsn * L::kStage);
                for (int idx = r; idx < (to - from) * NCH * 8; idx += kQpRows) {
                    const int t = from + idx / (NCH * 8), c = idx % (NCH * 8);
                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                     vst + (uint32_t)((t >> 3) * L::kGroup + (c >> 3) * 1024 +
                                                      (t & 7) * 128 + (c & 7) * 16)),
                                 "r"(0)
                                 : "memory");
                }
                ptx::fence_proxy_async_smem();
            }
            if (move && i > 0) {
                // O to the new reference, once P V of the tile before (and all
                // earlier) is in it: by now it mostly is
                wait_pv(i - 1);
                if (fail)
                    break;
                ptx::tc_fence_after();
                const float2 a2 = make_float2(alpha, alpha);
                uint32_t u[2][2][16];                    // 32 columns, and the next 32
                const uint32_t at = o_tm + lane_tm;
                ptx::tmem_ld16(at, u[0][0]);
                ptx::tmem_ld16(at + 16, u[0][1]);
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t (&now)[2][16] = u[c & 1], (&next)[2][16] = u[(c + 1) & 1];
                    ptx::tmem_wait_ld();
                    ptx::tmem_hold16(now[0]);
                    ptx::tmem_hold16(now[1]);
                    if (c + 1 < D / 32) {
                        ptx::tmem_ld16(at + (uint32_t)(32 * c + 32), next[0]);
                        ptx::tmem_ld16(at + (uint32_t)(32 * c + 48), next[1]);
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float2 y = ptx::mul2(make_float2(__uint_as_float(now[k][e]),
                                                                   __uint_as_float(now[k][e + 1])),
                                                       a2);
                            now[k][e] = __float_as_uint(y.x);
                            now[k][e + 1] = __float_as_uint(y.y);
                        }
                        ptx::tmem_st16(at + (uint32_t)(32 * c + 16 * k), now[k]);
                    }
                }
            }
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0)
                ptx::mbar_arrive(pready + 8u * pb);
        }
        if ((ntiles - 1) % kQpSets == set)
            wait_pv(ntiles - 1);
        else
            take_reference(ntiles - 1);
        // the sets' sums; with a split, the row's reference and sum for the
        // other CTAs (a warp that gave up takes part in the barriers too)
        ptx::barrier_or(1 + w4, 32 * kQpSets, false);    // (rows_s has been read, O is done)
        float *sums = reinterpret_cast<float *>(gen);    // (where the queries were)
        sums[set * kQpRows + r] = l;
        ptx::barrier_or(1 + w4, 32 * kQpSets, false);
        l = sums[r];
#pragma unroll
        for (int k = 1; k < kQpSets; ++k)
            l += sums[k * kQpRows + r];
        if (set == 0) {
            rows_s[r] = m_ref;
            rows_s[kQpRows + r] = l;
        }
        if (p.split == 1) {
            // a row of the output in shared memory, where the stages were
            // (16-byte unit u of row r at u ^ (r & 7)), then whole rows out
            if (!fail) {
                ptx::tc_fence_after();
                // (a sum that is not a number, from a non-finite query, stays one)
                const float inv = l == 0.f ? 0.f : __frcp_rn(l);
#pragma unroll 1
                for (int c = set; c < D / 32; c += kQpSets) {
                    uint32_t u[2][16];
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        ptx::tmem_ld16(o_tm + lane_tm + (uint32_t)(c * 32 + 16 * k), u[k]);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        ptx::tmem_hold16(u[k]);
                        uint32_t o[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            o[e] = ptx::pack_bf16x2(__uint_as_float(u[k][2 * e]) * inv,
                                                    __uint_as_float(u[k][2 * e + 1]) * inv);
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            asm volatile(
                                "st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                    base + (uint32_t)(L::k_off + r * D * 2) +
                                    ((uint32_t)((4 * c + 2 * k + e) ^ (r & 7)) << 4)),
                                "r"(o[4 * e]), "r"(o[4 * e + 1]), "r"(o[4 * e + 2]),
                                "r"(o[4 * e + 3])
                                : "memory");
                    }
                }
            }
            ptx::barrier_or(1 + w4, 32 * kQpSets, false);
            if (!fail) {
                constexpr int U = D / 8;                 // 16-byte units of a row
                constexpr int RW = 32 / U;               // rows a warp stores at a time
                for (int rr = w4 * 32 + set * RW + lane / U; rr < w4 * 32 + 32;
                     rr += kQpSets * RW) {
                    const int u = lane % U;
                    if (rr / G < ntok) {
                        uint4 *dst = reinterpret_cast<uint4 *>(
                            p.out +
                            ((int64_t)(q0 + tok0 + rr / G) * p.num_q_heads + h * G + rr % G) * D);
                        dst[u] = *reinterpret_cast<const uint4 *>(
                            gen + L::k_off + rr * D * 2 + ((u ^ (rr & 7)) << 4));
                    }
                }
            }
        } else {
            if (!fail) {
                ptx::tc_fence_after();
                // the accumulator to shared memory, where the stages were
                // (16-byte unit u of row r at u ^ (r & 31))
#pragma unroll 1
                for (int c = set; c < D / 16; c += kQpSets) {
                    uint32_t u[16];
                    ptx::tmem_ld16(o_tm + lane_tm + (uint32_t)(c * 16), u);
                    ptx::tmem_wait_ld();
                    ptx::tmem_hold16(u);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         base + (uint32_t)(L::k_off + r * D * 4) +
                                         ((uint32_t)((4 * c + k) ^ (r & 31)) << 4)),
                                     "r"(u[4 * k]), "r"(u[4 * k + 1]), "r"(u[4 * k + 2]),
                                     "r"(u[4 * k + 3])
                                     : "memory");
                }
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kQpWarpPV)
        ptx::tmem_dealloc(tmem, L::tmem_cols);
    if (p.split == 1) {
        // zeros for an invalid block and for a wait that ran out
        if (bad || *abort_flag != 0)
            zero_rows(ntok);
        return;
    }
    // ---- join the cluster's parts: row r by CTA r % split, a warp per row
    if (ntiles == 0 && tid < kQpRows) {
        rows_s[tid] = -INFINITY;
        rows_s[kQpRows + tid] = 0.f;
    }
    ptx::cluster_sync();
    const uint32_t rows_a = base + L::row_off, acc_a = base + L::k_off, flag_a = base + L::flag_off;
    bool lost = bad;
    for (int c = 0; c < p.split; ++c)
        lost |= ptx::ld_cluster_f32(ptx::map_cluster(flag_a, c)) != 0.f;
    for (int r = rank + p.split * warp; r < ntok * G; r += p.split * (kQpThreads / 32)) {
        float M = -INFINITY, sum = 0.f;
        for (int c = 0; c < p.split; ++c)
            M = fmaxf(M, ptx::ld_cluster_f32(ptx::map_cluster(rows_a + 4 * r, c)));
        float4 a[D / 128];
#pragma unroll
        for (int k = 0; k < D / 128; ++k)
            a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < p.split && !lost; ++c) {
            const float m = ptx::ld_cluster_f32(ptx::map_cluster(rows_a + 4 * r, c));
            const float ls = ptx::ld_cluster_f32(ptx::map_cluster(rows_a + 4 * (kQpRows + r), c));
            if (m == -INFINITY && ls == 0.f)
                continue;                                // no token of this part is seen
            const float f = ptx::ex2(m - M);
            sum += ptx::times_2_to(ls, m - M);
            const uint32_t row = ptx::map_cluster(acc_a + (uint32_t)(r * D * 4), c);
#pragma unroll
            for (int k = 0; k < D / 128; ++k) {
                const float4 v =
                    ptx::ld_cluster_f32x4(row + ((uint32_t)((lane + 32 * k) ^ (r & 31)) << 4));
                a[k].x = fmaf(v.x, f, a[k].x);
                a[k].y = fmaf(v.y, f, a[k].y);
                a[k].z = fmaf(v.z, f, a[k].z);
                a[k].w = fmaf(v.w, f, a[k].w);
            }
        }
        const float inv = sum == 0.f ? 0.f : __frcp_rn(sum);
        __nv_bfloat16 *dst =
            p.out + ((int64_t)(q0 + tok0 + r / G) * p.num_q_heads + h * G + r % G) * D + 4 * lane;
#pragma unroll
        for (int k = 0; k < D / 128; ++k)
            store4(dst + 128 * k, make_float4(a[k].x * inv, a[k].y * inv, a[k].z * inv, a[k].w * inv));
    }
    ptx::cluster_sync();                                 // the others may still be reading
}

}  // namespace pa
