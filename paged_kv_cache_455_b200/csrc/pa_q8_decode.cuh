// pa_q8_decode.cuh -- decode attention over a block-scaled E4M3 cache on the
// 5th-generation tensor cores (tcgen05.mma kind::f8f6f4, accumulators in
// tensor memory).
//
//   s_t = scale ks(t) (q . K_t),   o = sum_t p_t vs(t) V_t / sum_t p_t,
// p_t = exp(s_t - max s), K_t and V_t the codes of token t, ks(t) and vs(t)
// the scales of its block.
//
// Tile.  128 rows of K and of V: hpc KV heads (the largest of 4, 2, 1 that
// divides Hkv) times 128 / hpc consecutive tokens of one sequence, so a CTA
// reads whole token rows of its head group.  Rows 32 w .. 32 w + 31 belong to
// softmax warp w: 32 tokens of head w / (4 / hpc).  Both products take the
// cache as the A operand, straight from the stage the TMA filled:
//   S   [128 rows x NQ]  = K (K-major, 128 x d) * Q^T, NQ = the group's query
//       rows, each as two E4M3 parts; a row uses only its own head's columns
//       (the tensor cores have room: 128 x NQ x d per 2 * 128 * d bytes)
//   O^T [128 d x NP] += V_w^T (MN-major, 128 d x 32 tokens) * P_w, for each
//       warp w and half of d; P_w holds the warp's weights as three E5M2 parts,
//       MN-major too: a token's weights are consecutive, so the lane that has
//       the token stores them as one or two 16-byte words
// so no code is ever converted or moved by a thread, and the softmax of one
// tile is 32 tokens per warp, one per lane.
//
// Weights.  x_t = vs(t) 2^(s_t - m) with m a running reference per head and
// warp, raised to max_t (s_t + log2 vs(t)) whenever that has grown past m + 15
// (log2 units): x_t <= 2^15.  The three E5M2 parts are the value rounded to 3
// bits, the rest times 8 rounded to 3, and again; each part has accumulators of
// its own, so the factors of 8 come out at the end and all parts have the
// type's whole range: error 2^-9 of x_t down to x_t = 2^-14 and 2^-23 below,
// relative to a largest weight of at least 1, so that many small weights next
// to a large one are not lost.  The row sums take the fp32 weights 2^(s_t - m)
// (kept in range by kQ8Bias, and joined by times_2_to, for V scales from 2^-64 to
// 2^120 in any mixture).  Because m follows the weights with their scales, the errors are relative to
// what the output is made of, whatever the scales' spread.  A warp needs the
// maximum itself only for its first tile and when a vote finds a lane past the
// reference, and accumulators are rescaled only then.
//
// Warps: SETS x 4 softmax and epilogue, then one each for S, O^T, the TMA of K,
// the TMA of V with the block scales, and two for the query rows.  A tile's
// logits, softmax (~1100 cycles at G = 4) and second product follow one another,
// and together take longer than a tile's share of the memory bandwidth (2700
// cycles at d = 256, 1370 at d = 128), so two sets of warps take alternate tiles,
// each with accumulators and references of its own; they are joined at the
// segment's end.  With d = 256 and G = 8 tensor memory holds one set's
// accumulators only.
//
// Memory bounds it, behind the ends: setting up, the queries and the first tiles
// take ~5 us of a call, a segment's end ~2 us, a merge ~3 us.  Measured: 64
// sequences of up to 4K tokens, 16 query and 4 KV heads of 256, 267 MB: 52.6 us, 5.1
// TB/s; 8 of 8K, 134 MB: 33.9 us, 4.0 TB/s; 45 of up to 6K, 64 query and 8 KV heads of
// 128, 239 MB: 58.7 us, 4.1 TB/s.  One sequence, the same heads of 256: without a
// token 3.2 us, one tile 8.7, 100 tokens 12.3 (four tiles on as many CTAs, joined;
// 11.4 on one).
//
// Work is split as in decode_kernel: every CTA owns a contiguous range of the
// batch's tiles (mode 0), or whole segments (mode 1); a segment is the run of
// tiles of one sequence and head group.  The ranges are equal in the time they
// take: a segment's end costs a CTA about as much as end_tiles more tiles (its
// accumulators have to be read out before the next segment's products), so
// ranges are equal shares of the tiles plus end_tiles for every segment.  The pieces of a segment cut by
// range borders go to the workspace as fp32 (maximum, sum, accumulator).  Cut in
// a few pieces, the CTA whose piece is the last to arrive joins them after its
// range; cut in many (few long sequences), reading them all would take one SM
// longer than a launch (16 KB each at ~30 bytes a cycle: 19 pieces 6 us), and
// q8_merge_kernel joins them on all SMs.
#pragma once

#include "pa_kernels.cuh"
#include "pa_ptx8.cuh"

namespace pa {

constexpr int kQ8Tile = 128;              // rows of K and V per tile (MMA M)
constexpr int kQ8MaxSeqs = 16384;         // (the prefix of the tile counts is in shared memory)
constexpr int kQ8SmemStages = 6 * 32768;  // bytes of the stage ring
constexpr float kQ8Grow = 15.f;           // log2 growth that makes a rescale
// References are kept this much (log2) lower, so that weights without their V
// scale, 2^-120 of the others' with the largest one, and those 2^-30 of them
// are normal numbers; with the smallest, 2^-64, a million of 2^(64 + 15) still
// have a finite sum.
constexpr float kQ8Bias = 24.f;

struct Q8DecodeParams {
    __nv_bfloat16 *out;
    const __nv_bfloat16 *q;
    const float *k_scales, *v_scales;
    const int32_t *block_tables, *context_lens;
    int64_t len_stride;      // elements between context_lens
    float *pieces;           // mode 0: two slots per CTA
    unsigned long long *counters;   // mode 0: arrivals at the cut segment that starts in a
                                    // CTA's range, a line each (see segment_arrive)
    uint32_t epoch;          // mode 0: tag of this call's counts (never 0)
    int merge_later;         // mode 0: q8_merge_kernel joins the pieces
    int32_t *dev_status;
    int64_t num_blocks;
    int num_seqs, num_q_heads, num_kv_heads;
    int max_blocks, block_size, bs_log2;
    int ctx_cap;
    int hpc, hpc_log2;       // KV heads per tile
    int tt_log2;             // tokens per tile = 128 / hpc
    int box_log2;            // tokens per TMA box: 16, or 32 with blocks of 32
    int head_groups;
    int mode;                // 0: equal ranges, 1: whole segments
    int slot_floats;
    int end_tiles;           // tiles that a segment's end is counted as
    float scale_log2;
    uint64_t wait_ns;
    int withhold_cta;        // test hook, as in DecodeParams
};

// Per-stage metadata, written by V's TMA warp.
struct Q8Meta {
    int b, hg, j, ns;        // sequence, head group, tile in the segment, its tiles
    int n;                   // valid tokens of the tile
    int seg;                 // ordinal of the segment in this CTA's range
    int bad;                 // an invalid block id
    int pad;
    float ks[8], vs[8];      // scales of the tile's 16-row boxes
};

template <int D, int G>
struct Q8Smem {
    static constexpr int kStage = kQ8Tile * D;                       // K or V of a tile
    static constexpr int kStages = kQ8SmemStages / (2 * kStage);     // 3 (d 256), 6 (d 128)
    static constexpr int kQRows = 8 * G < 16 ? 16 : 8 * G;           // up to 4 heads, 2 parts
    static constexpr int kQBufs = (D == 256 && G == 8) ? 1 : 2;
    static constexpr int GP = G <= 4 ? 4 : 8;                        // rows of one weight part
    static constexpr int NP = 4 * GP;                                // 3 parts, padded
    static constexpr int kP = NP * 32;                               // bytes of a warp's weights
    // tensor memory columns: two S buffers of 64, then the sets' accumulators
    static constexpr int o_cols = 4 * (D / 128) * NP;
    static constexpr int kSets = 128 + 2 * o_cols <= 512 ? 2 : 1;
    static constexpr uint32_t tmem_cols = 128 + kSets * o_cols <= 256 ? 256u : 512u;
    static constexpr int kSoftmax = 4 * kSets;                       // warps
    static constexpr int kThreads = 32 * (kSoftmax + 8);
    static constexpr int v_off = kStages * kStage;
    static constexpr int q_off = kQ8SmemStages;
    static constexpr int p_off = q_off + kQBufs * kQRows * D;
    static constexpr int meta_off = p_off + 2 * 4 * kP;
    static constexpr int kflag_off = meta_off + kStages * (int)sizeof(Q8Meta);
    static constexpr int sf_off = kflag_off + 4 * 8;                 // query factors of 4 segments
    static constexpr int stat_off = sf_off + 4 * 4 * G * 4;          // [2][sets][4][m, l][G]
    static constexpr int fac_off = stat_off + 2 * kSets * 4 * 2 * G * 4;   // [sets][4][G]
    static constexpr int alpha_off = fac_off + kSets * 4 * G * 4;    // [sets][4][G]
    static constexpr int pend_off = (alpha_off + kSets * 4 * G * 4 + 15) / 16 * 16;
    static constexpr int bar_off = pend_off + 32;
    // a merge's weights lie where the queries and the weights of P were
    static_assert(meta_off - q_off >= 148 * 4 * G * 4, "room for a merge's weights");
    static constexpr int kBars = 5 * kStages + 8 + 2 * kQBufs + 5;
    static constexpr int flag_off = bar_off + 8 * kBars;   // abort, tensor memory, tiles done
    static constexpr int cbase_off = flag_off + 16;
    // (the prefix of the tile counts comes last, as long as the batch needs)
    static constexpr int bytes = 1024 + cbase_off;
    static_assert(bytes + 8 * (kQ8MaxSeqs / 32 + 1) <= kSmemBudget, "shared memory per CTA");
};

// Position in the batch's sequence of segments (whole warp, uniform).
struct Q8Walk {
    int b, hg;       // sequence, head group
    int ctx, nt;     // its effective length, tiles of the segment
    int g0;          // global index of the segment's first tile
    int ord;         // ordinal of the segment in the batch
};

// Length of sequence b as the caller gave it, and the length to process.
__device__ __forceinline__ int q8_len(int b, const Q8DecodeParams &p)
{
    return p.context_lens[b * p.len_stride];
}
__device__ __forceinline__ int q8_ctx(int b, const Q8DecodeParams &p)
{
    return b < p.num_seqs ? eff_ctx(q8_len(b, p), p.ctx_cap) : 0;
}

__device__ __forceinline__ int q8_tiles(int ctx, const Q8DecodeParams &p)
{
    return (ctx + (1 << p.tt_log2) - 1) >> p.tt_log2;
}

// For chunk c of 32 sequences, cbase[2 c] = tiles and cbase[2 c + 1] = segments
// before it; the totals come last.  Every thread of the CTA.
__device__ __forceinline__ void q8_prefix(const Q8DecodeParams &p, int *cbase)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
    const int nch = (p.num_seqs + 31) >> 5;
    for (int c = warp; c < nch; c += nwarps) {
        const int b = c * 32 + lane;
        int t = q8_tiles(q8_ctx(b, p), p);
        const int n = __popc(__ballot_sync(kFull, t > 0));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            t += __shfl_xor_sync(kFull, t, o);
        if (lane == 0) {
            cbase[2 * c + 2] = t * p.head_groups;
            cbase[2 * c + 3] = n * p.head_groups;
        }
    }
    __syncthreads();
    if (warp == 0) {
        int ct = 0, cn = 0;
        if (lane < 2)
            cbase[lane] = 0;
        for (int c0 = 0; c0 < nch; c0 += 32) {
            const int c = c0 + lane;
            int t = c < nch ? cbase[2 * c + 2] : 0, n = c < nch ? cbase[2 * c + 3] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(kFull, t, o), v = __shfl_up_sync(kFull, n, o);
                if (lane >= o) {
                    t += u;
                    n += v;
                }
            }
            if (c < nch) {
                cbase[2 * c + 2] = ct + t;
                cbase[2 * c + 3] = cn + n;
            }
            ct += __shfl_sync(kFull, t, 31);
            cn += __shfl_sync(kFull, n, 31);
        }
    }
    __syncthreads();
}

// The segment holding tile g, or with `weight` > 0 the one holding unit g of
// the sequence in which every segment is its tiles and then `weight` units
// (g below the total).
__device__ __forceinline__ Q8Walk q8_walk_at(int g, int weight, const Q8DecodeParams &p,
                                             const int *cbase, int lane)
{
    int c = 0, hi = ((p.num_seqs + 31) >> 5) - 1;        // the last chunk that starts at or before g
    while (c < hi) {
        const int mid = (c + hi + 1) >> 1;
        if (cbase[2 * mid] + weight * cbase[2 * mid + 1] <= g)
            c = mid;
        else
            hi = mid - 1;
    }
    const int b = c * 32 + lane;
    const int ctx = q8_ctx(b, p);
    const int nt = q8_tiles(ctx, p);
    int t = nt * p.head_groups;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, t, o);
        if (lane >= o)
            t += u;
    }
    const unsigned some = __ballot_sync(kFull, nt > 0);
    const int n = __popc(some & (0xffffffffu >> (31 - lane))) * p.head_groups;
    const int t0 = cbase[2 * c] + t - nt * p.head_groups;            // before this sequence
    const int n0 = cbase[2 * c + 1] + n - (nt > 0 ? p.head_groups : 0);
    const unsigned past = __ballot_sync(
        kFull, nt > 0 && t0 + weight * n0 + (nt + weight) * p.head_groups > g);
    const int src = past ? __ffs(past) - 1 : 31;
    Q8Walk w;
    w.b = c * 32 + src;
    w.ctx = __shfl_sync(kFull, ctx, src);
    w.nt = max(__shfl_sync(kFull, nt, src), 1);
    const int st = __shfl_sync(kFull, t0, src), sn = __shfl_sync(kFull, n0, src);
    w.hg = (g - st - weight * sn) / (w.nt + weight);
    w.g0 = st + w.hg * w.nt;
    w.ord = sn + w.hg;
    return w;
}

// Moves to the next segment (the batch must hold one).
__device__ __forceinline__ void q8_walk_next(Q8Walk &w, const Q8DecodeParams &p, int lane)
{
    w.g0 += w.nt;
    ++w.ord;
    if (++w.hg < p.head_groups)
        return;
    w.hg = 0;
    for (int b0 = w.b + 1; b0 < p.num_seqs; b0 += 32) {
        const int b = b0 + lane;
        const int ctx = q8_ctx(b, p);
        const unsigned some = __ballot_sync(kFull, ctx > 0);
        if (some) {
            const int src = __ffs(some) - 1;
            w.b = b0 + src;
            w.ctx = __shfl_sync(kFull, ctx, src);
            w.nt = q8_tiles(w.ctx, p);
            return;
        }
    }
}

// First tile of CTA x's range: of the `units` (tiles and segment ends), CTA x
// has [x units / C, (x + 1) units / C), and of those the tiles.
__device__ __forceinline__ int q8_range_begin(int x, int C, int T, int units,
                                              const Q8DecodeParams &p, const int *cbase, int lane)
{
    const int v = (int)((int64_t)x * units / C);
    if (x >= C || v >= units)
        return T;
    const Q8Walk w = q8_walk_at(v, p.end_tiles, p, cbase, lane);
    const int into = v - (w.g0 + p.end_tiles * w.ord);   // units into the segment
    if (p.mode == 0)
        return w.g0 + min(into, w.nt);
    return into == 0 ? w.g0 : w.g0 + w.nt;               // whole segments
}

// Two fp32 values to E5M2 codes, `lo` in byte 0 (nearest, ties to even).
__device__ __forceinline__ uint32_t e5m2x2(float lo, float hi)
{
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E5M2);
}

template <int D, int G>
__global__ void __launch_bounds__((Q8Smem<D, G>::kThreads), 1)
    q8_decode_kernel(const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const Q8DecodeParams p)
{
    using L = Q8Smem<D, G>;
    constexpr int S = L::kStages, QB = L::kQBufs, GP = L::GP, NP = L::NP, SETS = L::kSets;
    constexpr int HALVES = D / 128;
    constexpr int GROUP = 8 * D;                 // bytes between 8-row groups
    constexpr int W_S = L::kSoftmax, W_O = W_S + 1, W_K = W_S + 2, W_V = W_S + 3, W_Q = W_S + 4;
    extern __shared__ uint8_t smem_raw[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t raw = ptx::smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gen = smem_raw + (base - raw);
    Q8Meta *meta = reinterpret_cast<Q8Meta *>(gen + L::meta_off);
    volatile int *kflag = reinterpret_cast<volatile int *>(gen + L::kflag_off);
    float *sf = reinterpret_cast<float *>(gen + L::sf_off);
    float *stat = reinterpret_cast<float *>(gen + L::stat_off);
    float *fac_s = reinterpret_cast<float *>(gen + L::fac_off);
    float *alpha_s = reinterpret_cast<float *>(gen + L::alpha_off);
    // merges this CTA owes: first CTA, pieces, sequence, head group
    int4 *pend_s = reinterpret_cast<int4 *>(gen + L::pend_off);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gen + L::flag_off);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(gen + L::flag_off + 4);
    int *tiles_done = reinterpret_cast<int *>(gen + L::flag_off + 8);
    int *cbase = reinterpret_cast<int *>(gen + L::cbase_off);
    const uint32_t bars = base + L::bar_off;
    const uint32_t kfull = bars, kempty = kfull + 8 * S, vfull = kempty + 8 * S,
                   vempty = vfull + 8 * S, mfull = vempty + 8 * S, sfull = mfull + 8 * S,
                   sfree = sfull + 16, pready = sfree + 16, pvdone = pready + 16,
                   qfull = pvdone + 16, qempty = qfull + 8 * QB, ofree = qempty + 8 * QB,
                   xstat = ofree + 8, drain_s = xstat + 16, drain_o = drain_s + 8;
    const int hpc = p.hpc, sub_log2 = 2 - p.hpc_log2;   // 4 / hpc warps per head
    const int tt = 1 << p.tt_log2;

    if (tid == 0) {
        for (int i = 0; i < 5 * S; ++i)          // (stages: one arrival each)
            ptx::mbar_init(bars + 8 * i, 1);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(sfull + 8 * i, 2);    // the product, and the issuing warp
            ptx::mbar_init(sfree + 8 * i, 4);
            ptx::mbar_init(pready + 8 * i, 4);
            ptx::mbar_init(pvdone + 8 * i, 1);
        }
        for (int i = 0; i < QB; ++i) {
            ptx::mbar_init(qfull + 8 * i, 4);
            ptx::mbar_init(qempty + 8 * i, 1);
        }
        ptx::mbar_init(ofree, 4);
        ptx::mbar_init(xstat, 4);
        ptx::mbar_init(xstat + 8, 4);
        ptx::mbar_init(drain_s, 1);
        ptx::mbar_init(drain_o, 1);
        *abort_flag = 0;
        *tiles_done = 0;
        pend_s[0] = pend_s[1] = make_int4(0, 0, 0, 0);
    }
    ptx::fence_mbar_init();
    if (warp == W_S) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_holder), L::tmem_cols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    // What the kernel ahead wrote is visible behind this wait only, and it may
    // be any of the inputs: lengths that a small kernel raised, blocks that a
    // chunk's append filled or a copy cloned.  So nothing is read before it.
    // (Reading lengths, tables and full blocks before it took 49.7 us where this
    // takes 53.4, and 10.6 us where this takes 12.1; see above.)
    ptx::grid_wait_prerequisites();
    if (tid == 0)
        ptx::grid_launch_dependents();
    q8_prefix(p, cbase);                                // contains __syncthreads
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const uint32_t o_tm = tmem + 128;
    const int *totals = cbase + 2 * ((p.num_seqs + 31) >> 5);
    const int total = totals[0], units = total + p.end_tiles * totals[1];
    const int C = min((int)gridDim.x, max(total, 1));
    const int R0 = q8_range_begin(blockIdx.x, C, total, units, p, cbase, lane);
    const int R1 = q8_range_begin(blockIdx.x + 1, C, total, units, p, cbase, lane);
    const int nk = R1 - R0;
    const uint64_t lim = p.wait_ns;
    // Whole warp: true once the phase is complete; false when another warp has
    // given up or the bounded wait ran out.
    auto ready = [&](uint32_t bar, uint32_t parity) -> bool {
        if (__all_sync(kFull, ptx::mbar_test_wait(bar, parity)))
            return true;
        if (__any_sync(kFull, *abort_flag != 0))
            return false;
        return __all_sync(kFull, ptx::mbar_wait_bounded(bar, parity, lim));
    };
    // One thread: counts this CTA's piece of the cut segment [segS, segE), the
    // ord-th of the batch, in; whoever completes the count owes the merge.
    auto arrive_piece = [&](int segS, int segE, int ord, int b, int hg) {
        if (p.merge_later)
            return;
        const int before = p.end_tiles * ord;
        const int x0 = cta_of(segS + before, C, units);
        const int np = cta_of(segE - 1 + before, C, units) - x0 + 1;
        if (segment_arrive(p.counters + (int64_t)x0 * kLineWords, p.epoch) == np)
            pend_s[segS >= R0 ? 0 : 1] = make_int4(x0, np, b, hg);
    };
    auto give_up = [&]() {
        if (lane == 0) {
            report(p.dev_status, PA_DEV_WAIT_TIMEOUT);
            *abort_flag = 1;
        }
        __syncwarp();
    };

    if (warp == W_K || warp == W_V) {
        // ============================================== TMA and block scales
        // A tile of K (or V) comes as boxes of 16 or 32 tokens of one head.
        // Lane l serves box l % nb of tile l / nb of a batch of 32 / nb tiles;
        // a batch's block ids are fetched one batch ahead.
        const bool is_k = warp == W_K;
        const int nb_log2 = 7 - p.box_log2, nb = 1 << nb_log2;
        const int box = lane & (nb - 1), slot = lane >> nb_log2, batch = 32 >> nb_log2;
        const int row0 = box << p.box_log2;              // first row of the box in the tile
        const int bw = row0 >> 5;                        // its softmax warp
        const int bhead = bw >> sub_log2;
        const int btok = ((bw & ((1 << sub_log2) - 1)) << 5) + (row0 & 31);
        const uint32_t full = is_k ? kfull : vfull, empty = is_k ? kempty : vempty;
        const void *tmap = is_k ? static_cast<const void *>(&tmap_k)
                                : static_cast<const void *>(&tmap_v);
        struct Batch {
            int b, hg, j, ns, n, seg, id;
            bool active;
        };
        bool ok = true;
        int issued = 0;
        if (nk > 0) {
            if (lane == 0)
                ptx::prefetch_tensormap(tmap);
            const uint64_t policy = ptx::policy_evict_first();
            Q8Walk w = q8_walk_at(R0, 0, p, cbase, lane);
            int seg = 0;
            auto fill = [&](int g) {
                Batch d = {0, 0, 0, 1, 0, 0, -1, false};
                int t0 = 0;
#pragma unroll 1
                for (int i = 0; i < batch; ++i) {
                    if (g + i >= R1)
                        break;
                    if (g + i >= w.g0 + w.nt) {
                        q8_walk_next(w, p, lane);
                        ++seg;
                    }
                    if (slot == i) {
                        d.b = w.b;
                        d.hg = w.hg;
                        d.j = g + i - w.g0;
                        d.ns = w.nt;
                        d.seg = seg;
                        t0 = d.j << p.tt_log2;
                        d.n = min(tt, w.ctx - t0);
                        d.active = btok < d.n;
                    }
                }
                // one load for the whole batch, waited for by its first use
                if (d.active)
                    d.id = __ldg(p.block_tables + (int64_t)d.b * p.max_blocks +
                                 ((t0 + btok) >> p.bs_log2));
                return d;
            };
            Batch cur = fill(R0), nxt;
            for (int k0 = 0; ok && k0 < nk; k0 += batch, cur = nxt) {
                const bool valid = cur.active && cur.id >= 0 && (int64_t)cur.id < p.num_blocks;
                const int head = cur.hg * hpc + bhead;
                float ks = 0.f, vs = 0.f;
                if (valid && !is_k) {
                    const int64_t at = (int64_t)cur.id * p.num_kv_heads + head;
                    ks = __ldcg(p.k_scales + at);
                    vs = __ldcg(p.v_scales + at);
                }
                const unsigned vmask = __ballot_sync(kFull, valid);
                const unsigned bmask = __ballot_sync(kFull, cur.active && !valid);
                for (int i = 0; i < batch && k0 + i < nk; ++i) {
                    const int k = k0 + i, s = k % S;
                    if (__any_sync(kFull, *abort_flag != 0))
                        break;
                    if (k >= S &&
                        !__all_sync(kFull, ptx::mbar_wait_bounded(empty + 8 * s,
                                                                  (uint32_t)((k / S - 1) & 1),
                                                                  lim))) {
                        ok = false;
                        break;
                    }
                    // test hook: this CTA's second tile is never copied
                    const bool withhold = (int)blockIdx.x == p.withhold_cta && k == 1;
                    const int mine = __popc((vmask >> (i << nb_log2)) & ((1u << nb) - 1));
                    if (lane == 0)
                        ptx::mbar_expect_tx(full + 8 * s, (uint32_t)(mine << p.box_log2) * D);
                    __syncwarp();
                    if (slot == i && valid && !withhold) {
                        const int t0 = (cur.j << p.tt_log2) + btok;
                        const int row = cur.id * p.block_size + (t0 & (p.block_size - 1));
                        ptx::tma_load_5d(base + (uint32_t)((is_k ? 0 : L::v_off) + s * L::kStage +
                                                           row0 * D),
                                         tmap, 0, 0, 0, row >> 3, head, full + 8 * s, policy);
                    }
                    if (is_k) {
                        if (slot == i && box == 0)
                            kflag[s] = (cur.j == 0 || k == 0 ? 1 : 0) |
                                       (cur.j == cur.ns - 1 || k == nk - 1 ? 2 : 0);
                    } else {
                        if (slot == i) {
                            Q8Meta &m = meta[s];
                            if (box == 0) {
                                m.b = cur.b;
                                m.hg = cur.hg;
                                m.j = cur.j;
                                m.ns = cur.ns;
                                m.n = cur.n;
                                m.seg = cur.seg;
                                m.bad = ((bmask >> (i << nb_log2)) & ((1u << nb) - 1)) != 0;
                            }
                            m.ks[row0 >> 4] = ks;
                            m.vs[row0 >> 4] = vs;
                            if (p.box_log2 == 5) {
                                m.ks[(row0 >> 4) + 1] = ks;
                                m.vs[(row0 >> 4) + 1] = vs;
                            }
                        }
                    }
                    __syncwarp();
                    // (the arrivals release the flags, the metadata and the scales)
                    if (lane == 0) {
                        if (!is_k)
                            ptx::mbar_arrive(mfull + 8 * s);
                        ptx::mbar_arrive(full + 8 * s);
                    }
                    issued = k + 1;
                    if (i == 0)
                        nxt = fill(R0 + k0 + batch);
                }
                if (issued < min(k0 + batch, nk))
                    break;
            }
        }
        if (!ok)
            give_up();
        if (issued < nk) {
            // given up: let the copies in flight land before the CTA ends
            for (int k = max(0, issued - S); k < issued; ++k)
                ptx::mbar_wait_bounded(full + 8 * (k % S), (uint32_t)((k / S) & 1), lim);
        }
        __syncwarp();
    } else if (warp == W_S) {
        // ============================================================== S
        const uint32_t idesc = ptx::umma_idesc_f8(128, max(16, 2 * G * hpc), false, false, false,
                                                  false);
        bool ok = true;
        int seg = 0;
        for (int k = 0; k < nk; ++k) {
            const int s = k % S, qb = seg % QB;
            if (!(ok = ready(kfull + 8 * s, (uint32_t)((k / S) & 1))))
                break;
            const int flags = kflag[s];
            if ((flags & 1) && !(ok = ready(qfull + 8 * qb, (uint32_t)((seg / QB) & 1))))
                break;
            if (k >= 2 && !(ok = ready(sfree + 8 * (k & 1), (uint32_t)(((k >> 1) - 1) & 1))))
                break;
            ptx::tc_fence_after();
            const uint64_t ad = ptx::umma_desc_sw128(base + (uint32_t)(s * L::kStage), 16, GROUP);
            const uint64_t bd = ptx::umma_desc_sw128(
                base + (uint32_t)(L::q_off + qb * L::kQRows * D), 16, GROUP);
            if (ptx::elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk) {
                    const uint64_t off = (uint64_t)(((kk >> 2) * 1024 + (kk & 3) * 32) >> 4);
                    ptx::umma_f8_ss(tmem + (uint32_t)((k & 1) * 64), ad + off, bd + off, idesc,
                                    kk > 0);
                }
                ptx::umma_commit(sfull + 8 * (k & 1));
                ptx::umma_commit(kempty + 8 * s);
                if (flags & 2)
                    ptx::umma_commit(qempty + 8 * qb);
                // (passes on the query factors, seen with qfull)
                ptx::mbar_arrive(sfull + 8 * (k & 1));
            }
            __syncwarp();
            seg += flags >> 1;
        }
        if (!ok) {
            give_up();
            // products already issued finish before the memory goes
            if (ptx::elect_one())
                ptx::umma_commit(drain_s);
            __syncwarp();
            ptx::mbar_wait_bounded(drain_s, 0, lim);
        }
        __syncwarp();
    } else if (warp == W_O) {
        // ============================================================ O^T
        constexpr uint32_t idesc = ptx::umma_idesc_f8(128, NP, false, true, true, true);
        bool ok = true;
        for (int k = 0; k < nk; ++k) {
            const int s = k % S;
            if (!(ok = ready(mfull + 8 * s, (uint32_t)((k / S) & 1))))
                break;
            const int j = meta[s].j, seg = meta[s].seg;
            // a new segment: the epilogue of the one before has read O
            if ((j == 0 || k == 0) && seg > 0 &&
                !(ok = ready(ofree, (uint32_t)((seg - 1) & 1))))
                break;
            if (!(ok = ready(vfull + 8 * s, (uint32_t)((k / S) & 1)) &&
                       ready(pready + 8 * (k & 1), (uint32_t)((k >> 1) & 1))))
                break;
            ptx::tc_fence_after();
            const uint32_t vst = base + (uint32_t)(L::v_off + s * L::kStage);
            const uint32_t pst = base + (uint32_t)(L::p_off + (k & 1) * 4 * L::kP);
            const uint32_t acc = o_tm + (uint32_t)((k % SETS) * L::o_cols);
            const bool add = j >= SETS && k >= SETS;     // not the set's first tile
            if (ptx::elect_one()) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint64_t bd = ptx::umma_desc_plain(pst + w * L::kP, 128, 512);
#pragma unroll
                    for (int h = 0; h < HALVES; ++h)
                        ptx::umma_f8_ss(acc + (uint32_t)((w * HALVES + h) * NP),
                                        ptx::umma_desc_sw128(vst + w * 32 * D + h * 1024, 1024,
                                                             GROUP),
                                        bd, idesc, add);
                }
                ptx::umma_commit(vempty + 8 * s);
                ptx::umma_commit(pvdone + 8 * (k & 1));
            }
            __syncwarp();
        }
        if (!ok) {
            give_up();
            if (ptx::elect_one())
                ptx::umma_commit(drain_o);
            __syncwarp();
            ptx::mbar_wait_bounded(drain_o, 0, lim);
        }
        __syncwarp();
    } else if (warp >= W_Q) {
        // ====================================================== query rows
        // Row (h, g) of a segment is scaled by a power of two (largest
        // element in [128, 256)) and split into hi = e4m3(y) and
        // lo = e4m3(y - hi), as over the per-tensor FP8 cache; they become
        // rows (2 h) G + g and (2 h + 1) G + g of the B operand.
        bool ok = true;
        if (nk > 0) {
            constexpr int E = D / 32;                    // elements per lane
            Q8Walk w = q8_walk_at(R0, 0, p, cbase, lane);
            for (int seg = 0; w.g0 < R1; ++seg) {
                const int qb = seg % QB;
                if (__any_sync(kFull, *abort_flag != 0))
                    break;
                const int rows = hpc * G;
                const __nv_bfloat16 *src = p.q + ((int64_t)w.b * p.num_q_heads +
                                                  (int64_t)w.hg * rows) * D;
                constexpr int RW = G;                    // rows per warp, at most
                constexpr int RB = RW < 4 ? RW : 4;      // rows loaded at once
                bool free = seg < QB;
#pragma unroll 1
                for (int r0 = 0; r0 < RW; r0 += RB) {
                    uint32_t x[RB][E / 2];
#pragma unroll
                    for (int i = 0; i < RB; ++i) {
                        const int r = 4 * (r0 + i) + (warp - W_Q);
#pragma unroll
                        for (int e = 0; e < E / 2; ++e)
                            x[i][e] = 0;
                        if (r < rows) {
                            if constexpr (E == 8) {
                                const uint4 v = __ldg(
                                    reinterpret_cast<const uint4 *>(src + (int64_t)r * D) + lane);
                                x[i][0] = v.x;
                                x[i][1] = v.y;
                                x[i][2] = v.z;
                                x[i][3] = v.w;
                            } else {
                                const uint2 v = __ldg(
                                    reinterpret_cast<const uint2 *>(src + (int64_t)r * D) + lane);
                                x[i][0] = v.x;
                                x[i][1] = v.y;
                            }
                        }
                    }
                    if (!free) {
                        if (!__all_sync(kFull, ptx::mbar_wait_bounded(
                                                   qempty + 8 * qb,
                                                   (uint32_t)((seg / QB - 1) & 1), lim))) {
                            ok = false;
                            break;
                        }
                        free = true;
                    }
                    const uint32_t qst = base + (uint32_t)(L::q_off + qb * L::kQRows * D);
#pragma unroll
                    for (int i = 0; i < RB; ++i) {
                        const int r = 4 * (r0 + i) + (warp - W_Q);
                        if (r >= rows)
                            continue;
                        uint32_t top = 0;
#pragma unroll
                        for (int e = 0; e < E / 2; ++e)
                            top = max(top, max(x[i][e] << 16 & 0x7fffffffu, x[i][e] & 0x7fff0000u));
                        top = __reduce_max_sync(kFull, top);
                        const int ef = (int)(top >> 23);
                        const float sigma = __uint_as_float((uint32_t)min(254, 261 - ef) << 23);
                        uint32_t hi[E / 4], lo[E / 4];
#pragma unroll
                        for (int e = 0; e < E / 4; ++e) {
                            uint32_t h2[2], l2[2];
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                // (8 bits of a value below 256: exact in f16 but
                                // far below E4M3's quantum, and so is what is left)
                                const uint32_t y =
                                    ptx::pack_f16x2(ptx::bf16lo_to_f32(x[i][2 * e + k]) * sigma,
                                                    ptx::bf16hi_to_f32(x[i][2 * e + k]) * sigma);
                                h2[k] = f16x2_to_e4m3x2(y);
                                l2[k] = f16x2_to_e4m3x2(
                                    ptx::sub_f16x2(y, e4m3x2_to_f16x2(h2[k])));
                            }
                            hi[e] = h2[0] | (h2[1] << 16);
                            lo[e] = l2[0] | (l2[1] << 16);
                        }
                        const int h = r / G, g = r - h * G;
                        const int byte = lane * E;       // within the row
                        auto at = [&](int n) {
                            return qst + (uint32_t)((n >> 3) * GROUP + (byte >> 7) * 1024 +
                                                    (n & 7) * 128 +
                                                    ((((byte & 127) >> 4) ^ (n & 7)) << 4) +
                                                    (byte & 15));
                        };
                        const uint32_t ah = at(2 * h * G + g), al = at((2 * h + 1) * G + g);
                        if constexpr (E == 8) {
                            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(ah), "r"(hi[0]),
                                         "r"(hi[E / 4 - 1])
                                         : "memory");
                            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(al), "r"(lo[0]),
                                         "r"(lo[E / 4 - 1])
                                         : "memory");
                        } else {
                            asm volatile("st.shared.u32 [%0], %1;" ::"r"(ah), "r"(hi[0]) : "memory");
                            asm volatile("st.shared.u32 [%0], %1;" ::"r"(al), "r"(lo[0]) : "memory");
                        }
                        // A row with a non-finite element gives NaN logits.
                        // (Four segments' factors are kept: the buffer of
                        // segment seg is free, so S of an earlier one's last
                        // tile is done, and every tile but the two before it
                        // has been read with its factors.)
                        if (lane == 0)
                            sf[(seg & 3) * 4 * G + r] = ef < 255 ? p.scale_log2 / sigma
                                                                 : __int_as_float(0x7fc00000);
                    }
                }
                if (!ok)
                    break;
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    ptx::mbar_arrive(qfull + 8 * qb);
                if (w.g0 + w.nt >= R1)
                    break;
                q8_walk_next(w, p, lane);
            }
        }
        if (!ok)
            give_up();
    } else {
        // ================================================ softmax, epilogue
        const int set = warp >> 2, w4 = warp & 3, st = tid & 127;
        const int rows = hpc * G;
        // this CTA's counter starts the call at (epoch, 0), unless an arrival
        // has already counted in it
        if (p.mode == 0 && !p.merge_later && tid == 0)
            ptx::red_max_relaxed_gpu_u64(p.counters + (int64_t)blockIdx.x * kLineWords,
                                         (unsigned long long)p.epoch << 32);
        for (int b = blockIdx.x; set == 0 && b < p.num_seqs; b += gridDim.x) {
            const int len = q8_len(b, p);
            if (eff_ctx(len, p.ctx_cap) > 0)
                continue;
            if (len != 0 && tid == 0)
                report(p.dev_status, PA_DEV_BAD_CONTEXT);
            uint32_t *o = reinterpret_cast<uint32_t *>(p.out + (int64_t)b * p.num_q_heads * D);
            for (int i = tid; i < p.num_q_heads * D / 2; i += 128)
                o[i] = 0;
        }
        const int hl = w4 >> sub_log2;                    // this warp's head of the group
        const int tok0 = (w4 & ((1 << sub_log2) - 1)) << 5, tok = tok0 + lane;
        const uint32_t lane_tm = (uint32_t)(w4 * 32) << 16;
        const uint32_t acc_tm = o_tm + (uint32_t)(set * L::o_cols) + lane_tm;
        const int bar0 = 1 + 2 * set;
        float m[G], l[G], fac[G];
        bool fail = false, seg_bad = false;
        int exchanges = 0;
        const int ord0 = nk > 0 ? q8_walk_at(R0, 0, p, cbase, lane).ord : 0;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            if (!fail && !ready(bar, parity)) {
                fail = true;
                give_up();
            }
        };
        // Each iteration holds a barrier of the set's four warps, also for a
        // warp whose wait ran out; only what a barrier says ends the loop, so
        // that all four leave it together.
        for (int k = set; k < nk; k += SETS) {
            const int s = k % S;
            wait(sfull + 8 * (k & 1), (uint32_t)((k >> 1) & 1));
            wait(mfull + 8 * s, (uint32_t)((k / S) & 1));
            bool first = false, over = false;
            int n = 0, j = 0, seg = 0;
            float t[G], room = 0.f, lv = 0.f, vs = 0.f;
            bool seen = false;
            if (!fail) {
                n = meta[s].n;
                j = meta[s].j;
                seg = meta[s].seg;
                const int box = 2 * w4 + (lane >> 4);
                const float ks = meta[s].ks[box];
                vs = meta[s].vs[box];
                first = j < SETS || k < SETS;
                if (first) {
                    seg_bad = false;
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        fac[g] = sf[(seg & 3) * 4 * G + hl * G + g];
                        l[g] = 0.f;
                    }
                }
                seg_bad |= meta[s].bad != 0;
                ptx::tc_fence_after();
                uint32_t u[2 * G];
                ptx::tmem_ld<2 * G>(tmem + (uint32_t)((k & 1) * 64 + hl * 2 * G) + lane_tm, u);
                lv = fmaxf(ptx::lg2(vs), -64.f);
                room = kQ8Grow + kQ8Bias - lv;
                seen = tok < n;
                ptx::tmem_wait_ld();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    ptx::mbar_arrive(sfree + 8 * (k & 1));
                ptx::tmem_hold<2 * G>(u);
#pragma unroll
                for (int g = 0; g < G; ++g)
                    t[g] = (__uint_as_float(u[g]) + __uint_as_float(u[G + g])) * (fac[g] * ks);
                if (first) {
#pragma unroll
                    for (int g = 0; g < G; ++g)
                        m[g] = ptx::warp_max(seen ? t[g] + lv : -INFINITY) - kQ8Bias;
                }
                // (a warp without tokens so far has m = -inf: any token is over)
                float top = t[0] - m[0];
#pragma unroll
                for (int g = 1; g < G; ++g)
                    top = fmaxf(top, t[g] - m[g]);
                over = seen && top > room;
            }
            if (ptx::barrier_or(bar0, 128, over || fail)) {
                if (ptx::barrier_or(bar0 + 1, 128, fail))
                    break;
                // some lane of the set is past its reference: new references
                bool scale_o = false;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float mx = ptx::warp_max(seen ? t[g] + lv : -INFINITY) - kQ8Bias;
                    float al = 1.f;
                    if (mx > m[g] + kQ8Grow) {
                        // (from -inf there is nothing to rescale)
                        if (m[g] != -INFINITY) {
                            // (the sum may take a factor below the normal numbers)
                            const float root = ptx::ex2(0.5f * (m[g] - mx));
                            l[g] = l[g] * root * root;
                            al = root * root;
                            scale_o = true;
                        }
                        m[g] = mx;
                    }
                    if (lane == 0)
                        alpha_s[(set * 4 + w4) * G + g] = al;
                }
                if (ptx::barrier_or(bar0, 128, scale_o)) {
                    // the set's accumulators, once its product before is in
                    wait(pvdone + 8 * ((k - SETS) & 1), (uint32_t)(((k - SETS) >> 1) & 1));
                    ptx::tc_fence_after();
#pragma unroll 1
                    for (int w = 0; w < 4 && !fail; ++w) {
                        float al[G];
                        bool any = false;
#pragma unroll
                        for (int g = 0; g < G; ++g) {
                            al[g] = alpha_s[(set * 4 + w) * G + g];
                            any |= al[g] != 1.f;
                        }
                        if (!any)
                            continue;
#pragma unroll 1
                        for (int c = 0; c < HALVES * (NP / 16); ++c) {
                            const uint32_t at = acc_tm + (uint32_t)(w * HALVES * NP + c * 16);
                            uint32_t u[16];
                            ptx::tmem_ld16(at, u);
                            ptx::tmem_wait_ld();
                            ptx::tmem_hold16(u);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                u[i] = __float_as_uint(__uint_as_float(u[i]) *
                                                       ((i & (GP - 1)) < G ? al[(i & (GP - 1)) % G]
                                                                           : 1.f));
                            ptx::tmem_st16(at, u);
                        }
                        ptx::tmem_wait_st();
                    }
                    ptx::tc_fence_before();
                }
            }
            // weights of tile k - 2 have been used
            if (k >= 2)
                wait(pvdone + 8 * (k & 1), (uint32_t)(((k >> 1) - 1) & 1));
            const int nv = min(max(n - tok0, 0), 32);
            if (nv < 32)
                wait(vfull + 8 * s, (uint32_t)((k / S) & 1));
            if (!fail) {
                const uint32_t pw = base + (uint32_t)(L::p_off + ((k & 1) * 4 + w4) * L::kP +
                                                      (lane >> 3) * 128 + (lane & 7) * 16);
                float x[2 * ((G + 1) / 2)];
                const float vsx = seen ? vs * 0x1p-24f : 0.f;     // (2^-kQ8Bias)
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float e = ptx::ex2(seen ? t[g] - m[g] : -INFINITY);
                    l[g] += e;
                    x[g] = e * vsx;
                }
                if constexpr (G % 2)
                    x[G] = 0.f;
                uint32_t word[3][GP / 4];                 // part, four heads
#pragma unroll
                for (int q = 0; q < GP / 4; ++q)
                    word[0][q] = word[1][q] = word[2][q] = 0;
#pragma unroll
                for (int g = 0; g < G; g += 2) {
                    float x0 = x[g], x1 = x[g + 1];
#pragma unroll
                    for (int part = 0; part < 3; ++part) {
                        const uint32_t c = e5m2x2(x0, x1);
                        word[part][g / 4] |= c << (8 * (g & 3));
                        if (part < 2) {
                            // what is left, exactly, times 8 (a code is the
                            // upper byte of its f16)
                            const uint32_t f = ptx::prmt(c, 0, 0x1404);
                            x0 = (x0 - ptx::f16lo_to_f32(f)) * 8.f;
                            x1 = (x1 - ptx::f16hi_to_f32(f)) * 8.f;
                        }
                    }
                }
                auto put = [&](uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a),
                                 "r"(b), "r"(c), "r"(d)
                                 : "memory");
                };
                if constexpr (GP == 4) {
                    put(pw, word[0][0], word[1][0], word[2][0], 0);
                } else {
                    put(pw, word[0][0], word[0][GP / 4 - 1], word[1][0], word[1][GP / 4 - 1]);
                    put(pw + 512, word[2][0], word[2][GP / 4 - 1], 0, 0);
                }
                if (nv < 32) {
                    // V rows past the sequence hold whatever was there; their
                    // weight is 0, but 0 * NaN is NaN
                    const uint32_t vst = base + (uint32_t)(L::v_off + s * L::kStage + w4 * 32 * D);
#pragma unroll 1
                    for (int i = lane; i < (32 - nv) * (D / 16); i += 32) {
                        const int r = nv + i / (D / 16), c = i % (D / 16);
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                         vst + (uint32_t)((r >> 3) * GROUP + (c >> 3) * 1024 +
                                                          (r & 7) * 128 + (c & 7) * 16)),
                                     "r"(0)
                                     : "memory");
                    }
                }
                ptx::fence_proxy_async_smem();
            }
            const int ns = meta[s].ns, mb = meta[s].b, mhg = meta[s].hg;
            __syncwarp();
            if (!fail && lane == 0)
                ptx::mbar_arrive(pready + 8 * (k & 1));
            // the set's last tile of the segment's share of this range?
            const int left = min(ns - 1 - j, nk - 1 - k);     // tiles of the share after this
            if (left >= SETS)
                continue;
            const int share = min(j, k) + 1 + left;           // tiles of the share
            float *my = stat + ((seg & 1) * SETS + set) * 4 * 2 * G;
#pragma unroll
            for (int g = 0; g < G; ++g) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    l[g] += __shfl_xor_sync(kFull, l[g], o);
                if (lane == 0) {
                    my[w4 * 2 * G + g] = m[g];
                    my[w4 * 2 * G + G + g] = l[g] * 0x1p-24f;     // (as the weights)
                }
            }
            if (SETS > 1 && share > 1) {
                // (two barriers in turn: a set may hand over once more before
                // the other has taken the last one, but not twice, since its
                // second tile from then needs the accumulators)
                ++exchanges;
                if (left > 0) {
                    // the other set has the segment's last tile and joins both
                    // (a bad block of this set's tiles: marked in its sums)
                    if (seg_bad && lane == 0)
                        my[w4 * 2 * G + G] = -1.f;
                    __syncwarp();
                    if (lane == 0)
                        ptx::mbar_arrive(xstat + 8 * (exchanges & 1));
                    continue;
                }
                wait(xstat + 8 * (exchanges & 1), (uint32_t)(((exchanges - 1) >> 1) & 1));
            }
            // ---- the segment's share of this range is complete
            wait(pvdone + 8 * (k & 1), (uint32_t)((k >> 1) & 1));
            if (ptx::barrier_or(bar0, 128, fail)) {
                fail = true;
                break;
            }
            ptx::tc_fence_after();
            const int segS = R0 + k - j, segE = segS + ns;
            const bool complete = segS >= R0 && segE <= R1;
            float *ps = p.pieces + (int64_t)(2 * blockIdx.x + (segS >= R0 ? 1 : 0)) * p.slot_floats;
            const int nsets = share > 1 ? SETS : 1, e0 = share > 1 ? 0 : set;
            const float *both = stat + (seg & 1) * SETS * 4 * 2 * G;
            // Factors of this warp's accumulators in each set: 2^(m - M) over
            // the head row's sets and warps, over the sum when the segment is
            // complete.  Lane (and lane + 32) holds item x * G + g: head row g
            // in the x-th of the head's nx accumulators.
            const int nx = nsets << sub_log2, w0 = hl << sub_log2;
            float mi[2], li[2], fi[2], M = -INFINITY, sum = 0.f;
            bool marked = false;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int x = (lane + 32 * q) / G, g = lane % G;
                const int e = e0 + (x >> sub_log2), w = w0 + (x & ((1 << sub_log2) - 1));
                mi[q] = -INFINITY;
                li[q] = 0.f;
                if (x < nx) {
                    mi[q] = both[(e * 4 + w) * 2 * G + g];
                    li[q] = both[(e * 4 + w) * 2 * G + G + g];
                }
                marked |= li[q] == -1.f;
                M = fmaxf(M, mi[q]);
            }
            seg_bad |= __any_sync(kFull, marked);
#pragma unroll
            for (int o = G; o < 32; o <<= 1)
                M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                fi[q] = mi[q] == -INFINITY ? 0.f : ptx::ex2(mi[q] - M);
                // (what V scales far apart leave of an accumulator can vanish
                // next to another's, its sum cannot)
                sum += mi[q] == -INFINITY ? 0.f : ptx::times_2_to(li[q], mi[q] - M);
            }
#pragma unroll
            for (int o = G; o < 32; o <<= 1)
                sum += __shfl_xor_sync(kFull, sum, o);
            const float inv = !complete ? 1.f : (sum == 0.f ? 0.f : __frcp_rn(sum));
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int x = (lane + 32 * q) / G;
                const int e = e0 + (x >> sub_log2), w = w0 + (x & ((1 << sub_log2) - 1));
                if (x < nx && w == w4)
                    fac_s[(e * 4 + w) * G + lane % G] = fi[q] * inv;
            }
            if (!complete && w0 == w4 && lane < G)
                *reinterpret_cast<float2 *>(ps + rows * D + 2 * (hl * G + lane)) =
                    make_float2(M, sum);
            if (ptx::barrier_or(bar0, 128, false))
                break;                                        // (never: orders the factors)
            __nv_bfloat16 *oc = p.out + ((int64_t)mb * p.num_q_heads + (int64_t)mhg * rows) * D +
                                w4 * 32 + lane;
            float *op = ps + w4 * 32 + lane;
#pragma unroll 1
            for (int h = 0; h < hpc; ++h, oc += G * D, op += G * D) {
                float v[HALVES][G];
#pragma unroll
                for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
                    for (int g = 0; g < G; ++g)
                        v[hf][g] = 0.f;
                // two of the head's accumulators at a time (one, where that
                // would take 128 registers), all loads in flight
                constexpr int Y = HALVES * NP <= 32 ? 2 : 1;
                const int count = nsets << sub_log2;
#pragma unroll 1
                for (int x = 0; x < count; x += Y) {
                    uint32_t u[Y][HALVES][NP];
                    float f[Y][G];
#pragma unroll
                    for (int y = 0; y < Y; ++y) {
                        const int xx = x + y < count ? x + y : x;
                        const int e = e0 + (xx >> sub_log2);
                        const int w = (h << sub_log2) + (xx & ((1 << sub_log2) - 1));
                        const uint32_t at =
                            o_tm + lane_tm + (uint32_t)(e * L::o_cols + w * HALVES * NP);
                        // (an odd last one is loaded twice and counted once)
#pragma unroll
                        for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
                            for (int c = 0; c < NP / 16; ++c)
                                ptx::tmem_ld16(
                                    at + (uint32_t)(hf * NP + 16 * c),
                                    *reinterpret_cast<uint32_t(*)[16]>(&u[y][hf][16 * c]));
#pragma unroll
                        for (int g = 0; g < G; ++g)
                            f[y][g] = x + y < count ? fac_s[(e * 4 + w) * G + g] : 0.f;
                    }
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int y = 0; y < Y; ++y)
#pragma unroll
                        for (int hf = 0; hf < HALVES; ++hf) {
                            ptx::tmem_hold<NP>(u[y][hf]);
#pragma unroll
                            for (int g = 0; g < G; ++g)
                                v[hf][g] += f[y][g] *
                                            fmaf(fmaf(__uint_as_float(u[y][hf][2 * GP + g]), 0.125f,
                                                      __uint_as_float(u[y][hf][GP + g])),
                                                 0.125f, __uint_as_float(u[y][hf][g]));
                        }
                }
                if (complete) {
#pragma unroll
                    for (int g = 0; g < G; ++g)
#pragma unroll
                        for (int hf = 0; hf < HALVES; ++hf)
                            oc[g * D + hf * 128] = __float2bfloat16_rn(seg_bad ? 0.f : v[hf][g]);
                } else {
#pragma unroll
                    for (int g = 0; g < G; ++g)
#pragma unroll
                        for (int hf = 0; hf < HALVES; ++hf)
                            op[g * D + hf * 128] = v[hf][g];
                }
            }
            // O may be overwritten
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0)
                ptx::mbar_arrive(ofree);
            if (!complete) {
                if (st == 0)
                    ps[rows * D + 2 * rows] = seg_bad ? 1.f : 0.f;
                // the set's stores, then the arrival that releases them
                if (ptx::barrier_or(bar0, 128, false))
                    break;                                    // (never)
                if (st == 0)
                    arrive_piece(segS, segE, ord0 + seg, mb, mhg);
            } else if (seg_bad && st == 0) {
                report(p.dev_status, PA_DEV_BAD_BLOCK);
            }
            // (the other set may be past its next segment already)
            if (st == 0)
                atomicMax(tiles_done, k + 1);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == W_S)
        ptx::tmem_dealloc(tmem, L::tmem_cols);
    if (nk > 0 && *tiles_done < nk) {
        // a wait ran out: zeros for the segments that are not complete, and a
        // mark in their pieces
        const int rows = hpc * G;
        Q8Walk w = q8_walk_at(R0 + *tiles_done, 0, p, cbase, lane);
        while (true) {
            const int segE = w.g0 + w.nt;
            if (w.g0 >= R0 && segE <= R1) {
                __nv_bfloat16 *o = p.out + ((int64_t)w.b * p.num_q_heads + (int64_t)w.hg * rows) * D;
                for (int i = tid; i < rows * D; i += L::kThreads)
                    o[i] = __float2bfloat16_rn(0.f);
            } else if (tid == 0) {
                float *ps = p.pieces + (int64_t)(2 * blockIdx.x + (w.g0 >= R0 ? 1 : 0)) * p.slot_floats;
                ps[rows * D + 2 * rows] = 2.f;
                arrive_piece(w.g0, segE, w.ord, w.b, w.hg);
            }
            if (segE >= R1)
                break;
            q8_walk_next(w, p, lane);
        }
        __syncthreads();
    }
    // ---- the merges this CTA owes, all its threads:
    //   M = max_i m_i,  L = sum_i l_i 2^(m_i - M),  o = sum_i a_i 2^(m_i - M) / L
    // over the pieces i, in piece order, so that the result does not depend on
    // which arrival was the last.
    float *wt = reinterpret_cast<float *>(gen + L::q_off);        // [pieces][rows]
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const int4 pend = pend_s[i];
        const int x0 = pend.x, np = pend.y;
        if (np == 0)
            continue;
        const int rows = hpc * G;
        const float *first = p.pieces + (int64_t)2 * x0 * p.slot_floats;
        auto piece = [&](int c) {                        // slots 2 x0 + 1, then 2 (x0 + c)
            return first + (int64_t)(c == 0 ? 1 : 2 * c) * p.slot_floats;
        };
        float flag = 0.f;
        for (int c = tid; c < np; c += L::kThreads)
            flag = fmaxf(flag, __ldcg(piece(c) + rows * D + 2 * rows));
#pragma unroll 1
        for (int r = warp; r < rows; r += L::kThreads / 32) {
            const int at = rows * D + 2 * r;
            // (up to 32 pieces: loaded once)
            float2 ml = make_float2(-INFINITY, 0.f);
            if (lane < np)
                ml = __ldcg(reinterpret_cast<const float2 *>(piece(lane) + at));
            float M = ml.x, sum = 0.f;
            for (int c = lane + 32; c < np; c += 32)
                M = fmaxf(M, __ldcg(piece(c) + at));
            M = ptx::warp_max(M);
            for (int c = lane; c < np; c += 32) {
                if (c >= 32)
                    ml = __ldcg(reinterpret_cast<const float2 *>(piece(c) + at));
                const float f = ml.x == -INFINITY ? 0.f : ptx::ex2(ml.x - M);
                wt[c * rows + r] = f;
                if (ml.x != -INFINITY)
                    sum += ptx::times_2_to(ml.y, ml.x - M);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                sum += __shfl_xor_sync(kFull, sum, o);
            const float inv = sum == 0.f ? 0.f : __frcp_rn(sum);
            for (int c = lane; c < np; c += 32)
                wt[c * rows + r] *= inv;
        }
        const bool bad = __syncthreads_or(flag != 0.f);  // (also: the weights are in place)
        if (flag == 1.f)
            report(p.dev_status, PA_DEV_BAD_BLOCK);
        __nv_bfloat16 *o = p.out + ((int64_t)pend.z * p.num_q_heads + (int64_t)pend.w * rows) * D;
        // two float4s per thread at a time, eight pieces of each in flight
        const int units = rows * D / 4;
#pragma unroll 1
        for (int u = tid; u < units; u += 2 * L::kThreads) {
            const int u2 = u + L::kThreads < units ? u + L::kThreads : u;
            const int ra = u / (D / 4), rb = u2 / (D / 4);
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
            const float *src = piece(0);
            if (!bad) {
#pragma unroll 8
                for (int c = 0; c < np; ++c) {
                    const float4 va = __ldcg(reinterpret_cast<const float4 *>(src) + u);
                    const float4 vb = __ldcg(reinterpret_cast<const float4 *>(src) + u2);
                    src = first + (int64_t)2 * (c + 1) * p.slot_floats;
                    const float fa = wt[c * rows + ra], fb = wt[c * rows + rb];
                    a.x = fmaf(va.x, fa, a.x);
                    a.y = fmaf(va.y, fa, a.y);
                    a.z = fmaf(va.z, fa, a.z);
                    a.w = fmaf(va.w, fa, a.w);
                    b.x = fmaf(vb.x, fb, b.x);
                    b.y = fmaf(vb.y, fb, b.y);
                    b.z = fmaf(vb.z, fb, b.z);
                    b.w = fmaf(vb.w, fb, b.w);
                }
            }
            store4(o + 4 * u, a);
            if (u2 != u)
                store4(o + 4 * u2, b);
        }
        // the count starts again from nothing, whatever tag the next call has
        if (tid == 0)
            ptx::st_relaxed_gpu_u64(p.counters + (int64_t)x0 * kLineWords, 0);
        __syncthreads();
    }
}

constexpr int kQ8MaxCtas = 148;   // (a merge's weights have room for so many pieces)

// Joins the pieces of every cut segment of a batch of at most 32 sequences:
// CTA (segment, head, part) sums 128 elements of one head row, warp w taking
// pieces w, w + 4, ...  Which pieces a segment has follows from the lengths, so
// that is settled before the decode kernel has completed: this kernel starts
// behind that one's wait, and so behind whatever wrote the lengths.
constexpr int kQ8MergeThreads = 128;

__global__ void __launch_bounds__(kQ8MergeThreads) q8_merge_kernel(const Q8DecodeParams p, int ctas,
                                                                   int G, int D)
{
    constexpr int AHEAD = 6;                             // pieces loaded before their weights
    __shared__ float wt[kQ8MaxCtas];
    __shared__ float4 part_s[3][32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    ptx::grid_launch_dependents();
    const int parts = G * D / 128;
    const int part = blockIdx.x % parts, rest = blockIdx.x / parts;
    const int h = rest % p.hpc, seg = rest / p.hpc;
    const int b = seg / p.head_groups, hg = seg - b * p.head_groups;
    const int nt = q8_tiles(q8_ctx(lane, p), p);
    // units (see q8_range_begin) up to and with sequence `lane`
    const int size = nt > 0 ? (nt + p.end_tiles) * p.head_groups : 0;
    int incl = size, tiles = nt * p.head_groups;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFull, incl, o);
        if (lane >= o)
            incl += v;
        tiles += __shfl_xor_sync(kFull, tiles, o);
    }
    const int units = __shfl_sync(kFull, incl, 31);
    const int mine = __shfl_sync(kFull, nt, b);
    const int s0 = __shfl_sync(kFull, incl - size, b) + hg * (mine + p.end_tiles);
    const int C = min(ctas, max(tiles, 1));
    const int x0 = mine > 0 ? cta_of(s0, C, units) : 0;
    const int np = mine > 0 ? cta_of(s0 + mine - 1, C, units) - x0 + 1 : 1;
    const int rows = p.hpc * G, row = h * G + part * 128 / D;
    const float *first = p.pieces + (int64_t)2 * x0 * p.slot_floats;
    auto piece = [&](int c) {                            // slots 2 x0 + 1, then 2 (x0 + c)
        return first + (int64_t)(c == 0 ? 1 : 2 * c) * p.slot_floats;
    };
    const int off = h * G * D + part * 128 + 4 * lane;   // of this lane's four elements
    ptx::grid_wait_prerequisites();
    if (np == 1)
        return;                                          // whole, or empty: written already
    float4 v[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (warp + 4 * i < np)
            v[i] = __ldcg(reinterpret_cast<const float4 *>(piece(warp + 4 * i) + off));
    // every warp finds the row's maximum and sum; warp w keeps the weights of
    // its own pieces
    const int at = rows * D + 2 * row;
    float2 ml[(kQ8MaxCtas + 31) / 32];
    float M = -INFINITY, sum = 0.f, flag = 0.f;
#pragma unroll
    for (int i = 0; i < (kQ8MaxCtas + 31) / 32; ++i) {
        const int c = lane + 32 * i;
        ml[i] = make_float2(-INFINITY, 0.f);
        if (c < np) {
            ml[i] = __ldcg(reinterpret_cast<const float2 *>(piece(c) + at));
            flag = fmaxf(flag, __ldcg(piece(c) + rows * D + 2 * rows));
        }
        M = fmaxf(M, ml[i].x);
    }
    M = ptx::warp_max(M);
#pragma unroll
    for (int i = 0; i < (kQ8MaxCtas + 31) / 32; ++i) {
        sum += ml[i].x == -INFINITY ? 0.f : ptx::times_2_to(ml[i].y, ml[i].x - M);
        ml[i].x = ml[i].x == -INFINITY ? 0.f : ptx::ex2(ml[i].x - M);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(kFull, sum, o);
    const float inv = sum == 0.f ? 0.f : __frcp_rn(sum);
    const bool bad = __any_sync(kFull, flag != 0.f);
    if (flag == 1.f && h == 0 && part == 0 && warp == 0)
        report(p.dev_status, PA_DEV_BAD_BLOCK);
#pragma unroll
    for (int i = 0; i < (kQ8MaxCtas + 31) / 32; ++i)
        if (lane + 32 * i < np && (lane & 3) == warp)
            wt[lane + 32 * i] = ml[i].x * inv;
    __syncwarp();
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4 &x, float f) {
        a.x = fmaf(x.x, f, a.x);
        a.y = fmaf(x.y, f, a.y);
        a.z = fmaf(x.z, f, a.z);
        a.w = fmaf(x.w, f, a.w);
    };
    if (!bad) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (warp + 4 * i < np)
                add(v[i], wt[warp + 4 * i]);
#pragma unroll 6
        for (int c = warp + 4 * AHEAD; c < np; c += 4)
            add(__ldcg(reinterpret_cast<const float4 *>(piece(c) + off)), wt[c]);
    }
    if (warp > 0)
        part_s[warp - 1][lane] = a;
    __syncthreads();
    if (warp > 0)
        return;
#pragma unroll
    for (int i = 0; i < 3; ++i)
        add(part_s[i][lane], 1.f);
    store4(p.out + ((int64_t)b * p.num_q_heads + (int64_t)hg * rows) * D + off, a);
}

}  // namespace pa
