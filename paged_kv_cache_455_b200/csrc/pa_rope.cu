// pa_rope.cu -- cache writes that rotate queries and keys on the way, into
// pools of the input type (pa_rope_and_cache) or into E4M3 pools with one
// scale per (block, KV head) (pa_rope_and_cache_q8), and block copies that
// take the scales along (pa_copy_blocks_q8).
//
// Rotation.  With r = rot_dim, position p and pair i < r / 2, the elements
// (a, b) of pair i become
//     (a c - b s, b c + a s),   c = table[p][i], s = table[p][r / 2 + i],
// in fp32 with every product and sum rounded by itself (no contraction, so
// that the result does not depend on how the compiler fuses them); pairs are
// (i, i + r / 2), or (2 i, 2 i + 1) when interleaved.
//
// All three kernels only move data: HBM bounds them for prompts, launch and load
// latency for single tokens.  Measured, 16 query and 4 KV heads of 256, bf16:
//   pa_rope_and_cache     prompts, 487 MB read and written: 77 us, 6.3 TB/s (0.97
//                         of a plain copy's rate), 537 MB interleaved 85 us, 430 MB
//                         of fp32 67 us; 64 single tokens 2.3 us
//   pa_rope_and_cache_q8  8K tokens in chunks of up to 512, 205 MB: 40.5 us, 5.1 TB/s;
//                         256 single tokens 6.8 us
//   pa_copy_blocks_q8     3000 blocks of 32 tokens, 8 heads of 128, 394 MB: 60.3 us,
//                         6.5 TB/s; 48 blocks of 16 tokens 2.5 us; 512 blocks to pinned
//                         host memory and back 52 and 51 GB/s (one copy of as many
//                         bytes: 55)
// What keeps the second from the copy's rate is its chain of loads (a CTA of the
// cache part finds its sequence, then its block, and only then writes) and its
// arithmetic: the schedulers issue half of the time.  64 registers a thread for
// more CTAs per SM spill: 43 us.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "pa.h"
#include "pa_host.cuh"
#include "pa_kernels.cuh"

namespace {

// ---------------------------------------------------------------- rotation
// A row of d elements is cut into 16-byte chunks of VEC elements, and the
// chunks into units of two that one thread handles: for the half-split
// pairing, chunk u and the one r / 2 elements after it; for the interleaved
// one, and for what is not rotated, two consecutive chunks.  Either way a
// rotated unit u holds the pairs u * VEC .. u * VEC + VEC - 1, so its cosines
// and its sines are VEC consecutive floats each.
struct RotParams {
    const float *table;      // [max_position][rot]
    const int64_t *positions;
    int64_t max_position;
    int rot;
    int interleaved;
};

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4 u, float (&x)[4])
    {
        x[0] = __uint_as_float(u.x);
        x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z);
        x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4])
    {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4 u, float (&x)[8])
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = pa::ptx::bf16lo_to_f32(w[i]);
            x[2 * i + 1] = pa::ptx::bf16hi_to_f32(w[i]);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8])
    {
        return make_uint4(pa::ptx::pack_bf16x2(x[0], x[1]), pa::ptx::pack_bf16x2(x[2], x[3]),
                          pa::ptx::pack_bf16x2(x[4], x[5]), pa::ptx::pack_bf16x2(x[6], x[7]));
    }
};

// The two chunks of unit u; true if the unit is rotated.
template <int VEC>
__device__ __forceinline__ bool unit_chunks(int u, int rot, bool interleaved, int &c0, int &c1)
{
    const int half = rot / (2 * VEC);
    if (u < half && !interleaved) {
        c0 = u;
        c1 = u + half;
    } else {
        c0 = 2 * u;
        c1 = 2 * u + 1;
    }
    return u < half;
}

template <int VEC>
struct Angles {
    float c[VEC], s[VEC];

    // Cosines and sines of unit u at position pos (in range).
    __device__ __forceinline__ void load(const RotParams &p, int64_t pos, int u)
    {
        const float4 *row = reinterpret_cast<const float4 *>(p.table + pos * p.rot);
        const int half4 = p.rot / 8;
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const float4 a = __ldg(row + u * (VEC / 4) + i);
            const float4 b = __ldg(row + half4 + u * (VEC / 4) + i);
            c[4 * i] = a.x;
            c[4 * i + 1] = a.y;
            c[4 * i + 2] = a.z;
            c[4 * i + 3] = a.w;
            s[4 * i] = b.x;
            s[4 * i + 1] = b.y;
            s[4 * i + 2] = b.z;
            s[4 * i + 3] = b.w;
        }
    }

    // Rotates the unit's elements x (chunk 0) and y (chunk 1).
    __device__ __forceinline__ void apply(float (&x)[VEC], float (&y)[VEC], bool interleaved) const
    {
        if (!interleaved) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float a = x[i], b = y[i];
                x[i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
                y[i] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                const float a = x[2 * i], b = x[2 * i + 1];
                x[2 * i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
                x[2 * i + 1] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
                const float e = y[2 * i], f = y[2 * i + 1];
                const int j = VEC / 2 + i;
                y[2 * i] = __fsub_rn(__fmul_rn(e, c[j]), __fmul_rn(f, s[j]));
                y[2 * i + 1] = __fadd_rn(__fmul_rn(f, c[j]), __fmul_rn(e, s[j]));
            }
        }
    }
};

// ------------------------------------------------------- pa_rope_and_cache
struct RopeParams {
    RotParams rot;
    const void *query, *key, *value;
    void *query_out, *k_pool, *v_pool;
    int64_t q_stride, qo_stride, k_stride, v_stride;   // bytes between tokens
    const int64_t *slot_mapping;
    int32_t *dev_status;
    int64_t num_slots;
    int num_tokens, num_q_heads, num_kv_heads;
    int row_bytes;
    int units_log2;          // threads per row (units) = d / (2 VEC), a power of two
};

// One thread handles unit u of ROWS rows of one token: the rows are the
// token's query heads, key heads and value heads.  The loads of all its rows
// are issued before the first is used.
template <typename T, int ROWS>
__global__ void __launch_bounds__(256) rope_cache_kernel(const RopeParams p)
{
    constexpr int VEC = Vec<T>::N;
    // launched as a programmatic dependent; it does not let its own dependent
    // start early: a decode kernel reads the cached rows of all but each
    // sequence's last token before it waits, and a call may store more
    pa::ptx::grid_wait_prerequisites();
    const int units = 1 << p.units_log2;
    const int rows = p.num_q_heads + 2 * p.num_kv_heads;
    const int groups = (rows + ROWS - 1) / ROWS;
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int u = (int)(x & (units - 1));
    const int64_t tg = x >> p.units_log2;
    const int64_t t = tg / groups;
    const int g = (int)(tg - t * groups);
    if (t >= p.num_tokens)
        return;
    int c0, c1;
    const bool turned = unit_chunks<VEC>(u, p.rot.rot, p.rot.interleaved != 0, c0, c1);
    uint4 a[ROWS], b[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int r = g + i * groups;
        if (r >= rows)
            continue;
        const uint8_t *src;
        if (r < p.num_q_heads)
            src = static_cast<const uint8_t *>(p.query) + t * p.q_stride + (int64_t)r * p.row_bytes;
        else if (r < p.num_q_heads + p.num_kv_heads)
            src = static_cast<const uint8_t *>(p.key) + t * p.k_stride +
                  (int64_t)(r - p.num_q_heads) * p.row_bytes;
        else
            src = static_cast<const uint8_t *>(p.value) + t * p.v_stride +
                  (int64_t)(r - p.num_q_heads - p.num_kv_heads) * p.row_bytes;
        // (plain loads: query_out may be query itself)
        a[i] = reinterpret_cast<const uint4 *>(src)[c0];
        b[i] = reinterpret_cast<const uint4 *>(src)[c1];
    }
    const int64_t slot = p.slot_mapping[t];
    bool bad_pos = false;
    Angles<VEC> ang;
    if (p.rot.rot > 0) {
        const int64_t pos = p.rot.positions[t];
        bad_pos = pos < 0 || pos >= p.rot.max_position;
        if (turned && !bad_pos)
            ang.load(p.rot, pos, u);
    }
    const bool bad_slot = slot >= p.num_slots;
    if (u == 0 && g == 0) {
        if (bad_pos)
            pa::report(p.dev_status, PA_DEV_BAD_POSITION);
        if (bad_slot)
            pa::report(p.dev_status, PA_DEV_BAD_SLOT);
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int r = g + i * groups;
        if (r >= rows)
            continue;
        const bool is_q = r < p.num_q_heads;
        const bool is_v = r >= p.num_q_heads + p.num_kv_heads;
        if (!is_q && (slot < 0 || bad_slot || bad_pos))
            continue;
        if (is_q && bad_pos) {
            a[i] = make_uint4(0, 0, 0, 0);
            b[i] = make_uint4(0, 0, 0, 0);
        } else if (turned && !is_v) {
            float xa[VEC], xb[VEC];
            Vec<T>::unpack(a[i], xa);
            Vec<T>::unpack(b[i], xb);
            ang.apply(xa, xb, p.rot.interleaved != 0);
            a[i] = Vec<T>::pack(xa);
            b[i] = Vec<T>::pack(xb);
        }
        uint8_t *dst;
        if (is_q)
            dst = static_cast<uint8_t *>(p.query_out) + t * p.qo_stride + (int64_t)r * p.row_bytes;
        else if (!is_v)
            dst = static_cast<uint8_t *>(p.k_pool) +
                  (slot * p.num_kv_heads + (r - p.num_q_heads)) * p.row_bytes;
        else
            dst = static_cast<uint8_t *>(p.v_pool) +
                  (slot * p.num_kv_heads + (r - p.num_q_heads - p.num_kv_heads)) * p.row_bytes;
        reinterpret_cast<uint4 *>(dst)[c0] = a[i];
        reinterpret_cast<uint4 *>(dst)[c1] = b[i];
    }
}

// ---------------------------------------------------- pa_rope_and_cache_q8
struct RopeQ8Params {
    RotParams rot;
    const __nv_bfloat16 *query, *key, *value;
    __nv_bfloat16 *query_out;
    uint8_t *k_pool, *v_pool;
    float *k_scales, *v_scales;
    int64_t q_stride, qo_stride, k_stride, v_stride;   // elements between tokens
    const int32_t *cu_q_lens, *block_tables, *context_lens;
    int64_t len_stride;      // elements between context_lens
    int32_t *dev_status;
    int64_t num_blocks;
    int64_t ctx_cap;
    int total_q, max_q_len, num_seqs, max_blocks;
    int num_q_heads, num_kv_heads;
    int bs_log2;
    int write_ctas;          // CTAs of the cache part; the query part follows
    int query_rows;          // rows per thread of it, at most kQ8QueryRows
};

constexpr int kQ8QueryRows = 4;      // query rows per thread

// Two fp32 values to E4M3 codes, `lo` in byte 0 (nearest, ties to even,
// saturating to +-448, NaN to NaN).
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi)
{
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3) &
           0xffffu;
}

// The smallest 2^e, -64 <= e <= 120, with amax <= 448 * 2^e (448 = 1.75 * 2^8;
// amax is finite and >= 0).
__device__ __forceinline__ float block_scale(float amax)
{
    const uint32_t bits = __float_as_uint(amax);
    int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = min(max(e, -64), 120);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ float finite_abs(float x)
{
    const float y = fabsf(x);
    return y <= 3.402823466e38f ? y : 0.f;   // infinities and NaN do not count
}

// Last b in [0, n) with cu[b] / bs + 2 b <= u, whole warp (u >= 0; b = 0 if
// there is none).  Sequence b touches at most n_b / bs + 2 blocks, so unit
// numbers cu[b] / bs + 2 b + i name every touched block i of every sequence
// once.
__device__ __forceinline__ int find_sequence(const int32_t *cu, int n, int bs_log2, int u, int lane)
{
    int lo = 0, len = n;
    while (len > 1) {
        const int step = (len + 31) >> 5;
        const int i = lane * step;
        const bool le = i < len && (__ldg(cu + lo + i) >> bs_log2) + 2 * (lo + i) <= u;
        const int k = max(__popc(__ballot_sync(pa::kFull, le)) - 1, 0);
        lo += k * step;
        len = min(step, len - k * step);
    }
    return lo;
}

// Cache part: one CTA of 128 threads per (touched block of a sequence, KV
// head, K or V).  The CTA owns its block: it rotates the sequence's new rows
// in it (D / 16 threads per row, RPT rows per thread, kept in registers),
// finds their largest magnitude, settles the block's scale, requantises the
// rows already there if the scale grew, and stores the new codes.  No two
// CTAs touch the same codes or scale, so there are no atomics and the result
// does not depend on timing.
// Query part: 128 threads rotate 128 / (D / 16) rows at a time, query_rows times.
template <int D, int RPT>
__global__ void __launch_bounds__(128) rope_cache_q8_kernel(const RopeQ8Params p)
{
    constexpr int UNITS = D / 16;            // threads per row
    constexpr int RPB = 128 / UNITS;         // rows per pass of the CTA
    using V8 = Vec<__nv_bfloat16>;
    // With one new token per sequence the next kernel, a decode mostly, may set
    // itself up now; it reads nothing before this grid has completed.  (Not before
    // the wait: a kernel that starts then could run beside one further ahead.)
    pa::ptx::grid_wait_prerequisites();
    if (p.max_q_len == 1)
        pa::ptx::grid_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int u = tid % UNITS, rl = tid / UNITS;
    const bool inter = p.rot.interleaved != 0;
    int c0, c1;
    const bool turned = unit_chunks<8>(u, p.rot.rot, inter, c0, c1);

    if ((int)blockIdx.x >= p.write_ctas) {
        // ---------------------------------------------------- query part
        // all rows are asked for before the first is turned
        constexpr int QR = kQ8QueryRows;
        const int real = min(p.cu_q_lens[p.num_seqs], p.total_q);
        const int64_t row0 = (int64_t)((int)blockIdx.x - p.write_ctas) * (RPB * p.query_rows) + rl;
        int64_t t = row0 / p.num_q_heads;
        int h = (int)(row0 - t * p.num_q_heads);
        int64_t tok[QR], pos[QR];
        int head[QR];
        uint4 a[QR], c[QR];
#pragma unroll
        for (int i = 0; i < QR; ++i) {
            tok[i] = i < p.query_rows ? t : real;
            head[i] = h;
            a[i] = c[i] = make_uint4(0, 0, 0, 0);
            pos[i] = 0;
            if (tok[i] < real) {
                const uint4 *src =
                    reinterpret_cast<const uint4 *>(p.query + t * p.q_stride + (int64_t)h * D);
                a[i] = src[c0];
                c[i] = src[c1];
                if (p.rot.rot > 0)
                    pos[i] = p.rot.positions[t];
            }
            for (h += RPB; h >= p.num_q_heads; h -= p.num_q_heads)
                ++t;
        }
#pragma unroll
        for (int i = 0; i < QR; ++i) {
            if (tok[i] >= real)
                continue;
            if (p.rot.rot > 0 && (pos[i] < 0 || pos[i] >= p.rot.max_position)) {
                if (u == 0 && head[i] == 0)
                    pa::report(p.dev_status, PA_DEV_BAD_POSITION);
                a[i] = c[i] = make_uint4(0, 0, 0, 0);
            } else if (turned) {
                Angles<8> ang;
                ang.load(p.rot, pos[i], u);
                float xa[8], xb[8];
                V8::unpack(a[i], xa);
                V8::unpack(c[i], xb);
                ang.apply(xa, xb, inter);
                a[i] = V8::pack(xa);
                c[i] = V8::pack(xb);
            }
            uint4 *dst = reinterpret_cast<uint4 *>(p.query_out + tok[i] * p.qo_stride +
                                                   (int64_t)head[i] * D);
            dst[c0] = a[i];
            dst[c1] = c[i];
        }
        return;
    }

    // -------------------------------------------------------- cache part
    const int kv = blockIdx.x & 1;
    const int hx = (blockIdx.x >> 1) % p.num_kv_heads;
    const int unit = (blockIdx.x >> 1) / p.num_kv_heads;
    const int bs = 1 << p.bs_log2;
    // with at most one new token per sequence, sequence b touches one block
    int b = unit, i = 0;
    if (p.max_q_len > 1) {
        b = find_sequence(p.cu_q_lens, p.num_seqs, p.bs_log2, unit, lane);
        i = unit - ((p.cu_q_lens[b] >> p.bs_log2) + 2 * b);
    }
    const int q0 = p.cu_q_lens[b], n = p.cu_q_lens[b + 1] - q0;
    const int ctx = p.context_lens[b * p.len_stride];
    auto bad_sequence = [&](int first_row, int rows, int len) {
        return rows < 0 || first_row < 0 || (int64_t)first_row + rows > p.total_q ||
               rows > p.max_q_len || rows > len || len > p.ctx_cap;
    };
    if (blockIdx.x == 0) {
        // this CTA reports for the whole batch (a sequence with invalid rows
        // may have no CTA of its own)
        bool bad = false;
        for (int x = tid; x < p.num_seqs; x += 128) {
            const int a = p.cu_q_lens[x];
            bad |= bad_sequence(a, p.cu_q_lens[x + 1] - a,
                                p.context_lens[x * p.len_stride]);
        }
        if (bad)
            pa::report(p.dev_status, PA_DEV_BAD_CONTEXT);
    }
    if (bad_sequence(q0, n, ctx))
        return;
    const int start = ctx - n;               // position of the first new token
    const int64_t first = (int64_t)(start >> p.bs_log2) + i;   // logical block
    if (n == 0 || i < 0 || (first << p.bs_log2) >= ctx)
        return;
    const int lb = (int)first;
    const int id = p.block_tables[(int64_t)b * p.max_blocks + lb];
    const int r0 = max(start - (lb << p.bs_log2), 0);          // new rows [r0, r1) of the block
    const int r1 = min(ctx - (lb << p.bs_log2), bs);
    const int64_t t0 = (int64_t)q0 + (lb << p.bs_log2) - start;   // token of row 0
    // the rows are asked for before the block's number is looked at
    uint4 a[RPT], c[RPT];
    int64_t pos[RPT];
    bool have[RPT];
    {
        const __nv_bfloat16 *src = kv ? p.value : p.key;
        const int64_t stride = kv ? p.v_stride : p.k_stride;
#pragma unroll
        for (int k = 0; k < RPT; ++k) {
            const int r = rl + k * RPB;
            have[k] = r >= r0 && r < r1;
            a[k] = c[k] = make_uint4(0, 0, 0, 0);
            pos[k] = 0;
            if (have[k]) {
                const uint4 *row =
                    reinterpret_cast<const uint4 *>(src + (t0 + r) * stride + (int64_t)hx * D);
                a[k] = __ldg(row + c0);
                c[k] = __ldg(row + c1);
                if (p.rot.rot > 0)
                    pos[k] = p.rot.positions[t0 + r];
            }
        }
    }
    if (id < 0 || (int64_t)id >= p.num_blocks) {
        if (tid == 0 && kv == 0 && hx == 0)
            pa::report(p.dev_status, PA_DEV_BAD_BLOCK);
        return;
    }
    float *scale_at = (kv ? p.v_scales : p.k_scales) + (int64_t)id * p.num_kv_heads + hx;
    const float old = *scale_at;
    uint8_t *block = (kv ? p.v_pool : p.k_pool) +
                     ((int64_t)id * bs * p.num_kv_heads + hx) * D;
    const int64_t row_bytes = (int64_t)p.num_kv_heads * D;

    float xa[RPT][8], xb[RPT][8];
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < RPT; ++k) {
        V8::unpack(a[k], xa[k]);
        V8::unpack(c[k], xb[k]);
        if (p.rot.rot > 0 && have[k]) {
            if (pos[k] < 0 || pos[k] >= p.rot.max_position) {
                // the token is not stored (its value row neither)
                if (u == 0 && kv == 0 && hx == 0)
                    pa::report(p.dev_status, PA_DEV_BAD_POSITION);
                have[k] = false;
            } else if (turned && kv == 0) {
                Angles<8> ang;
                ang.load(p.rot, pos[k], u);
                ang.apply(xa[k], xb[k], inter);
            }
        }
        if (have[k]) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                amax = fmaxf(amax, fmaxf(fabsf(xa[k][e]), fabsf(xb[k][e])));   // (not NaN)
        }
    }
    if (amax > 3.402823466e38f) {            // an infinity: again, without them
        amax = 0.f;
#pragma unroll
        for (int k = 0; k < RPT; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (have[k])
                    amax = fmaxf(amax, fmaxf(finite_abs(xa[k][e]), finite_abs(xb[k][e])));
    }
    __shared__ float wmax[4];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(pa::kFull, amax, o));
    if (lane == 0)
        wmax[warp] = amax;
    __syncthreads();                         // (also: every thread has read the old scale)
    amax = fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3]));
    const float want = block_scale(amax);
    const float s = r0 == 0 ? want : fmaxf(old, want);
    if (tid == 0)
        *scale_at = s;
    if (r0 > 0 && s != old) {
        // the scale grew: requantise the rows already there, 16 codes a thread
        const float ratio = __fdiv_rn(old, s);
        for (int x = tid; x < r0 * (D / 16); x += 128) {
            uint4 *at = reinterpret_cast<uint4 *>(block + (x / (D / 16)) * row_bytes) + x % (D / 16);
            const uint4 in = *at;
            const uint32_t w[4] = {in.x, in.y, in.z, in.w};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t f0 = pa::e4m3x2_to_f16x2(w[k]), f1 = pa::e4m3x2_to_f16x2(w[k] >> 16);
                o[k] = e4m3_pair(pa::ptx::f16lo_to_f32(f0) * ratio, pa::ptx::f16hi_to_f32(f0) * ratio) |
                       (e4m3_pair(pa::ptx::f16lo_to_f32(f1) * ratio,
                                  pa::ptx::f16hi_to_f32(f1) * ratio) << 16);
            }
            *at = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    // x / s: for a power of two (every scale this kernel makes) the product
    // with the reciprocal is the same number
    const bool pow2 = (__float_as_uint(s) & 0x807fffffu) == 0 && s >= 0x1p-64f && s <= 0x1p120f;
    if (pow2) {
        const float inv = __fdiv_rn(1.f, s);
#pragma unroll
        for (int k = 0; k < RPT; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xa[k][e] *= inv;
                xb[k][e] *= inv;
            }
    } else {
#pragma unroll
        for (int k = 0; k < RPT; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xa[k][e] = __fdiv_rn(xa[k][e], s);
                xb[k][e] = __fdiv_rn(xb[k][e], s);
            }
    }
#pragma unroll
    for (int k = 0; k < RPT; ++k) {
        if (!have[k])
            continue;
        uint8_t *row = block + (rl + k * RPB) * row_bytes;
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            o[e / 4] = e4m3_pair(xa[k][e], xa[k][e + 1]) |
                       (e4m3_pair(xa[k][e + 2], xa[k][e + 3]) << 16);
            o[2 + e / 4] = e4m3_pair(xb[k][e], xb[k][e + 1]) |
                           (e4m3_pair(xb[k][e + 2], xb[k][e + 3]) << 16);
        }
        *reinterpret_cast<uint2 *>(row + 8 * c0) = make_uint2(o[0], o[1]);
        *reinterpret_cast<uint2 *>(row + 8 * c1) = make_uint2(o[2], o[3]);
    }
}

// ------------------------------------------------------- pa_copy_blocks_q8
struct CopyQ8Params {
    const uint8_t *src_k, *src_v;
    uint8_t *dst_k, *dst_v;
    const float *src_ks, *src_vs;
    float *dst_ks, *dst_vs;
    const int64_t *block_mapping;
    int32_t *dev_status;
    int64_t src_blocks, dst_blocks;
    int64_t block_bytes;
    int num_pairs, num_kv_heads;
};

// One CTA per (pair, pool, 8 KB chunk of the block); the CTA of chunk 0 copies
// the block's scales too.
__global__ void __launch_bounds__(256) copy_blocks_q8_kernel(const CopyQ8Params p, int chunks)
{
    pa::ptx::grid_wait_prerequisites();
    const int pair = blockIdx.x / (2 * chunks);
    const int rest = blockIdx.x - pair * 2 * chunks;
    const int kv = rest / chunks;
    const int chunk = rest - kv * chunks;
    const int64_t src = p.block_mapping[2 * (int64_t)pair];
    const int64_t dst = p.block_mapping[2 * (int64_t)pair + 1];
    if (src < 0 || src >= p.src_blocks || dst < 0 || dst >= p.dst_blocks) {
        if (threadIdx.x == 0 && kv == 0 && chunk == 0)
            pa::report(p.dev_status, PA_DEV_BAD_BLOCK);
        return;
    }
    const uint4 *from =
        reinterpret_cast<const uint4 *>((kv ? p.src_v : p.src_k) + src * p.block_bytes);
    uint4 *to = reinterpret_cast<uint4 *>((kv ? p.dst_v : p.dst_k) + dst * p.block_bytes);
    const int64_t n16 = p.block_bytes >> 4;
    const int64_t c0 = (int64_t)chunk * 512 + threadIdx.x, c1 = c0 + 256;
    uint4 a, b;
    if (c0 < n16)
        a = __ldcg(from + c0);
    if (c1 < n16)
        b = __ldcg(from + c1);
    if (c0 < n16)
        to[c0] = a;
    if (c1 < n16)
        to[c1] = b;
    if (chunk == 0)
        for (int h = threadIdx.x; h < p.num_kv_heads; h += 256)
            (kv ? p.dst_vs : p.dst_ks)[dst * p.num_kv_heads + h] =
                __ldcg((kv ? p.src_vs : p.src_ks) + src * p.num_kv_heads + h);
}

// ------------------------------------------------------------------- host
int log2_exact(int v)
{
    int s = 0;
    while ((1 << s) < v)
        ++s;
    return (1 << s) == v ? s : -1;
}

// Arguments both rotary cache writes share; strides in elements, `es` their
// size.
pa_status check_rope(const void *query_out, int64_t qo_stride, const void *query, int64_t q_stride,
                     const void *key, int64_t k_stride, const void *value, int64_t v_stride,
                     const int64_t *positions, const float *cos_sin, int rot_dim,
                     int64_t max_position, int num_tokens, int num_q_heads, int num_kv_heads,
                     int head_dim, int es)
{
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16 != 0)
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0)
        return PA_OK;
    if (!key || !value || !pa::aligned16(key) || !pa::aligned16(value))
        return PA_ERR_INVALID_ARG;
    if (num_q_heads > 0 &&
        (!query || !query_out || !pa::aligned16(query) || !pa::aligned16(query_out)))
        return PA_ERR_INVALID_ARG;
    if (rot_dim > 0 && (!positions || !cos_sin || !pa::aligned16(cos_sin) || max_position <= 0))
        return PA_ERR_INVALID_ARG;
    const int64_t kv = (int64_t)num_kv_heads * head_dim, q = (int64_t)num_q_heads * head_dim;
    if (k_stride < kv || v_stride < kv || k_stride * es % 16 || v_stride * es % 16)
        return PA_ERR_INVALID_ARG;
    if (num_q_heads > 0 &&
        (q_stride < q || qo_stride < q || q_stride * es % 16 || qo_stride * es % 16))
        return PA_ERR_INVALID_ARG;
    return PA_OK;
}

template <typename T>
pa_status launch_rope(RopeParams &p, int head_dim, void *stream)
{
    const int units = head_dim / (2 * Vec<T>::N);
    p.units_log2 = log2_exact(units);
    const int rows = p.num_q_heads + 2 * p.num_kv_heads;
    // Four rows per thread reuse a token's angles and keep more loads in
    // flight, one row per thread fills the GPU: four once that still leaves
    // every SM two full waves of threads.
    const bool many = (int64_t)p.num_tokens * units * ((rows + 3) / 4) >= 148 * 2048 * 2;
    const int groups = many ? (rows + 3) / 4 : rows;
    const int64_t blocks = ((int64_t)p.num_tokens * units * groups + 255) / 256;
    if (blocks > INT32_MAX)
        return PA_ERR_INVALID_ARG;
    return many ? pa::launch_dependent(rope_cache_kernel<T, 4>, (unsigned)blocks, 256, 0, stream, p)
                : pa::launch_dependent(rope_cache_kernel<T, 1>, (unsigned)blocks, 256, 0, stream, p);
}

}  // namespace

extern "C" {

pa_status pa_rope_and_cache(void *query_out, int64_t query_out_stride, const void *query,
                            int64_t query_stride, const void *key, int64_t key_stride,
                            const void *value, int64_t value_stride, void *k_pool, void *v_pool,
                            const int64_t *slot_mapping, const int64_t *positions,
                            const float *cos_sin, int rot_dim, int64_t max_position,
                            int interleaved, int num_tokens, int num_q_heads, int num_kv_heads,
                            int head_dim, int block_size, int64_t num_blocks, pa_dtype dtype,
                            int32_t *dev_status, void *stream)
{
    if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads <= 0 || num_blocks <= 0)
        return PA_ERR_INVALID_ARG;
    if (dtype != PA_DTYPE_F32 && dtype != PA_DTYPE_BF16)
        return PA_ERR_UNSUPPORTED;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return PA_ERR_UNSUPPORTED;
    if (log2_exact(block_size) < 0 || block_size < 4 || block_size > 32)
        return PA_ERR_UNSUPPORTED;
    const int es = dtype == PA_DTYPE_F32 ? 4 : 2;
    const pa_status st = check_rope(query_out, query_out_stride, query, query_stride, key,
                                    key_stride, value, value_stride, positions, cos_sin, rot_dim,
                                    max_position, num_tokens, num_q_heads, num_kv_heads, head_dim,
                                    es);
    if (st != PA_OK || num_tokens == 0)
        return st;
    if (!k_pool || !v_pool || !slot_mapping || !pa::aligned16(k_pool) || !pa::aligned16(v_pool))
        return PA_ERR_INVALID_ARG;
    RopeParams p;
    p.rot = RotParams{cos_sin, positions, max_position, rot_dim, interleaved};
    p.query = query;
    p.key = key;
    p.value = value;
    p.query_out = query_out;
    p.k_pool = k_pool;
    p.v_pool = v_pool;
    p.q_stride = query_stride * es;
    p.qo_stride = query_out_stride * es;
    p.k_stride = key_stride * es;
    p.v_stride = value_stride * es;
    p.slot_mapping = slot_mapping;
    p.dev_status = dev_status;
    p.num_slots = num_blocks * block_size;
    p.num_tokens = num_tokens;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.row_bytes = head_dim * es;
    return dtype == PA_DTYPE_F32 ? launch_rope<float>(p, head_dim, stream)
                                 : launch_rope<__nv_bfloat16>(p, head_dim, stream);
}

pa_status pa_rope_and_cache_q8(void *query_out, int64_t query_out_stride, const void *query,
                               int64_t query_stride, const void *key, int64_t key_stride,
                               const void *value, int64_t value_stride, void *k_pool, void *v_pool,
                               float *k_scales, float *v_scales, const int32_t *cu_q_lens,
                               int total_q, int max_q_len, const int32_t *block_tables,
                               int max_blocks_per_seq, const int32_t *context_lens, int num_seqs,
                               const int64_t *positions, const float *cos_sin, int rot_dim,
                               int64_t max_position, int interleaved, int num_q_heads,
                               int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                               int32_t *dev_status, void *stream)
{
    return pa_rope_and_cache_q8_strided(
        query_out, query_out_stride, query, query_stride, key, key_stride, value, value_stride,
        k_pool, v_pool, k_scales, v_scales, cu_q_lens, total_q, max_q_len, block_tables,
        max_blocks_per_seq, context_lens, 1, num_seqs, positions, cos_sin, rot_dim, max_position,
        interleaved, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, dev_status,
        stream);
}

pa_status pa_rope_and_cache_q8_strided(
    void *query_out, int64_t query_out_stride, const void *query, int64_t query_stride,
    const void *key, int64_t key_stride, const void *value, int64_t value_stride, void *k_pool,
    void *v_pool, float *k_scales, float *v_scales, const int32_t *cu_q_lens, int total_q,
    int max_q_len, const int32_t *block_tables, int max_blocks_per_seq,
    const int32_t *context_lens, int64_t context_lens_stride, int num_seqs,
    const int64_t *positions, const float *cos_sin, int rot_dim, int64_t max_position,
    int interleaved, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
    int64_t num_blocks, int32_t *dev_status, void *stream)
{
    if (total_q < 0 || num_seqs < 0 || max_q_len < 0 || num_q_heads < 0 || num_kv_heads <= 0 ||
        num_blocks <= 0 || max_blocks_per_seq <= 0 || context_lens_stride < 0)
        return PA_ERR_INVALID_ARG;
    if ((head_dim != 128 && head_dim != 256) || (block_size != 16 && block_size != 32))
        return PA_ERR_UNSUPPORTED;
    const bool nothing = total_q == 0 || num_seqs == 0 || max_q_len == 0;
    pa_status st = check_rope(query_out, query_out_stride, query, query_stride, key, key_stride,
                              value, value_stride, positions, cos_sin, rot_dim, max_position,
                              nothing ? 0 : total_q, num_q_heads, num_kv_heads, head_dim, 2);
    if (st != PA_OK || nothing)
        return st;
    if (!k_pool || !v_pool || !k_scales || !v_scales || !cu_q_lens || !block_tables ||
        !context_lens || !pa::aligned16(k_pool) || !pa::aligned16(v_pool))
        return PA_ERR_INVALID_ARG;
    RopeQ8Params p;
    p.rot = RotParams{cos_sin, positions, max_position, rot_dim, interleaved};
    p.query = static_cast<const __nv_bfloat16 *>(query);
    p.key = static_cast<const __nv_bfloat16 *>(key);
    p.value = static_cast<const __nv_bfloat16 *>(value);
    p.query_out = static_cast<__nv_bfloat16 *>(query_out);
    p.k_pool = static_cast<uint8_t *>(k_pool);
    p.v_pool = static_cast<uint8_t *>(v_pool);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.q_stride = query_stride;
    p.qo_stride = query_out_stride;
    p.k_stride = key_stride;
    p.v_stride = value_stride;
    p.cu_q_lens = cu_q_lens;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.len_stride = context_lens_stride;
    p.dev_status = dev_status;
    p.num_blocks = num_blocks;
    p.ctx_cap = (int64_t)max_blocks_per_seq * block_size;
    p.total_q = total_q;
    p.max_q_len = max_q_len;
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.bs_log2 = log2_exact(block_size);
    // touched blocks: one per sequence with single tokens; else the unit
    // numbers of find_sequence
    const int64_t units = max_q_len == 1 ? num_seqs
                                         : (int64_t)total_q / block_size + 2 * (int64_t)num_seqs;
    const int64_t write = units * num_kv_heads * 2;
    // nothing to do for the queries when they are not rotated in place
    const bool rotate_q = num_q_heads > 0 && !(rot_dim == 0 && query == query_out);
    // Four rows a thread once they fill the GPU several times over, one for the
    // few rows of single tokens: 8K new tokens of 16 query heads of 256 took
    // 45 us with four and 49 us with two one after the other, 256 tokens 9.6 us
    // with four and 8.5 us with one (these with a copy of the lengths).
    const int64_t query_ctas = (int64_t)total_q * num_q_heads / (128 / (head_dim / 16));
    p.query_rows = query_ctas >= 148 * 16 * 4 ? kQ8QueryRows : 1;
    const int rows_per_cta = 128 / (head_dim / 16) * p.query_rows;
    const int64_t qctas =
        rotate_q ? ((int64_t)total_q * num_q_heads + rows_per_cta - 1) / rows_per_cta : 0;
    if (write + qctas > INT32_MAX)
        return PA_ERR_INVALID_ARG;
    p.write_ctas = (int)write;
    const unsigned grid = (unsigned)(write + qctas);
    if (head_dim == 128)
        return block_size == 16
                   ? pa::launch_dependent(rope_cache_q8_kernel<128, 1>, grid, 128, 0, stream, p)
                   : pa::launch_dependent(rope_cache_q8_kernel<128, 2>, grid, 128, 0, stream, p);
    return block_size == 16
               ? pa::launch_dependent(rope_cache_q8_kernel<256, 2>, grid, 128, 0, stream, p)
               : pa::launch_dependent(rope_cache_q8_kernel<256, 4>, grid, 128, 0, stream, p);
}

pa_status pa_copy_blocks_q8(void *dst_k_pool, void *dst_v_pool, float *dst_k_scales,
                            float *dst_v_scales, int64_t dst_num_blocks, const void *src_k_pool,
                            const void *src_v_pool, const float *src_k_scales,
                            const float *src_v_scales, int64_t src_num_blocks,
                            const int64_t *block_mapping, int num_pairs, int block_size,
                            int num_kv_heads, int head_dim, int32_t *dev_status, void *stream)
{
    if (num_pairs < 0 || src_num_blocks <= 0 || dst_num_blocks <= 0 || num_kv_heads <= 0)
        return PA_ERR_INVALID_ARG;
    if ((head_dim != 128 && head_dim != 256) || (block_size != 16 && block_size != 32))
        return PA_ERR_UNSUPPORTED;
    if (num_pairs == 0)
        return PA_OK;
    const void *ptrs[9] = {dst_k_pool,   dst_v_pool,   src_k_pool,   src_v_pool,  dst_k_scales,
                           dst_v_scales, src_k_scales, src_v_scales, block_mapping};
    for (const void *ptr : ptrs)
        if (!ptr)
            return PA_ERR_INVALID_ARG;
    for (int i = 0; i < 4; ++i)
        if (!pa::aligned16(ptrs[i]))
            return PA_ERR_INVALID_ARG;
    for (int i = 0; i < 9; ++i) {
        if ((i & 2) && ptrs[i] == ptrs[i - 2])
            continue;                    // copies within one pool
        if (!pa::device_addressable(ptrs[i]))
            return PA_ERR_INVALID_ARG;   // e.g. pageable host memory
    }
    CopyQ8Params p;
    p.src_k = static_cast<const uint8_t *>(src_k_pool);
    p.src_v = static_cast<const uint8_t *>(src_v_pool);
    p.dst_k = static_cast<uint8_t *>(dst_k_pool);
    p.dst_v = static_cast<uint8_t *>(dst_v_pool);
    p.src_ks = src_k_scales;
    p.src_vs = src_v_scales;
    p.dst_ks = dst_k_scales;
    p.dst_vs = dst_v_scales;
    p.block_mapping = block_mapping;
    p.dev_status = dev_status;
    p.src_blocks = src_num_blocks;
    p.dst_blocks = dst_num_blocks;
    p.block_bytes = (int64_t)block_size * num_kv_heads * head_dim;
    p.num_pairs = num_pairs;
    p.num_kv_heads = num_kv_heads;
    const int64_t chunks = (p.block_bytes + 8191) / 8192;
    const int64_t blocks = (int64_t)num_pairs * 2 * chunks;
    if (blocks > INT32_MAX)
        return PA_ERR_INVALID_ARG;
    return pa::launch_dependent(copy_blocks_q8_kernel, (unsigned)blocks, 256, 0, stream, p,
                                (int)chunks);
}

}  // extern "C"
