// attend.cu -- sparse attention of one decode step over 4-bit rows named by
// slot ids (include/hisparse_rows4.h, hisparse_attend).
//
// The mathematics.  With s = scale * log2(e) * (q . row), a running reference
// m of the row maximum, l = sum 2^(s - m) and O = sum 2^(s - m) * latent over
// the rows seen so far; when s outgrows m by more than 8, m moves and l and O
// are multiplied by 2^(m_old - m_new).  Then out = O / l and lse = (m +
// log2 l) ln 2.  A row's latent part is key and value at once, so a tile of
// rows is decoded once and used by both products.
//
// Exactness.  A latent value (e2m1 times e4m3) has at most six significant
// bits, so the decoded tile is exact in f16, scaled by 2^-7 (see decode8).
// A query row is multiplied by a power of two that brings its largest value
// to [1, 2), and is then exact in f16 down to 2^-22 of that; the rope parts
// stay in the model's type.  Scores, sums and O are 32-bit; probabilities
// enter the second product as f16 (relative step 2^-11).
//
// One CTA takes up to 64 heads of one request over a range of its rows, 64
// rows a tile, two tiles in flight:
//   warps 4-11   fetch the tile's packed rows into registers one tile ahead,
//                decode them to f16 in shared memory (128-byte swizzle);
//   warp 12      one thread issues the MMAs (M = 64 heads): S = Q K^T into
//                tensor memory, then O += P V, the same tile read as V with
//                the rows as the k dimension;
//   warps 0-3    softmax: read S, move the reference, write P as f16 over the
//                tile's rope part (S no longer needs it), keep l.
// O takes 256 columns of tensor memory: M = 64 uses 16 of each warp's 32
// lanes, so values 0-255 sit in the lower and 256-511 in the upper 16.
//
// The rows of a request are split over several CTAs when there are few
// (request, head tile) pairs; a second launch joins the parts.  With weights,
// the scores (base 2) go to the workspace and a last launch adds up each
// row's probabilities over the heads.
#include <cfloat>

#include "rows4.cuh"
#include "tcgen05.cuh"

namespace hs {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int TILE = 64;          // rows a tile
constexpr int HEADS = 64;         // heads a CTA
constexpr int AT_NT = 416;        // 4 softmax, 8 decode warps and the MMA warp
constexpr int SOFTMAX_WARPS = 4, DECODE_WARPS = 8, MMA_WARP = 12;
constexpr uint32_t BLOCK = 64 * 128;             // 64 values of 64 rows, swizzled
constexpr uint32_t OPERAND = 9 * BLOCK;          // 576 values of 64 rows
constexpr uint32_t ROPE_BLOCK = 8 * BLOCK;
constexpr uint32_t TMEM_S = 256;                 // column of S; 64 columns a stage
constexpr float kMoveAbove = 8.0f;               // base-2 growth that moves the reference

struct AttendSmem {
    uint64_t full[2], empty[2], scored[2], weighed[2], drained;
    uint32_t tmem;
    int gave_up;
    uint64_t valid[2];        // bit i: row i of the stage's tile is named
    float factor[HEADS];      // scale * log2(e) * the query's power of two
};
constexpr size_t AT_SMEM = 3 * OPERAND + sizeof(AttendSmem);

// Row that an id names, or null (nothing, or an id out of range, whose status
// bit is set in *bad).
__device__ __forceinline__ const uint8_t *row_of(const AttendLaunch &a, int r, int32_t id, int *bad)
{
    if (id < 0) {
        if (id != -1) *bad |= 1 << kStatusBadIndex;
        return nullptr;
    }
    if (id & kResidentFlag) {
        const int64_t n = id & (kResidentFlag - 1);
        if (n < a.res_count) return a.res + n * a.res_stride;
        *bad |= 1 << kStatusBadResident;
        return nullptr;
    }
    if (id < a.D) return a.rows + (int64_t)r * a.req_stride + (int64_t)id * a.row_stride;
    *bad |= 1 << kStatusBadIndex;
    return nullptr;
}

__device__ __forceinline__ uint4 ld_row_v4(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t ld_row_u16(const void *p)
{
    uint16_t v;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ void st_smem_v4(uint32_t at, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ void st_smem_u32(uint32_t at, uint32_t v)
{
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// 16-byte unit u (8 values) of row i in a swizzled block
__device__ __forceinline__ uint32_t swizzled(uint32_t block, int i, int u)
{
    return block + i * 128 + ((u ^ (i & 7)) << 4);
}

// Eight codes (a 32-bit word of a row) times scale, as f16, in the order 0 4 1
// 5 2 6 3 7: the codes of a pair are then 16 bits apart in the word as they
// are in the result.  A code's bits, put at the top of f16's exponent and
// mantissa (sign 15, exponent 11-10, mantissa 9), read as its value times
// 2^-14, subnormal included; the scale comes with 2^7 of that, the result
// keeps 2^-7.  Exact: at most six significant bits, at least 2^-17.
__device__ __forceinline__ uint4 decode8(uint32_t w, __half2 scale)
{
    auto pair = [&](uint32_t sign, uint32_t rest) {
        const uint32_t b = (sign & 0x80008000u) | (rest & 0x0E000E00u);
        const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&b), scale);
        return *reinterpret_cast<const uint32_t *>(&v);
    };
    return make_uint4(pair(w << 12, w << 9), pair(w << 8, w << 5), pair(w << 4, w << 1), pair(w, w >> 3));
}

// A thread's share of a packed row: a quarter of its 16-byte chunks.
struct RowPart {
    uint4 codes[4], rope[2];
    uint32_t scales[4];
};

__device__ __forceinline__ void fetch(RowPart &p, const uint8_t *row, int quarter)
{
    if (row) {
#pragma unroll
        for (int j = 0; j < 4; ++j) p.codes[j] = ld_row_v4(row + (j * 4 + quarter) * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) p.scales[j] = ld_row_u16(row + kScaleAt + (j * 4 + quarter) * 2);
#pragma unroll
        for (int j = 0; j < 2; ++j) p.rope[j] = ld_row_v4(row + kRopeAt + (j * 4 + quarter) * 16);
    } else {     // zeros: nothing of it reaches a result
#pragma unroll
        for (int j = 0; j < 4; ++j) p.codes[j] = make_uint4(0, 0, 0, 0), p.scales[j] = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) p.rope[j] = make_uint4(0, 0, 0, 0);
    }
}

__device__ __forceinline__ void decode(const RowPart &p, uint32_t stage, int i, int quarter)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t s2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2) : "h"((uint16_t)p.scales[j]));
        const __half2 s = __hmul2(*reinterpret_cast<__half2 *>(&s2), __half2half2(__ushort_as_half(0x5800)));  // 2^7
        const __half2 lo = __low2half2(s), hi = __high2half2(s);
        const uint32_t block = stage + (2 * j + (quarter >> 1)) * BLOCK;
        const int u = (quarter & 1) * 4;
        st_smem_v4(swizzled(block, i, u), decode8(p.codes[j].x, lo));
        st_smem_v4(swizzled(block, i, u + 1), decode8(p.codes[j].y, lo));
        st_smem_v4(swizzled(block, i, u + 2), decode8(p.codes[j].z, hi));
        st_smem_v4(swizzled(block, i, u + 3), decode8(p.codes[j].w, hi));
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) st_smem_v4(swizzled(stage + ROPE_BLOCK, i, j * 4 + quarter), p.rope[j]);
}

template <int DT>
__device__ __forceinline__ float2 pair_to_float(uint32_t w)
{
    if (DT == kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

template <int DT>
__device__ __forceinline__ uint32_t floats_to_pair(float x, float y)
{
    if (DT == kBf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// A power of two as float
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Query rows [h0, h0 + 64) into shared memory, by whole warps; rows past H
// are zero.
template <int DT>
__device__ __forceinline__ void stage_queries(const AttendLaunch &a, int r, int h0, uint32_t dst, float *factor,
                                              int warp, int lane)
{
    for (int i = warp; i < HEADS; i += AT_NT / 32) {
        const int h = h0 + i;
        uint4 v[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)}, rope = make_uint4(0, 0, 0, 0);
        if (h < a.H) {
            const uint8_t *q = a.q + (int64_t)r * a.q_rs + (int64_t)h * a.q_hs;
            v[0] = ld_dev_v4(q + lane * 16);
            v[1] = ld_dev_v4(q + 512 + lane * 16);
            if (lane < 8) rope = ld_dev_v4(q + kLatent * 2 + lane * 16);
        }
        uint32_t m = 0;   // magnitudes compare as integers
#pragma unroll
        for (int half = 0; half < 2; ++half)
            m = __vmaxu2(m, __vmaxu2(__vmaxu2(v[half].x & 0x7FFF7FFFu, v[half].y & 0x7FFF7FFFu),
                                     __vmaxu2(v[half].z & 0x7FFF7FFFu, v[half].w & 0x7FFF7FFFu)));
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(rope.x & 0x7FFF7FFFu, rope.y & 0x7FFF7FFFu),
                                 __vmaxu2(rope.z & 0x7FFF7FFFu, rope.w & 0x7FFF7FFFu)));
        uint32_t top = max(m >> 16, m & 0xFFFFu);
        top = __reduce_max_sync(0xffffffffu, top);
        // exponent of the largest value; 0 for none and for infinities and
        // NaN, which pass through as they are
        int e = (int)(__float_as_uint(pair_to_float<DT>(top).x) >> 23) - 127;
        if (top == 0 || e == 128) e = 0;
        e = max(e, -119);
        const float up = exp2i(7 - e), up_rope = exp2i(-e);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float2 x0 = pair_to_float<DT>(v[half].x), x1 = pair_to_float<DT>(v[half].y);
            const float2 x2 = pair_to_float<DT>(v[half].z), x3 = pair_to_float<DT>(v[half].w);
            // the order of decode8
            const uint4 h = make_uint4(floats_to_pair<kF16>(x0.x * up, x2.x * up), floats_to_pair<kF16>(x0.y * up, x2.y * up),
                                       floats_to_pair<kF16>(x1.x * up, x3.x * up), floats_to_pair<kF16>(x1.y * up, x3.y * up));
            const int unit = half * 32 + lane;
            st_smem_v4(swizzled(dst + (unit >> 3) * BLOCK, i, unit & 7), h);
        }
        if (lane < 8) {
            uint4 h;
            float2 x = pair_to_float<DT>(rope.x);
            h.x = floats_to_pair<DT>(x.x * up_rope, x.y * up_rope);
            x = pair_to_float<DT>(rope.y);
            h.y = floats_to_pair<DT>(x.x * up_rope, x.y * up_rope);
            x = pair_to_float<DT>(rope.z);
            h.z = floats_to_pair<DT>(x.x * up_rope, x.y * up_rope);
            x = pair_to_float<DT>(rope.w);
            h.w = floats_to_pair<DT>(x.x * up_rope, x.y * up_rope);
            st_smem_v4(swizzled(dst + ROPE_BLOCK, i, lane), h);
        }
        if (lane == 0) factor[i] = a.scale * kLog2e * exp2i(e);
    }
}

// Parts of the workspace, in floats.
struct AttendParts {
    int splits, tiles_per_split;
    float *lse2;      // [R][H] log2 of the sums, for the weights
    float *ml;        // [splits][R][H][2] reference and sum of each part
    float *o;         // [splits][R][H][512] 2^-7 O of each part
    float *scores;    // [R][H][k] base-2 scores, for the weights
};

// The warp's 16 heads' value, kept by the threads of a 16x256b fragment
// (rows lane / 4 and lane / 4 + 8), for the head of lane % 16.
__device__ __forceinline__ float by_lane(float a, float b, int lane)
{
    const float x = __shfl_sync(0xffffffffu, a, (lane & 7) * 4), y = __shfl_sync(0xffffffffu, b, (lane & 7) * 4);
    return (lane & 8) ? y : x;
}

template <int DT>
__global__ void __launch_bounds__(AT_NT, 1) attend_kernel(const __grid_constant__ AttendLaunch a,
                                                          const __grid_constant__ AttendParts w)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    AttendSmem &sm = *reinterpret_cast<AttendSmem *>(smem + 3 * OPERAND);
    const uint32_t q_at = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int head_tiles = (a.H + HEADS - 1) / HEADS;
    const int ht = blockIdx.x % head_tiles;
    const int split = (blockIdx.x / head_tiles) % w.splits;
    const int r = blockIdx.x / head_tiles / w.splits;
    const int h0 = ht * HEADS;
    const int k0 = split * w.tiles_per_split * TILE;
    const int rows = min(a.k - k0, w.tiles_per_split * TILE);
    const int tiles = (rows + TILE - 1) / TILE;

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&sm.full[s]), DECODE_WARPS);
            mbar_init(smem_u32(&sm.empty[s]), 1);
            mbar_init(smem_u32(&sm.scored[s]), 1);
            mbar_init(smem_u32(&sm.weighed[s]), SOFTMAX_WARPS);
        }
        mbar_init(smem_u32(&sm.drained), 1);
        sm.gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == MMA_WARP) tmem_alloc_all(smem_u32(&sm.tmem));
    stage_queries<DT>(a, r, h0, q_at, sm.factor, warp, lane);
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    volatile int *gave_up = &sm.gave_up;

    if (warp >= SOFTMAX_WARPS && warp < MMA_WARP) {
        // ---- fetch and decode -----------------------------------------------
        const int dw = warp - SOFTMAX_WARPS, i = dw * 8 + (lane & 7), quarter = lane >> 3;
        const int32_t *ids = a.ids + (int64_t)r * a.ids_stride + k0;
        auto id_at = [&](int t) { return t * TILE + i < rows ? ids[t * TILE + i] : -1; };
        RowPart next;
        int bad = 0;
        const uint8_t *row = row_of(a, r, id_at(0), &bad);
        fetch(next, row, quarter);
        int32_t id = id_at(1);
        for (int t = 0; t < tiles; ++t) {
            const RowPart part = next;
            const uint32_t named = __ballot_sync(0xffffffffu, row != nullptr) & 0xFFu;
            row = row_of(a, r, id, &bad);
            fetch(next, row, quarter);
            id = id_at(t + 2);
            const int s = t & 1;
            const bool free = t < 2 || mbar_wait(smem_u32(&sm.empty[s]), ((t >> 1) - 1) & 1, gave_up);
            if (!__all_sync(0xffffffffu, free)) break;
            decode(part, q_at + (1 + s) * OPERAND, i, quarter);
            if (lane == 0) reinterpret_cast<uint8_t *>(&sm.valid[s])[dw] = (uint8_t)named;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.full[s]));
        }
        if (bad && a.status) atomicOr(a.status + r, bad);
    } else if (warp == MMA_WARP) {
        // ---- MMA issue -----------------------------------------------------------
        if (lane == 0) {
            constexpr uint32_t qk = mma_desc(HEADS, TILE, false, false);
            constexpr uint32_t qk_rope = mma_desc(HEADS, TILE, DT == kBf16, false);
            constexpr uint32_t pv = mma_desc(HEADS, 256, false, true);
            const uint64_t q_desc = smem_desc(q_at, 16, 1024);
            bool ok = true;
            for (int t0 = 0; ok && t0 < tiles; t0 += 2) {
                const int n = min(2, tiles - t0);
                for (int s = 0; ok && s < n; ++s) {       // S = Q K^T
                    ok = mbar_wait(smem_u32(&sm.full[s]), (t0 >> 1) & 1, gave_up);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t k_desc = smem_desc(q_at + (1 + s) * OPERAND, 16, 1024);
                    const uint32_t d = tmem + TMEM_S + s * TILE;
#pragma unroll
                    for (int b = 0; b < 9; ++b)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {     // 16 values a step: 32 bytes
                            const uint64_t off = (b * BLOCK + x * 32) >> 4;
                            mma_f16(d, q_desc + off, k_desc + off, b < 8 ? qk : qk_rope, b + x > 0);
                        }
                    mma_commit(smem_u32(&sm.scored[s]));
                }
                for (int s = 0; ok && s < n; ++s) {       // O += P V
                    ok = mbar_wait(smem_u32(&sm.weighed[s]), (t0 >> 1) & 1, gave_up);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t stage = q_at + (1 + s) * OPERAND;
                    const uint64_t p_desc = smem_desc(stage + ROPE_BLOCK, 16, 1024);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint64_t v_desc = smem_desc(stage + half * 4 * BLOCK, BLOCK, 1024);
#pragma unroll
                        for (int x = 0; x < 4; ++x)       // 16 rows a step
                            mma_f16(tmem + (half ? 16u << 16 : 0u), p_desc + ((x * 32) >> 4),
                                    v_desc + ((x * 2048) >> 4), pv, t0 + s + x > 0);
                    }
                    mma_commit(smem_u32(&sm.empty[s]));
                }
            }
            if (!ok) {     // let what was issued end before the CTA goes
                mma_commit(smem_u32(&sm.drained));
                const uint32_t bar = smem_u32(&sm.drained);
                for (int i = 0; i < (1 << 20) && !mbar_try(bar, 0); ++i) {}
            }
        }
        __syncwarp();
    } else {
        // ---- softmax --------------------------------------------------------------
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        const int g = lane >> 2, c2 = (lane & 3) * 2;     // fragment row and column
        const int i0 = warp * 16 + g, i1 = i0 + 8;
        const float f0 = sm.factor[i0], f1 = sm.factor[i1];
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
        float *sc0 = nullptr, *sc1 = nullptr;
        if (a.weights) {
            const int64_t at = ((int64_t)r * a.H + h0) * a.k + k0;
            if (h0 + i0 < a.H) sc0 = w.scores + at + (int64_t)i0 * a.k;
            if (h0 + i1 < a.H) sc1 = w.scores + at + (int64_t)i1 * a.k;
        }
        bool ok = true;
        for (int t = 0; t < tiles; ++t) {
            const int s = t & 1;
            const uint32_t parity = (t >> 1) & 1;
            ok = mbar_wait(smem_u32(&sm.full[s]), parity, gave_up) &&
                 mbar_wait(smem_u32(&sm.scored[s]), parity, gave_up);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            uint32_t v[32];
            tmem_ld_16x64(lanes + TMEM_S + s * TILE, v);
            const uint64_t named = sm.valid[s] >> c2;
            tmem_wait_ld();
            float x[32];
            float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const bool on = (named >> (8 * j + b)) & 1u;
                    x[4 * j + b] = on ? __uint_as_float(v[4 * j + b]) * f0 : -INFINITY;
                    x[4 * j + 2 + b] = on ? __uint_as_float(v[4 * j + 2 + b]) * f1 : -INFINITY;
                    top0 = fmaxf(top0, x[4 * j + b]);
                    top1 = fmaxf(top1, x[4 * j + 2 + b]);
                }
            if (a.weights) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const int c = t * TILE + 8 * j + c2 + b;
                        if (c < rows) {
                            if (sc0) sc0[c] = x[4 * j + b];
                            if (sc1) sc1[c] = x[4 * j + 2 + b];
                        }
                    }
            }
            top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, 1));
            top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, 1));
            top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, 2));
            top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, 2));
            if (__any_sync(0xffffffffu, top0 > m0 + kMoveAbove || top1 > m1 + kMoveAbove)) {
                const float n0 = fmaxf(m0, top0), n1 = fmaxf(m1, top1);
                const float d0 = n0 == -INFINITY ? 1.0f : exp2f(m0 - n0), d1 = n1 == -INFINITY ? 1.0f : exp2f(m1 - n1);
                m0 = n0;
                m1 = n1;
                l0 *= d0;
                l1 *= d1;
                if (t > 0) {      // O so far, once the product before this one is done
                    const float d = by_lane(d0, d1, lane);
                    ok = mbar_wait(smem_u32(&sm.empty[s ^ 1]), ((t - 1) >> 1) & 1, gave_up);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 256; c += 32) {
                        tmem_ld_32x32(lanes + c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * d);
                        tmem_st_32x32(lanes + c, v);
                    }
                    tmem_wait_st();
                }
            }
            const float r0 = m0 == -INFINITY ? 0.0f : m0, r1 = m1 == -INFINITY ? 0.0f : m1;
            const uint32_t p_at = q_at + (1 + s) * OPERAND + ROPE_BLOCK;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float p00 = exp2f(x[4 * j] - r0), p01 = exp2f(x[4 * j + 1] - r0);
                const float p10 = exp2f(x[4 * j + 2] - r1), p11 = exp2f(x[4 * j + 3] - r1);
                l0 += p00 + p01;
                l1 += p10 + p11;
                st_smem_u32(swizzled(p_at, i0, j) + c2 * 2, floats_to_pair<kF16>(p00, p01));
                st_smem_u32(swizzled(p_at, i1, j) + c2 * 2, floats_to_pair<kF16>(p10, p11));
            }
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.weighed[s]));
        }
        // the last product, then O / l or this part's O, m and l
        if (__all_sync(0xffffffffu, ok))
            ok = mbar_wait(smem_u32(&sm.empty[(tiles - 1) & 1]), ((tiles - 1) >> 1) & 1, gave_up);
        if (__all_sync(0xffffffffu, ok)) {
            tc_fence_after();
            l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
            l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
            const int h = h0 + warp * 16 + (lane & 15), d0 = (lane >> 4) * 256;
            const float l = by_lane(l0, l1, lane), m = by_lane(m0, m1, lane);
            const int64_t rh = (int64_t)r * a.H + h;
            const bool whole = w.splits == 1;
            float *part = w.o + ((int64_t)split * a.R * a.H + rh) * kLatent + d0;
            uint8_t *out = a.out + (int64_t)r * a.out_rs + (int64_t)h * a.out_hs + d0 * 2;
            const float inv = l == 0.0f ? 0.0f : 128.0f / l;
            if (lane < 16 && h < a.H) {
                if (whole) {
                    const float l2 = l == 0.0f ? -INFINITY : m + log2f(l);
                    if (a.lse) a.lse[rh] = l2 * kLn2;
                    if (a.weights) w.lse2[rh] = l2;
                } else {
                    float *ml = w.ml + ((int64_t)split * a.R * a.H + rh) * 2;
                    ml[0] = m;
                    ml[1] = l;
                }
            }
#pragma unroll 1
            for (int c = 0; c < 256; c += 32) {
                uint32_t v[32];
                tmem_ld_32x32(lanes + c, v);
                tmem_wait_ld();
                if (h < a.H) {
#pragma unroll
                    for (int u = 0; u < 32; u += 8) {     // back to value order
                        const float y0 = __uint_as_float(v[u]), y4 = __uint_as_float(v[u + 1]);
                        const float y1 = __uint_as_float(v[u + 2]), y5 = __uint_as_float(v[u + 3]);
                        const float y2 = __uint_as_float(v[u + 4]), y6 = __uint_as_float(v[u + 5]);
                        const float y3 = __uint_as_float(v[u + 6]), y7 = __uint_as_float(v[u + 7]);
                        if (whole) {
                            st_v4(out + (c + u) * 2,
                                  make_uint4(floats_to_pair<DT>(y0 * inv, y1 * inv), floats_to_pair<DT>(y2 * inv, y3 * inv),
                                             floats_to_pair<DT>(y4 * inv, y5 * inv), floats_to_pair<DT>(y6 * inv, y7 * inv)));
                        } else {
                            *reinterpret_cast<float4 *>(part + c + u) = make_float4(y0, y1, y2, y3);
                            *reinterpret_cast<float4 *>(part + c + u + 4) = make_float4(y4, y5, y6, y7);
                        }
                    }
                }
            }
            tc_fence_before();
        }
    }
    __syncthreads();
    if (tid == 0 && sm.gave_up && a.status) record_status(a.status, r, kStatusAttendTimeout);
    if (warp == MMA_WARP) tmem_free_all(tmem);
}

// ---- joining the parts -------------------------------------------------------------

constexpr int JN_NT = 128;     // 4 values a thread

template <int DT>
__global__ void __launch_bounds__(JN_NT) join_kernel(const __grid_constant__ AttendLaunch a,
                                                     const __grid_constant__ AttendParts w)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t rh = blockIdx.x, RH = (int64_t)a.R * a.H;
    const int r = (int)(rh / a.H), h = (int)(rh - (int64_t)r * a.H), tid = threadIdx.x;
    float top = -INFINITY;
    for (int s = 0; s < w.splits; ++s) top = fmaxf(top, w.ml[(s * RH + rh) * 2]);
    const float ref = top == -INFINITY ? 0.0f : top;
    float l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s = 0; s < w.splits; ++s) {
        const float f = exp2f(w.ml[(s * RH + rh) * 2] - ref);
        l = fmaf(f, w.ml[(s * RH + rh) * 2 + 1], l);
        const float4 p = *reinterpret_cast<const float4 *>(w.o + (s * RH + rh) * kLatent + tid * 4);
        o.x = fmaf(f, p.x, o.x);
        o.y = fmaf(f, p.y, o.y);
        o.z = fmaf(f, p.z, o.z);
        o.w = fmaf(f, p.w, o.w);
    }
    const float inv = l == 0.0f ? 0.0f : 128.0f / l;
    uint8_t *out = a.out + (int64_t)r * a.out_rs + (int64_t)h * a.out_hs;
    *reinterpret_cast<uint2 *>(out + tid * 8) =
        make_uint2(floats_to_pair<DT>(o.x * inv, o.y * inv), floats_to_pair<DT>(o.z * inv, o.w * inv));
    if (tid == 0) {
        const float l2 = l == 0.0f ? -INFINITY : ref + log2f(l);
        if (a.lse) a.lse[rh] = l2 * kLn2;
        if (a.weights) w.lse2[rh] = l2;
    }
}

// ---- weights -----------------------------------------------------------------------

constexpr int WT_NT = 128;

__global__ void __launch_bounds__(WT_NT) weights_kernel(const __grid_constant__ AttendLaunch a,
                                                        const __grid_constant__ AttendParts w)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int r = blockIdx.y, i = blockIdx.x * WT_NT + threadIdx.x;
    if (i >= a.k) return;
    int bad = 0;
    if (!row_of(a, r, a.ids[(int64_t)r * a.ids_stride + i], &bad)) return;
    const int64_t pos = a.positions[(int64_t)r * a.positions_stride + i];
    if (pos < 0 || pos >= a.weights_tokens) {
        if (a.status) record_status(a.status, r, kStatusBadPosition);
        return;
    }
    const float *s = w.scores + (int64_t)r * a.H * a.k + i, *lse2 = w.lse2 + (int64_t)r * a.H;
    float sum = 0.0f;
#pragma unroll 8
    for (int h = 0; h < a.H; ++h) sum += exp2f(s[(int64_t)h * a.k] - lse2[h]);
    atomicAdd(a.weights + (int64_t)r * a.weights_stride + pos, sum);
}

// How many parts each request's rows are split into: the count for which the
// waves of CTAs (one on each SM) take the fewest tiles, counting a CTA's own
// start and end as three.
int choose_splits(int64_t units, int tiles, int num_sms)
{
    int best = 1;
    int64_t best_cost = INT64_MAX;
    for (int s = 1; s <= tiles && s <= 64; ++s) {
        const int per = (tiles + s - 1) / s;
        if ((tiles + per - 1) / per != s) continue;       // the same parts as a smaller s
        const int64_t waves = (units * s + num_sms - 1) / num_sms;
        const int64_t cost = waves * (per + 3);
        if (cost < best_cost) best_cost = cost, best = s;
    }
    return best;
}

int64_t up4(int64_t n) { return (n + 3) / 4 * 4; }

AttendParts lay_out(int32_t R, int32_t H, int32_t k, bool weights, int num_sms, uint8_t *ws, int64_t *bytes)
{
    AttendParts p;
    const int tiles = (k + TILE - 1) / TILE;
    const int64_t RH = (int64_t)R * H;
    p.splits = choose_splits((int64_t)R * ((H + HEADS - 1) / HEADS), tiles, num_sms);
    p.tiles_per_split = (tiles + p.splits - 1) / p.splits;
    float *f = reinterpret_cast<float *>(ws);
    int64_t n = 0;
    p.lse2 = f + n;
    n += up4(RH);
    p.ml = f + n;
    n += p.splits > 1 ? up4(2 * p.splits * RH) : 0;
    p.o = f + n;
    n += p.splits > 1 ? p.splits * RH * kLatent : 0;
    p.scores = f + n;
    n += weights ? up4(RH * k) : 0;
    *bytes = n * 4;
    return p;
}

template <class... Args>
cudaError_t launch_after(void (*kernel)(Args...), dim3 grid, int threads, cudaStream_t s, const AttendLaunch &a,
                         const AttendParts &w)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, w);
}

template <int DT>
cudaError_t launch_dt(const AttendLaunch &a, const AttendParts &w, cudaStream_t s)
{
    cudaError_t e = cudaFuncSetAttribute(attend_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)AT_SMEM);
    if (e != cudaSuccess) return e;
    const unsigned ctas = (unsigned)(a.R * ((a.H + HEADS - 1) / HEADS) * w.splits);
    attend_kernel<DT><<<ctas, AT_NT, AT_SMEM, s>>>(a, w);
    e = cudaGetLastError();
    if (e == cudaSuccess && w.splits > 1)
        e = launch_after(join_kernel<DT>, dim3((unsigned)(a.R * a.H)), JN_NT, s, a, w);
    if (e == cudaSuccess && a.weights)
        e = launch_after(weights_kernel, dim3((a.k + WT_NT - 1) / WT_NT, a.R), WT_NT, s, a, w);
    return e;
}

}  // namespace

int64_t attend_workspace_bytes(int32_t R, int32_t H, int32_t k, bool weights, int num_sms)
{
    int64_t bytes = 0;
    lay_out(R, H, k, weights, num_sms, nullptr, &bytes);
    return bytes;
}

cudaError_t launch_attend(const AttendLaunch &a, int num_sms, cudaStream_t s)
{
    int64_t bytes;
    const AttendParts w = lay_out(a.R, a.H, a.k, a.weights != nullptr, num_sms, a.workspace, &bytes);
    return a.dtype == kBf16 ? launch_dt<kBf16>(a, w, s) : launch_dt<kF16>(a, w, s);
}

}  // namespace hs
