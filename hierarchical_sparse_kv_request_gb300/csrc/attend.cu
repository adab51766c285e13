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
// rows a tile, three tiles in flight:
//   warps 4-19   fetch a tile's packed rows into registers one tile ahead,
//                decode them to f16 in shared memory (128-byte swizzle);
//   warp 20      issues the MMAs (M = 64 heads): S = Q K^T, then O += P V of
//                the tile before, its rows now the k dimension;
//   warps 0-3    softmax: read S, move the reference, write P as f16 over the
//                tile's rope part (S no longer needs it), keep l.
// M = 64 uses 16 of the 32 lanes of each warp's part of tensor memory: O fills
// the upper 16 (512 columns), S (two tiles) and the queries the lower.  With
// the queries there, an MMA of the first product reads 2 KB of shared memory
// in its 32 cycles instead of 4 KB, which would take all of its bandwidth and
// leave the decoding warps none (measured: 45.9 -> XX us for 32 requests, 128
// heads, 2,048 rows).
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
constexpr int SOFTMAX_WARPS = 4, DECODE_WARPS = 16, MMA_WARP = SOFTMAX_WARPS + DECODE_WARPS;
constexpr int AT_NT = (MMA_WARP + 1) * 32;
constexpr uint32_t BLOCK = 64 * 128;             // 64 values of 64 rows, swizzled
constexpr uint32_t OPERAND = 9 * BLOCK;          // 576 values of 64 rows
constexpr uint32_t ROPE_BLOCK = 8 * BLOCK;
constexpr int STAGES = 3;                        // tiles in shared memory
constexpr uint32_t TMEM_UPPER = 16u << 16;       // O: the upper lanes, column = value
constexpr uint32_t TMEM_Q = 2 * TILE;            // lower lanes: S of two tiles, then the queries
constexpr float kMoveAbove = 8.0f;               // base-2 growth that moves the reference

struct AttendSmem {
    uint64_t full[STAGES], empty[STAGES], scored[2], weighed[2], queries, drained;
    uint32_t tmem;
    int gave_up;
    __align__(16) uint8_t valid[STAGES][16];   // bit b of byte n: row 4 n + b of the stage's tile is named
    float factor[HEADS];      // scale * log2(e) * the query's power of two
};
constexpr size_t AT_SMEM = STAGES * OPERAND + sizeof(AttendSmem);

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
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t ld_row_u16(const void *p)
{
    uint16_t v;
    asm volatile("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ void st_smem_v4(uint32_t at, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint4 ld_smem_v4(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
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

// A decode warp's four rows, as its threads hold them: half a warp takes the
// 256 bytes of codes of one row (chunk c = lane % 16; two loads for four
// rows), a quarter the rope part of one, so every load is whole sectors of a
// few rows.
struct RowPart {
    uint4 codes[2], rope;
    uint32_t scales[2];
};

// row: this lane's rope row (lane / 8 of the warp's four), or null.
__device__ __forceinline__ void fetch(RowPart &p, const uint8_t *row, int lane)
{
    const int c = lane & 15;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint8_t *src = reinterpret_cast<const uint8_t *>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), (2 * j + (lane >> 4)) * 8));
        p.codes[j] = make_uint4(0, 0, 0, 0);     // of no row: nothing of it reaches a result
        p.scales[j] = 0;
        if (src) {
            p.codes[j] = ld_row_v4(src + c * 16);
            p.scales[j] = ld_row_u16(src + kScaleAt + c * 2);
        }
    }
    p.rope = make_uint4(0, 0, 0, 0);
    if (row) p.rope = ld_row_v4(row + kRopeAt + (lane & 7) * 16);
}

// i0: the warp's first row in the tile.  A thread's four words go to four
// units of one row and block; lanes start at different words, so that the 8
// lanes that store at once go to 8 different units.
__device__ __forceinline__ void decode(const RowPart &p, uint32_t stage, int i0, int lane)
{
    const int c = lane & 15, turn = (c >> 1) & 3;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int i = i0 + 2 * j + (lane >> 4);
        uint32_t s2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2) : "h"((uint16_t)p.scales[j]));
        const __half2 s = __hmul2(*reinterpret_cast<__half2 *>(&s2), __half2half2(__ushort_as_half(0x5800)));   // 2^7
        const __half2 lo = __low2half2(s), hi = __high2half2(s);
        const uint4 v = p.codes[j];
        uint4 a = (turn & 1) ? make_uint4(v.y, v.z, v.w, v.x) : v;
        a = (turn & 2) ? make_uint4(a.z, a.w, a.x, a.y) : a;       // word (w + turn) % 4 in place w
        const uint32_t row = stage + (c >> 1) * BLOCK + i * 128;
        auto put = [&](uint32_t word, int w) {
            const int n = (w + turn) & 3;
            st_smem_v4(row + ((((c & 1) * 4 + n) ^ (i & 7)) << 4), decode8(word, n & 2 ? hi : lo));
        };
        put(a.x, 0);
        put(a.y, 1);
        put(a.z, 2);
        put(a.w, 3);
    }
    st_smem_v4(swizzled(stage + ROPE_BLOCK, i0 + (lane >> 3), lane & 7), p.rope);
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

// Query rows [h0, h0 + 64) into shared memory, by whole warps (QROWS rows
// each, all their loads in flight); rows past H are zero.
constexpr int QROWS = (HEADS + AT_NT / 32 - 1) / (AT_NT / 32);

template <int DT>
__device__ __forceinline__ void stage_queries(const AttendLaunch &a, int r, int h0, uint32_t dst, float *factor,
                                              int warp, int lane)
{
    uint4 v[QROWS][2], rope[QROWS];
#pragma unroll
    for (int n = 0; n < QROWS; ++n) {
        const int i = warp + n * (AT_NT / 32), h = h0 + i;
        v[n][0] = v[n][1] = rope[n] = make_uint4(0, 0, 0, 0);
        if (i < HEADS && h < a.H) {
            const uint8_t *q = a.q + (int64_t)r * a.q_rs + (int64_t)h * a.q_hs;
            v[n][0] = ld_row_v4(q + lane * 16);
            v[n][1] = ld_row_v4(q + 512 + lane * 16);
            if (lane < 8) rope[n] = ld_row_v4(q + kLatent * 2 + lane * 16);
        }
    }
#pragma unroll
    for (int n = 0; n < QROWS; ++n) {
        const int i = warp + n * (AT_NT / 32);
        if (i >= HEADS) break;
        uint32_t m = 0;   // magnitudes compare as integers
#pragma unroll
        for (int part = 0; part < 3; ++part) {
            const uint4 x = part < 2 ? v[n][part] : rope[n];
            m = __vmaxu2(m, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                     __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
        }
        const uint32_t top = __reduce_max_sync(0xffffffffu, max(m >> 16, m & 0xFFFFu));
        // exponent of the largest value; 0 for none and for infinities and
        // NaN, which pass through as they are
        int e = (int)(__float_as_uint(pair_to_float<DT>(top).x) >> 23) - 127;
        if (top == 0 || e == 128) e = 0;
        e = max(e, -119);
        const float up = exp2i(-e), u7 = exp2i(7 - e);    // the latter: decode8's 2^7
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float2 x0 = pair_to_float<DT>(v[n][half].x), x1 = pair_to_float<DT>(v[n][half].y);
            const float2 x2 = pair_to_float<DT>(v[n][half].z), x3 = pair_to_float<DT>(v[n][half].w);
            // the order of decode8
            const uint4 h = make_uint4(floats_to_pair<kF16>(x0.x * u7, x2.x * u7), floats_to_pair<kF16>(x0.y * u7, x2.y * u7),
                                       floats_to_pair<kF16>(x1.x * u7, x3.x * u7), floats_to_pair<kF16>(x1.y * u7, x3.y * u7));
            const int unit = half * 32 + lane;
            st_smem_v4(swizzled(dst + (unit >> 3) * BLOCK, i, unit & 7), h);
        }
        if (lane < 8) {
            auto scaled = [&](uint32_t w) {
                const float2 x = pair_to_float<DT>(w);
                return floats_to_pair<DT>(x.x * up, x.y * up);
            };
            st_smem_v4(swizzled(dst + ROPE_BLOCK, i, lane),
                       make_uint4(scaled(rope[n].x), scaled(rope[n].y), scaled(rope[n].z), scaled(rope[n].w)));
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

template <int DT>
__global__ void __launch_bounds__(AT_NT, 1) attend_kernel(const __grid_constant__ AttendLaunch a,
                                                          const __grid_constant__ AttendParts w)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    // this call's own next launch may be placed now; it waits for this grid
    if (w.splits > 1 || a.weights) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    AttendSmem &sm = *reinterpret_cast<AttendSmem *>(smem + STAGES * OPERAND);
    const uint32_t stages = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int head_tiles = (a.H + HEADS - 1) / HEADS;
    const int ht = blockIdx.x % head_tiles;
    const int split = (blockIdx.x / head_tiles) % w.splits;
    const int r = blockIdx.x / head_tiles / w.splits;
    const int h0 = ht * HEADS;
    const int k0 = split * w.tiles_per_split * TILE;
    const int rows = min(a.k - k0, w.tiles_per_split * TILE);
    const int tiles = (rows + TILE - 1) / TILE;

    const bool decodes = warp >= SOFTMAX_WARPS && warp < MMA_WARP;
    const int dw = warp - SOFTMAX_WARPS;      // its rows of a tile: 4 dw to 4 dw + 3
    const int32_t *ids = a.ids + (int64_t)r * a.ids_stride + k0;
    auto id_at = [&](int t) {
        const int n = t * TILE + dw * 4 + (lane >> 3);
        return n < rows ? ids[n] : -1;
    };
    RowPart next;
    const uint8_t *row = nullptr;
    int32_t id = -1;
    int bad = 0;
    if (decodes) {       // the first tile's rows are on their way while the queries are staged
        row = row_of(a, r, id_at(0), &bad);
        id = id_at(1);
        fetch(next, row, lane);
    }
    const uint32_t q_at = stages + (STAGES - 1) * OPERAND;   // the queries, until they are in tensor memory
    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&sm.full[s]), DECODE_WARPS);
            mbar_init(smem_u32(&sm.empty[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&sm.scored[s]), 1);
            mbar_init(smem_u32(&sm.weighed[s]), SOFTMAX_WARPS);
        }
        mbar_init(smem_u32(&sm.queries), SOFTMAX_WARPS);
        mbar_init(smem_u32(&sm.drained), 1);
        sm.gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == MMA_WARP) tmem_alloc_all(smem_u32(&sm.tmem));
    stage_queries<DT>(a, r, h0, q_at, sm.factor, warp, lane);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    volatile int *gave_up = &sm.gave_up;
    auto all = [](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };

    if (decodes) {
        // ---- fetch and decode -----------------------------------------------
        int s = 0, phase = 1;     // the phase whose end frees stage s
#pragma unroll 2
        for (int t = 0; t < tiles; ++t) {
            const RowPart now = next;
            const uint32_t named = __ballot_sync(0xffffffffu, row != nullptr);    // lanes 0, 8, 16, 24
            row = row_of(a, r, id, &bad);
            fetch(next, row, lane);
            id = id_at(t + 2);
            const bool free = t < STAGES - 1    ? true
                              : t == STAGES - 1 ? mbar_wait(smem_u32(&sm.queries), 0, gave_up)
                                                : mbar_wait(smem_u32(&sm.empty[s]), phase, gave_up);
            if (!all(free)) break;
            decode(now, stages + s * OPERAND, dw * 4, lane);
            if (lane == 0)
                sm.valid[s][dw] = (uint8_t)((named & 1u) | (named >> 7 & 2u) | (named >> 14 & 4u) | (named >> 21 & 8u));
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.full[s]));
            if (++s == STAGES) s = 0, phase ^= 1;
        }
        if (bad && a.status) atomicOr(a.status + r, bad);
    } else if (warp == MMA_WARP) {
        // ---- MMA issue -----------------------------------------------------------
        constexpr uint32_t qk = mma_desc(HEADS, TILE, false, false);
        constexpr uint32_t qk_rope = mma_desc(HEADS, TILE, DT == kBf16, false);
        constexpr uint32_t pv = mma_desc(HEADS, 256, false, true);
        bool ok = all(mbar_wait(smem_u32(&sm.queries), 0, gave_up));
        int s = 0, s_pv = 0, phase = 0;
        for (int t = 0; ok && t <= tiles; ++t) {
            if (t < tiles) {            // S(t) = Q K^T
                if (!(ok = all(mbar_wait(smem_u32(&sm.full[s]), phase, gave_up)))) break;
                tc_fence_after();
                const uint64_t k_desc = smem_desc(stages + s * OPERAND, 16, 1024);
                const uint32_t d = tmem + (t & 1) * TILE;
                if (elect_one()) {
#pragma unroll
                    for (int b = 0; b < 9; ++b)
#pragma unroll
                        for (int x = 0; x < 4; ++x)      // 16 values a step: 32 bytes, 8 columns
                            mma_f16_ts(d, tmem + TMEM_Q + (b * 4 + x) * 8, k_desc + ((b * BLOCK + x * 32) >> 4),
                                       b < 8 ? qk : qk_rope, b + x > 0);
                    mma_commit(smem_u32(&sm.scored[t & 1]));
                }
                __syncwarp();
                if (++s == STAGES) s = 0, phase ^= 1;
            }
            if (t > 0) {                // O += P(t - 1) V
                if (!(ok = all(mbar_wait(smem_u32(&sm.weighed[(t - 1) & 1]), ((t - 1) >> 1) & 1, gave_up)))) break;
                tc_fence_after();
                const uint32_t stage = stages + s_pv * OPERAND;
                const uint64_t p_desc = smem_desc(stage + ROPE_BLOCK, 16, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint64_t v_desc = smem_desc(stage + half * 4 * BLOCK, BLOCK, 1024);
#pragma unroll
                        for (int x = 0; x < 4; ++x)       // 16 rows a step
                            mma_f16(tmem + TMEM_UPPER + half * 256, p_desc + ((x * 32) >> 4),
                                    v_desc + ((x * 2048) >> 4), pv, t - 1 + x > 0);
                    }
                    mma_commit(smem_u32(&sm.empty[s_pv]));
                }
                __syncwarp();
                if (++s_pv == STAGES) s_pv = 0;
            }
        }
        if (!ok) {     // let what was issued end before the CTA goes
            if (elect_one()) mma_commit(smem_u32(&sm.drained));
            const uint32_t bar = smem_u32(&sm.drained);
            for (int i = 0; i < (1 << 20) && !mbar_try(bar, 0); ++i) {}
        }
        __syncwarp();
    } else {
        // ---- softmax --------------------------------------------------------------
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        {   // the queries of this warp's 16 heads: 16 columns (32 values) at a time
            const int i = warp * 16 + (lane & 15);
#pragma unroll 2
            for (int c = 0; c < 18; ++c) {
                uint32_t v[16];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint4 x = ld_smem_v4(swizzled(q_at + (c >> 1) * BLOCK, i, (c & 1) * 4 + u));
                    v[4 * u] = x.x, v[4 * u + 1] = x.y, v[4 * u + 2] = x.z, v[4 * u + 3] = x.w;
                }
                // (the upper lanes get them too: O starts there later)
                tmem_st_32x16(lanes + TMEM_Q + c * 16, v);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.queries));
        }
        const int g = lane >> 2, c2 = (lane & 3) * 2;     // fragment row and column
        const int vs = (c2 >> 2) * 8 + (c2 & 3);          // its bit in valid's 16-bit pieces
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
        int s = 0, phase = 0, s_before = 0, phase_before = 0;     // of tile t, of tile t - 1
        for (int t = 0; t < tiles; ++t) {
            ok = all(mbar_wait(smem_u32(&sm.full[s]), phase, gave_up) &&
                     mbar_wait(smem_u32(&sm.scored[t & 1]), (t >> 1) & 1, gave_up));
            if (!ok) break;
            tc_fence_after();
            uint32_t v[32];
            tmem_ld_16x64(lanes + (t & 1) * TILE, v);
            const uint4 valid = *reinterpret_cast<const uint4 *>(sm.valid[s]);
            const uint32_t named[4] = {valid.x >> vs, valid.y >> vs, valid.z >> vs, valid.w >> vs};
            tmem_wait_ld();
            float (&x)[32] = reinterpret_cast<float (&)[32]>(v);
            float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const bool on = (named[j >> 1] >> ((j & 1) * 16 + b)) & 1u;
                    x[4 * j + b] = on ? x[4 * j + b] * f0 : -INFINITY;
                    x[4 * j + 2 + b] = on ? x[4 * j + 2 + b] * f1 : -INFINITY;
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
                    ok = all(mbar_wait(smem_u32(&sm.empty[s_before]), phase_before, gave_up));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < kLatent; c += 64) {
                        uint32_t o[32];
                        tmem_ld_16x64(lanes + TMEM_UPPER + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            o[j] = __float_as_uint(__uint_as_float(o[j]) * (j & 2 ? d1 : d0));
                        tmem_st_16x64(lanes + TMEM_UPPER + c, o);
                    }
                    tmem_wait_st();
                }
            }
            const float r0 = m0 == -INFINITY ? 0.0f : m0, r1 = m1 == -INFINITY ? 0.0f : m1;
            const uint32_t p_at = stages + s * OPERAND + ROPE_BLOCK;
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
            if (lane == 0) mbar_arrive(smem_u32(&sm.weighed[t & 1]));
            s_before = s, phase_before = phase;
            if (++s == STAGES) s = 0, phase ^= 1;
        }
        // the last product, then O / l or this part's O, m and l
        if (ok) ok = all(mbar_wait(smem_u32(&sm.empty[s_before]), phase_before, gave_up));
        if (ok) {
            tc_fence_after();
            l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
            l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
            const bool whole = w.splits == 1, odd = lane & 1;
            // columns hold values in decode8's order: after an exchange with
            // its neighbour, this thread holds values d, d + 1 of each eight
            const int d = (lane & 2) + (odd ? 4 : 0);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int h = h0 + (half ? i1 : i0);
                const float l = half ? l1 : l0, m = half ? m1 : m0;
                if ((lane & 3) || h >= a.H) continue;
                const int64_t rh = (int64_t)r * a.H + h;
                if (whole) {
                    const float l2 = l == 0.0f ? -INFINITY : m + log2f(l);
                    if (a.lse) a.lse[rh] = l2 * kLn2;
                    if (a.weights) w.lse2[rh] = l2;
                } else {
                    *reinterpret_cast<float2 *>(w.ml + ((int64_t)split * a.R * a.H + rh) * 2) = make_float2(m, l);
                }
            }
            const float inv0 = l0 == 0.0f ? 0.0f : 128.0f / l0, inv1 = l1 == 0.0f ? 0.0f : 128.0f / l1;
            const bool on0 = h0 + i0 < a.H, on1 = h0 + i1 < a.H;
            const int64_t rh0 = (int64_t)r * a.H + h0 + i0;
            float *o0 = w.o + ((int64_t)split * a.R * a.H + rh0) * kLatent + d, *o1 = o0 + 8 * kLatent;
            uint8_t *out0 = a.out + (int64_t)r * a.out_rs + (int64_t)(h0 + i0) * a.out_hs + d * 2, *out1 = out0 + 8 * a.out_hs;
#pragma unroll 1
            for (int c = 0; c < kLatent; c += 64) {
                uint32_t v[32];
                tmem_ld_16x64(lanes + TMEM_UPPER + c, v);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const float x = __uint_as_float(v[4 * j + 2 * half]), y = __uint_as_float(v[4 * j + 2 * half + 1]);
                        const float got = __shfl_xor_sync(0xffffffffu, odd ? x : y, 1);
                        const float lo = odd ? got : x, hi = odd ? y : got;
                        if (!(half ? on1 : on0)) continue;
                        if (whole) {
                            const float inv = half ? inv1 : inv0;
                            *reinterpret_cast<uint32_t *>((half ? out1 : out0) + (c + 8 * j) * 2) =
                                floats_to_pair<DT>(lo * inv, hi * inv);
                        } else {
                            *reinterpret_cast<float2 *>((half ? o1 : o0) + c + 8 * j) = make_float2(lo, hi);
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

// out = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s.  A CTA joins one
// (request, head), 4 values a thread; lane s of each warp holds part s's
// factor.  Bound by latency: the references, then all of the parts at once.
constexpr int JN_NT = 128;
constexpr int MAX_SPLITS = 32;     // one lane each

template <int DT>
__global__ void __launch_bounds__(JN_NT) join_kernel(const __grid_constant__ AttendLaunch a,
                                                     const __grid_constant__ AttendParts w)
{
    const int64_t rh = blockIdx.x, RH = (int64_t)a.R * a.H;
    const int r = (int)(rh / a.H), h = (int)(rh - (int64_t)r * a.H), tid = threadIdx.x, lane = tid & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float2 ml = make_float2(-INFINITY, 0.0f);
    if (lane < w.splits) ml = *reinterpret_cast<const float2 *>(w.ml + (lane * RH + rh) * 2);
    const float *o_part = w.o + rh * kLatent + tid * 4;
    constexpr int AHEAD = 8;
    float4 p[AHEAD];
#pragma unroll
    for (int s = 0; s < AHEAD; ++s)
        if (s < w.splits) p[s] = *reinterpret_cast<const float4 *>(o_part + s * RH * kLatent);
    float top = ml.x;
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float factor = exp2f(ml.x - (top == -INFINITY ? 0.0f : top));
    float l = factor * ml.y;
    for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s0 = 0; s0 < w.splits; s0 += AHEAD) {
#pragma unroll
        for (int s = 0; s < AHEAD; ++s) {
            if (s0 + s >= w.splits) break;
            const float f = __shfl_sync(0xffffffffu, factor, s0 + s);
            o.x = fmaf(f, p[s].x, o.x);
            o.y = fmaf(f, p[s].y, o.y);
            o.z = fmaf(f, p[s].z, o.z);
            o.w = fmaf(f, p[s].w, o.w);
            if (s0 + s + AHEAD < w.splits)
                p[s] = *reinterpret_cast<const float4 *>(o_part + (s0 + s + AHEAD) * RH * kLatent);
        }
    }
    const float inv = l == 0.0f ? 0.0f : 128.0f / l;
    uint8_t *out = a.out + (int64_t)r * a.out_rs + (int64_t)h * a.out_hs;
    *reinterpret_cast<uint2 *>(out + tid * 8) =
        make_uint2(floats_to_pair<DT>(o.x * inv, o.y * inv), floats_to_pair<DT>(o.z * inv, o.w * inv));
    if (tid == 0) {
        const float l2 = l == 0.0f ? -INFINITY : top + log2f(l);
        if (a.lse) a.lse[rh] = l2 * kLn2;
        if (a.weights) w.lse2[rh] = l2;
    }
}

// ---- weights -----------------------------------------------------------------------

// weights[position] += sum over the heads of 2^(score - lse2).  A CTA takes 64
// rows of a request: a warp reads 64 scores of a head (256 bytes) at a time,
// the 8 warps take the heads in turn, and their sums meet in shared memory in
// a fixed order.  Bound by reading the scores once.
constexpr int WT_NT = 256, WT_ROWS = 64, WT_WARPS = WT_NT / 32;

__global__ void __launch_bounds__(WT_NT) weights_kernel(const __grid_constant__ AttendLaunch a,
                                                        const __grid_constant__ AttendParts w)
{
    __shared__ float sums[WT_WARPS][WT_ROWS];
    const int r = blockIdx.y, i0 = blockIdx.x * WT_ROWS, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c0 = i0 + lane, c1 = c0 + 32;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float *s = w.scores + (int64_t)r * a.H * a.k, *lse2 = w.lse2 + (int64_t)r * a.H;
    const bool on0 = c0 < a.k, on1 = c1 < a.k;
    float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll 8
    for (int h = warp; h < a.H; h += WT_WARPS) {
        const float ref = lse2[h];
        const float x0 = on0 ? s[(int64_t)h * a.k + c0] : -INFINITY, x1 = on1 ? s[(int64_t)h * a.k + c1] : -INFINITY;
        sum0 += exp2f(x0 - ref);
        sum1 += exp2f(x1 - ref);
    }
    sums[warp][lane] = sum0;
    sums[warp][lane + 32] = sum1;
    __syncthreads();
    const int i = i0 + threadIdx.x;
    if (threadIdx.x >= WT_ROWS || i >= a.k) return;
    int bad = 0;
    if (!row_of(a, r, a.ids[(int64_t)r * a.ids_stride + i], &bad)) return;
    const int64_t pos = a.positions[(int64_t)r * a.positions_stride + i];
    if (pos < 0 || pos >= a.weights_tokens) {
        if (a.status) record_status(a.status, r, kStatusBadPosition);
        return;
    }
    float sum = 0.0f;
#pragma unroll
    for (int x = 0; x < WT_WARPS; ++x) sum += sums[x][threadIdx.x];
    atomicAdd(a.weights + (int64_t)r * a.weights_stride + pos, sum);
}

// How many parts each request's rows are split into: the count for which the
// waves of CTAs (one on each SM) take the fewest tiles, counting a CTA's own
// start and end as three.
int choose_splits(int64_t units, int tiles, int num_sms)
{
    int best = 1;
    int64_t best_cost = INT64_MAX;
    for (int s = 1; s <= tiles && s <= MAX_SPLITS; ++s) {
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
        e = launch_after(weights_kernel, dim3((a.k + WT_ROWS - 1) / WT_ROWS, a.R), WT_NT, s, a, w);
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
