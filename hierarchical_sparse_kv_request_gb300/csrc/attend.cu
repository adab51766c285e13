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
// The rows of a request are split over the CTAs of a cluster when there are
// few (request, head tile) pairs.  At the end the CTAs of a cluster share out
// the heads: every CTA writes its part of a head's O from tensor memory into
// the shared memory of the CTA that joins it (writes, as nothing waits for
// them; reading took several times as long).  With weights, the scores
// (base 2) go to the workspace and a second launch adds up each row's
// probabilities over the heads.
#include <atomic>
#include <cfloat>
#include <mutex>

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

constexpr int MAX_SPLITS = 16;                   // CTAs a cluster
// At the end, where the tiles were: a part of a head's O a slot (no bank
// conflict between 8 slots).
constexpr int SLOTS = HEADS + MAX_SPLITS - 1;
constexpr uint32_t O_STRIDE = (kLatent + 8) * 4;
static_assert(SLOTS * O_STRIDE <= STAGES * OPERAND, "O fits where the tiles were");

struct AttendSmem {
    uint64_t full[STAGES], empty[STAGES], scored[2], weighed[2], fetched[SOFTMAX_WARPS], queries, drained;
    uint32_t tmem;
    int gave_up;
    __align__(16) uint8_t valid[STAGES][16];   // bit b of byte n: row 4 n + b of the stage's tile is named
    float factor[HEADS];      // |scale| * log2(e) * the query's power of two, > 0
    float2 ml[SLOTS];         // at the end: reference and sum of each slot (see join)
};
// Queries on their way to tensor memory start at the last stage and reach a
// little past it.
constexpr uint32_t Q_AT = (STAGES - 1) * OPERAND, MISC_AT = STAGES * OPERAND + HEADS * 16;
constexpr size_t AT_SMEM = MISC_AT + sizeof(AttendSmem);

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

__device__ __forceinline__ uint2 ld_smem_v2(uint32_t at)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
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

// Eight codes (a 32-bit word of a row) times scale, as f16, in the order 0 2 4
// 6 1 3 5 7.  The high byte of an f16 holds its sign, exponent and two bits of
// mantissa: a code's sign in bit 7 and its other bits in 3-1 read as its value
// times 2^-14, subnormal included, and four codes (the even, the odd) are
// placed so at once.  The scale comes with 2^7 of that, the result keeps
// 2^-7.  Exact: at most six significant bits, at least 2^-17.
__device__ __forceinline__ uint4 decode8(uint32_t w, __half2 scale)
{
    const uint32_t even = ((w << 4) & 0x80808080u) | ((w << 1) & 0x0E0E0E0Eu);
    const uint32_t odd = (w & 0x80808080u) | ((w >> 3) & 0x0E0E0E0Eu);
    auto pair = [&](uint32_t bytes, uint32_t select) {
        const uint32_t b = __byte_perm(bytes, 0, select);     // bytes 4-7 are 0
        const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&b), scale);
        return *reinterpret_cast<const uint32_t *>(&v);
    };
    return make_uint4(pair(even, 0x1404), pair(even, 0x3424), pair(odd, 0x1404), pair(odd, 0x3424));
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

// 2^x; less than 2^-126 is 0
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A power of two as float
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// ---- queries -------------------------------------------------------------------------

// A softmax warp brings its 16 heads' queries into shared memory (as they
// are; the last stage is still free) and writes them, scaled, to tensor
// memory in the fragments of a 16x256b store.
constexpr uint32_t Q_STRIDE = kRowValues * 2 + 16;     // no bank conflict between 8 heads

__device__ __forceinline__ void fetch_queries(const AttendLaunch &a, int r, int h0, uint32_t dst, uint32_t bar,
                                              int warp, int lane)
{
    const int heads = min(max(a.H - h0 - warp * 16, 0), 16);
    if (lane == 0) {
        mbar_init(bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(heads * kRowValues * 2) : "memory");
    }
    __syncwarp();
    if (lane < heads) {
        const int i = warp * 16 + lane;
        const uint8_t *src = a.q + (int64_t)r * a.q_rs + (int64_t)(h0 + i) * a.q_hs;
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst + i * Q_STRIDE),
                     "l"(src), "r"(kRowValues * 2), "r"(bar)
                     : "memory");
    }
}

// Largest magnitudes, by halves, of m and 8 values (NaN does not count).
template <int DT>
__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y)
{
    uint32_t z;
    if (DT == kBf16)
        asm("max.bf16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
    else
        asm("max.f16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
    return z;
}

template <int DT>
__device__ __forceinline__ uint32_t magnitude(uint32_t m, uint4 x)
{
    return max2<DT>(m, max2<DT>(max2<DT>(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), max2<DT>(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
}

template <int DT>
__device__ __forceinline__ void place_queries(const AttendLaunch &a, int h0, uint32_t src, uint32_t tmem, float *factor,
                                              int warp, int lane)
{
    const int g = lane >> 2, q = lane & 3, i0 = warp * 16 + g;
    const uint32_t at[2] = {src + i0 * Q_STRIDE, src + (i0 + 8) * Q_STRIDE};
    const bool on[2] = {h0 + i0 < a.H, h0 + i0 + 8 < a.H};
    uint32_t m[2] = {0, 0};      // (of no head: of whatever is there, and not used)
#pragma unroll 1
    for (int n = 0; n < kRowValues / 32; n += 3) {
        uint4 x[6];
#pragma unroll
        for (int j = 0; j < 6; ++j) x[j] = ld_smem_v4(at[j & 1] + ((n + (j >> 1)) * 4 + q) * 16);
#pragma unroll
        for (int j = 0; j < 6; ++j) m[j & 1] = magnitude<DT>(m[j & 1], x[j]);
    }
    float up[2], u7[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t x = m[half];
        x = max2<DT>(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = max2<DT>(x, __shfl_xor_sync(0xffffffffu, x, 2));
        const uint32_t top = max(x >> 16, x & 0xFFFFu);
        // exponent of the largest value; 0 for none and for infinities, which
        // pass through as they are (as NaN does)
        int e = (int)(__float_as_uint(pair_to_float<DT>(top).x) >> 23) - 127;
        if (top == 0 || e == 128) e = 0;
        e = max(e, -119);      // (2^(7 - e) is a float)
        // with the sign of the scale, so that the factor of the scores is
        // positive; u7: decode8's 2^7
        up[half] = copysignf(exp2i(-e), a.scale);
        u7[half] = 128.0f * up[half];
        if (q == 0) factor[i0 + 8 * half] = fmaxf(fabsf(a.scale) * kLog2e * exp2i(e), FLT_MIN);
    }
    // Latent columns 8 j + 2 q and + 1 hold the even (q even) or the odd
    // values of the eight at 16 j + 8 (q / 2): the order of decode8.
    const uint32_t pick = q & 1 ? 0x7632 : 0x5410;
#pragma unroll 1
    for (int c = 0; c < kLatent / 2; c += 64) {
        uint32_t v[32];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            uint4 x[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) x[n] = ld_smem_v4(at[n & 1] + (c + 8 * (j + (n >> 1))) * 4 + (q >> 1) * 16);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int half = n & 1, to = 4 * (j + (n >> 1)) + 2 * half;
                const float2 y = pair_to_float<DT>(__byte_perm(x[n].x, x[n].y, pick));
                const float2 z = pair_to_float<DT>(__byte_perm(x[n].z, x[n].w, pick));
                v[to] = on[half] ? floats_to_pair<kF16>(y.x * u7[half], y.y * u7[half]) : 0u;
                v[to + 1] = on[half] ? floats_to_pair<kF16>(z.x * u7[half], z.y * u7[half]) : 0u;
            }
        }
        tmem_st_16x64(tmem + c, v);
    }
    uint32_t v[16];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const uint2 x = ld_smem_v2(at[half] + kLatent * 2 + (8 * j + 2 * q) * 4);
            const float2 y = pair_to_float<DT>(x.x), z = pair_to_float<DT>(x.y);
            v[4 * j + 2 * half] = on[half] ? floats_to_pair<DT>(y.x * up[half], y.y * up[half]) : 0u;
            v[4 * j + 2 * half + 1] = on[half] ? floats_to_pair<DT>(z.x * up[half], z.y * up[half]) : 0u;
        }
    tmem_st_16x32(tmem + kLatent / 2, v);
    tmem_wait_st();
}

// How a call is cut up, and its workspace.
struct AttendParts {
    int splits, tiles_per_split;
    float *lse2;            // [R][H] log2 of the sums, for the weights
    float *scores;          // [R][H][score_stride] base-2 scores, for the weights
    int64_t score_stride;   // whole tiles
};

// This CTA's shared-memory address `at` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t at, int rank)
{
    uint32_t y;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(y) : "r"(at), "r"(rank));
    return y;
}

__device__ __forceinline__ void st_cluster_v2(uint32_t at, uint32_t x, uint32_t y)
{
    asm volatile("st.shared::cluster.v2.u32 [%0], {%1,%2};" ::"r"(at), "r"(x), "r"(y) : "memory");
}

__device__ __forceinline__ void cluster_sync_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int DT>
__global__ void __launch_bounds__(AT_NT, 1) attend_kernel(const __grid_constant__ AttendLaunch a,
                                                          const __grid_constant__ AttendParts w)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    // this call's own next launch may be placed now; it waits for this grid
    if (a.weights) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    AttendSmem &sm = *reinterpret_cast<AttendSmem *>(smem + MISC_AT);
    const uint32_t stages = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int head_tiles = (a.H + HEADS - 1) / HEADS;
    const int split = blockIdx.x % w.splits;          // the CTA's rank in its cluster
    const int ht = (blockIdx.x / w.splits) % head_tiles;
    const int r = blockIdx.x / w.splits / head_tiles;
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
    if (decodes) {
        const int32_t id0 = id_at(0);
        id = id_at(1);
        row = row_of(a, r, id0, &bad);
        fetch(next, row, lane);
    } else if (warp < SOFTMAX_WARPS) {
        fetch_queries(a, r, h0, stages + Q_AT, smem_u32(&sm.fetched[warp]), warp, lane);
    } else {
        if (lane == 0) {
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
        __syncwarp();
        tmem_alloc_all(smem_u32(&sm.tmem));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    volatile int *gave_up = &sm.gave_up;
    auto all = [](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };

    // softmax threads: reference and sum of heads lane / 4 and lane / 4 + 8 of
    // the warp's 16
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
    if (decodes) {
        // ---- fetch and decode -----------------------------------------------
        int s = 0, phase = 1;     // the phase whose end frees stage s
#pragma unroll 1
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
                if (elect_one()) {
                    uint64_t k_desc = smem_desc(stages + s * OPERAND, 16, 1024);
                    uint32_t q_col = tmem + TMEM_Q;
                    const uint32_t d = tmem + (t & 1) * TILE;
#pragma unroll 1
                    for (int b = 0; b < 9; ++b, k_desc += BLOCK >> 4, q_col += 32) {
                        const uint32_t kind = b < 8 ? qk : qk_rope;
#pragma unroll
                        for (int x = 0; x < 4; ++x)      // 16 values a step: 32 bytes, 8 columns
                            mma_f16_ts(d, q_col + x * 8, k_desc + ((x * 32) >> 4), kind, b + x > 0);
                    }
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
#pragma unroll 1
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
        bool ok = all(mbar_wait(smem_u32(&sm.fetched[warp]), 0, gave_up));
        for (int i = 0; !ok && i < (1 << 20) && !mbar_try(smem_u32(&sm.fetched[warp]), 0); ++i) {}
        place_queries<DT>(a, h0, stages + Q_AT, lanes + TMEM_Q, sm.factor, warp, lane);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.queries));
        const int g = lane >> 2, c2 = (lane & 3) * 2;     // fragment row and column
        const int vs = (c2 >> 2) * 8 + (c2 & 3);          // its bit in valid's 16-bit pieces
        const int i0 = warp * 16 + g, i1 = i0 + 8;
        const float f0 = sm.factor[i0], f1 = sm.factor[i1];
        float *sc0 = nullptr, *sc1 = nullptr;
        if (a.weights) {
            float *at = w.scores + ((int64_t)r * a.H + h0) * w.score_stride + k0 + c2;
            if (h0 + i0 < a.H) sc0 = at + (int64_t)i0 * w.score_stride;
            if (h0 + i1 < a.H) sc1 = at + (int64_t)i1 * w.score_stride;
        }
        int s = 0, phase = 0, s_before = 0, phase_before = 0;     // of tile t, of tile t - 1
        for (int t = 0; ok && t < tiles; ++t) {
            ok = all(mbar_wait(smem_u32(&sm.full[s]), phase, gave_up) &&
                     mbar_wait(smem_u32(&sm.scored[t & 1]), (t >> 1) & 1, gave_up));
            if (!ok) break;
            tc_fence_after();
            uint32_t v[32];
            tmem_ld_16x64(lanes + (t & 1) * TILE, v);
            const uint4 valid = *reinterpret_cast<const uint4 *>(sm.valid[s]);
            tmem_wait_ld();
            float (&x)[32] = reinterpret_cast<float (&)[32]>(v);     // 1 / f0, 1 / f1 of the scores
            if ((valid.x & valid.y & valid.z & valid.w) != 0x0F0F0F0Fu) {
                const uint32_t named[4] = {valid.x >> vs, valid.y >> vs, valid.z >> vs, valid.w >> vs};
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        if (!((named[j >> 1] >> ((j & 1) * 16 + b)) & 1u)) x[4 * j + b] = x[4 * j + 2 + b] = -INFINITY;
            }
            if (a.weights) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = t * TILE + 8 * j;
                    if (sc0) *reinterpret_cast<float2 *>(sc0 + c) = make_float2(x[4 * j] * f0, x[4 * j + 1] * f0);
                    if (sc1) *reinterpret_cast<float2 *>(sc1 + c) = make_float2(x[4 * j + 2] * f1, x[4 * j + 3] * f1);
                }
            }
            float top0 = fmaxf(x[0], x[1]), top1 = fmaxf(x[2], x[3]);
#pragma unroll
            for (int j = 1; j < 8; ++j) {
                top0 = fmaxf(top0, fmaxf(x[4 * j], x[4 * j + 1]));
                top1 = fmaxf(top1, fmaxf(x[4 * j + 2], x[4 * j + 3]));
            }
            top0 *= f0;
            top1 *= f1;
            top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, 1));
            top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, 1));
            top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, 2));
            top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, 2));
            if (__any_sync(0xffffffffu, top0 > m0 + kMoveAbove || top1 > m1 + kMoveAbove)) {
                const float n0 = fmaxf(m0, top0), n1 = fmaxf(m1, top1);
                const float d0 = n0 == -INFINITY ? 1.0f : ex2(m0 - n0), d1 = n1 == -INFINITY ? 1.0f : ex2(m1 - n1);
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
            const float r0 = m0 == -INFINITY ? 0.0f : -m0, r1 = m1 == -INFINITY ? 0.0f : -m1;
            // unit j of row i0: bits 6-4 of the address are j ^ (i0 & 7)
            const uint32_t p_at = stages + s * OPERAND + ROPE_BLOCK + i0 * 128 + (g << 4) + c2 * 2;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float p00 = ex2(fmaf(x[4 * j], f0, r0)), p01 = ex2(fmaf(x[4 * j + 1], f0, r0));
                const float p10 = ex2(fmaf(x[4 * j + 2], f1, r1)), p11 = ex2(fmaf(x[4 * j + 3], f1, r1));
                l0 += p00 + p01;
                l1 += p10 + p11;
                st_smem_u32(p_at ^ (j << 4), floats_to_pair<kF16>(p00, p01));
                st_smem_u32((p_at ^ (j << 4)) + 8 * 128, floats_to_pair<kF16>(p10, p11));
            }
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.weighed[t & 1]));
            s_before = s, phase_before = phase;
            if (++s == STAGES) s = 0, phase ^= 1;
        }
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    }

    // ---- join ----------------------------------------------------------------------
    // Head i is joined by CTA i % splits.  Part p of its m-th head (head p' + m
    // splits, p' its own rank) comes to slot p + m splits of its shared memory,
    // once every CTA's last product is done and the tiles are free.
    const int last = tiles - 1, heads = min(HEADS, a.H - h0);
    const bool done = all(mbar_wait(smem_u32(&sm.empty[last % STAGES]), (last / STAGES) & 1, gave_up));
    tc_fence_after();
    if (w.splits > 1) cluster_sync_all();
    if (done && warp < MMA_WARP && (warp & 3) * 16 < heads) {
        const int i0 = (warp & 3) * 16 + (lane >> 2), i1 = i0 + 8;
        const int to0 = i0 % w.splits, to1 = i1 % w.splits;
        const int slot0 = i0 - to0 + split, slot1 = i1 - to1 + split;
        if (warp < SOFTMAX_WARPS && (lane & 3) == 0) {
            if (i0 < heads) st_cluster_v2(in_cta(smem_u32(&sm.ml[slot0]), to0), __float_as_uint(m0), __float_as_uint(l0));
            if (i1 < heads) st_cluster_v2(in_cta(smem_u32(&sm.ml[slot1]), to1), __float_as_uint(m1), __float_as_uint(l1));
        }
        const uint32_t upper = tmem + ((uint32_t)((warp & 3) * 32) << 16) + TMEM_UPPER;
        const uint32_t at0 = in_cta(stages + slot0 * O_STRIDE + (lane & 3) * 8, to0);
        const uint32_t at1 = in_cta(stages + slot1 * O_STRIDE + (lane & 3) * 8, to1);
#pragma unroll 1
        for (int c = (warp >> 2) * 64; c < kLatent; c += (MMA_WARP / 4) * 64) {
            uint32_t v[32];
            tmem_ld_16x64(upper + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (i0 < heads) st_cluster_v2(at0 + (c + 8 * j) * 4, v[4 * j], v[4 * j + 1]);
                if (i1 < heads) st_cluster_v2(at1 + (c + 8 * j) * 4, v[4 * j + 2], v[4 * j + 3]);
            }
        }
        tc_fence_before();
    }
    if (w.splits > 1)
        cluster_sync_all();
    else
        __syncthreads();
    // out = sum_p 2^(m_p - m) O_p / sum_p 2^(m_p - m) l_p, half a head's values a warp
    const int mine = (heads - split + w.splits - 1) / w.splits;
    for (int n = warp; n < 2 * mine; n += AT_NT / 32) {
        const int slot = (n >> 1) * w.splits, d = (n & 1) * 256 + lane * 8;
        float2 ml = make_float2(-INFINITY, 0.0f);      // lane p: part p
        if (lane < w.splits) ml = sm.ml[slot + lane];
        float top = ml.x;
        for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        float factor = ex2(ml.x - (top == -INFINITY ? 0.0f : top));
        float l = factor * ml.y;
        for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
        factor *= l == 0.0f ? 0.0f : 128.0f / l;       // decode8's 2^7
        float o[8] = {};
        const uint32_t at = stages + slot * O_STRIDE + d * 4;
#pragma unroll 2
        for (int p = 0; p < w.splits; ++p) {
            const uint4 x = ld_smem_v4(at + p * O_STRIDE), y = ld_smem_v4(at + p * O_STRIDE + 16);
            const float f = __shfl_sync(0xffffffffu, factor, p);
            // columns are in decode8's order: the even values, then the odd
            o[0] = fmaf(f, __uint_as_float(x.x), o[0]);
            o[2] = fmaf(f, __uint_as_float(x.y), o[2]);
            o[4] = fmaf(f, __uint_as_float(x.z), o[4]);
            o[6] = fmaf(f, __uint_as_float(x.w), o[6]);
            o[1] = fmaf(f, __uint_as_float(y.x), o[1]);
            o[3] = fmaf(f, __uint_as_float(y.y), o[3]);
            o[5] = fmaf(f, __uint_as_float(y.z), o[5]);
            o[7] = fmaf(f, __uint_as_float(y.w), o[7]);
        }
        const int h = h0 + split + slot;
        st_v4(a.out + (int64_t)r * a.out_rs + (int64_t)h * a.out_hs + d * 2,
              make_uint4(floats_to_pair<DT>(o[0], o[1]), floats_to_pair<DT>(o[2], o[3]),
                         floats_to_pair<DT>(o[4], o[5]), floats_to_pair<DT>(o[6], o[7])));
        if (lane == 0 && !(n & 1)) {
            const int64_t rh = (int64_t)r * a.H + h;
            const float l2 = l == 0.0f ? -INFINITY : top + log2f(l);
            if (a.lse) a.lse[rh] = l2 * kLn2;
            if (a.weights) w.lse2[rh] = l2;
        }
    }
    if (tid == 0 && sm.gave_up && a.status) record_status(a.status, r, kStatusAttendTimeout);
    if (warp == MMA_WARP) tmem_free_all(tmem);
}

// ---- weights -----------------------------------------------------------------------

// weights[position] += sum over the heads of 2^(score - lse2).  A CTA takes 64
// rows of a request: a warp reads 64 scores of a head (256 bytes) at a time,
// the 8 warps take the heads in turn, and their sums meet in shared memory in
// a fixed order.  Bound by reading the scores once.
constexpr int WT_NT = 256, WT_ROWS = TILE, WT_WARPS = WT_NT / 32;

__global__ void __launch_bounds__(WT_NT) weights_kernel(const __grid_constant__ AttendLaunch a,
                                                        const __grid_constant__ AttendParts w)
{
    __shared__ float sums[WT_WARPS][WT_ROWS];
    const int r = blockIdx.y, i0 = blockIdx.x * WT_ROWS, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float *s = w.scores + (int64_t)r * a.H * w.score_stride, *lse2 = w.lse2 + (int64_t)r * a.H;
    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll 8
    for (int h = warp; h < a.H; h += WT_WARPS) {
        const float ref = lse2[h];
        const float2 x = *reinterpret_cast<const float2 *>(s + h * w.score_stride + i0 + 2 * lane);
        sum.x += ex2(x.x - ref);
        sum.y += ex2(x.y - ref);
    }
    *reinterpret_cast<float2 *>(&sums[warp][2 * lane]) = sum;
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
    float total = 0.0f;
#pragma unroll
    for (int x = 0; x < WT_WARPS; ++x) total += sums[x][threadIdx.x];
    atomicAdd(a.weights + (int64_t)r * a.weights_stride + pos, total);
}

// ---- host ----------------------------------------------------------------------------

// Clusters of each size that the device holds at once (0: none), for the
// attention kernel; found once per device.
struct Capacity {
    int clusters[MAX_SPLITS + 1];
};

template <int DT>
cudaError_t prepare_kernel()
{
    cudaError_t e = cudaFuncSetAttribute(attend_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)AT_SMEM);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(attend_kernel<DT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e;
}

void fill_launch(cudaLaunchConfig_t &cfg, cudaLaunchAttribute &attr, unsigned ctas, int splits, cudaStream_t s)
{
    cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(AT_NT);
    cfg.dynamicSmemBytes = AT_SMEM;
    cfg.stream = s;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)splits;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
}

// Capacity of the current device; also sets the kernels' attributes there.
cudaError_t capacity(const Capacity **out)
{
    constexpr int kDevices = 64;
    static Capacity cap[kDevices];
    static std::atomic<int> state[kDevices];      // 0: not known, 1: being found, 2: known
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kDevices) return cudaErrorInvalidDevice;
    if (state[dev].load(std::memory_order_acquire) != 2) {
        static std::mutex one;
        std::lock_guard<std::mutex> lock(one);
        if (state[dev].load(std::memory_order_acquire) != 2) {
            e = prepare_kernel<kBf16>();
            if (e == cudaSuccess) e = prepare_kernel<kF16>();
            cudaFuncAttributes fa;
            if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, weights_kernel);   // loads it
            if (e != cudaSuccess) return e;
            for (int c = 1; c <= MAX_SPLITS; ++c) {
                cudaLaunchConfig_t cfg;
                cudaLaunchAttribute attr;
                fill_launch(cfg, attr, c, c, nullptr);
                int n = 0;
                if (cudaOccupancyMaxActiveClusters(&n, attend_kernel<kBf16>, &cfg) != cudaSuccess) {
                    cudaGetLastError();
                    n = 0;
                }
                cap[dev].clusters[c] = n;
            }
            if (cap[dev].clusters[1] < 1) return cudaErrorInvalidConfiguration;
            state[dev].store(2, std::memory_order_release);
        }
    }
    *out = &cap[dev];
    return cudaSuccess;
}

// How many parts each request's rows are split into, one for each CTA of a
// cluster: the count for which the waves of clusters take the fewest tiles,
// counting a CTA's own start and end as three.
int choose_splits(int64_t units, int tiles, const Capacity &cap)
{
    int best = 1;
    int64_t best_cost = INT64_MAX;
    for (int s = 1; s <= tiles && s <= MAX_SPLITS; ++s) {
        const int per = (tiles + s - 1) / s;
        if (cap.clusters[s] < 1 || (tiles + per - 1) / per != s) continue;
        const int64_t waves = (units + cap.clusters[s] - 1) / cap.clusters[s];
        const int64_t cost = waves * (per + 3);
        if (cost < best_cost) best_cost = cost, best = s;
    }
    return best;
}

int64_t up4(int64_t n) { return (n + 3) / 4 * 4; }

AttendParts lay_out(int32_t R, int32_t H, int32_t k, bool weights, const Capacity &cap, uint8_t *ws, int64_t *bytes)
{
    AttendParts p = {};
    const int64_t RH = (int64_t)R * H;
    const int tiles = (k + TILE - 1) / TILE;
    p.splits = choose_splits((int64_t)R * ((H + HEADS - 1) / HEADS), tiles, cap);
    p.tiles_per_split = (tiles + p.splits - 1) / p.splits;
    p.score_stride = (int64_t)tiles * TILE;
    float *f = reinterpret_cast<float *>(ws);
    int64_t n = 4;          // never empty
    p.lse2 = f + n;
    n += weights ? up4(RH) : 0;
    p.scores = f + n;
    n += weights ? RH * p.score_stride : 0;
    *bytes = n * 4;
    return p;
}

template <int DT>
cudaError_t launch_dt(const AttendLaunch &a, const AttendParts &w, cudaStream_t s)
{
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr;
    fill_launch(cfg, attr, (unsigned)(a.R * ((a.H + HEADS - 1) / HEADS) * w.splits), w.splits, s);
    cudaError_t e = cudaLaunchKernelEx(&cfg, attend_kernel<DT>, a, w);
    if (e == cudaSuccess && a.weights) {
        cfg = {};
        cfg.gridDim = dim3((unsigned)(w.score_stride / WT_ROWS), (unsigned)a.R);
        cfg.blockDim = dim3(WT_NT);
        cfg.stream = s;
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, weights_kernel, a, w);
    }
    return e;
}

}  // namespace

cudaError_t attend_workspace_bytes(int32_t R, int32_t H, int32_t k, bool weights, int64_t *bytes)
{
    const Capacity *cap;
    const cudaError_t e = capacity(&cap);
    if (e == cudaSuccess) lay_out(R, H, k, weights, *cap, nullptr, bytes);
    return e;
}

cudaError_t launch_attend(const AttendLaunch &a, int64_t workspace_bytes, bool *too_small, cudaStream_t s)
{
    const Capacity *cap;
    const cudaError_t e = capacity(&cap);
    if (e != cudaSuccess) return e;
    int64_t bytes;
    const AttendParts w = lay_out(a.R, a.H, a.k, a.weights != nullptr, *cap, a.workspace, &bytes);
    *too_small = workspace_bytes < bytes;
    if (*too_small) return cudaSuccess;
    return a.dtype == kBf16 ? launch_dt<kBf16>(a, w, s) : launch_dt<kF16>(a, w, s);
}

}  // namespace hs
