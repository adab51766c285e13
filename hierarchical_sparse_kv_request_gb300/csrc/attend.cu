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
// At the end a part of a head's O takes a slot where the tiles were (the stride
// keeps the bank conflicts of a 16x256b fragment to two ways).
constexpr uint32_t O_STRIDE = (kLatent + 4) * 4;
constexpr int SLOTS = (STAGES * OPERAND + HEADS * 64) / O_STRIDE;
static_assert(SLOTS >= HEADS + MAX_SPLITS - 1, "the parts that a CTA joins");

struct AttendSmem {
    uint64_t full[STAGES], empty[STAGES], scored[2], weighed[2], fetched[SOFTMAX_WARPS], queries, drained;
    uint32_t tmem;
    int gave_up;
    __align__(16) uint8_t valid[STAGES][16];   // bit b of byte n: row 4 n + b of the stage's tile is named
    float factor[HEADS];      // |scale| * log2(e) * the query's power of two, > 0
    float2 ml[HEADS + MAX_SPLITS];   // at the end: reference and sum of each part of the CTA's
                                     // heads, then its factor
    uint32_t top[HEADS];      // largest magnitude in each query, as its 16 bits
};
// Queries on their way to tensor memory start at the last stage and reach a
// little past it.
constexpr uint32_t Q_AT = (STAGES - 1) * OPERAND, MISC_AT = STAGES * OPERAND + HEADS * 64;
constexpr size_t AT_SMEM = MISC_AT + sizeof(AttendSmem);

// An id as it is, or -1 if it names nothing or is out of range (then its status
// bit is set in *bad).
__device__ __forceinline__ int32_t checked_id(const AttendLaunch &a, int32_t id, int *bad)
{
    if (id == -1) return -1;
    const int64_t n = id & (kResidentFlag - 1);
    const bool resident = id >= 0 && (id & kResidentFlag);
    if (id >= 0 && n < (resident ? a.res_count : a.D)) return id;
    *bad |= 1 << (resident ? kStatusBadResident : kStatusBadIndex);
    return -1;
}

// The row that a checked id names; for -1, the request's row 0 (hot), which is
// there too.
__device__ __forceinline__ const uint8_t *row_of(const AttendLaunch &a, const uint8_t *hot, int32_t id)
{
    if (a.res_count > 0 && id >= 0 && (id & kResidentFlag))
        return a.res + (int64_t)(id & (kResidentFlag - 1)) * a.res_stride;
    return hot + (int64_t)max(id, 0) * a.row_stride;
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

__device__ __forceinline__ void st_smem_v2(uint32_t at, uint32_t x, uint32_t y)
{
    asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(at), "r"(x), "r"(y) : "memory");
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

// A decode warp has four rows of a tile.  Lane: bit 0 and bits 4-3 are a
// number c of 0-7, bits 2-1 the row; the thread takes 16-byte chunks c and c + 8
// of the row's codes and c of its rope part.  So a load of the warp is 128
// contiguous bytes of each row, and the 8 lanes that store at once (four rows,
// two chunks) go to 8 different swizzled units: no bank conflict.
struct RowPart {
    uint4 codes[2], rope;
    uint32_t scales;     // of the two chunks, two e4m3 each
};

__device__ __forceinline__ int lane_row(int lane) { return (lane >> 1) & 3; }
__device__ __forceinline__ int lane_chunk(int lane) { return (lane & 1) + ((lane >> 3) << 1); }

// id: of the lane's row, checked.  For no row (-1) the scales become 0, and with
// them the values of the second product; its scores are masked.
__device__ __forceinline__ void fetch(RowPart &p, const AttendLaunch &a, const uint8_t *hot, int32_t id, int lane)
{
    const int c = lane_chunk(lane);
    const uint8_t *row = row_of(a, hot, id), *src = row + c * 16;
    p.codes[0] = ld_row_v4(src);
    p.codes[1] = ld_row_v4(src + 128);
    p.rope = ld_row_v4(src + kRopeAt);
    const uint32_t s0 = ld_row_u16(row + kScaleAt + c * 2), s1 = ld_row_u16(row + kScaleAt + 16 + c * 2);
    p.scales = id >= 0 ? s0 | (s1 << 16) : 0u;
}

// at: where the first word goes (see decode_at).
__device__ __forceinline__ void decode(const RowPart &p, uint32_t at, uint32_t rope_at)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t s2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2) : "h"((uint16_t)(p.scales >> (16 * j))));
        const __half2 s = __hmul2(*reinterpret_cast<__half2 *>(&s2), __half2half2(__ushort_as_half(0x5800)));   // 2^7
        const __half2 lo = __low2half2(s), hi = __high2half2(s);
        const uint32_t to = at + j * 4 * BLOCK;
        st_smem_v4(to, decode8(p.codes[j].x, lo));
        st_smem_v4(to ^ 16, decode8(p.codes[j].y, lo));
        st_smem_v4(to ^ 32, decode8(p.codes[j].z, hi));
        st_smem_v4(to ^ 48, decode8(p.codes[j].w, hi));
    }
    st_smem_v4(rope_at, p.rope);
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

// A softmax warp has its 16 heads' queries copied to shared memory (as they
// are; the last stage is still free).  Then the warps of each quarter of tensor
// memory (warp % 4), five of them, find the heads' largest magnitudes and write
// the queries, scaled, in the fragments of a 16x256b store.
constexpr uint32_t Q_STRIDE = kRowValues * 2 + 64;     // no bank conflict between neighbours
constexpr int QUARTER_WARPS = MMA_WARP / 4;

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
__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y)      // (the signs mean nothing)
{
    uint32_t z;
    if (DT == kBf16)
        asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
    else
        asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
    return z;
}

template <int DT>
__device__ __forceinline__ uint32_t magnitude(uint32_t m, uint4 x)
{
    return max2<DT>(m, max2<DT>(max2<DT>(x.x, x.y), max2<DT>(x.z, x.w)));
}

// The largest magnitudes (see top) of heads lane / 4 and lane / 4 + 8 of the
// quarter; share: the warp's part of the values.
template <int DT>
__device__ __forceinline__ void measure_queries(uint32_t src, uint32_t *top, int quarter, int share, int lane)
{
    const int i0 = quarter * 16 + (lane >> 2);
    const uint32_t at = src + i0 * Q_STRIDE + (lane & 3) * 16;
    uint32_t m[2] = {0, 0};      // (of no head: of whatever is there, and not used)
#pragma unroll 1
    for (int n = share; n < kRowValues / 32; n += QUARTER_WARPS)
#pragma unroll
        for (int half = 0; half < 2; ++half)
            m[half] = magnitude<DT>(m[half], ld_smem_v4(at + half * 8 * Q_STRIDE + n * 64));
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t x = max2<DT>(m[half], __shfl_xor_sync(0xffffffffu, m[half], 1));
        x = max2<DT>(x, __shfl_xor_sync(0xffffffffu, x, 2));
        x &= 0x7FFF7FFFu;
        if ((lane & 3) == 0) atomicMax(top + i0 + 8 * half, max(x >> 16, x & 0xFFFFu));
    }
}

// Two values times a power of two, exactly: 2^n for bf16, 2^n in two steps for
// f16, whose own powers reach 2^15.
template <int DT>
struct PowerOfTwo {
    uint32_t f[2];
    __device__ __forceinline__ PowerOfTwo(int n, bool negative)
    {
        const float s = negative ? -1.0f : 1.0f;
        if (DT == kBf16) {
            f[0] = floats_to_pair<DT>(s * exp2i(n), s * exp2i(n));
        } else {
            const int a = max(min(n, 15), -14);
            f[0] = floats_to_pair<DT>(s * exp2i(a), s * exp2i(a));
            f[1] = floats_to_pair<DT>(exp2i(n - a), exp2i(n - a));
        }
    }
    __device__ __forceinline__ uint32_t times(uint32_t x) const
    {
        uint32_t y;
        if (DT == kBf16) {
            asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(f[0]));
        } else {
            asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(f[0]));
            asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(y), "r"(f[1]));
        }
        return y;
    }
};

template <int DT>
__device__ __forceinline__ void place_queries(const AttendLaunch &a, int h0, uint32_t src, uint32_t tmem, const uint32_t *top,
                                              float *factor, int quarter, int share, int lane)
{
    const int q = lane & 3, i0 = quarter * 16 + (lane >> 2);
    const uint32_t at = src + i0 * Q_STRIDE;
    int e[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int i = i0 + 8 * half;
        // exponent of the largest value; 0 for none and for infinities, which
        // pass through as they are (as NaN does)
        e[half] = (int)(__float_as_uint(pair_to_float<DT>(top[i]).x) >> 23) - 127;
        if (top[i] == 0 || e[half] == 128) e[half] = 0;
        // (2^(7 - e) is representable, in one step or two)
        e[half] = max(e[half], DT == kBf16 ? -119 : -23);
        if (q == 0 && share == 0) factor[i] = fmaxf(fabsf(a.scale) * kLog2e * exp2i(e[half]), FLT_MIN);
    }
    // with the sign of the scale, so that the factor of the scores is positive
    const bool neg = a.scale < 0.0f;
    const bool on[2] = {h0 + i0 < a.H, h0 + i0 + 8 < a.H};
    // 8 columns a time.  Latent columns 8 j + 2 q and + 1 hold the even (q
    // even) or the odd values of the eight at 16 j + 8 (q / 2), the order of
    // decode8, with its 2^7; rope columns their values in order.
    const PowerOfTwo<DT> up7[2] = {{7 - e[0], neg}, {7 - e[1], neg}};
    const uint32_t pick = q & 1 ? 0x7632 : 0x5410;
#pragma unroll 1
    for (int j = share; j < kLatent / 16; j += QUARTER_WARPS) {
        uint32_t v[4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const uint4 x = ld_smem_v4(at + half * 8 * Q_STRIDE + j * 32 + (q >> 1) * 16);
            uint32_t lo = up7[half].times(__byte_perm(x.x, x.y, pick)), hi = up7[half].times(__byte_perm(x.z, x.w, pick));
            if (DT == kBf16) {
                const float2 y = pair_to_float<DT>(lo), z = pair_to_float<DT>(hi);
                lo = floats_to_pair<kF16>(y.x, y.y);
                hi = floats_to_pair<kF16>(z.x, z.y);
            }
            v[2 * half] = on[half] ? lo : 0u;
            v[2 * half + 1] = on[half] ? hi : 0u;
        }
        tmem_st_16x8(tmem + j * 8, v);
    }
    if (share < 4) {
        const PowerOfTwo<DT> up[2] = {{-e[0], neg}, {-e[1], neg}};
        uint32_t v[4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const uint2 x = ld_smem_v2(at + half * 8 * Q_STRIDE + kLatent * 2 + share * 32 + q * 8);
            v[2 * half] = on[half] ? up[half].times(x.x) : 0u;
            v[2 * half + 1] = on[half] ? up[half].times(x.y) : 0u;
        }
        tmem_st_16x8(tmem + kLatent / 2 + share * 8, v);
    }
    tmem_wait_st();
}

// How a call is cut up, and its workspace.
struct AttendParts {
    int splits, tiles_per_split;
    float *lse2;            // [R][H] log2 of the sums, for the weights
    // Base-2 scores, for the weights: [R][head_blocks][tiles] blocks of 16 heads
    // by 64 rows, each as a softmax warp holds it: [8][32 lanes][4], the
    // fragments of a 16x256b load.
    float4 *scores;
    int64_t head_blocks;
    int tiles;
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

__device__ __forceinline__ void st_cluster_v4(uint32_t at, uint4 v)
{
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

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
        const int n = t * TILE + dw * 4 + lane_row(lane);
        return n < rows ? ids[n] : -1;
    };
    const uint8_t *hot = a.rows + (int64_t)r * a.req_stride;
    RowPart part[2];                      // of tiles t (even) and t + 1
    int32_t id[2] = {-1, -1}, id2 = -1;   // theirs (checked), and of tile t + 2
    int bad = 0;
    const int heads = min(HEADS, a.H - h0);
    if (decodes) {
        id[0] = id_at(0);
        id[1] = id_at(1);
        id2 = id_at(2);
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
            mbar_init(smem_u32(&sm.queries), MMA_WARP);
            mbar_init(smem_u32(&sm.drained), 1);
            sm.gave_up = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        sm.top[lane] = sm.top[lane + 32] = 0;
        __syncwarp();
        tmem_alloc_all(smem_u32(&sm.tmem));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    volatile int *gave_up = &sm.gave_up;
    auto all = [](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };
    bool ok = true;

    // ---- the queries, while the first tiles' rows are on their way -----------------
    if (decodes) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            id[u] = checked_id(a, id[u], &bad);
            fetch(part[u], a, hot, id[u], lane);
        }
    }
    const int quarter = warp & 3, share = warp >> 2;
    const bool serves = warp < MMA_WARP && quarter * 16 < heads;     // the quarter has heads
    if (serves) {
        ok = all(mbar_wait(smem_u32(&sm.fetched[quarter]), 0, gave_up));
        for (int i = 0; !ok && i < (1 << 20) && !mbar_try(smem_u32(&sm.fetched[quarter]), 0); ++i) {}
        measure_queries<DT>(stages + Q_AT, sm.top, quarter, share, lane);
    }
    __syncthreads();
    if (warp < MMA_WARP) {
        // (the rows of a quarter without heads stay as they are: what they give
        // stays in that quarter)
        if (serves)
            place_queries<DT>(a, h0, stages + Q_AT, tmem + ((uint32_t)(quarter * 32) << 16) + TMEM_Q, sm.top, sm.factor,
                              quarter, share, lane);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.queries));
    }
    // softmax threads: reference and sum of heads lane / 4 and lane / 4 + 8 of
    // the warp's 16
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
    if (decodes) {
        // ---- fetch and decode -----------------------------------------------
        int s = 0, phase = 1;     // the phase whose end frees stage s
        const int i = dw * 4 + lane_row(lane), c = lane_chunk(lane);
        const uint32_t at = stages + (c >> 1) * BLOCK + i * 128 + ((((c & 1) * 4) ^ (i & 7)) << 4);
        const uint32_t rope_at = swizzled(stages + ROPE_BLOCK, i, c);
        for (int t = 0; ok && t < tiles; t += 2) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (t + u >= tiles) break;
                ok = all(t + u < STAGES - 1    ? true
                         : t + u == STAGES - 1 ? mbar_wait(smem_u32(&sm.queries), 0, gave_up)
                                               : mbar_wait(smem_u32(&sm.empty[s]), phase, gave_up));
                if (!ok) break;
                decode(part[u], at + s * OPERAND, rope_at + s * OPERAND);
                const uint32_t named = __ballot_sync(0xffffffffu, id[u] >= 0);      // rows: lanes 0, 2, 4, 6
                if (lane == 0)
                    sm.valid[s][dw] = (uint8_t)((named & 1u) | (named >> 1 & 2u) | (named >> 2 & 4u) | (named >> 3 & 8u));
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.full[s]));
                if (++s == STAGES) s = 0, phase ^= 1;
                id[u] = checked_id(a, id2, &bad);
                if (t + u + 2 < tiles) fetch(part[u], a, hot, id[u], lane);
                id2 = id_at(t + u + 3);
            }
        }
        if (bad && a.status) atomicOr(a.status + r, bad);
    } else if (warp == MMA_WARP) {
        // ---- MMA issue -----------------------------------------------------------
        constexpr uint32_t qk = mma_desc(HEADS, TILE, false, false);
        constexpr uint32_t qk_rope = mma_desc(HEADS, TILE, DT == kBf16, false);
        constexpr uint32_t pv = mma_desc(HEADS, 256, false, true);
        ok = all(mbar_wait(smem_u32(&sm.queries), 0, gave_up));
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
        ok = ok && all(mbar_wait(smem_u32(&sm.queries), 0, gave_up));     // for the factors
        const int g = lane >> 2, c2 = (lane & 3) * 2;     // fragment row and column
        const int vs = (c2 >> 2) * 8 + (c2 & 3);          // its bit in valid's 16-bit pieces
        const int i0 = warp * 16 + g, i1 = i0 + 8;
        const float f0 = sm.factor[i0], f1 = sm.factor[i1];
        float4 *sc = nullptr;       // this thread's place in the warp's score blocks
        if (a.weights && h0 + warp * 16 < a.H)
            sc = w.scores + (((int64_t)r * w.head_blocks + h0 / 16 + warp) * w.tiles + split * w.tiles_per_split) * 256 + lane;
        int s = 0, phase = 0, s_before = 0, phase_before = 0;     // of tile t, of tile t - 1
        for (int t = 0; ok && t < tiles; ++t) {
            ok = all(mbar_wait(smem_u32(&sm.full[s]), phase, gave_up) &&
                     mbar_wait(smem_u32(&sm.scored[t & 1]), (t >> 1) & 1, gave_up));
            if (!ok) break;
            tc_fence_after();
            if (!serves) {          // no head to weigh
                if (lane == 0) mbar_arrive(smem_u32(&sm.weighed[t & 1]));
                s_before = s, phase_before = phase;
                if (++s == STAGES) s = 0, phase ^= 1;
                continue;
            }
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
            if (sc) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    sc[j * 32] = make_float4(x[4 * j] * f0, x[4 * j + 1] * f0, x[4 * j + 2] * f1, x[4 * j + 3] * f1);
                sc += 256;
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
    // Head i is joined by CTA i % splits (its `mine` heads: split + m splits).
    // O goes from tensor memory to slot i of this CTA's shared memory, where
    // the tiles were, and the other CTAs' heads from there to slots behind the
    // owner's own, 512 bytes a store; or, where these do not all fit, straight
    // from tensor memory to slot p + m splits of the owner (part p), which
    // takes twice as long (32 bytes of a row at a time: 64 KB to a neighbour
    // 7.9 thousand cycles against 4).
    const int last = tiles - 1, mine = (heads - split + w.splits - 1) / w.splits;
    const bool staged = w.splits > 1 && heads + (w.splits - 1) * ((heads + w.splits - 1) / w.splits) <= SLOTS;
    auto part_slot = [&](int owner, int m, int p) {      // part p of the owner's m-th head
        return !staged        ? p + m * w.splits
               : p == owner   ? owner + m * w.splits
                              : heads + m * (w.splits - 1) + (p < owner ? p : p - 1);
    };
    const bool done = all(mbar_wait(smem_u32(&sm.empty[last % STAGES]), (last / STAGES) & 1, gave_up));
    tc_fence_after();
    if (w.splits > 1) cluster_arrive();       // this CTA's tiles are free
    if (w.splits > 1 && !staged) cluster_wait();
    if (done && serves) {
        const uint32_t upper = tmem + ((uint32_t)(quarter * 32) << 16) + TMEM_UPPER;
        uint32_t at[2];
        bool on[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = quarter * 16 + (lane >> 2) + 8 * half, owner = i % w.splits;
            on[half] = i < heads;
            at[half] = stages + (staged ? i : part_slot(owner, i / w.splits, split)) * O_STRIDE + (lane & 3) * 8;
            if (!staged) at[half] = in_cta(at[half], owner);
        }
#pragma unroll 1
        for (int c = share; c < kLatent / 32; c += QUARTER_WARPS) {
            uint32_t v[16];
            tmem_ld_16x32(upper + c * 32, v);
            tmem_wait_ld();
#pragma unroll
            for (int half = 0; half < 2; ++half)
                if (on[half]) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (staged)
                            st_smem_v2(at[half] + c * 128 + j * 32, v[4 * j + 2 * half], v[4 * j + 2 * half + 1]);
                        else
                            st_cluster_v2(at[half] + c * 128 + j * 32, v[4 * j + 2 * half], v[4 * j + 2 * half + 1]);
                    }
                }
        }
        tc_fence_before();
    }
    if (staged) {
        __syncthreads();
        cluster_wait();
#pragma unroll 1
        for (int n = warp; n < heads * 2; n += AT_NT / 32) {       // half a head's values a warp
            const int i = n >> 1, owner = i % w.splits;
            if (owner == split) continue;
            const uint32_t src = stages + i * O_STRIDE + (n & 1) * 1024 + lane * 16;
            const uint32_t dst = in_cta(stages + part_slot(owner, i / w.splits, split) * O_STRIDE + (n & 1) * 1024 + lane * 16, owner);
            const uint4 x = ld_smem_v4(src), y = ld_smem_v4(src + 512);
            st_cluster_v4(dst, x);
            st_cluster_v4(dst + 512, y);
        }
    }
    if (warp < SOFTMAX_WARPS && (lane & 3) == 0) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = warp * 16 + (lane >> 2) + 8 * half, owner = i % w.splits;
            if (i < heads)
                st_cluster_v2(in_cta(smem_u32(&sm.ml[i - owner + split]), owner), __float_as_uint(half ? m1 : m0),
                              __float_as_uint(half ? l1 : l0));
        }
    }
    if (w.splits > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    // out = sum_p 2^(m_p - m) O_p / sum_p 2^(m_p - m) l_p: first the parts'
    // factors, a thread a part, then the sums, half a head's values a warp
    int group = 1;       // threads a head
    while (group < w.splits) group *= 2;
    if (tid < (mine * group + 31) / 32 * 32) {
        const int m = tid / group, p = tid % group;
        const bool on = m < mine && p < w.splits;
        float2 ml = on ? sm.ml[m * w.splits + p] : make_float2(-INFINITY, 0.0f);
        float top = ml.x;
#pragma unroll 1
        for (int x = 1; x < group; x *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        const float f = ex2(ml.x - (top == -INFINITY ? 0.0f : top));
        float l = f * ml.y;
#pragma unroll 1
        for (int x = 1; x < group; x *= 2) l += __shfl_xor_sync(0xffffffffu, l, x);
        if (on) sm.ml[m * w.splits + p].x = l == 0.0f ? 0.0f : f * (128.0f / l);        // decode8's 2^7
        if (on && p == 0) {
            const int64_t rh = (int64_t)r * a.H + h0 + split + m * w.splits;
            const float l2 = l == 0.0f ? -INFINITY : top + log2f(l);
            if (a.lse) a.lse[rh] = l2 * kLn2;
            if (a.weights) w.lse2[rh] = l2;
        }
    }
    __syncthreads();
    // Columns are in decode8's order: of eight values the even in one 16-byte
    // unit, the odd in the next, here in neighbouring lanes.
#pragma unroll 1
    for (int n = warp; n < 2 * mine; n += AT_NT / 32) {
        const int m = n >> 1, d = (n & 1) * 256 + lane * 4;      // its place in the slot, and 128 on
        float o[2][4] = {};
#pragma unroll 2
        for (int p = 0; p < w.splits; ++p) {
            const uint32_t at = stages + part_slot(split, m, p) * O_STRIDE + d * 4;
            const float f = sm.ml[m * w.splits + p].x;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint4 x = ld_smem_v4(at + u * 512);
                o[u][0] = fmaf(f, __uint_as_float(x.x), o[u][0]);
                o[u][1] = fmaf(f, __uint_as_float(x.y), o[u][1]);
                o[u][2] = fmaf(f, __uint_as_float(x.z), o[u][2]);
                o[u][3] = fmaf(f, __uint_as_float(x.w), o[u][3]);
            }
        }
        uint8_t *out = a.out + (int64_t)r * a.out_rs + (int64_t)(h0 + split + m * w.splits) * a.out_hs + d * 2;
        const bool odd = lane & 1;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            // even lane: values 0-3 of its eight; odd lane: 4-7
            const float g0 = __shfl_xor_sync(0xffffffffu, odd ? o[u][0] : o[u][2], 1);
            const float g1 = __shfl_xor_sync(0xffffffffu, odd ? o[u][1] : o[u][3], 1);
            *reinterpret_cast<uint2 *>(out + u * 256) =
                odd ? make_uint2(floats_to_pair<DT>(g0, o[u][2]), floats_to_pair<DT>(g1, o[u][3]))
                    : make_uint2(floats_to_pair<DT>(o[u][0], g0), floats_to_pair<DT>(o[u][1], g1));
        }
    }
    if (tid == 0 && sm.gave_up && a.status) record_status(a.status, r, kStatusAttendTimeout);
    if (warp == MMA_WARP) tmem_free_all(tmem);
}

// ---- weights -----------------------------------------------------------------------

// weights[position] += sum over the heads of 2^(score - lse2).  A CTA takes the
// 64 rows of a tile, warp j eight of them: it reads the j-th 512 bytes of every
// block of 16 heads, a thread two rows by two heads at a time; then the 8
// threads of a row meet, always in the same order.  Bound by reading the
// scores once.
constexpr int WT_NT = 256;

__global__ void __launch_bounds__(WT_NT) weights_kernel(const __grid_constant__ AttendLaunch a,
                                                        const __grid_constant__ AttendParts w)
{
    const int t = blockIdx.x, r = blockIdx.y, j = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
    const int i = t * TILE + 8 * j + 2 * (lane & 3) + (g & 1);      // this thread's row in the end (g < 2)
    int32_t pos = -1;
    bool on = g < 2 && i < a.k;
    if (on) {     // (inputs: they do not wait for the launch before)
        int bad = 0;
        on = checked_id(a, a.ids[(int64_t)r * a.ids_stride + i], &bad) >= 0;
        if (on) pos = a.positions[(int64_t)r * a.positions_stride + i];
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float4 *s = w.scores + ((int64_t)r * w.head_blocks * w.tiles + t) * 256 + j * 32 + lane;
    const float *lse2 = w.lse2 + (int64_t)r * a.H;
    float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll 8
    for (int b = 0; b < (int)w.head_blocks; ++b) {
        const float4 x = s[(int64_t)b * w.tiles * 256];
        const int h = b * 16 + g;
        const float ref0 = h < a.H ? lse2[h] : INFINITY, ref1 = h + 8 < a.H ? lse2[h + 8] : INFINITY;
        sum0 += ex2(x.x - ref0) + ex2(x.z - ref1);
        sum1 += ex2(x.y - ref0) + ex2(x.w - ref1);
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        sum0 += __shfl_xor_sync(0xffffffffu, sum0, o);
        sum1 += __shfl_xor_sync(0xffffffffu, sum1, o);
    }
    if (!on) return;
    if (pos < 0 || pos >= a.weights_tokens) {
        if (a.status) record_status(a.status, r, kStatusBadPosition);
        return;
    }
    atomicAdd(a.weights + (int64_t)r * a.weights_stride + pos, g & 1 ? sum1 : sum0);
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
    p.tiles = tiles;
    p.head_blocks = (H + 15) / 16;
    float *f = reinterpret_cast<float *>(ws);
    int64_t n = 4;          // never empty
    p.lse2 = f + n;
    n += weights ? up4(RH) : 0;
    p.scores = reinterpret_cast<float4 *>(f + n);
    n += weights ? R * p.head_blocks * tiles * 1024 : 0;
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
        cfg.gridDim = dim3((unsigned)w.tiles, (unsigned)a.R);
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
