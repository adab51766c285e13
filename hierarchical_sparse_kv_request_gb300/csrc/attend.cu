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
// to [1, 2) ([2, 4) from 2^127 on).  Its latent part, with another 2^7, is then
// exact in f16 down to 2^-22 of that value, its rope part in bf16, or in f16 down
// to 2^-14; below, values round to multiples of 2^-31 and 2^-24 of it, the latter
// the step of a 32-bit number that size.
// Scores, sums and O are 32-bit; probabilities enter the second product as f16,
// relative to the reference (the largest lies between it and 2^8 times it): half
// a step is 2^-11 of a probability, and below 2^-14 of the reference 2^-25 of
// the latter (less is dropped; l keeps all in 32 bits).  The product's other
// operand is f16 and the two have one type, that with the most bits at its rate.
// The error of out against 64 bits is that of the plain 32-bit form in bf16, and
// a quarter more in f16 (2.6 against 2.1 x 10^-4, 37 requests of 40 heads).
//
// One CTA takes up to 64 heads of one request over a range of its rows, 64
// rows a tile, three tiles in shared memory:
//   warps 4-19   fetch a tile's packed rows into registers one tile ahead,
//                decode them to f16 in shared memory (128-byte swizzle);
//   warp 20      issues the MMAs (M = 64 heads): S = Q K^T, then O += P V of
//                the tile before, its rows now the k dimension;
//   warps 0-3    softmax: read S, move the reference, write P as f16 over the
//                tile's rope part (S no longer needs it), keep l.
// O of 64 heads takes half of tensor memory, and with 128 heads nothing would be
// left for S.  M = 64 uses 16 of the 32 lanes of each warp's part of it: O fills
// the upper 16 (512 columns), S (two tiles) and the queries the lower.  With
// the queries there, an MMA of the first product reads 2 KB of shared memory
// in its 32 cycles instead of 4 KB, which would take all of its bandwidth and
// leave the decoding warps none.
//
// The rows of a request are split over the CTAs of a cluster when there are
// few (request, head tile) pairs.  At the end the CTAs of a cluster share out
// the heads, and every CTA sends its part of a head's O to the shared memory of
// the CTA that joins it.  With weights, the scores (base 2, 32 bits) go to the
// workspace, and each row's probabilities over the heads, which need the heads'
// final sums, are added up from there: by the CTA itself where it has all heads
// and rows of a request (256 requests of 64 heads, at that time: 150 us, 158
// with a launch for it), else by a second launch.
//
// What bounds it.  The two products of a tile take 2,176 cycles of the tensor
// pipe; measured, a tile takes some 2,650, as shared memory serves their
// operands (1,200 cycles), the decoded tile's stores (580) and the fetches.  A
// CTA's start (ids, then rows; queries) takes some 10 thousand cycles to the
// first scores, its end 7 to 10 thousand with a join, 4 without.  Measured on
// GB300, 2,048 rows, GPU time: 32 requests of 128 heads 33 us (553 TFLOP/s), with
// weights 41; 32 of 16 heads 20; one request of 16 heads 10; 256 requests of 64
// heads with weights 142.
#include <atomic>
#include <mutex>

#include "attend.cuh"

namespace hs {
namespace {

constexpr int HEADS = 64;         // heads a CTA
constexpr int SOFTMAX_WARPS = 4, DECODE_WARPS = 16, MMA_WARP = SOFTMAX_WARPS + DECODE_WARPS;
constexpr int AT_NT = (MMA_WARP + 1) * 32;
constexpr uint32_t BLOCK = 64 * 128;             // 64 values of 64 rows, swizzled
constexpr uint32_t OPERAND = 9 * BLOCK;          // 576 values of 64 rows
constexpr uint32_t ROPE_BLOCK = 8 * BLOCK;
constexpr int STAGES = 3;                        // tiles in shared memory
constexpr uint32_t TMEM_UPPER = 16u << 16;       // O: the upper lanes, column = value
constexpr uint32_t TMEM_Q = 2 * TILE;            // lower lanes: S of two tiles, then the queries

// At the end a part of a head's O takes a slot where the tiles were.
constexpr int SLOTS = (STAGES * OPERAND + HEADS * 64) / O_STRIDE;
static_assert(SLOTS >= HEADS + MAX_SPLITS - 1, "the parts that a CTA joins");

// See AttendParts::split_inv: n * (65536 / splits + 1 - f) >> 16, f < 1, is exact
// while n < 65536 / splits.
constexpr uint32_t inverse_of(int splits) { return 65536u / (unsigned)splits + 1u; }
static_assert((HEADS + MAX_SPLITS) * MAX_SPLITS <= 65536, "");

struct AttendSmem {
    uint64_t full[STAGES], empty[STAGES], scored[2], weighed[2], fetched[SOFTMAX_WARPS], queries, drained, known, joined;
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

// 16-byte unit u (8 values) of row i in a swizzled block
__device__ __forceinline__ uint32_t swizzled(uint32_t block, int i, int u)
{
    return block + i * 128 + ((u ^ (i & 7)) << 4);
}

// A decode warp has four rows of a tile.  Half a warp takes the 256 bytes of
// codes of a row (16 bytes a thread; rows lane / 16 and + 2), a quarter the rope
// part of one of its two.  So eight neighbouring threads load 128 contiguous
// bytes (32 bytes of each of four rows, measured: 39.7 against 35.9 us for 32
// requests, 128 heads, 2,048 rows) and store eight units of a row and block.
struct RowPart {
    uint4 codes[2], rope;
    uint32_t scales[2];  // two e4m3 each
};

__device__ __forceinline__ const uint8_t *shfl_ptr(const uint8_t *p, int lane)
{
    return reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(p), lane));
}

// row: of the warp's n-th, in lane first + n.  Nothing here waits for what it
// loads.
__device__ __forceinline__ void fetch(RowPart &p, const uint8_t *row, int first, int lane)
{
    const int c = lane & 15;
    const uint8_t *src[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        src[j] = shfl_ptr(row, first + (lane >> 4) + 2 * j);
        p.codes[j] = ld_row_v4(src[j] + c * 16);
    }
    p.rope = ld_row_v4((lane & 8 ? src[1] : src[0]) + kRopeAt + (lane & 7) * 16);
#pragma unroll
    for (int j = 0; j < 2; ++j) p.scales[j] = ld_row_u16(src[j] + kScaleAt + c * 2);
}

// named: bit n is set if the warp's row n is one.  The values of no row are 0 (by
// its scales) for the second product; its scores are masked.  at: where the
// thread's first word goes, for each of its rows.
__device__ __forceinline__ void decode(const RowPart &p, uint32_t named, const uint32_t (&at)[2], uint32_t rope_at, int lane)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t s2;
        const bool on = named >> ((lane >> 4) + 2 * j) & 1u;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2) : "h"((uint16_t)(on ? p.scales[j] : 0u)));
        const __half2 s = __hmul2(*reinterpret_cast<__half2 *>(&s2), __half2half2(__ushort_as_half(0x5800)));   // 2^7
        const __half2 lo = __low2half2(s), hi = __high2half2(s);
        st_smem_v4(at[j], decode8(p.codes[j].x, lo));
        st_smem_v4(at[j] + 2 * BLOCK, decode8(p.codes[j].y, lo));
        st_smem_v4(at[j] + 4 * BLOCK, decode8(p.codes[j].z, hi));
        st_smem_v4(at[j] + 6 * BLOCK, decode8(p.codes[j].w, hi));
    }
    st_smem_v4(rope_at, p.rope);
}

// ---- queries -------------------------------------------------------------------------

// A softmax warp has its 16 heads' queries copied to shared memory (as they
// are; the last stage is still free).  Then the warps of each quarter of tensor
// memory (warp % 4), five of them, find the heads' largest magnitudes and write
// the queries, scaled, in the fragments of a 16x256b store.
constexpr uint32_t Q_STRIDE = kRowValues * 2 + 32;     // no bank conflict between neighbours
constexpr int QUARTER_WARPS = MMA_WARP / 4;

__device__ __forceinline__ void fetch_queries(const AttendLaunch &a, int r, int h0, uint32_t dst, uint32_t bar,
                                              int warp, int lane)
{
    const int heads = min(max(a.H - h0 - warp * 16, 0), 16);
    if (lane == 0) {
        mbar_init(bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        mbar_expect(bar, heads * kRowValues * 2);
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

// The largest magnitudes (see top) of heads lane / 4 and lane / 4 + 8 of the
// quarter; share: the warp's part of the values.
template <int DT>
__device__ __forceinline__ void measure_queries(uint32_t src, uint32_t *top, int quarter, int share, int lane)
{
    const int i0 = quarter * 16 + (lane >> 2);
    const uint32_t at = src + i0 * Q_STRIDE + (lane & 1) * 16 + (lane & 2) * 32;     // 32 bytes of 128
    uint32_t m[2] = {0, 0};      // (of no head: of whatever is there, and not used)
#pragma unroll 1
    for (int n = share; n < kRowValues / 64; n += QUARTER_WARPS)
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                m[half] = magnitude<DT>(m[half], ld_smem_v4(at + half * 8 * Q_STRIDE + n * 128 + u * 32));
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t x = max2<DT>(m[half], __shfl_xor_sync(0xffffffffu, m[half], 1));
        x = max2<DT>(x, __shfl_xor_sync(0xffffffffu, x, 2));
        x &= 0x7FFF7FFFu;
        if ((lane & 3) == 0) atomicMax(top + i0 + 8 * half, max(x >> 16, x & 0xFFFFu));
    }
}

template <int DT>
__device__ __forceinline__ void place_queries(const AttendLaunch &a, int heads, uint32_t src, uint32_t tmem, const uint32_t *top,
                                              float *factor, int quarter, int share, int lane)
{
    const int q = lane & 3, i0 = quarter * 16 + (lane >> 2);
    uint32_t at[2];
    int e[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int i = min(i0 + 8 * half, heads - 1);      // (no head: the last one once more)
        at[half] = src + i * Q_STRIDE;
        e[half] = query_exponent<DT>(top[i]);
        if (q == 0 && share == 0) factor[i0 + 8 * half] = query_factor(a, e[half]);
    }
    // with the sign of the scale, so that the factor of the scores is positive,
    // and NaN if it is: the scores of rows, not of holes, become so
    const float sign = a.scale != a.scale ? a.scale : copysignf(1.0f, a.scale);
    // Four of the quarter's warps take 64 columns each, the fifth the rope part.
    // Latent columns 8 j + 2 q and + 1 hold the even (q even) or the odd values
    // of the eight in unit 2 j + q / 2, the order of decode8, with its 2^7; rope
    // columns their values in order.
    static_assert(QUARTER_WARPS == 5, "");
    if (share < 4) {
        const PowerOfTwo<DT> up7[2] = {{7 - e[0], sign}, {7 - e[1], sign}};
        const uint32_t pick = q & 1 ? 0x7632 : 0x5410;
        uint32_t v[32];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                // units of one block of 8 are 64 bytes apart
                const uint4 x = ld_smem_v4(at[half] + unit_values(share * 16 + (j >> 2) * 8 + (q >> 1)) * 2 + (j & 3) * 128);
                uint32_t lo = up7[half].times(__byte_perm(x.x, x.y, pick)), hi = up7[half].times(__byte_perm(x.z, x.w, pick));
                if (DT == kBf16) {
                    const float2 f = pair_to_float<DT>(lo), g = pair_to_float<DT>(hi);
                    lo = floats_to_pair<kF16>(f.x, f.y);
                    hi = floats_to_pair<kF16>(g.x, g.y);
                }
                v[4 * j + 2 * half] = lo;
                v[4 * j + 2 * half + 1] = hi;
            }
        tmem_st_16x64(tmem + share * 64, v);
    } else {
        const PowerOfTwo<DT> up[2] = {{-e[0], sign}, {-e[1], sign}};
        uint32_t v[16];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint2 x = ld_smem_v2(at[half] + kLatent * 2 + j * 32 + q * 8);
                v[4 * j + 2 * half] = up[half].times(x.x);
                v[4 * j + 2 * half + 1] = up[half].times(x.y);
            }
        tmem_st_16x32(tmem + kLatent / 2, v);
    }
    tmem_wait_st();
}

// ---- weights -----------------------------------------------------------------------

// weights[position] += sum over the heads of 2^(score - lse2), for eight rows a
// warp, the j-th of tile t: it reads the j-th 512 bytes of every block of 16 heads,
// a thread two rows by two heads at a time; then the 8 threads of a row meet,
// always in the same order, and two of them (lane / 4 < 2) have a row each.
struct WeightRow {
    int32_t id, pos;      // of this thread's row in the end
    __device__ __forceinline__ void load(const AttendLaunch &a, int r, int t, int j, int lane)
    {
        const int i = t * TILE + 8 * j + 2 * (lane & 3) + (lane >> 2 & 1);
        const bool on = lane < 8 && i < a.k;
        id = on ? a.ids[(int64_t)r * a.ids_stride + i] : -1;
        pos = on ? a.positions[(int64_t)r * a.positions_stride + i] : -1;
    }
    // sum0, sum1: of rows 2 (lane % 4) and + 1 over this thread's heads
    __device__ __forceinline__ void add(const AttendLaunch &a, int r, float sum0, float sum1, int lane) const
    {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            sum0 += __shfl_xor_sync(0xffffffffu, sum0, o);
            sum1 += __shfl_xor_sync(0xffffffffu, sum1, o);
        }
        int bad = 0;
        if (checked_id(a, id, &bad) < 0) return;
        if (pos >= 0 && pos < a.weights_tokens)
            atomicAdd(a.weights + (int64_t)r * a.weights_stride + pos, lane & 4 ? sum1 : sum0);
        else if (a.status)
            record_status(a.status, r, kStatusBadPosition);
    }
};

__device__ __forceinline__ void add_weight(float &sum0, float &sum1, float score0, float score1, float lse2)
{
    sum0 += ex2(score0 - lse2);
    sum1 += ex2(score1 - lse2);
}

__device__ __forceinline__ const float4 *scores_at(const AttendParts &w, int r, int t, int j, int lane)
{
    return w.scores + ((int64_t)r * w.head_blocks * w.tiles + t) * 256 + j * 32 + lane;
}

// A score is read once and then only in the way of others in L2 (256 requests of
// 64 heads: 148.6 -> 142.3 us).
__device__ __forceinline__ float4 ld_once_v4(const float4 *p)
{
    uint64_t policy;
    float4 v;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    asm volatile("ld.global.L2::cache_hint.v4.f32 {%0,%1,%2,%3}, [%4], %5;" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p), "l"(policy) : "memory");
    return v;
}

// A CTA takes the 64 rows of a tile.  Bound by reading the scores once.
constexpr int WT_NT = 256;

__global__ void __launch_bounds__(WT_NT, 6) weights_kernel(const __grid_constant__ AttendLaunch a,
                                                           const __grid_constant__ AttendParts w)
{
    const int t = blockIdx.x, r = blockIdx.y, j = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
    WeightRow row;
    row.load(a, r, t, j, lane);      // (inputs, ahead of the wait: see launch_behind)
    after_launch_before();
    const float4 *s = scores_at(w, r, t, j, lane);
    const float *lse2 = w.lse2 + (int64_t)r * a.H;
    float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll 4
    for (int b = 0; b < (int)w.head_blocks; ++b) {
        const float4 x = ld_once_v4(s + (int64_t)b * w.tiles * 256);
        const int h = b * 16 + g;
        if (h < a.H) add_weight(sum0, sum1, x.x, x.y, lse2[h]);
        if (h + 8 < a.H) add_weight(sum0, sum1, x.z, x.w, lse2[h + 8]);
    }
    row.add(a, r, sum0, sum1, lane);
}

// The same by a CTA that has all heads and rows of request r and has written
// their scores; ml[head].y: its lse2.  The next eight rows' loads are under way
// while a warp adds up.
__device__ __forceinline__ void add_own_weights(const AttendLaunch &a, const AttendParts &w, int r, const float2 *ml, int warp,
                                                int lane)
{
    constexpr int BLOCKS = HEADS / 16, WARPS = AT_NT / 32;
    const int pieces = w.tiles * 8;
    float ref[BLOCKS][2];
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b) {
        ref[b][0] = ml[b * 16 + (lane >> 2)].y;
        ref[b][1] = ml[b * 16 + (lane >> 2) + 8].y;
    }
    float4 next[BLOCKS];
    WeightRow next_row;
    auto load = [&](int n) {
        const float4 *s = scores_at(w, r, n >> 3, n & 7, lane);
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b)
            next[b] = b < w.head_blocks ? ld_once_v4(s + (int64_t)b * w.tiles * 256) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        next_row.load(a, r, n >> 3, n & 7, lane);
    };
    if (warp < pieces) load(warp);
#pragma unroll 1
    for (int n = warp; n < pieces; n += WARPS) {
        float4 x[BLOCKS];
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) x[b] = next[b];
        const WeightRow row = next_row;
        if (n + WARPS < pieces) load(n + WARPS);
        float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
            const int h = b * 16 + (lane >> 2);
            if (h < a.H) add_weight(sum0, sum1, x[b].x, x[b].y, ref[b][0]);
            if (h + 8 < a.H) add_weight(sum0, sum1, x[b].z, x[b].w, ref[b][1]);
        }
        row.add(a, r, sum0, sum1, lane);
    }
}

// ---- out -------------------------------------------------------------------------

// O of a quarter's heads times their factors (ml[head].x), from tensor memory to
// out: four units a time whose values are 32 neighbours, one unit a thread of
// the four that have a head's fragment.
template <int DT>
__device__ __forceinline__ void store_out(const AttendLaunch &a, int r, int h0, int heads, uint32_t o_at, const float2 *ml,
                                          int quarter, int share, int lane)
{
    const int q = lane & 3, i0 = quarter * 16 + (lane >> 2);
    const float f[2] = {ml[i0].x, ml[i0 + 8].x};
    uint8_t *out = a.out + (int64_t)r * a.out_rs + (int64_t)(h0 + i0) * a.out_hs + q * 16;
#pragma unroll 1
    for (int n = share; n < 16; n += QUARTER_WARPS) {      // units n and the three that follow by 16
        uint32_t v[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) tmem_ld_16x8(o_at + (n + 16 * j) * 8, v[j]);
        tmem_wait_ld();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            // Of unit j this thread has values 0 2, 4 6, 1 3 or 5 7, by q.
            uint32_t x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[j] = floats_to_pair<DT>(__uint_as_float(v[j][2 * half]) * f[half], __uint_as_float(v[j][2 * half + 1]) * f[half]);
            // threads q and q ^ 2 swap: q keeps units 0 and 1 or 2 and 3, with
            // values 0-3 (q even) or 4-7
            const bool hi = q & 2;
            uint32_t y[2][2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? x[j] : x[j + 2], 2), own = hi ? x[j + 2] : x[j];
                const uint32_t even = hi ? got : own, odd = hi ? own : got;
                y[j][0] = __byte_perm(even, odd, 0x5410);
                y[j][1] = __byte_perm(even, odd, 0x7632);
            }
            // threads q and q ^ 1 swap: q keeps unit q
            const bool second = q & 1;
            const uint32_t g0 = __shfl_xor_sync(0xffffffffu, second ? y[0][0] : y[1][0], 1);
            const uint32_t g1 = __shfl_xor_sync(0xffffffffu, second ? y[0][1] : y[1][1], 1);
            const uint4 z = second ? make_uint4(g0, g1, y[1][0], y[1][1]) : make_uint4(y[0][0], y[0][1], g0, g1);
            if (i0 + 8 * half < heads) *reinterpret_cast<uint4 *>(out + half * 8 * a.out_hs + unit_values(n) * 2) = z;
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(AT_NT, 1) attend_kernel(const __grid_constant__ AttendLaunch a,
                                                          const __grid_constant__ AttendParts w)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    AttendSmem &sm = *reinterpret_cast<AttendSmem *>(smem + MISC_AT);
    const uint32_t stages = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int split = blockIdx.x;        // the CTA's rank in its cluster
    const int h0 = blockIdx.y * HEADS, r = blockIdx.z;
    const int k0 = split * w.rows_per_split;
    const int rows = min(a.k - k0, w.rows_per_split);
    const int tiles = (rows + TILE - 1) / TILE;

    const bool decodes = warp >= SOFTMAX_WARPS && warp < MMA_WARP;
    const int dw = warp - SOFTMAX_WARPS;      // its rows of a tile: 4 dw to 4 dw + 3
    // Decode warps take the ids of eight tiles at once: lane has row lane % 4 of
    // the warp's in tile lane / 4 of the eight.
    const int32_t *ids = a.ids + (int64_t)r * a.ids_stride + k0;
    auto ids_at = [&](int t) {
        const int n = (t + (lane >> 2)) * TILE + dw * 4 + (lane & 3);
        return n < rows ? ids[n] : -1;
    };
    const uint8_t *hot = a.rows + (int64_t)r * a.req_stride, *row = hot;
    RowPart next;               // of tile t + 1
    uint32_t named = 0;         // bit n: lane n's id names a row
    int32_t id = -1;            // of the next eight tiles
    int bad = 0;
    const int heads = min(HEADS, a.H - h0);
    const Join join{stages, smem_u32(&sm.known), smem_u32(&sm.joined), sm.ml, heads, w.splits, split, w.split_inv, staged_slots(heads, w.splits) <= SLOTS};
    if (decodes) {
        after_launch_before();
        id = ids_at(0);
    } else if (warp < SOFTMAX_WARPS) {
        after_launch_before();
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
            mbar_init(smem_u32(&sm.known), 1);
            mbar_init(smem_u32(&sm.joined), 1);
            sm.gave_up = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            mbar_expect(smem_u32(&sm.known), join.parts() * 8);
            mbar_expect(smem_u32(&sm.joined), join.parts() * kLatent * 4);
        }
        sm.top[lane] = sm.top[lane + 32] = 0;
        __syncwarp();
        tmem_alloc_all(smem_u32(&sm.tmem));
        after_launch_before();
        // this call's own next launch may be placed now: after this wait, as it
        // reads inputs ahead of its own (see launch_behind)
        if (a.weights && !w.whole) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (w.splits > 1) cluster_arrive();       // its mbarriers are there
    const uint32_t tmem = sm.tmem;
    volatile int *gave_up = &sm.gave_up;
    auto all = [](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };
    bool ok = true;

    // ---- the queries, while the first tile's rows are on their way -----------------
    auto name_rows = [&](int t) {      // of the eight tiles from t on; their ids are in id
        id = checked_id(a, id, &bad);
        row = row_of(a, hot, id);
        named = __ballot_sync(0xffffffffu, id >= 0);
        id = ids_at(t + 8);
    };
    if (decodes) {
        name_rows(0);
        fetch(next, row, 0, lane);
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
            place_queries<DT>(a, heads, stages + Q_AT, tmem + ((uint32_t)(quarter * 32) << 16) + TMEM_Q, sm.top, sm.factor,
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
        // word w of a row's 16-byte chunk c is unit c % 8 of block 2 w + c / 8
        const int c = lane & 15, i = dw * 4 + (lane >> 4);
        const uint32_t to0 = swizzled(stages + (c >> 3) * BLOCK, i, c & 7), to1 = swizzled(stages + (c >> 3) * BLOCK, i + 2, c & 7);
        const uint32_t rope_to = swizzled(stages + ROPE_BLOCK, i + (lane & 8 ? 2 : 0), lane & 7);
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
            const RowPart now = next;
            const uint32_t now_named = named >> ((t & 7) * 4) & 15u;
            if (((t + 1) & 7) == 0) name_rows(t + 1);
            fetch(next, row, ((t + 1) & 7) * 4, lane);      // (after the last tile: row 0)
            ok = ok && all(t < STAGES - 1    ? true
                           : t == STAGES - 1 ? mbar_wait(smem_u32(&sm.queries), 0, gave_up)
                                             : mbar_wait(smem_u32(&sm.empty[s]), phase, gave_up));
            if (!ok) break;
            const uint32_t to[2] = {to0 + s * OPERAND, to1 + s * OPERAND};
            decode(now, now_named, to, rope_to + s * OPERAND, lane);
            if (lane == 0) sm.valid[s][dw] = (uint8_t)now_named;
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
            sc = w.scores + (((int64_t)r * w.head_blocks + h0 / 16 + warp) * w.tiles + k0 / TILE) * 256 + lane;
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
            if (sc) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    sc[j * 32] = make_float4(x[4 * j] * f0, x[4 * j + 1] * f0, x[4 * j + 2] * f1, x[4 * j + 3] * f1);
                sc += 256;
            }
            s_before = s, phase_before = phase;
            if (++s == STAGES) s = 0, phase ^= 1;
        }
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    }

    const bool keeps = warp < SOFTMAX_WARPS && (lane & 3) == 0;      // a thread with references and sums
    if (w.splits > 1) {
        cluster_wait();
        if (keeps) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = warp * 16 + (lane >> 2) + 8 * half;
                if (i < heads) join.send_ml(i, half ? m1 : m0, half ? l1 : l0);
            }
        }
    }
    const int last = tiles - 1;
    const bool done = all(mbar_wait(smem_u32(&sm.empty[last % STAGES]), (last / STAGES) & 1, gave_up));
    tc_fence_after();
    const uint32_t o_at = tmem + ((uint32_t)(quarter * 32) << 16) + TMEM_UPPER;
    if (w.splits == 1) {
        // ---- out from tensor memory ------------------------------------------------
        if (keeps) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = warp * 16 + (lane >> 2) + 8 * half;
                const float m = half ? m1 : m0, l = half ? l1 : l0;
                sm.ml[i] = make_float2(out_factor(l), log2_sum(m, l));
                if (i < heads) store_lse(a, w, (int64_t)r * a.H + h0 + i, sm.ml[i].y);
            }
        }
        __syncthreads();
        if (done && serves) store_out<DT>(a, r, h0, heads, o_at, sm.ml, quarter, share, lane);
        if (a.weights && w.whole) add_own_weights(a, w, r, sm.ml, warp, lane);
        tc_fence_before();
        __syncthreads();
    } else {
        // ---- join (see attend.cuh): O from tensor memory to where the tiles were ---
        cluster_arrive();       // this CTA's tiles are free: the last product is done with them
        if (!join.staged) cluster_wait();
        if (serves) {       // (also if a wait gave up: the others wait for as many bytes)
            uint32_t at[2], bar[2];
            bool on[2], local[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = quarter * 16 + (lane >> 2) + 8 * half, m = join.over_splits(i), owner = i - m * w.splits;
                on[half] = i < heads;
                local[half] = join.staged || owner == split;
                at[half] = (join.staged ? stages + i * O_STRIDE : join.place(owner, m)) + (lane & 3) * 8;
                if (!local[half]) at[half] = in_cta(at[half], owner);
                bar[half] = in_cta(join.joined, owner);
            }
#pragma unroll 1
            for (int c = share; c < kLatent / 64; c += QUARTER_WARPS) {
                uint32_t v[32];
                tmem_ld_16x64(o_at + c * 64, v);
                tmem_wait_ld();
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    if (on[half]) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const uint32_t to = at[half] + c * 256 + j * 32;
                            if (local[half])
                                st_smem_v2(to, v[4 * j + 2 * half], v[4 * j + 2 * half + 1]);
                            else
                                send_v2(to, v[4 * j + 2 * half], v[4 * j + 2 * half + 1], bar[half]);
                        }
                    }
            }
        }
        tc_fence_before();
        __syncthreads();
        if (join.staged) {
            cluster_wait();
            join.send(warp, AT_NT / 32, lane);
        }
        // No CTA leaves before the others have sent it their parts, whatever
        // has gone wrong: a part that is late is waited for once more.
        cluster_arrive();
        bool here = true;
        if (warp * 32 < join.count(split) * 16) {
            here = mbar_wait(join.known, 0, gave_up);
            join.factors(a, w, (int64_t)r * a.H + h0, tid);
        }
        here = mbar_wait(join.joined, 0, gave_up) && here;
        __syncthreads();
        if (join.count(split) * 4 <= AT_NT / 32)
            join.finish<DT, 1>(a, r, h0, warp, AT_NT / 32, lane);
        else
            join.finish<DT, 4>(a, r, h0, warp, AT_NT / 32, lane);
        cluster_wait();
        for (int i = 0; !here && i < (1 << 20) && !(mbar_try(join.known, 0) && mbar_try(join.joined, 0)); ++i) {}
    }
    if (tid == 0 && sm.gave_up && a.status) record_status(a.status, r, kStatusAttendTimeout);
    if (warp == MMA_WARP) tmem_free_all(tmem);
}

// ---- host ----------------------------------------------------------------------------

// Clusters of each size that a device holds at once (0: none).
struct Capacity {
    int clusters[MAX_SPLITS + 1];
};

// Sets the kernel's attributes on the current device (which also loads it) and
// fills in cap.
template <class Kernel>
cudaError_t prepare(Kernel kernel, Capacity *cap)
{
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)AT_SMEM);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    for (int c = 1; e == cudaSuccess && c <= MAX_SPLITS; ++c) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr;
        cfg.gridDim = dim3(c);
        cfg.blockDim = dim3(AT_NT);
        cfg.dynamicSmemBytes = AT_SMEM;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = c;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        cap->clusters[c] = n;
    }
    return e != cudaSuccess ? e : cap->clusters[1] < 1 ? cudaErrorInvalidConfiguration : cudaSuccess;
}

// What a device holds of the kernel, found once per device.
cudaError_t capacity(const Capacity **out)
{
    constexpr int kDevices = 64;
    static Capacity cap[kDevices];
    static std::atomic<bool> known[kDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kDevices) return cudaErrorInvalidDevice;
    if (!known[dev].load(std::memory_order_acquire)) {
        static std::mutex one;
        std::lock_guard<std::mutex> lock(one);
        if (!known[dev].load(std::memory_order_acquire)) {
            e = prepare(attend_kernel<kBf16>, &cap[dev]);
            if (e == cudaSuccess) e = prepare(attend_kernel<kF16>, &cap[dev]);
            cudaFuncAttributes fa;
            if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, weights_kernel);   // loads it
            if (e != cudaSuccess) return e;
            known[dev].store(true, std::memory_order_release);
        }
    }
    *out = &cap[dev];
    return cudaSuccess;
}

// How many parts the rows of `units` head tiles, `tiles` tiles each, are split
// into, one for each CTA of a cluster: the count for which the waves of clusters
// take the fewest tiles, counting a CTA's own start and end as kFixedTiles (some
// 22 thousand cycles, a tile 2,650).  Measured with 8 against 3, 2,048 rows of 64
// heads: 100 requests 53.5 against 75.6 us, 160 requests 98 against 123.
constexpr int kFixedTiles = 8;

int choose_splits(int64_t units, int tiles, const Capacity &cap, int64_t *cost)
{
    int best = 1;
    *cost = INT64_MAX;
    for (int s = 1; s <= tiles && s <= MAX_SPLITS; ++s) {
        const int per = (tiles + s - 1) / s;
        if (cap.clusters[s] < 1 || (tiles + per - 1) / per != s) continue;
        const int64_t waves = (units + cap.clusters[s] - 1) / cap.clusters[s];
        if (waves * (per + kFixedTiles) < *cost) *cost = waves * (per + kFixedTiles), best = s;
    }
    return best;
}

// How many of the R requests go ahead in whole waves of unsplit head tiles, in a
// launch of their own, before the rest: 0 if that takes no fewer tiles.  (160
// requests of 64 heads, 2,048 rows: 152 and then 8, split, 73.5 against 97 us in
// one launch; 100 of 128 heads 84 against 95.)
int32_t requests_ahead(int32_t R, int head_tiles, int tiles, const Capacity &cap)
{
    const int32_t wave = cap.clusters[1] / head_tiles;
    if (wave < 1 || R <= wave || R % wave == 0) return 0;
    int64_t all, rest;
    choose_splits((int64_t)R * head_tiles, tiles, cap, &all);
    choose_splits((int64_t)(R % wave) * head_tiles, tiles, cap, &rest);
    return R / wave * (int64_t)(tiles + kFixedTiles) + rest < all ? R - R % wave : 0;
}

// Whole 128-byte lines of floats (scores at odd 16 bytes: 151.6 against 148.6 us).
int64_t whole_lines(int64_t n) { return (n + 31) / 32 * 32; }

// The workspace of a call.
AttendParts lay_out(int32_t R, int32_t H, int32_t k, bool weights, uint8_t *ws, int64_t *bytes)
{
    AttendParts p = {};
    p.tiles = (k + TILE - 1) / TILE;
    p.head_blocks = (H + 15) / 16;
    float *f = reinterpret_cast<float *>(ws);
    int64_t n = 32;         // never empty
    p.lse2 = f + n;
    n += weights ? whole_lines((int64_t)R * H) : 0;
    p.scores = reinterpret_cast<float4 *>(f + n);
    n += weights ? R * p.head_blocks * p.tiles * 1024 : 0;
    *bytes = n * 4;
    return p;
}

// Requests first to first + count - 1 of a call.
cudaError_t launch_requests(AttendLaunch a, AttendParts w, int32_t first, int32_t count, const Capacity &cap, cudaStream_t s)
{
    a.R = count;
    a.q += first * a.q_rs;
    a.rows += first * a.req_stride;
    a.ids += first * a.ids_stride;
    a.out += first * a.out_rs;
    if (a.lse) a.lse += (int64_t)first * a.H;
    if (a.status) a.status += first;
    if (a.weights) {
        a.weights += first * a.weights_stride;
        a.positions += first * a.positions_stride;
        w.lse2 += (int64_t)first * a.H;
        w.scores += first * w.head_blocks * w.tiles * 256;
    }
    const int head_tiles = (a.H + HEADS - 1) / HEADS;
    int64_t cost;
    w.splits = choose_splits((int64_t)count * head_tiles, w.tiles, cap, &cost);
    w.split_inv = inverse_of(w.splits);
    w.rows_per_split = (w.tiles + w.splits - 1) / w.splits * TILE;
    w.whole = w.splits == 1 && a.H <= HEADS;
    const cudaError_t e = launch_behind(a.dtype == kBf16 ? attend_kernel<kBf16> : attend_kernel<kF16>,
                                        dim3(w.splits, head_tiles, count), AT_NT, AT_SMEM, w.splits, s, a, w);
    if (e != cudaSuccess || !a.weights || w.whole) return e;
    return launch_behind(weights_kernel, dim3(w.tiles, count), WT_NT, 0, 1, s, a, w);
}

}  // namespace

void attend_workspace_bytes(int32_t R, int32_t H, int32_t k, bool weights, int64_t *bytes)
{
    lay_out(R, H, k, weights, nullptr, bytes);
}

cudaError_t launch_attend(const AttendLaunch &a, int64_t workspace_bytes, bool *too_small, cudaStream_t s)
{
    const Capacity *cap;
    cudaError_t e = capacity(&cap);
    if (e != cudaSuccess) return e;
    int64_t bytes;
    const AttendParts w = lay_out(a.R, a.H, a.k, a.weights != nullptr, a.workspace, &bytes);
    *too_small = workspace_bytes < bytes;
    if (*too_small) return cudaSuccess;
    const int32_t ahead = requests_ahead(a.R, (a.H + HEADS - 1) / HEADS, w.tiles, *cap);
    if (ahead) e = launch_requests(a, w, 0, ahead, *cap, s);
    return e == cudaSuccess ? launch_requests(a, w, ahead, a.R - ahead, *cap, s) : e;
}

}  // namespace hs
