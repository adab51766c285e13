// attend.cuh -- the parts of the attention kernel (attend.cu) that stand for
// themselves: ids and rows, decoding, queries as f16, and the join of what the
// CTAs of a cluster have worked on.
#pragma once

#include <cfloat>

#include "rows4.cuh"
#include "tcgen05.cuh"

namespace hs {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int TILE = 64;          // rows a tile
constexpr float kMoveAbove = 8.0f;               // base-2 growth that moves the softmax's reference
constexpr int MAX_SPLITS = 16;                   // CTAs a cluster

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

// (straight into 32 bits: widening it would wait for it)
__device__ __forceinline__ uint32_t ld_row_u16(const void *p)
{
    uint32_t v;
    asm volatile("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=r"(v) : "l"(p));
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

// The first of the eight values that unit u (8 columns) of a decoded row holds:
// units are numbered so that a row's 16-byte pieces, which have four times eight
// values, go to neighbouring units, one word of each at a time.
__host__ __device__ constexpr int unit_values(int u)
{
    return ((u >> 3 & 1) * 8 + (u & 7)) * 32 + (u >> 4) * 8;
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

// Two values times a power of two and a sign (or NaN), exactly: 2^n for bf16, 2^n
// in two steps for f16, whose own powers reach 2^15.
template <int DT>
struct PowerOfTwo {
    uint32_t f[2];
    __device__ __forceinline__ PowerOfTwo(int n, float s)
    {
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

// A query is multiplied by 2^-e (latent: 2^(7 - e), decode8's 2^7) and the sign
// of the scale; top: the 16 bits of its largest magnitude.  e is that one's
// exponent, or 0 where there is none and for infinities, which pass through as
// they are (as NaN does); 2^-e and 2^(7 - e) have to be normal, f16's in two
// steps (so bf16's largest exponent, 127, counts as 126).
template <int DT>
__device__ __forceinline__ int query_exponent(uint32_t top)
{
    const int e = (int)(__float_as_uint(pair_to_float<DT>(top).x) >> 23) - 127;
    return min(max(top == 0 || e == 128 ? 0 : e, DT == kBf16 ? -119 : -23), 126);
}

// What the products of such a query have to be multiplied by to be base-2
// scores; positive.  (The power of two first: the largest scales times log2(e)
// are infinite, and the smallest lose bits.)
__device__ __forceinline__ float query_factor(const AttendLaunch &a, int e)
{
    return fmaxf(fabsf(a.scale) * exp2i(e) * kLog2e, FLT_MIN);
}

// How a call is cut up, and its workspace.
struct AttendParts {
    int splits;             // CTAs a request's (or head tile's) rows are split over: a cluster
    int rows_per_split;
    uint32_t split_inv;     // n / splits = n * split_inv >> 16 for n below HEADS + MAX_SPLITS
    float *lse2;            // [R][H] log2 of the sums, for the weights
    // Base-2 scores, for the weights: [R][head_blocks][tiles] blocks of 16 heads
    // by 64 rows, each as a warp holds it: [8][32 lanes][4], where lane's four
    // are head lane / 4 by rows 8 j + 2 (lane % 4) and + 1, then head lane / 4 + 8
    // by the same rows.
    float4 *scores;
    int64_t head_blocks;
    int tiles;
    bool whole;             // a CTA has all of a request: it adds up the weights itself
};

// This CTA's shared-memory address `at` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t at, int rank)
{
    uint32_t y;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(y) : "r"(at), "r"(rank));
    return y;
}

// Stores to a CTA of the cluster; its mbarrier `bar` counts the bytes as they
// arrive.
__device__ __forceinline__ void send_v2(uint32_t at, uint32_t x, uint32_t y, uint32_t bar)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1,%2}, [%3];" ::"r"(at), "r"(x), "r"(y),
                 "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void send_v4(uint32_t at, uint4 v, uint32_t bar)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1,%2,%3,%4}, [%5];" ::"r"(at), "r"(v.x),
                 "r"(v.y), "r"(v.z), "r"(v.w), "r"(bar)
                 : "memory");
}

// The cluster's barrier, for what has been waited for already (a release of all
// that a CTA has written takes some 1,400 cycles).
__device__ __forceinline__ void cluster_arrive()
{
    __syncwarp();      // (.aligned: the warp together)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait()
{
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Log2 of a head's whole sum, from its reference and sum, and where it goes.
__device__ __forceinline__ float log2_sum(float m, float l) { return l == 0.0f ? -INFINITY : m + log2f(l); }

__device__ __forceinline__ void store_lse(const AttendLaunch &a, const AttendParts &w, int64_t rh, float l2)
{
    if (a.lse) a.lse[rh] = l2 * kLn2;
    if (a.weights) w.lse2[rh] = l2;
}

// What a head's O is multiplied by at the end: 1 / l, and decode8's 2^7; l is
// normal or 0 (its largest term is at least 2^-8), and the quotient's error of
// two steps of 2^-23 small beside out's type.
__device__ __forceinline__ float out_factor(float l) { return l == 0.0f ? 0.0f : __fdividef(128.0f, l); }

// ---- join ------------------------------------------------------------------------
//
// Every CTA of a cluster has, for each of its heads, a part of O and its
// reference and sum; head i is joined by CTA i % splits, whose m-th head is its
// rank + m splits.  Parts are slots of 512 floats in shared memory, values in
// the columns' order (unit_values, decode8).  `staged`: a CTA's own parts are in
// slots 0 to heads - 1 first, and are sent on from there (512 bytes a store, 64 KB
// to a neighbour: 3.8 thousand cycles); else they go to their owner at once, 32
// bytes of a row at a time, straight from fragments (7.9 thousand).  What a CTA gets from the others comes behind its own: for each
// of its heads, one slot for each of the others, in their order.
constexpr uint32_t O_STRIDE = (kLatent + 8) * 4;     // (no bank conflicts between a fragment's rows)

// Slots that a staged join of so many heads and CTAs takes at most.
__host__ __device__ constexpr int staged_slots(int heads, int splits)
{
    return heads + (splits - 1) * ((heads + splits - 1) / splits);
}

struct Join {
    uint32_t slots;      // shared-memory address of slot 0
    uint32_t known, joined;     // and of the mbarriers that count what the others send: references
                                // and sums, parts of O
    float2 *ml;          // [mine][splits] reference and sum of each part, the own first
    int heads, splits, rank;
    uint32_t split_inv;
    bool staged;

    __host__ __device__ __forceinline__ int over_splits(int n) const { return (int)(n * split_inv >> 16); }
    __host__ __device__ __forceinline__ int count(int owner) const { return over_splits(heads - owner + splits - 1); }
    // The own part of the CTA's m-th head, and the first that another sends it.
    __host__ __device__ __forceinline__ uint32_t own(int m) const { return slots + (staged ? rank + m * splits : m) * O_STRIDE; }
    __host__ __device__ __forceinline__ uint32_t others(int owner, int m) const
    {
        return slots + ((staged ? heads : count(owner)) + m * (splits - 1)) * O_STRIDE;
    }
    // Where this CTA's part of owner's m-th head goes: in owner, if that is another.
    __host__ __device__ __forceinline__ uint32_t place(int owner, int m) const
    {
        return owner == rank ? own(m) : others(owner, m) + (rank - (rank > owner)) * O_STRIDE;
    }
    // Where this CTA's reference and sum of head i go in owner's ml: a head's own
    // first, then the others' in the order of their parts.
    __host__ __device__ __forceinline__ int ml_at(int i, int owner) const
    {
        return owner == rank ? i - owner : i - owner + rank + (rank < owner);
    }
    // What the others send a CTA.
    __host__ __device__ __forceinline__ uint32_t parts() const { return count(rank) * (splits - 1); }
    // Staged parts to their owners.  Every CTA's slots must be free to take them.
    __device__ __forceinline__ void send(int warp, int warps, int lane) const
    {
#pragma unroll 2
        for (int n = warp; n < heads * 2; n += warps) {       // half a head's values a warp
            const int i = n >> 1, m = over_splits(i), owner = i - m * splits;
            if (owner == rank) continue;
            const uint32_t off = (n & 1) * 1024 + lane * 16, bar = in_cta(joined, owner);
            const uint32_t src = slots + i * O_STRIDE + off, dst = in_cta(place(owner, m) + off, owner);
            const uint4 x = ld_smem_v4(src), y = ld_smem_v4(src + 512);
            send_v4(dst, x, bar);
            send_v4(dst + 512, y, bar);
        }
    }
    // A head's reference and sum to its owner.
    __device__ __forceinline__ void send_ml(int i, float m, float l) const
    {
        const int owner = i - over_splits(i) * splits;
        if (owner == rank)
            ml[ml_at(i, owner)] = make_float2(m, l);
        else
            send_v2(in_cta(smem_u32(&ml[ml_at(i, owner)]), owner), __float_as_uint(m), __float_as_uint(l),
                    in_cta(known, owner));
    }
    // Once all references and sums are here: each part's factor 2^(m_p - m) / sum_p
    // 2^(m_p - m) l_p, and lse, of heads rh + ...; 16 threads a head.
    __device__ __forceinline__ void factors(const AttendLaunch &a, const AttendParts &w, int64_t rh, int tid) const
    {
        static_assert(MAX_SPLITS == 16, "");
        const int m = tid >> 4, p = tid & 15;
        const bool on = m < count(rank);
        const float2 x = on && p < splits ? ml[m * splits + p] : make_float2(-INFINITY, 0.0f);
        float top = x.x;
#pragma unroll
        for (int o = 1; o < 16; o *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float f = ex2(x.x - (top == -INFINITY ? 0.0f : top));
        float l = f * x.y;
#pragma unroll
        for (int o = 1; o < 16; o *= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (on && p < splits) ml[m * splits + p].x = f * out_factor(l);
        if (on && p == 0) store_lse(a, w, rh + rank + m * splits, log2_sum(top, l));
    }
    // Once all parts are here too, their sums.  A warp takes U quarters of a head's
    // values at a time (1 of few heads, 4 of many: 33.0 against 34.4 us for 32
    // requests of 128 heads, where a CTA has 32), two threads a unit, whose values are 128 neighbours of out a
    // quarter.  Of eight values the even are in one 16-byte piece and the odd in
    // the next, here in neighbouring lanes.
    template <int DT, int U>
    __device__ __forceinline__ void finish(const AttendLaunch &a, int r, int h0, int warp, int warps, int lane) const
    {
        const int mine = count(rank);
#pragma unroll 1
        for (int n = warp * U; n < 4 * mine; n += warps * U) {
            const int m = n >> 2, unit0 = (lane >> 3) * 16 + (lane >> 1 & 3);
            auto unit = [&](int u) { return unit0 + ((n + u) & 1) * 8 + ((n + u) >> 1 & 1) * 4; };
            const float2 *f = ml + m * splits;
            const uint32_t off = (lane & 1) * 16;
            float o[U][4] = {};
            auto add = [&](uint32_t at, float f) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const uint4 x = ld_smem_v4(at + unit(u) * 32);
                    o[u][0] = fmaf(f, __uint_as_float(x.x), o[u][0]);
                    o[u][1] = fmaf(f, __uint_as_float(x.y), o[u][1]);
                    o[u][2] = fmaf(f, __uint_as_float(x.z), o[u][2]);
                    o[u][3] = fmaf(f, __uint_as_float(x.w), o[u][3]);
                }
            };
            add(own(m) + off, f[0].x);
            uint32_t at = others(rank, m) + off;
#pragma unroll (U == 1 ? 3 : 1)
            for (int p = 1; p < splits; ++p, at += O_STRIDE) add(at, f[p].x);
            uint8_t *out = a.out + (int64_t)r * a.out_rs + (int64_t)(h0 + rank + m * splits) * a.out_hs;
            const bool odd = lane & 1;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // even lane: values 0-3 of its eight; odd lane: 4-7
                const float g0 = __shfl_xor_sync(0xffffffffu, odd ? o[u][0] : o[u][2], 1);
                const float g1 = __shfl_xor_sync(0xffffffffu, odd ? o[u][1] : o[u][3], 1);
                *reinterpret_cast<uint2 *>(out + unit_values(unit(u)) * 2 + odd * 8) =
                    odd ? make_uint2(floats_to_pair<DT>(g0, o[u][2]), floats_to_pair<DT>(g1, o[u][3]))
                        : make_uint2(floats_to_pair<DT>(o[u][0], g0), floats_to_pair<DT>(o[u][1], g1));
            }
        }
    }
};

}  // namespace hs
