// rows.cu -- KV rows normalised and stored by slot, and read back
// (include/hisparse_pages.h, hisparse_norm_rows, hisparse_gather_rows).
//
// The mathematics.  y = x w / sqrt(mean x^2 + eps): the product t = x w of two 16-bit
// values is exact in 32 bits (as long as it is a normal number there), so y = t f has one rounding of its own and those of the one
// factor f = 1 / sqrt, and the largest |y| of a group is that of t, times f.  Then per
// group of 128 values a power of two s and e4m3 codes of t (f / s), per group of 16 an
// e4m3 scale and e2m1 codes, or y in 16 bits.  Codes and scales are those of unlimited
// precision (a y within 2^-42 of a border between two counts as on it): worked out with f
// too small and too large by what it may be off, and, where that makes a difference, with
// pairs of numbers.
//
// Bound by HBM: 1,152 bytes of values and 416 to 1,152 of row, each moved once; nothing
// is kept between rows; and, next to it, by instructions.  A warp works on a whole row.  For
// codes a lane has 16 neighbouring values: a group of 16 is a lane's own, one of 128 eight
// lanes', its scale worked out once a lane, and the codes' stores are contiguous (8 values
// of each half a lane, whose loads are, took 1.5 us more for the first case below).  Products
// of 16-bit pairs go straight into 32 bits.
// Not kept: values read with the hint that they leave L2 first (2 to 6 % less for 65,536
// rows, 3 to 6 % more for 16,384 and for 196,608 and up).  GPU time there and back, at slots
// in no order: 262,144 rows of 656 bytes 157 us, 0.89 of the copy rate (152.3 without the
// second look); 70,001 of 416 38.4, 0.80 (36.8).  norm_kernel and gather_kernel alone, 262,144
// rows: of 416 bytes 71 and 69 us, of 656 83 and 75, of 1,152 89 and 89; without a weight
// 66, 76 and 89.
#include "pages.cuh"

namespace hs {
namespace {

constexpr int ROWS_NT = 128;                     // threads a CTA
constexpr int NORM_CTAS = 14, GATHER_CTAS = 16;  // CTAs an SM (norm, 262,144 rows of 656
                                                 // bytes: 12 90 us, 14 and 16 83)
constexpr int ROWS_A_CTA = ROWS_NT / 32;

template <int DT>
__device__ __forceinline__ void unpack16(const uint4 &v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 p = pair_to_float<DT>(w[j]);
        x[2 * j] = p.x;
        x[2 * j + 1] = p.y;
    }
}

template <int DT>
__device__ __forceinline__ uint4 pack16(const float (&x)[8])
{
    return make_uint4(floats_to_pair<DT>(x[0], x[1]), floats_to_pair<DT>(x[2], x[3]), floats_to_pair<DT>(x[4], x[5]), floats_to_pair<DT>(x[6], x[7]));
}

// sum + a[k] b[k], k = 0, 1, and a[k] b[k], of 16-bit pairs, in 32 bits.
template <int DT>
__device__ __forceinline__ float fma16(uint32_t a, uint32_t b, int k, float c)
{
    const uint16_t x = (uint16_t)(a >> (16 * k)), y = (uint16_t)(b >> (16 * k));
    float d;
    if (DT == kBf16)
        asm("fma.rn.f32.bf16 %0, %1, %2, %3;" : "=f"(d) : "h"(x), "h"(y), "f"(c));
    else
        asm("fma.rn.f32.f16 %0, %1, %2, %3;" : "=f"(d) : "h"(x), "h"(y), "f"(c));
    return d;
}

// Largest magnitude of the 16 values of LANES neighbouring lanes; NaN if one is.
template <int LANES>
__device__ __forceinline__ float largest(const float (&t)[16])
{
    auto max3 = [](float x, float y, float z) {
        float m;
        asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(fabsf(x)), "f"(fabsf(y)), "f"(fabsf(z)));
        return m;
    };
    float m = fabsf(t[15]);
#pragma unroll
    for (int j = 0; j < 14; j += 2) m = j ? max3(m, t[j], t[j + 1]) : max3(t[0], t[1], t[15]);
    m = max3(m, t[14], t[14]);
#pragma unroll
    for (int d = 1; d < LANES; d *= 2) {
        const float o = __shfl_xor_sync(0xffffffffu, m, d);
        m = max3(m, o, o);
    }
    return m;
}

// The exponent k of the least power of two with m <= 448 2^k = 1.75 2^(k + 8), from the
// bits of m; -126 at least.
__device__ __forceinline__ int scale_exponent(uint32_t m)
{
    return max((int)(m >> 23) - 127 - 8 + ((m & 0x7FFFFFu) > 0x600000u), -126);
}

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// x with the sign of y: of a 0, which sums and products of two numbers lose.
__device__ __forceinline__ float signed_as(float x, float y)
{
    return __uint_as_float((__float_as_uint(x) & 0x7FFFFFFFu) | (__float_as_uint(y) & 0x80000000u));
}

// How far t f / scale may be from what it stands for: 13 roundings of 2^-24 (of the sum of
// squares 10, of which the root halves what they come to; the mean, the root 2, 1 / scale 2,
// the products 3).  Codes and scales that are the same this far to both sides are those of
// unlimited precision; a row with others, one in a hundred, is done again with twice the
// bits (exact_row).  (Without that, counted over random rows as in perf/more_operators.py, 255
// of 5.4 x 10^8 8-bit codes, 87 of 5.4 x 10^8 4-bit ones and 13 of 3.4 x 10^7 of their scales
// are the next one.)
constexpr float LOW = 1.0f - 13.0f / (1 << 24), HIGH = 1.0f + 13.0f / (1 << 24);

// Values t f, those from 16 lane on, to a row.  NORM: whether a code or scale may be the
// one next to it; nothing is stored if the warp has one.
template <bool NORM>
__device__ __forceinline__ bool store8(uint8_t *dst, float (&t)[16], float f, int lane)
{
    const float top = largest<8>(t) * f;
    const uint32_t m = __float_as_uint(top);
    // infinities have the exponent of 2^128: 2^120, and their codes clip to 448
    const int k = scale_exponent(min(m, 0x7F800000u));
    float by = f * power_of_two(-k);            // (exact: a power of two)
    const bool far = !(by <= FLT_MAX);          // a group of zeros, or next to it
    if (far) {
        by = power_of_two(-k);
#pragma unroll
        for (int j = 0; j < 16; ++j) t[j] *= f;
    }
    uint32_t c[4];
    bool near = false;
    if (NORM) {
        const float low = by * LOW, high = by * HIGH;
        near = scale_exponent(min(__float_as_uint(top * LOW), 0x7F800000u)) != scale_exponent(min(__float_as_uint(top * HIGH), 0x7F800000u));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            c[j] = e4m3x4(t[4 * j] * low, t[4 * j + 1] * low, t[4 * j + 2] * low, t[4 * j + 3] * low);
            near |= c[j] != e4m3x4(t[4 * j] * high, t[4 * j + 1] * high, t[4 * j + 2] * high, t[4 * j + 3] * high);
        }
        if (__any_sync(0xffffffffu, near)) return true;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = e4m3x4(t[4 * j] * by, t[4 * j + 1] * by, t[4 * j + 2] * by, t[4 * j + 3] * by);
    }
    st_v4(dst + lane * 16, make_uint4(c[0], c[1], c[2], c[3]));
    if ((lane & 7) == 0) *reinterpret_cast<float *>(dst + kRow8ScaleAt + (lane >> 3) * 4) = top != top ? top : power_of_two(k);
    return false;
}

__device__ __forceinline__ uint32_t e2m1x8(const float (&q)[16], int j)
{
    uint32_t out;
    asm("{\n"
        ".reg .b8 b0, b1, b2, b3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        "mov.b32 %0, {b0, b1, b2, b3};\n"
        "}"
        : "=r"(out)
        : "f"(q[j]), "f"(q[j + 1]), "f"(q[j + 2]), "f"(q[j + 3]), "f"(q[j + 4]), "f"(q[j + 5]), "f"(q[j + 6]), "f"(q[j + 7]));
    return out;
}

// The same.  Not NORM: f is 1 and t has a 16-bit type's value, and may lie on a border
// between two codes: then the product's rounding is taken out (see rows4.cu), which would
// move numbers next to a border onto it.
template <bool NORM>
__device__ __forceinline__ bool store4(uint8_t *dst, float (&t)[16], float f, int lane)
{
    const float top = largest<1>(t) * f, sixth = __fdiv_rn(top, 6.0f);
    uint16_t e8;
    bool near = false;
    if (NORM) {
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e8) : "f"(sixth * LOW), "f"(sixth * HIGH));
        near = (e8 & 0xFFu) != e8 >> 8;
    } else {
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e8) : "f"(0.0f), "f"(sixth));
    }
    const float scale = __low2float(scale_half2(e8 & 0xFFu));
    uint2 c;
    if (NORM) {      // (approximate, and one step of Newton's method; scale >= 2^-9 or 0)
        float inv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
        inv = fmaf(inv, fmaf(-scale, inv, 1.0f), inv);
        const float by = f * (scale == 0.0f ? 0.0f : inv), low = by * LOW, high = by * HIGH;
        float q[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) q[j] = t[j] * low;
        c = make_uint2(e2m1x8(q, 0), e2m1x8(q, 8));
#pragma unroll
        for (int j = 0; j < 16; ++j) q[j] = t[j] * high;
        near |= c.x != e2m1x8(q, 0) || c.y != e2m1x8(q, 8);
        if (__any_sync(0xffffffffu, near)) return true;
    } else {
        const float inv = scale == 0.0f ? 0.0f : __frcp_rn(scale);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            t[j] = signed_as(__fadd_rn(__fmaf_rn(t[j], inv, 48.0f), -48.0f), t[j]);
        }
        c = make_uint2(e2m1x8(t, 0), e2m1x8(t, 8));
    }
    *reinterpret_cast<uint2 *>(dst + lane * 8) = c;
    dst[kScaleAt + lane] = (uint8_t)e8;
    return false;
}

// 1 / sqrt(v), by one step of Newton's method from the approximate root, off by about
// 2^-23; 0 for infinity.
__device__ __forceinline__ float inverse_root(float v)
{
    const float r = rsqrtf(v), e = fmaf(-v * r, r, 1.0f);
    return v <= FLT_MAX ? fmaf(0.5f * r, e, r) : r;
}

// A sum of two numbers, the second less than half a step of the first: 47 bits or more.
struct Twice {
    float hi, lo;
};

// x + y, y small against x (infinities and NaN stay what they are).
__device__ __forceinline__ Twice together(float x, float y)
{
    if (!(fabsf(x) <= FLT_MAX)) return {x, 0.0f};
    const float h = __fadd_rn(x, y);
    return {h, __fsub_rn(y, __fsub_rn(h, x))};
}

__device__ __forceinline__ Twice plus(const Twice &x, const Twice &y)
{
    const float s = __fadd_rn(x.hi, y.hi), b = __fsub_rn(s, x.hi);
    return together(s, __fadd_rn(__fadd_rn(__fsub_rn(x.hi, __fsub_rn(s, b)), __fsub_rn(y.hi, b)), __fadd_rn(x.lo, y.lo)));
}

__device__ __forceinline__ Twice times(const Twice &x, float y)
{
    const float h = __fmul_rn(x.hi, y);
    return together(h, __fmaf_rn(x.lo, y, __fmaf_rn(x.hi, y, -h)));
}

// x / y: what the approximate quotient leaves, once.
__device__ __forceinline__ Twice over(const Twice &x, float y)
{
    const float inv = __frcp_rn(y), h = __fmul_rn(x.hi, inv);
    return together(h, __fmul_rn(__fadd_rn(__fmaf_rn(-h, y, x.hi), x.lo), inv));
}

// 1 / sqrt(v): a step of Newton's method, its difference kept apart.  (Below 2^-100 v.lo has
// lost its bits, and r^2 may be too large.)
__device__ __forceinline__ Twice inverse_root(const Twice &v)
{
    if (v.hi < 0x1p-100f) return {inverse_root(v.hi), 0.0f};
    const float r = inverse_root(v.hi), p = __fmul_rn(r, r), pl = __fmaf_rn(r, r, -p);
    const float e = __fsub_rn(__fmaf_rn(-v.hi, p, 1.0f), __fmaf_rn(v.hi, pl, __fmul_rn(v.lo, p)));
    return together(r, __fmul_rn(__fmul_rn(0.5f, r), e));
}

// In 32 bits, cut off, with the last bit set if that is not exact: rounded again to fewer
// bits it gives what x does.  A pair here is off by 12 roundings of 2^-47 (of the sum of
// squares 11, halved by the root; the mean, the root 2, the products 3): nearer than 2^-42 to a
// number of 24 bits, which borders between codes are, x counts as that number.  (Without
// that a y that lies on a border, as with rows of one magnitude and eps 0, got the code below.)
__device__ __forceinline__ float to_odd(const Twice &x)
{
    const uint32_t h = __float_as_uint(x.hi), l = __float_as_uint(x.lo);
    return !(fabsf(x.lo) > fabsf(x.hi) * 0x1p-42f) ? x.hi : __uint_as_float((h - ((h ^ l) >> 31)) | 1u);
}

// The row that value i goes to or comes from; -1: none.
__device__ __forceinline__ int64_t row_of_value(const RowsLaunch &a, int64_t i)
{
    const int64_t s = a.slots ? a.slots[i] : i;
    return s < a.num_rows ? s : -1;
}

// Codes and scales of the warp's row, normalised, with twice the bits.  (Its root is a
// number: with another, codes are the same to both sides.)
template <int DT, int ROW>
__device__ __noinline__ void exact_row(const RowsLaunch &a)
{
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * ROWS_A_CTA + (threadIdx.x >> 5);
    const uint8_t *src = a.values + i * a.value_stride;
    uint8_t *dst = a.rows + row_of_value(a, i) * a.row_stride;
    float t[16];
    Twice sums[4] = {};
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        float x[8], w[8];
        unpack16<DT>(ld_dev_v4(src + half * 16 + lane * 32), x);
        unpack16<DT>(ld_dev_v4(a.weight + half * 16 + lane * 32), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sums[j & 3] = plus(sums[j & 3], {x[j] * x[j], 0.0f});      // (exact)
            t[half * 8 + j] = x[j] * w[j];
        }
    }
    Twice sum = plus(plus(sums[0], sums[1]), plus(sums[2], sums[3]));
#pragma unroll
    for (int d = 1; d < 32; d *= 2)
        sum = plus(sum, {__shfl_xor_sync(0xffffffffu, sum.hi, d), __shfl_xor_sync(0xffffffffu, sum.lo, d)});
    const Twice f = inverse_root(plus({sum.hi / kLatent, sum.lo / kLatent}, {a.eps, 0.0f}));
    const Twice top = times(f, largest<ROW == kRow8 ? 8 : 1>(t));
    if (ROW == kRow8) {
        // (448 is even: a top above a border is above it when its last bit is set)
        const int k = scale_exponent(min(__float_as_uint(to_odd(top)), 0x7F800000u));
        const float by = power_of_two(-k);      // (f times this may be too much: see store8)
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const Twice y = times(f, t[j]);
            t[j] = signed_as(to_odd({y.hi * by, y.lo * by}), t[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = e4m3x4(t[4 * j], t[4 * j + 1], t[4 * j + 2], t[4 * j + 3]);
        st_v4(dst + lane * 16, make_uint4(c[0], c[1], c[2], c[3]));
        if ((lane & 7) == 0) *reinterpret_cast<float *>(dst + kRow8ScaleAt + (lane >> 3) * 4) = top.hi != top.hi ? top.hi : power_of_two(k);
    } else {
        uint16_t e8;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e8) : "f"(0.0f), "f"(to_odd(over(top, 6.0f))));
        const float scale = __low2float(scale_half2(e8 & 0xFFu));
        const Twice g = scale == 0.0f ? Twice{0.0f, 0.0f} : over(f, scale);
#pragma unroll
        for (int j = 0; j < 16; ++j) t[j] = signed_as(to_odd(times(g, t[j])), t[j]);
        *reinterpret_cast<uint2 *>(dst + lane * 8) = make_uint2(e2m1x8(t, 0), e2m1x8(t, 8));
        dst[kScaleAt + lane] = (uint8_t)e8;
    }
}

template <int DT, int ROW, bool NORM>
__global__ void __launch_bounds__(ROWS_NT, NORM_CTAS) norm_kernel(const __grid_constant__ RowsLaunch a)
{
    // A lane's two pieces of 8 values: 16 neighbouring ones, or of each half of the row
    constexpr int LANE = ROW == kRow16 ? 16 : 32, NEXT = ROW == kRow16 ? 512 : 16;
    after_launch_before();
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * ROWS_A_CTA + (threadIdx.x >> 5);
    if (i >= a.n) return;      // the same for the whole warp
    const uint8_t *src = a.values + i * a.value_stride;
    // (ahead of the slot, which would be one more wait)
    const uint4 v[2] = {ld_dev_v4(src + lane * LANE), ld_dev_v4(src + NEXT + lane * LANE)};
    uint4 rope;
    if (lane < 8) rope = ld_dev_v4(src + kLatent * 2 + lane * 16);
    const int64_t row = row_of_value(a, i);
    if (row < 0) return;
    uint8_t *dst = a.rows + row * a.row_stride;
    if (lane < 8) st_v4(dst + rope_at(ROW) + lane * 16, rope);
    float t[16], f = 1.0f;
    if (NORM) {
        float sums[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const uint4 w4 = ld_dev_v4(a.weight + half * NEXT + lane * LANE);
            const uint32_t x[4] = {v[half].x, v[half].y, v[half].z, v[half].w}, w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sums[j & 3] = fma16<DT>(x[j >> 1], x[j >> 1], j & 1, sums[j & 3]);
                t[half * 8 + j] = fma16<DT>(x[j >> 1], w[j >> 1], j & 1, -0.0f);
            }
        }
        float sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
#pragma unroll
        for (int d = 1; d < 32; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        f = inverse_root(fmaf(sum, 1.0f / kLatent, a.eps));
    } else {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float x[8];
            unpack16<DT>(v[half], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) t[half * 8 + j] = x[j];
        }
    }
    if (ROW == kRow16) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = t[half * 8 + j] * f;
            st_v4(dst + half * 512 + lane * 16, pack16<DT>(x));
        }
    } else if (ROW == kRow8) {
        if (store8<NORM>(dst, t, f, lane)) exact_row<DT, ROW>(a);
    } else {
        if (store4<NORM>(dst, t, f, lane)) exact_row<DT, ROW>(a);
    }
}

template <int DT, int ROW>
__global__ void __launch_bounds__(ROWS_NT, GATHER_CTAS) gather_kernel(const __grid_constant__ RowsLaunch a)
{
    after_launch_before();
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * ROWS_A_CTA + (threadIdx.x >> 5);
    if (i >= a.n) return;
    const int64_t row = row_of_value(a, i);
    if (row < 0) return;
    const uint8_t *src = a.rows + row * a.row_stride;
    uint8_t *dst = a.values + i * a.value_stride;
    uint4 rope;
    if (lane < 8) rope = ld_dev_v4(src + rope_at(ROW) + lane * 16);
    uint4 v[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) v[half] = load_latent8<DT, ROW>(src, half * 32 + lane);
#pragma unroll
    for (int half = 0; half < 2; ++half) st_v4(dst + half * 512 + lane * 16, v[half]);
    if (lane < 8) st_v4(dst + kLatent * 2 + lane * 16, rope);
}

template <class Kernel>
cudaError_t launch(Kernel kernel, const RowsLaunch &a, cudaStream_t s)
{
    return launch_behind(kernel, dim3((unsigned)((a.n + ROWS_A_CTA - 1) / ROWS_A_CTA)), ROWS_NT, 0, 1, s, a);
}

}  // namespace

template <int DT, int ROW>
static cudaError_t launch_norm(const RowsLaunch &a, cudaStream_t s)
{
    return a.weight ? launch(norm_kernel<DT, ROW, true>, a, s) : launch(norm_kernel<DT, ROW, false>, a, s);
}

cudaError_t launch_norm_rows(const RowsLaunch &a, cudaStream_t s)
{
    const bool b = a.dtype == kBf16;
    if (a.row_bytes == kRow4) return b ? launch_norm<kBf16, kRow4>(a, s) : launch_norm<kF16, kRow4>(a, s);
    if (a.row_bytes == kRow8) return b ? launch_norm<kBf16, kRow8>(a, s) : launch_norm<kF16, kRow8>(a, s);
    return b ? launch_norm<kBf16, kRow16>(a, s) : launch_norm<kF16, kRow16>(a, s);
}

cudaError_t launch_gather_rows(const RowsLaunch &a, cudaStream_t s)
{
    const bool b = a.dtype == kBf16;
    if (a.row_bytes == kRow4) return b ? launch(gather_kernel<kBf16, kRow4>, a, s) : launch(gather_kernel<kF16, kRow4>, a, s);
    if (a.row_bytes == kRow8) return b ? launch(gather_kernel<kBf16, kRow8>, a, s) : launch(gather_kernel<kF16, kRow8>, a, s);
    return b ? launch(gather_kernel<kBf16, kRow16>, a, s) : launch(gather_kernel<kF16, kRow16>, a, s);
}

}  // namespace hs
