// rows.cu -- KV rows normalised and stored by slot, and read back
// (include/hisparse_pages.h, hisparse_norm_rows, hisparse_gather_rows).
//
// The mathematics.  y = x w / sqrt(mean x^2 + eps): the product x w of two
// 16-bit values is exact in 32 bits, so y has one rounding of its own and those
// of the one factor 1 / sqrt.  Then per group of 128 values a power of two and
// e4m3 codes, per group of 16 an e4m3 scale and e2m1 codes, or y in 16 bits.
//
// Bound by HBM: 1,152 bytes of values and 416 to 1,152 of row, each moved once;
// nothing is kept between rows.  A warp works on a whole row: a lane holds 8
// neighbouring values of each half of the latent part, so every load and store of
// the warp is contiguous (512 bytes of values, 256 of e4m3 codes), a group of 16
// is two neighbouring lanes, one of 128 half a warp.
#include "pages.cuh"

namespace hs {
namespace {

constexpr int ROWS_NT = 128, ROWS_CTAS = 14;     // threads a CTA, CTAs an SM
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

// Largest magnitude of the 8 values of `lanes` neighbouring lanes; NaN if one is
// (as integers, a NaN's magnitude is the largest).
template <int LANES>
__device__ __forceinline__ uint32_t top_bits(const float (&y)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(y[j]) & 0x7FFFFFFFu);
#pragma unroll
    for (int d = 1; d < LANES; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    return m;
}

// The exponent k of the least power of two with m <= 448 2^k = 1.75 2^(k + 8),
// from the bits of m; -126 at least.
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

// 8 values to a row: those from 256 half + 8 lane on.
__device__ __forceinline__ void store8(uint8_t *dst, const float (&y)[8], int half, int lane)
{
    const uint32_t m = top_bits<16>(y);
    // infinities have the exponent of 2^128: 2^120, and their codes clip to 448
    const int k = scale_exponent(min(m, 0x7F800000u));
    const float inv = power_of_two(-k);
    const bool nan = m > 0x7F800000u;
    *reinterpret_cast<uint2 *>(dst + half * 256 + lane * 8) =
        make_uint2(e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                   e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
    if ((lane & 15) == 0)
        *reinterpret_cast<float *>(dst + kRow8ScaleAt + (half * 2 + (lane >> 4)) * 4) = nan ? __uint_as_float(0x7FC00000u) : power_of_two(k);
}

// normed: y is any 32-bit number, and y * (1 / scale) as good as the quotient;
// else it has a 16-bit type's value, and may lie on a border between two codes:
// then the product's rounding is taken out (see rows4.cu), which would move
// numbers next to a border onto it.
__device__ __forceinline__ void store4(uint8_t *dst, const float (&y)[8], int half, int lane, bool normed)
{
    const float top = __uint_as_float(top_bits<2>(y));
    uint16_t e8;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e8) : "f"(0.0f), "f"(__fdiv_rn(top, 6.0f)));
    const float scale = __low2float(scale_half2(e8 & 0xFFu));
    const float inv = scale == 0.0f ? 0.0f : __frcp_rn(scale);
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float t = normed ? y[j] * inv : __fadd_rn(__fmaf_rn(y[j], inv, 48.0f), -48.0f);
        q[j] = __uint_as_float((__float_as_uint(t) & 0x7FFFFFFFu) | (__float_as_uint(y[j]) & 0x80000000u));
    }
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
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    *reinterpret_cast<uint32_t *>(dst + half * 128 + lane * 4) = out;
    if (!(lane & 1)) dst[kScaleAt + half * 16 + (lane >> 1)] = (uint8_t)e8;
}

// The row that value i goes to or comes from; -1: none.
__device__ __forceinline__ int64_t row_of_value(const RowsLaunch &a, int64_t i)
{
    const int64_t s = a.slots ? a.slots[i] : i;
    return s < a.num_rows ? s : -1;
}

template <int DT, int ROW>
__global__ void __launch_bounds__(ROWS_NT, ROWS_CTAS) norm_kernel(const __grid_constant__ RowsLaunch a)
{
    after_launch_before();
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * ROWS_A_CTA + (threadIdx.x >> 5);
    if (i >= a.n) return;      // the same for the whole warp
    const int64_t row = row_of_value(a, i);
    if (row < 0) return;
    const uint8_t *src = a.values + i * a.value_stride;
    uint8_t *dst = a.rows + row * a.row_stride;
    const uint4 v[2] = {ld_dev_v4(src + lane * 16), ld_dev_v4(src + 512 + lane * 16)};
    uint4 rope;
    if (lane < 8) rope = ld_dev_v4(src + kLatent * 2 + lane * 16);
    float y[2][8];
    unpack16<DT>(v[0], y[0]);
    unpack16<DT>(v[1], y[1]);
    if (a.weight) {
        float sum = 0.0f;
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(y[half][j], y[half][j], sum);
#pragma unroll
        for (int d = 1; d < 32; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const float f = __frcp_rn(__fsqrt_rn(fmaf(sum, 1.0f / kLatent, a.eps)));
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float w[8];
            unpack16<DT>(ld_dev_v4(a.weight + half * 512 + lane * 16), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[half][j] = y[half][j] * w[j] * f;
        }
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        if (ROW == kRow16)
            st_v4(dst + half * 512 + lane * 16, pack16<DT>(y[half]));
        else if (ROW == kRow8)
            store8(dst, y[half], half, lane);
        else
            store4(dst, y[half], half, lane, a.weight != nullptr);
    }
    if (lane < 8) st_v4(dst + rope_at(ROW) + lane * 16, rope);
}

template <int DT, int ROW>
__global__ void __launch_bounds__(ROWS_NT, ROWS_CTAS) gather_kernel(const __grid_constant__ RowsLaunch a)
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

cudaError_t launch_norm_rows(const RowsLaunch &a, cudaStream_t s)
{
    const bool b = a.dtype == kBf16;
    if (a.row_bytes == kRow4) return b ? launch(norm_kernel<kBf16, kRow4>, a, s) : launch(norm_kernel<kF16, kRow4>, a, s);
    if (a.row_bytes == kRow8) return b ? launch(norm_kernel<kBf16, kRow8>, a, s) : launch(norm_kernel<kF16, kRow8>, a, s);
    return b ? launch(norm_kernel<kBf16, kRow16>, a, s) : launch(norm_kernel<kF16, kRow16>, a, s);
}

cudaError_t launch_gather_rows(const RowsLaunch &a, cudaStream_t s)
{
    const bool b = a.dtype == kBf16;
    if (a.row_bytes == kRow4) return b ? launch(gather_kernel<kBf16, kRow4>, a, s) : launch(gather_kernel<kF16, kRow4>, a, s);
    if (a.row_bytes == kRow8) return b ? launch(gather_kernel<kBf16, kRow8>, a, s) : launch(gather_kernel<kF16, kRow8>, a, s);
    return b ? launch(gather_kernel<kBf16, kRow16>, a, s) : launch(gather_kernel<kF16, kRow16>, a, s);
}

}  // namespace hs
