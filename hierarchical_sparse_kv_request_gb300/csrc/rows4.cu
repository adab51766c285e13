// rows4.cu -- packing of KV rows to 4 bits and back, and the C entry points
// of include/hisparse_rows4.h that take no handle.
//
// A row's latent values are quantised in groups of 16: scale = the e4m3 value
// nearest to (largest magnitude) / 6, code = the e2m1 value nearest to value
// / scale.  Both kernels are bound by HBM (1152 bytes of values and 416 of
// row per row, each moved once); they keep no state between rows.
//
// A warp works on whole rows: a lane holds 8 consecutive values of each half
// of the latent part, so every load and store of the warp is contiguous (512
// bytes of values, 128 bytes of codes), and a group is two neighbouring lanes.
#include "hisparse_rows4.h"

#include "rows4.cuh"

namespace hs {
namespace {

// A row a warp, and as many CTAs as that takes: measured 125 us for 262,144
// rows packed and unpacked (the bytes alone take 121), 138 with two rows a warp in
// a loop over the rows.
constexpr int ROWS_NT = 128, ROWS_CTAS = 16;     // threads a CTA, CTAs an SM
constexpr int ROWS_A_CTA = ROWS_NT / 32;

template <int DT>
__device__ __forceinline__ float2 pair_to_float(uint32_t w)
{
    if (DT == kBf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// value / scale rounded to a multiple of 2^-18, with the value's sign also at
// 0.  inv is 1 / scale correctly rounded; the product may be off a border
// between two codes by an ulp where value / scale lies on it, and adding and
// taking off 48 rounds it back onto the border (|value / scale| <= 12 unless
// it clips anyway).  A value that is not on a border is at least 2^-11
// (relative) away from it: values have at most 11 significant bits, borders
// times scales 7.
__device__ __forceinline__ float quotient(float x, float inv)
{
    const float t = __fadd_rn(__fmaf_rn(x, inv, 48.0f), -48.0f);
    return __uint_as_float((__float_as_uint(t) & 0x7FFFFFFFu) | (__float_as_uint(x) & 0x80000000u));
}

template <int DT>
__device__ __forceinline__ uint32_t pack8(const uint4 &v, float inv)
{
    const float2 a = pair_to_float<DT>(v.x), b = pair_to_float<DT>(v.y);
    const float2 c = pair_to_float<DT>(v.z), d = pair_to_float<DT>(v.w);
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
        : "f"(quotient(a.x, inv)), "f"(quotient(a.y, inv)), "f"(quotient(b.x, inv)),
          "f"(quotient(b.y, inv)), "f"(quotient(c.x, inv)), "f"(quotient(c.y, inv)),
          "f"(quotient(d.x, inv)), "f"(quotient(d.y, inv)));
    return out;
}

template <int DT>
__global__ void __launch_bounds__(ROWS_NT, ROWS_CTAS) pack_kernel(const uint8_t *values, int64_t vstride, int64_t n,
                                                                  uint8_t *rows, int64_t rstride)
{
    after_launch_before();
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * ROWS_A_CTA + (threadIdx.x >> 5);
    if (i >= n) return;     // the same for the whole warp
    const uint8_t *src = values + i * vstride;
    uint8_t *dst = rows + i * rstride;
    const uint4 v[2] = {ld_dev_v4(src + lane * 16), ld_dev_v4(src + 512 + lane * 16)};
    uint4 rope;
    if (lane < 8) rope = ld_dev_v4(src + kLatent * 2 + lane * 16);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const uint4 x = v[half];
        // magnitudes compare as integers, and a NaN's is the largest
        uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                              __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
        const uint32_t top = max(m >> 16, m & 0xFFFFu);
        const float amax = pair_to_float<DT>(top).x;
        // amax has at most 11 significant bits and a border between two
        // scales times 6 at most 7: the division's rounding cannot move the
        // quotient across a border
        uint16_t e8;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e8) : "f"(0.0f), "f"(__fdiv_rn(amax, 6.0f)));
        const float scale = __low2float(scale_half2(e8 & 0xFFu));
        const float inv = scale == 0.0f ? 0.0f : __frcp_rn(scale);
        *reinterpret_cast<uint32_t *>(dst + half * 128 + lane * 4) = pack8<DT>(x, inv);
        if (!(lane & 1)) dst[kScaleAt + half * 16 + (lane >> 1)] = (uint8_t)e8;
    }
    if (lane < 8) st_v4(dst + kRopeAt + lane * 16, rope);
}

// Eight values of a row from a word of codes and their scale.
template <int DT>
__device__ __forceinline__ uint4 unpack8(uint32_t codes, __half2 scale)
{
    uint32_t h[4];
    codes_to_half2(codes, h);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2 p = __hmul2(*reinterpret_cast<__half2 *>(&h[j]), scale);
        if (DT == kBf16) {
            const __nv_bfloat162 b = __float22bfloat162_rn(__half22float2(p));
            h[j] = *reinterpret_cast<const uint32_t *>(&b);
        } else {
            h[j] = *reinterpret_cast<const uint32_t *>(&p);
        }
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}

template <int DT>
__global__ void __launch_bounds__(ROWS_NT, ROWS_CTAS) unpack_kernel(const uint8_t *rows, int64_t rstride, int64_t n,
                                                                    uint8_t *values, int64_t vstride)
{
    after_launch_before();
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * ROWS_A_CTA + (threadIdx.x >> 5);
    if (i >= n) return;
    const uint8_t *src = rows + i * rstride;
    uint8_t *dst = values + i * vstride;
    uint32_t c[2], e8[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        c[half] = *reinterpret_cast<const uint32_t *>(src + half * 128 + lane * 4);
        e8[half] = src[kScaleAt + half * 16 + (lane >> 1)];
    }
    uint4 rope;
    if (lane < 8) rope = ld_dev_v4(src + kRopeAt + lane * 16);
#pragma unroll
    for (int half = 0; half < 2; ++half)
        st_v4(dst + half * 512 + lane * 16, unpack8<DT>(c[half], scale_half2(e8[half])));
    if (lane < 8) st_v4(dst + kLatent * 2 + lane * 16, rope);
}

unsigned rows_grid(int64_t n) { return (unsigned)((n + ROWS_A_CTA - 1) / ROWS_A_CTA); }

}  // namespace

cudaError_t launch_pack_rows(const void *values, int64_t value_stride, int32_t dtype, int64_t n,
                             void *rows, int64_t row_stride, cudaStream_t s)
{
    auto *v = static_cast<const uint8_t *>(values);
    auto *d = static_cast<uint8_t *>(rows);
    if (dtype == kBf16)
        return launch_behind(pack_kernel<kBf16>, dim3(rows_grid(n)), ROWS_NT, 0, 1, s, v, value_stride * 2, n, d, row_stride);
    return launch_behind(pack_kernel<kF16>, dim3(rows_grid(n)), ROWS_NT, 0, 1, s, v, value_stride * 2, n, d, row_stride);
}

cudaError_t launch_unpack_rows(const void *rows, int64_t row_stride, int64_t n, void *values,
                               int64_t value_stride, int32_t dtype, cudaStream_t s)
{
    auto *d = static_cast<const uint8_t *>(rows);
    auto *v = static_cast<uint8_t *>(values);
    if (dtype == kBf16)
        return launch_behind(unpack_kernel<kBf16>, dim3(rows_grid(n)), ROWS_NT, 0, 1, s, d, row_stride, n, v, value_stride * 2);
    return launch_behind(unpack_kernel<kF16>, dim3(rows_grid(n)), ROWS_NT, 0, 1, s, d, row_stride, n, v, value_stride * 2);
}

}  // namespace hs

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

uint64_t apart(int64_t stride) { return stride < 0 ? 0u - (uint64_t)stride : (uint64_t)stride; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? HISPARSE_OK : HISPARSE_ERR_CUDA; }

int check_rows(const void *values, int64_t value_stride, int32_t dtype, int64_t n, const void *rows,
               int64_t row_stride)
{
    if (n < 0 || (dtype != HISPARSE_BF16 && dtype != HISPARSE_F16)) return HISPARSE_ERR_INVALID_ARG;
    if (value_stride < HISPARSE_ROW4_VALUES || value_stride % 8 != 0) return HISPARSE_ERR_INVALID_ARG;
    if (row_stride < HISPARSE_ROW4_BYTES || row_stride % 16 != 0) return HISPARSE_ERR_INVALID_ARG;
    if (n > 0 && (!values || !rows)) return HISPARSE_ERR_INVALID_ARG;
    if (n > HISPARSE_MAX_PACKED_ROWS) return HISPARSE_ERR_UNSUPPORTED;
    if (!aligned16(values) || !aligned16(rows)) return HISPARSE_ERR_ALIGNMENT;
    return HISPARSE_OK;
}

int check_attend_sizes(int32_t R, int32_t H, int32_t k)
{
    if (R < 1 || H < 1 || k < 1) return HISPARSE_ERR_INVALID_ARG;
    if (R > HISPARSE_MAX_REQUESTS || H > HISPARSE_MAX_HEADS || k > HISPARSE_MAX_TOP_K)
        return HISPARSE_ERR_UNSUPPORTED;
    return HISPARSE_OK;
}

}  // namespace

extern "C" {

int hisparse_pack_rows(const void *values, int64_t value_stride, int32_t dtype, int64_t n,
                       void *rows, int64_t row_stride, void *stream)
{
    const int rc = check_rows(values, value_stride, dtype, n, rows, row_stride);
    if (rc != HISPARSE_OK || n == 0) return rc;
    return cuda_status(hs::launch_pack_rows(values, value_stride, dtype, n, rows, row_stride,
                                            static_cast<cudaStream_t>(stream)));
}

int hisparse_unpack_rows(const void *rows, int64_t row_stride, int64_t n, void *values,
                         int64_t value_stride, int32_t dtype, void *stream)
{
    const int rc = check_rows(values, value_stride, dtype, n, rows, row_stride);
    if (rc != HISPARSE_OK || n == 0) return rc;
    return cuda_status(hs::launch_unpack_rows(rows, row_stride, n, values, value_stride, dtype,
                                              static_cast<cudaStream_t>(stream)));
}

int hisparse_attend_workspace(int32_t num_requests, int32_t num_heads, int32_t top_k,
                              int32_t with_weights, int64_t *bytes)
{
    if (!bytes) return HISPARSE_ERR_INVALID_ARG;
    *bytes = 0;
    const int rc = check_attend_sizes(num_requests, num_heads, top_k);
    if (rc != HISPARSE_OK) return rc;
    hs::attend_workspace_bytes(num_requests, num_heads, top_k, with_weights != 0, bytes);
    return HISPARSE_OK;
}

int hisparse_attend(const hisparse_attend_args *p, void *stream)
{
    if (!p) return HISPARSE_ERR_INVALID_ARG;
    const hisparse_attend_args &a = *p;
    const int rc = check_attend_sizes(a.num_requests, a.num_heads, a.top_k);
    if (rc != HISPARSE_OK) return rc;
    if (a.dtype != HISPARSE_BF16 && a.dtype != HISPARSE_F16) return HISPARSE_ERR_INVALID_ARG;
    if (!a.q || !a.rows || !a.slot_ids || !a.out || !a.workspace || a.rows_per_request < 1 ||
        a.ids_stride < a.top_k)
        return HISPARSE_ERR_INVALID_ARG;
    // (the stride of a dimension of one is not used and means nothing)
    if (a.num_requests > 1 && (a.q_request_stride % 8 != 0 || a.out_request_stride % 8 != 0 || a.request_stride % 16 != 0))
        return HISPARSE_ERR_INVALID_ARG;
    if (a.num_heads > 1 && (a.q_head_stride % 8 != 0 || a.out_head_stride % 8 != 0)) return HISPARSE_ERR_INVALID_ARG;
    if ((a.num_requests > 1 && apart(a.out_request_stride) < HISPARSE_ROW4_LATENT) ||
        (a.num_heads > 1 && apart(a.out_head_stride) < HISPARSE_ROW4_LATENT))
        return HISPARSE_ERR_INVALID_ARG;      // heads of out would overlap
    if (a.row_stride < HISPARSE_ROW4_BYTES || a.row_stride % 16 != 0) return HISPARSE_ERR_INVALID_ARG;
    if (a.resident_count < 0 || (a.resident_count > 0 && !a.resident_rows)) return HISPARSE_ERR_INVALID_ARG;
    if (a.resident_count > 0 && (a.resident_stride < HISPARSE_ROW4_BYTES || a.resident_stride % 16 != 0))
        return HISPARSE_ERR_INVALID_ARG;
    if (a.weights && (!a.positions || a.weights_tokens < 0 || a.weights_stride < a.weights_tokens ||
                      a.positions_stride < a.top_k))
        return HISPARSE_ERR_INVALID_ARG;
    if (!aligned16(a.q) || !aligned16(a.rows) || !aligned16(a.resident_rows) || !aligned16(a.out) ||
        !aligned16(a.workspace))
        return HISPARSE_ERR_ALIGNMENT;
    if (a.workspace_bytes < 16) return HISPARSE_ERR_CAPACITY;
    hs::AttendLaunch l;
    l.R = a.num_requests;
    l.H = a.num_heads;
    l.k = a.top_k;
    l.D = a.rows_per_request;
    l.dtype = a.dtype;
    l.q = static_cast<const uint8_t *>(a.q);
    l.q_rs = a.q_request_stride * 2;
    l.q_hs = a.q_head_stride * 2;
    l.rows = static_cast<const uint8_t *>(a.rows);
    l.row_stride = a.row_stride;
    l.req_stride = a.request_stride;
    l.res = static_cast<const uint8_t *>(a.resident_rows);
    l.res_stride = a.resident_stride;
    l.res_count = a.resident_count;
    l.ids = a.slot_ids;
    l.ids_stride = a.ids_stride;
    l.scale = a.scale;
    l.out = static_cast<uint8_t *>(a.out);
    l.out_rs = a.out_request_stride * 2;
    l.out_hs = a.out_head_stride * 2;
    l.lse = a.lse;
    l.weights = a.weights;
    l.weights_stride = a.weights_stride;
    l.weights_tokens = a.weights_tokens;
    l.positions = a.positions;
    l.positions_stride = a.positions_stride;
    l.status = a.status;
    l.workspace = static_cast<uint8_t *>(a.workspace);
    bool too_small = false;
    const cudaError_t e = hs::launch_attend(l, a.workspace_bytes, &too_small, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess && too_small ? HISPARSE_ERR_CAPACITY : cuda_status(e);
}

int hisparse_evict_select(int32_t num_requests, int32_t rows_per_request, const float *weights,
                          int64_t weights_stride, int64_t weights_tokens, const int32_t *slot2tok,
                          const int32_t *seq_lens, int32_t keep_recent, int32_t n,
                          const int32_t *want, int32_t *out_slots, int32_t *out_counts, void *stream)
{
    if ((!weights && weights_tokens != 0) || !slot2tok || !seq_lens || !out_slots || !out_counts)
        return HISPARSE_ERR_INVALID_ARG;
    if (num_requests < 1 || rows_per_request < 1 || weights_tokens < 0 ||
        weights_stride < weights_tokens || keep_recent < 0 || n < 1 ||
        n > rows_per_request)
        return HISPARSE_ERR_INVALID_ARG;
    if (rows_per_request > HISPARSE_MAX_DEVICE_BUFFER || num_requests > HISPARSE_MAX_REQUESTS)
        return HISPARSE_ERR_UNSUPPORTED;
    hs::EvictLaunch e = {};
    e.R = num_requests;
    e.D = rows_per_request;
    e.n = n;
    e.weights = weights;
    e.weights_stride = weights_stride;
    e.weights_tokens = weights_tokens;
    e.slot2tok = slot2tok;
    e.seq_lens = seq_lens;
    e.keep_recent = keep_recent;
    e.want = want;
    e.out_slots = out_slots;
    e.out_counts = out_counts;
    return cuda_status(hs::launch_evict(e, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
