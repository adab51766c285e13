// attend.cu -- sparse attention of one decode step over 4-bit rows named by
// slot ids (include/hisparse_rows4.h, hisparse_attend).
//
// Three launches: scores of every (request, head, row) into the workspace,
// then per (request, head) the softmax and the weighted sum of the latent
// parts, then (with weights) per (request, row) the sum of the heads'
// probabilities.
#include <cfloat>

#include "rows4.cuh"

namespace hs {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Row that an id names, or null (nothing, or an id out of range).
__device__ __forceinline__ const uint8_t *row_of(const AttendLaunch &a, int r, int32_t id, int *bad)
{
    if (id < 0) {
        if (id != -1) *bad = kStatusBadIndex;
        return nullptr;
    }
    if (id & kResidentFlag) {
        const int64_t n = id & (kResidentFlag - 1);
        if (n < a.res_count) return a.res + n * a.res_stride;
        *bad = kStatusBadResident;
        return nullptr;
    }
    if (id < a.D) return a.rows + (int64_t)r * a.req_stride + (int64_t)id * a.row_stride;
    *bad = kStatusBadIndex;
    return nullptr;
}

__device__ __forceinline__ float value16(const uint8_t *p, int i, int dtype)
{
    return dtype == kBf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i])
                          : __half2float(reinterpret_cast<const __half *>(p)[i]);
}

__device__ __forceinline__ float latent_value(const uint8_t *row, int d)
{
    const uint32_t code = (row[d >> 1] >> ((d & 1) * 4)) & 15u;
    uint32_t h[4];
    codes_to_half2(code, h);
    return __half2float(__low2half(*reinterpret_cast<__half2 *>(&h[0]))) *
           __low2float(scale_half2(row[kScaleAt + (d >> 4)]));
}

constexpr int SC_NT = 256, SC_ROWS = 16;

// Scores in base-2 units: scores[(r * H + h) * k + i].
__global__ void __launch_bounds__(SC_NT) scores_kernel(AttendLaunch a, float *scores)
{
    __shared__ float x[SC_ROWS][kRowValues + 1];
    __shared__ int valid[SC_ROWS];
    const int r = blockIdx.y, i0 = blockIdx.x * SC_ROWS;
    const int nr = min(SC_ROWS, a.k - i0);
    for (int j = threadIdx.x; j < nr; j += SC_NT) {
        int bad = 0;
        const uint8_t *row = row_of(a, r, a.ids[(int64_t)r * a.ids_stride + i0 + j], &bad);
        if (bad && a.status) record_status(a.status, r, bad);
        valid[j] = row != nullptr;
    }
    for (int e = threadIdx.x; e < nr * kRowValues; e += SC_NT) {
        const int j = e / kRowValues, d = e % kRowValues;
        int bad = 0;
        const uint8_t *row = row_of(a, r, a.ids[(int64_t)r * a.ids_stride + i0 + j], &bad);
        x[j][d] = !row ? 0.0f : d < kLatent ? latent_value(row, d) : value16(row + kRopeAt, d - kLatent, a.dtype);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.H * nr; e += SC_NT) {
        const int h = e / nr, j = e % nr;
        const uint8_t *q = a.q + r * a.q_rs + h * a.q_hs;
        float s = 0.0f;
        for (int d = 0; d < kRowValues; ++d) s = fmaf(value16(q, d, a.dtype), x[j][d], s);
        scores[((int64_t)r * a.H + h) * a.k + i0 + j] = valid[j] ? s * (a.scale * kLog2e) : -INFINITY;
    }
}

constexpr int SM_NT = 256;

__global__ void __launch_bounds__(SM_NT) softmax_kernel(AttendLaunch a, const float *scores, float *lse2)
{
    __shared__ float red[SM_NT / 32];
    __shared__ float p[SM_NT];
    const int r = blockIdx.y, h = blockIdx.x, tid = threadIdx.x;
    const float *s = scores + ((int64_t)r * a.H + h) * a.k;
    float top = -INFINITY;
    for (int i = tid; i < a.k; i += SM_NT) top = fmaxf(top, s[i]);
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((tid & 31) == 0) red[tid >> 5] = top;
    __syncthreads();
    for (int w = 0; w < SM_NT / 32; ++w) top = fmaxf(top, red[w]);
    const float ref = top == -INFINITY ? 0.0f : top;
    float total = 0.0f, o0 = 0.0f, o1 = 0.0f;
    for (int i0 = 0; i0 < a.k; i0 += SM_NT) {
        __syncthreads();
        p[tid] = i0 + tid < a.k ? exp2f(s[i0 + tid] - ref) : 0.0f;
        __syncthreads();
        for (int j = 0; j < SM_NT && i0 + j < a.k; ++j) {
            int bad = 0;
            const uint8_t *row = row_of(a, r, a.ids[(int64_t)r * a.ids_stride + i0 + j], &bad);
            if (!row) continue;
            total += p[j];
            o0 = fmaf(p[j], latent_value(row, 2 * tid), o0);
            o1 = fmaf(p[j], latent_value(row, 2 * tid + 1), o1);
        }
    }
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    uint8_t *out = a.out + r * a.out_rs + h * a.out_hs;
    if (a.dtype == kBf16)
        reinterpret_cast<__nv_bfloat162 *>(out)[tid] = __floats2bfloat162_rn(o0 * inv, o1 * inv);
    else
        reinterpret_cast<__half2 *>(out)[tid] = __floats2half2_rn(o0 * inv, o1 * inv);
    if (tid == 0) {
        const float l2 = total == 0.0f ? -INFINITY : ref + log2f(total);
        if (a.lse) a.lse[(int64_t)r * a.H + h] = l2 * kLn2;
        lse2[(int64_t)r * a.H + h] = l2;
    }
}

constexpr int WT_NT = 128;

__global__ void __launch_bounds__(WT_NT) weights_kernel(AttendLaunch a, const float *scores, const float *lse2)
{
    const int r = blockIdx.y, i = blockIdx.x * WT_NT + threadIdx.x;
    if (i >= a.k) return;
    int bad = 0;
    if (!row_of(a, r, a.ids[(int64_t)r * a.ids_stride + i], &bad)) return;
    const int64_t pos = a.positions[(int64_t)r * a.positions_stride + i];
    if (pos < 0 || pos >= a.weights_tokens) {
        if (a.status) record_status(a.status, r, kStatusBadPosition);
        return;
    }
    float w = 0.0f;
    for (int h = 0; h < a.H; ++h) {
        const int64_t rh = (int64_t)r * a.H + h;
        w += exp2f(scores[rh * a.k + i] - lse2[rh]);
    }
    atomicAdd(a.weights + (int64_t)r * a.weights_stride + pos, w);
}

}  // namespace

int64_t attend_workspace_bytes(int32_t R, int32_t H, int32_t k, bool weights, int num_sms)
{
    (void)weights;
    (void)num_sms;
    return ((int64_t)R * H * k + (int64_t)R * H) * 4;
}

cudaError_t launch_attend(const AttendLaunch &a, int num_sms, cudaStream_t s)
{
    (void)num_sms;
    float *scores = reinterpret_cast<float *>(a.workspace);
    float *lse2 = scores + (int64_t)a.R * a.H * a.k;
    scores_kernel<<<dim3((a.k + SC_ROWS - 1) / SC_ROWS, a.R), SC_NT, 0, s>>>(a, scores);
    softmax_kernel<<<dim3(a.H, a.R), SM_NT, 0, s>>>(a, scores, lse2);
    if (a.weights) weights_kernel<<<dim3((a.k + WT_NT - 1) / WT_NT, a.R), WT_NT, 0, s>>>(a, scores, lse2);
    return cudaGetLastError();
}

}  // namespace hs
