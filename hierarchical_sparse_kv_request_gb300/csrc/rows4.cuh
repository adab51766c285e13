// rows4.cuh -- the 4-bit row format (include/hisparse_rows4.h) on the device,
// and the launchers of the kernels that work on such rows.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "hs_common.cuh"

namespace hs {

constexpr int kLatent = 512, kRope = 64, kRowValues = kLatent + kRope;
constexpr int kScaleAt = 256, kRopeAt = 288;
constexpr int kBf16 = 0, kF16 = 1;
constexpr int kStatusAttendTimeout = 9;

// 8 codes (one 32-bit word of a row) as four f16 pairs in value order:
// pair j holds codes 2j and 2j + 1.
__device__ __forceinline__ void codes_to_half2(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n"
        ".reg .b8 b0, b1, b2, b3;\n"
        "mov.b32 {b0, b1, b2, b3}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n"
        "}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// The value of an e4m3 byte as f16, in both halves (exact).
__device__ __forceinline__ __half2 scale_half2(uint32_t e4m3)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(e4m3 | (e4m3 << 8))));
    return *reinterpret_cast<__half2 *>(&h);
}

cudaError_t launch_pack_rows(const void *values, int64_t value_stride, int32_t dtype, int64_t n,
                             void *rows, int64_t row_stride, cudaStream_t s);
cudaError_t launch_unpack_rows(const void *rows, int64_t row_stride, int64_t n, void *values,
                               int64_t value_stride, int32_t dtype, cudaStream_t s);

// Arguments of the attention kernels (see hisparse_attend_args).
struct AttendLaunch {
    int32_t R, H, k, D, dtype;
    const uint8_t *q;            // strides in bytes
    int64_t q_rs, q_hs;
    const uint8_t *rows;
    int64_t row_stride, req_stride;
    const uint8_t *res;
    int64_t res_stride, res_count;
    const int32_t *ids;
    int64_t ids_stride;
    float scale;
    uint8_t *out;                // strides in bytes
    int64_t out_rs, out_hs;
    float *lse;
    float *weights;
    int64_t weights_stride, weights_tokens;
    const int32_t *positions;
    int64_t positions_stride;
    int32_t *status;
    uint8_t *workspace;
};
// Workspace of a call.
void attend_workspace_bytes(int32_t R, int32_t H, int32_t k, bool weights, int64_t *bytes);
// Launches nothing and sets *too_small if the workspace is too small.  The first
// call on a device also loads the attention kernels and finds how many of their
// clusters it holds.
cudaError_t launch_attend(const AttendLaunch &a, int64_t workspace_bytes, bool *too_small, cudaStream_t s);

// A launch that may be set up while the stream's last kernel ends; the kernel
// reads and writes nothing before after_launch_before(), which waits for that
// one's completion.  (70,001 rows packed and unpacked, call after call: 33.2
// against 38.1 us.)  One exception: weights_kernel reads its ids and positions
// ahead of its wait.  It always follows attend_kernel, which lets it start only
// once every CTA has waited for the launch before; whatever wrote those two
// arrays is complete by then, and attend_kernel does not write them.  cluster:
// CTAs along x.
template <class... P, class... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, unsigned cluster, cudaStream_t s,
                          const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

__device__ __forceinline__ void after_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Arguments of the eviction kernel.  With st.tok2slot the chosen slots are
// freed in that hot state (slot2tok is then st.slot2tok); without, slot2tok
// is the caller's.
struct EvictLaunch {
    int32_t R, D, n;
    const float *weights;
    int64_t weights_stride, weights_tokens;
    const int32_t *slot2tok;
    const int32_t *seq_lens;
    int32_t keep_recent;
    const int32_t *want;
    int32_t *out_slots, *out_counts;   // may be null (only with st)
    HotState st;
    const int64_t *host_off;
    uint32_t protect_calls;
};
cudaError_t launch_evict(const EvictLaunch &a, cudaStream_t s);

}  // namespace hs
