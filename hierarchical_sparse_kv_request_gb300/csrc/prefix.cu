// prefix.cu -- attention of a whole batch over a prefix that its requests share
// (include/hisparse_pages.h, hisparse_attend_prefix).
//
// The mathematics.  With s = scale * log2(e) * (q . row), a running maximum m, l =
// sum 2^(s - m) and O = sum 2^(s - m) * latent over the rows; a part comes in as
// one more row of score part_lse * log2(e) and value part.  out = O / l, lse = (m +
// log2 l) ln 2.
//
// A warp a head of a request: a lane has 18 values of the query and 16 of O.
#include "pages.cuh"

namespace hs {
namespace {

constexpr int PX_NT = 128;

template <int DT, int ROW>
__global__ void __launch_bounds__(PX_NT) prefix_kernel(const __grid_constant__ PrefixLaunch a)
{
    after_launch_before();
    const int lane = threadIdx.x & 31;
    const int64_t n = (int64_t)blockIdx.x * (PX_NT / 32) + (threadIdx.x >> 5);
    if (n >= (int64_t)a.R * a.H) return;
    const int r = (int)(n / a.H), h = (int)(n % a.H);
    const uint8_t *src = a.q + r * a.q_rs + h * a.q_hs;
    auto expand = [](uint4 v, float *x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 p = pair_to_float<DT>(w[j]);
            x[2 * j] = p.x;
            x[2 * j + 1] = p.y;
        }
    };
    float q[16], o[16] = {};
    expand(ld_dev_v4(src + lane * 16), q);
    expand(ld_dev_v4(src + 512 + lane * 16), q + 8);
    const float2 q_rope = pair_to_float<DT>(*reinterpret_cast<const uint32_t *>(src + 1024 + lane * 4));
    float m = -INFINITY, l = 0.0f;
    bool bad = false;
    for (int t = 0; t < a.len; ++t) {
        const int32_t page = a.table[t / a.bs];
        const int64_t row = (int64_t)page * a.bs + t % a.bs;
        if (page < 0 || row >= a.num_rows) {
            bad |= page != -1;
            continue;
        }
        const uint8_t *p = a.rows + row * a.row_stride;
        float x[16];
        expand(load_latent8<DT, ROW>(p, lane), x);
        expand(load_latent8<DT, ROW>(p, lane + 32), x + 8);
        const float2 rope = pair_to_float<DT>(*reinterpret_cast<const uint32_t *>(p + rope_at(ROW) + lane * 4));
        float s = q_rope.x * rope.x + q_rope.y * rope.y;
#pragma unroll
        for (int j = 0; j < 16; ++j) s = fmaf(q[j], x[j], s);
#pragma unroll
        for (int d = 1; d < 32; d *= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= a.scale * kLog2e;
        const float top = fmaxf(m, s), f = top == -INFINITY ? 1.0f : exp2f(m - top), w = top == -INFINITY ? 0.0f : exp2f(s - top);
        m = top;
        l = l * f + w;
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = o[j] * f + w * x[j];
    }
    if (a.part) {
        const float s = a.part_lse[n] * kLog2e;
        const uint8_t *p = a.part + r * a.part_rs + h * a.part_hs;
        float x[16];
        expand(ld_dev_v4(p + lane * 16), x);
        expand(ld_dev_v4(p + 512 + lane * 16), x + 8);
        const float top = fmaxf(m, s), f = top == -INFINITY ? 1.0f : exp2f(m - top), w = top == -INFINITY ? 0.0f : exp2f(s - top);
        m = top;
        l = l * f + w;
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = o[j] * f + w * x[j];
    }
    __syncwarp();
    const float f = l == 0.0f ? 0.0f : 1.0f / l;
    uint8_t *dst = a.out + r * a.out_rs + h * a.out_hs;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = floats_to_pair<DT>(o[8 * half + 2 * j] * f, o[8 * half + 2 * j + 1] * f);
        st_v4(dst + half * 512 + lane * 16, make_uint4(w[0], w[1], w[2], w[3]));
    }
    if (lane == 0) {
        if (a.lse) a.lse[n] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
        if (bad && a.status) record_status(a.status, r, kStatusBadResident);
    }
}

template <int DT>
cudaError_t launch(const PrefixLaunch &a, cudaStream_t s)
{
    const dim3 grid((unsigned)(((int64_t)a.R * a.H + PX_NT / 32 - 1) / (PX_NT / 32)));
    auto kernel = a.row_bytes == kRow4 ? prefix_kernel<DT, kRow4> : a.row_bytes == kRow8 ? prefix_kernel<DT, kRow8> : prefix_kernel<DT, kRow16>;
    return launch_behind(kernel, grid, PX_NT, 0, 1, s, a);
}

}  // namespace

void attend_prefix_workspace_bytes(int32_t R, int32_t H, int32_t len, int64_t *bytes) { *bytes = 16; }

cudaError_t launch_attend_prefix(const PrefixLaunch &a, cudaStream_t s)
{
    return a.dtype == kBf16 ? launch<kBf16>(a, s) : launch<kF16>(a, s);
}

}  // namespace hs
