// pages.cuh -- launchers of the resident pages' kernels (include/hisparse_pages.h)
// and the rows' formats on the device.
#pragma once

#include "attend.cuh"

namespace hs {

constexpr int kRow4 = 416, kRow8 = 656, kRow16 = 1152;
constexpr int kRow8ScaleAt = 512;      // 4 floats behind the codes

// Where a row's rope values begin.
__host__ __device__ constexpr int rope_at(int row_bytes) { return row_bytes - kRope * 2; }

// Latent values 8 u to 8 u + 7 of a row, each rounded to DT once.
// Its bytes (zeros stand for zeros),
template <int ROW>
struct Latent8 {
    uint4 whole;         // of a 16-bit row
    uint2 codes;
    float scale;         // of an 8-bit row
    uint32_t scale4;     // of a 4-bit one
    __device__ __forceinline__ Latent8() : whole(make_uint4(0, 0, 0, 0)), codes(make_uint2(0, 0)), scale(0.0f), scale4(0) {}
    __device__ __forceinline__ void fetch(const uint8_t *row, int u)
    {
        if (ROW == kRow16) {
            whole = ld_dev_v4(row + u * 16);
        } else if (ROW == kRow8) {
            codes = *reinterpret_cast<const uint2 *>(row + u * 8);
            scale = *reinterpret_cast<const float *>(row + kRow8ScaleAt + (u >> 4) * 4);
        } else {
            codes.x = *reinterpret_cast<const uint32_t *>(row + u * 4);
            scale4 = row[kScaleAt + (u >> 1)];
        }
    }
};

// and its values.
template <int DT, int ROW>
__device__ __forceinline__ uint4 latent8(const Latent8<ROW> &x)
{
    if (ROW == kRow16) return x.whole;
    uint32_t h[4];
    if (ROW == kRow4) {
        codes_to_half2(x.codes.x, h);
        const __half2 scale = scale_half2(x.scale4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {      // (exact in f16: see decode8)
            const __half2 p = __hmul2(*reinterpret_cast<__half2 *>(&h[j]), scale);
            const float2 f = __half22float2(p);
            h[j] = DT == kBf16 ? floats_to_pair<DT>(f.x, f.y) : *reinterpret_cast<const uint32_t *>(&p);
        }
    } else {
        const uint32_t w[4] = {x.codes.x & 0xFFFFu, x.codes.x >> 16, x.codes.y & 0xFFFFu, x.codes.y >> 16};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t p;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(p) : "h"((uint16_t)w[j]));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&p));
            h[j] = floats_to_pair<DT>(f.x * x.scale, f.y * x.scale);
        }
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}

template <int DT, int ROW>
__device__ __forceinline__ uint4 load_latent8(const uint8_t *row, int u)
{
    Latent8<ROW> x;
    x.fetch(row, u);
    return latent8<DT, ROW>(x);
}

// Arguments of the block table kernels (see hisparse_page_tables_args).
struct TablesLaunch {
    int32_t R, W, bs, shared_count;
    const int32_t *lens;
    int32_t *tables;
    int64_t tables_stride;
    int32_t *held;
    int32_t *free_list;
    int32_t free_capacity;
    int32_t *free_count;
    const int32_t *shared;
    const int32_t *new_tokens;
    int32_t *offsets, *slots, *positions;
    int32_t tokens;
    int32_t *status;
};
cudaError_t launch_page_tables(const TablesLaunch &a, cudaStream_t s);

// Arguments of the row kernels; strides in bytes.
struct RowsLaunch {
    uint8_t *values;
    int64_t value_stride, n;
    int32_t dtype;
    const uint8_t *weight;       // null: no norm
    float eps;
    uint8_t *rows;
    int64_t row_stride, num_rows;
    int32_t row_bytes;
    const int32_t *slots;        // null: slot i is i
};
cudaError_t launch_norm_rows(const RowsLaunch &a, cudaStream_t s);
cudaError_t launch_gather_rows(const RowsLaunch &a, cudaStream_t s);

// Arguments of the prefix attention's kernels (see hisparse_attend_prefix_args).
struct PrefixLaunch {
    int32_t R, H, dtype, row_bytes;
    const uint8_t *q;            // strides in bytes
    int64_t q_rs, q_hs;
    const uint8_t *rows;
    int64_t row_stride, num_rows;
    const int32_t *table;
    int32_t bs, len;
    float scale;
    const uint8_t *part;
    int64_t part_rs, part_hs;
    const float *part_lse;
    uint8_t *out;
    int64_t out_rs, out_hs;
    float *lse;
    int32_t *status;
    uint8_t *workspace;
};
void attend_prefix_workspace_bytes(int32_t R, int32_t H, int32_t len, int64_t *bytes);
cudaError_t launch_attend_prefix(const PrefixLaunch &a, cudaStream_t s);

}  // namespace hs
