// pages.cu -- the C entry points of include/hisparse_pages.h: host checks, then
// the launchers (pages.cuh).
#include "hisparse_pages.h"

#include "pages.cuh"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

uint64_t apart(int64_t stride) { return stride < 0 ? 0u - (uint64_t)stride : (uint64_t)stride; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? HISPARSE_OK : HISPARSE_ERR_CUDA; }

bool known_format(int32_t row_bytes)
{
    return row_bytes == HISPARSE_ROW4_BYTES || row_bytes == HISPARSE_ROW8_BYTES || row_bytes == HISPARSE_ROW16_BYTES;
}

bool known_type(int32_t dtype) { return dtype == HISPARSE_BF16 || dtype == HISPARSE_F16; }

int check_rows(const void *values, int64_t value_stride, int32_t dtype, int64_t n, const void *rows,
               int64_t row_stride, int32_t row_bytes, int64_t num_rows, const int32_t *slots)
{
    if (n < 0 || num_rows < 0 || !known_type(dtype) || !known_format(row_bytes)) return HISPARSE_ERR_INVALID_ARG;
    if (value_stride < HISPARSE_ROW4_VALUES || value_stride % 8 != 0) return HISPARSE_ERR_INVALID_ARG;
    if (row_stride < row_bytes || row_stride % 16 != 0) return HISPARSE_ERR_INVALID_ARG;
    if (n > 0 && (!values || (!rows && num_rows > 0) || (!slots && num_rows < n))) return HISPARSE_ERR_INVALID_ARG;
    if (n > HISPARSE_MAX_PACKED_ROWS) return HISPARSE_ERR_UNSUPPORTED;
    if (!aligned16(values) || !aligned16(rows)) return HISPARSE_ERR_ALIGNMENT;
    return HISPARSE_OK;
}

int check_prefix_sizes(int32_t R, int32_t H, int32_t len)
{
    if (R < 1 || H < 1 || len < 0) return HISPARSE_ERR_INVALID_ARG;
    if (R > HISPARSE_MAX_REQUESTS || H > HISPARSE_MAX_HEADS || len > HISPARSE_MAX_PREFIX) return HISPARSE_ERR_UNSUPPORTED;
    return HISPARSE_OK;
}

// Strides of [R][H][values] (elements); those of a dimension of one are not looked at.
bool good_strides(int32_t R, int32_t H, int64_t request, int64_t head, bool written)
{
    if ((R > 1 && request % 8 != 0) || (H > 1 && head % 8 != 0)) return false;
    return !written || ((R <= 1 || apart(request) >= HISPARSE_ROW4_LATENT) && (H <= 1 || apart(head) >= HISPARSE_ROW4_LATENT));
}

}  // namespace

extern "C" {

int hisparse_page_tables(const hisparse_page_tables_args *p, void *stream)
{
    if (!p) return HISPARSE_ERR_INVALID_ARG;
    const hisparse_page_tables_args &a = *p;
    if (a.num_requests < 1 || a.max_blocks < 1 || a.block_size < 1 || a.free_capacity < 1) return HISPARSE_ERR_INVALID_ARG;
    if (!a.lens || !a.tables || !a.held || !a.free_list || !a.free_count) return HISPARSE_ERR_INVALID_ARG;
    if (a.num_shared < 0 || a.num_shared > a.max_blocks || (a.num_shared > 0 && !a.shared)) return HISPARSE_ERR_INVALID_ARG;
    if (a.num_requests > 1 && a.tables_stride < a.max_blocks) return HISPARSE_ERR_INVALID_ARG;
    if (a.new_tokens && (a.num_tokens < 0 || !a.offsets || (a.num_tokens > 0 && !a.slots))) return HISPARSE_ERR_INVALID_ARG;
    if (a.num_requests > HISPARSE_MAX_REQUESTS || a.max_blocks > HISPARSE_MAX_TABLE_BLOCKS ||
        a.block_size > HISPARSE_RESIDENT_FLAG || (a.new_tokens && a.num_tokens > HISPARSE_RESIDENT_FLAG) ||
        (int64_t)a.num_requests * a.max_blocks > INT32_MAX)
        return HISPARSE_ERR_UNSUPPORTED;
    hs::TablesLaunch l;
    l.R = a.num_requests;
    l.W = a.max_blocks;
    l.bs = a.block_size;
    l.shared_count = a.num_shared;
    l.lens = a.lens;
    l.tables = a.tables;
    l.tables_stride = a.tables_stride;
    l.held = a.held;
    l.free_list = a.free_list;
    l.free_capacity = a.free_capacity;
    l.free_count = a.free_count;
    l.shared = a.shared;
    l.new_tokens = a.new_tokens;
    l.offsets = a.offsets;
    l.slots = a.slots;
    l.positions = a.positions;
    l.tokens = a.new_tokens ? a.num_tokens : 0;
    l.status = a.status;
    return cuda_status(hs::launch_page_tables(l, static_cast<cudaStream_t>(stream)));
}

int hisparse_norm_rows(const void *values, int64_t value_stride, int32_t dtype, int64_t n,
                       const void *weight, float eps, void *rows, int64_t row_stride,
                       int32_t row_bytes, int64_t num_rows, const int32_t *slots, void *stream)
{
    if (!(eps >= 0.0f)) return HISPARSE_ERR_INVALID_ARG;
    const int rc = check_rows(values, value_stride, dtype, n, rows, row_stride, row_bytes, num_rows, slots);
    if (rc != HISPARSE_OK) return rc;
    if (!aligned16(weight)) return HISPARSE_ERR_ALIGNMENT;
    if (n == 0 || num_rows == 0) return HISPARSE_OK;
    const hs::RowsLaunch l = {static_cast<uint8_t *>(const_cast<void *>(values)), value_stride * 2, n, dtype,
                              static_cast<const uint8_t *>(weight), eps, static_cast<uint8_t *>(rows), row_stride,
                              num_rows, row_bytes, slots};
    return cuda_status(hs::launch_norm_rows(l, static_cast<cudaStream_t>(stream)));
}

int hisparse_gather_rows(const void *rows, int64_t row_stride, int32_t row_bytes, int64_t num_rows,
                         const int32_t *slots, int64_t n, void *values, int64_t value_stride,
                         int32_t dtype, void *stream)
{
    const int rc = check_rows(values, value_stride, dtype, n, rows, row_stride, row_bytes, num_rows, slots);
    if (rc != HISPARSE_OK || n == 0 || num_rows == 0) return rc;
    const hs::RowsLaunch l = {static_cast<uint8_t *>(values), value_stride * 2, n, dtype, nullptr, 0.0f,
                              static_cast<uint8_t *>(const_cast<void *>(rows)), row_stride, num_rows, row_bytes, slots};
    return cuda_status(hs::launch_gather_rows(l, static_cast<cudaStream_t>(stream)));
}

int hisparse_attend_prefix_workspace(int32_t num_requests, int32_t num_heads, int32_t prefix_len, int64_t *bytes)
{
    if (!bytes) return HISPARSE_ERR_INVALID_ARG;
    *bytes = 0;
    const int rc = check_prefix_sizes(num_requests, num_heads, prefix_len);
    if (rc == HISPARSE_OK) hs::attend_prefix_workspace_bytes(num_requests, num_heads, prefix_len, bytes);
    return rc;
}

int hisparse_attend_prefix(const hisparse_attend_prefix_args *p, void *stream)
{
    if (!p) return HISPARSE_ERR_INVALID_ARG;
    const hisparse_attend_prefix_args &a = *p;
    const int rc = check_prefix_sizes(a.num_requests, a.num_heads, a.prefix_len);
    if (rc != HISPARSE_OK) return rc;
    if (!known_type(a.dtype) || !known_format(a.row_bytes) || !a.q || !a.out || !a.workspace || a.block_size < 1 ||
        a.num_rows < 0 || (a.num_rows > 0 && !a.rows) || (a.prefix_len > 0 && !a.table) || !a.part != !a.part_lse)
        return HISPARSE_ERR_INVALID_ARG;
    if (a.row_stride < a.row_bytes || a.row_stride % 16 != 0) return HISPARSE_ERR_INVALID_ARG;
    if (!good_strides(a.num_requests, a.num_heads, a.q_request_stride, a.q_head_stride, false) ||
        !good_strides(a.num_requests, a.num_heads, a.out_request_stride, a.out_head_stride, true) ||
        (a.part && !good_strides(a.num_requests, a.num_heads, a.part_request_stride, a.part_head_stride, false)))
        return HISPARSE_ERR_INVALID_ARG;
    if (!aligned16(a.q) || !aligned16(a.rows) || !aligned16(a.part) || !aligned16(a.out) || !aligned16(a.workspace))
        return HISPARSE_ERR_ALIGNMENT;
    int64_t bytes;
    hs::attend_prefix_workspace_bytes(a.num_requests, a.num_heads, a.prefix_len, &bytes);
    if (a.workspace_bytes < bytes) return HISPARSE_ERR_CAPACITY;
    hs::PrefixLaunch l;
    l.R = a.num_requests;
    l.H = a.num_heads;
    l.dtype = a.dtype;
    l.row_bytes = a.row_bytes;
    l.q = static_cast<const uint8_t *>(a.q);
    l.q_rs = a.q_request_stride * 2;
    l.q_hs = a.q_head_stride * 2;
    l.rows = static_cast<const uint8_t *>(a.rows);
    l.row_stride = a.row_stride;
    l.num_rows = a.num_rows;
    l.table = a.table;
    l.bs = a.block_size;
    l.len = a.prefix_len;
    l.scale = a.scale;
    l.part = static_cast<const uint8_t *>(a.part);
    l.part_rs = a.part_request_stride * 2;
    l.part_hs = a.part_head_stride * 2;
    l.part_lse = a.part_lse;
    l.out = static_cast<uint8_t *>(a.out);
    l.out_rs = a.out_request_stride * 2;
    l.out_hs = a.out_head_stride * 2;
    l.lse = a.lse;
    l.status = a.status;
    l.workspace = static_cast<uint8_t *>(a.workspace);
    return cuda_status(hs::launch_attend_prefix(l, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
