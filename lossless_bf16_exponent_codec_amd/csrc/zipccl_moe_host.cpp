// Host layer of the mixture-of-experts operators: argument checks and launches.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "zipccl.h"
#include "zipccl_moe_internal.h"

using namespace zc;

namespace {

static_assert(ZIPCCL_MAX_EXPERTS == kMaxExperts && ZIPCCL_MAX_TOP_K == kMaxTopK && ZIPCCL_ROW_PAD == kQuantPad &&
              ZIPCCL_MOE_SORT_WORKSPACE_BYTES == kSortWorkspace, "the header states the limits");

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

zipccl_status hip_status(hipError_t e) { return e == hipSuccess ? ZIPCCL_OK : ZIPCCL_ERR_HIP; }

constexpr uint64_t kMaxCount = 1ull << 31;     // choices, rows: 32-bit signed indices
constexpr uint64_t kMaxRowLen = 1ull << 28;
constexpr uint64_t kMaxSumLen = 131071;        // 128 * 128 * this stays below 2^31
constexpr uint64_t kMaxTiles = 1ull << 24;     // workgroups of one launch
constexpr uint64_t kMaxByteStride = 1ull << 24;  // of the product's rows: 255 of them stay within 32 bits
constexpr uint64_t kMaxStride = 1ull << 40;    // values
constexpr uint64_t kMaxSpan = 1ull << 60;      // rows * stride: 8 bytes times it stay within 64 bits

bool is_dtype(int d) { return d == ZIPCCL_BF16 || d == ZIPCCL_FP32; }
// Whether a row stride is too large: by itself, or for the address of the last row.
bool too_far(uint64_t rows, uint64_t stride) { return stride >= kMaxStride || (rows > 1 && stride > kMaxSpan / rows); }
uintptr_t value_bytes(int dtype) { return dtype == ZIPCCL_FP32 ? 4 : 2; }

// A matrix of `rows` rows of row_len values at a row stride.
zipccl_status check_rows(const void* p, uint64_t rows, uint64_t row_len, uint64_t stride, int dtype)
{
    if (rows > 0 && !p) return ZIPCCL_ERR_INVALID;
    if (rows > 1 && stride < row_len) return ZIPCCL_ERR_INVALID;
    if (too_far(rows, stride)) return ZIPCCL_ERR_SIZE;
    if (p && !aligned(p, value_bytes(dtype))) return ZIPCCL_ERR_ALIGN;
    return ZIPCCL_OK;
}

// The token side that every operator with slots has.
zipccl_status check_slots(const int32_t* slots, uint64_t tokens, int top_k, uint64_t nrows, uint64_t row_len,
                          const uint32_t* status)
{
    if (top_k < 1 || top_k > kMaxTopK || row_len < 1) return ZIPCCL_ERR_INVALID;
    if (tokens >= kMaxCount || tokens * uint64_t(top_k) >= kMaxCount || nrows >= kMaxCount || row_len > kMaxRowLen)
        return ZIPCCL_ERR_SIZE;
    if (tokens > 0 && !slots) return ZIPCCL_ERR_INVALID;
    if (!aligned(slots, 4) || (status && !aligned(status, 4))) return ZIPCCL_ERR_ALIGN;
    return ZIPCCL_OK;
}

// n choices split over the sort's workgroups, in groups of 64 per wave: one workgroup (one
// launch) up to 2048 choices (5.1 us at 2048 over 256 experts, 6.7 as two launches; at 4096
// 7.6 and 7.2), else the fewest groups that leave at most 128 workgroups (131072 choices
// over 256 experts: 9.0 us, as at 64 workgroups, 12.6 at 32; 524288 over 64: 12.2 at 128, 17
// at 64, 26 at 32), and past 16 groups as many workgroups as the workspace has counts for.
void split_choices(SortArgs& a)
{
    constexpr uint32_t kOneBlock = 2 * kSortThreads, kBlocks = 128;
    uint64_t groups = 1;
    const uint64_t most = a.n <= kOneBlock ? 1 : kBlocks;
    while (groups < 16 && (a.n + groups * kSortThreads - 1) / (groups * kSortThreads) > most) groups *= 2;
    const uint64_t even = (a.n + uint64_t(kSortMaxBlocks) * kSortThreads - 1) / (uint64_t(kSortMaxBlocks) * kSortThreads);
    if (groups < even) groups = even;
    a.per_block = uint32_t(groups * kSortThreads);
    a.blocks = uint32_t((a.n + uint64_t(a.per_block) - 1) / a.per_block);
    if (a.blocks == 0) a.blocks = 1;
}

}  // namespace

extern "C" {

zipccl_status zipccl_moe_sort(const void* experts, int id_bytes, uint64_t stride, uint64_t tokens, int top_k,
                              int num_experts, int32_t* offsets, int32_t* rows, int32_t* slots, void* workspace,
                              uint64_t workspace_bytes, uint32_t* status, void* stream)
{
    if ((id_bytes != 4 && id_bytes != 8) || top_k < 1 || top_k > kMaxTopK || num_experts < 1 ||
        num_experts > kMaxExperts || !offsets || !workspace)
        return ZIPCCL_ERR_INVALID;
    if (tokens >= kMaxCount || tokens * uint64_t(top_k) >= kMaxCount || too_far(tokens, stride) ||
        workspace_bytes < kSortWorkspace)
        return ZIPCCL_ERR_SIZE;
    if (tokens > 0 && (!experts || !rows || !slots)) return ZIPCCL_ERR_INVALID;
    if (tokens > 1 && stride < uint64_t(top_k)) return ZIPCCL_ERR_INVALID;
    if (!aligned(experts, uintptr_t(id_bytes)) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(slots, 4) ||
        !aligned(workspace, 256) || (status && !aligned(status, 4)))
        return ZIPCCL_ERR_ALIGN;
    SortArgs a{};
    a.ids = experts;
    a.offsets = offsets;
    a.rows = rows;
    a.slots = slots;
    a.hist = static_cast<uint32_t*>(workspace);
    a.status = status;
    a.stride = stride;
    a.n = uint32_t(tokens * uint64_t(top_k));
    a.top_k = uint32_t(top_k);
    a.experts = uint32_t(num_experts);
    a.wide_ids = id_bytes == 8;
    split_choices(a);
    return hip_status(launch_moe_sort(a, static_cast<hipStream_t>(stream)));
}

zipccl_status zipccl_moe_dispatch(const void* x, uint64_t x_stride, const int32_t* slots, uint64_t tokens, int top_k,
                                  uint64_t row_len, int dtype, void* y, uint64_t y_rows, uint64_t y_stride,
                                  uint32_t* status, void* stream)
{
    if (!is_dtype(dtype)) return ZIPCCL_ERR_INVALID;
    if (zipccl_status r = check_slots(slots, tokens, top_k, y_rows, row_len, status)) return r;
    if (zipccl_status r = check_rows(x, tokens, row_len, x_stride, dtype)) return r;
    if (zipccl_status r = check_rows(y, y_rows, row_len, y_stride, dtype)) return r;
    if (tokens == 0) return ZIPCCL_OK;
    RowsArgs a{};
    a.src = static_cast<const uint8_t*>(x);
    a.dst = static_cast<uint8_t*>(y);
    a.slots = slots;
    a.status = status;
    a.src_stride = x_stride * value_bytes(dtype);
    a.dst_stride = y_stride * value_bytes(dtype);
    a.tokens = tokens;
    a.nrows = uint32_t(y_rows);
    a.row_len = uint32_t(row_len);
    a.top_k = uint32_t(top_k);
    a.fp32 = dtype == ZIPCCL_FP32;
    return hip_status(launch_moe_dispatch(a, static_cast<hipStream_t>(stream)));
}

zipccl_status zipccl_moe_combine(const void* y, uint64_t y_rows, uint64_t y_stride, const int32_t* slots,
                                 const float* weights, uint64_t tokens, int top_k, uint64_t row_len, int dtype,
                                 void* out, uint64_t out_stride, uint32_t* status, void* stream)
{
    if (!is_dtype(dtype)) return ZIPCCL_ERR_INVALID;
    if (zipccl_status r = check_slots(slots, tokens, top_k, y_rows, row_len, status)) return r;
    if (zipccl_status r = check_rows(y, y_rows, row_len, y_stride, dtype)) return r;
    if (zipccl_status r = check_rows(out, tokens, row_len, out_stride, dtype)) return r;
    if (!aligned(weights, 4)) return ZIPCCL_ERR_ALIGN;
    if (tokens == 0) return ZIPCCL_OK;
    RowsArgs a{};
    a.src = static_cast<const uint8_t*>(y);
    a.dst = static_cast<uint8_t*>(out);
    a.slots = slots;
    a.weights = weights;
    a.status = status;
    a.src_stride = y_stride * value_bytes(dtype);
    a.dst_stride = out_stride * value_bytes(dtype);
    a.tokens = tokens;
    a.nrows = uint32_t(y_rows);
    a.row_len = uint32_t(row_len);
    a.top_k = uint32_t(top_k);
    a.fp32 = dtype == ZIPCCL_FP32;
    return hip_status(launch_moe_combine(a, static_cast<hipStream_t>(stream)));
}

zipccl_status zipccl_moe_dispatch_backward(const void* dy, uint64_t dy_rows, uint64_t dy_stride, const int32_t* slots,
                                           uint64_t tokens, int top_k, uint64_t row_len, int dtype, void* dx,
                                           uint64_t dx_stride, uint32_t* status, void* stream)
{
    return zipccl_moe_combine(dy, dy_rows, dy_stride, slots, nullptr, tokens, top_k, row_len, dtype, dx, dx_stride,
                              status, stream);
}

zipccl_status zipccl_moe_combine_backward(const void* dout, uint64_t dout_stride, const void* y, uint64_t y_rows,
                                          uint64_t y_stride, const int32_t* slots, const float* weights,
                                          uint64_t tokens, int top_k, uint64_t row_len, int dtype, void* dy,
                                          uint64_t dy_stride, float* dweights, uint32_t* status, void* stream)
{
    if (!is_dtype(dtype)) return ZIPCCL_ERR_INVALID;
    if (zipccl_status r = check_slots(slots, tokens, top_k, y_rows, row_len, status)) return r;
    if (zipccl_status r = check_rows(dout, tokens, row_len, dout_stride, dtype)) return r;
    if (zipccl_status r = check_rows(y, y_rows, row_len, y_stride, dtype)) return r;
    if (zipccl_status r = check_rows(dy, y_rows, row_len, dy_stride, dtype)) return r;
    if (tokens > 0 && (!weights || !dweights)) return ZIPCCL_ERR_INVALID;
    if (!aligned(weights, 4) || !aligned(dweights, 4)) return ZIPCCL_ERR_ALIGN;
    if (tokens == 0) return ZIPCCL_OK;
    RowsArgs a{};
    a.src = static_cast<const uint8_t*>(y);
    a.grad = static_cast<const uint8_t*>(dout);
    a.dst = static_cast<uint8_t*>(dy);
    a.slots = slots;
    a.weights = weights;
    a.grad_weights = dweights;
    a.status = status;
    a.src_stride = y_stride * value_bytes(dtype);
    a.grad_stride = dout_stride * value_bytes(dtype);
    a.dst_stride = dy_stride * value_bytes(dtype);
    a.tokens = tokens;
    a.nrows = uint32_t(y_rows);
    a.row_len = uint32_t(row_len);
    a.top_k = uint32_t(top_k);
    a.fp32 = dtype == ZIPCCL_FP32;
    return hip_status(launch_moe_combine_backward(a, static_cast<hipStream_t>(stream)));
}

zipccl_status zipccl_quantize_rows(const void* x, uint64_t x_stride, uint64_t tokens, uint64_t row_len,
                                   const int32_t* slots, int top_k, void* q, uint64_t q_rows, uint64_t q_stride,
                                   float* scales, uint32_t* status, void* stream)
{
    if (slots) {
        if (zipccl_status r = check_slots(slots, tokens, top_k, q_rows, row_len, status)) return r;
    } else {
        if (row_len < 1 || q_rows < tokens) return ZIPCCL_ERR_INVALID;
        if (q_rows >= kMaxCount || row_len > kMaxRowLen) return ZIPCCL_ERR_SIZE;
        if (status && !aligned(status, 4)) return ZIPCCL_ERR_ALIGN;
    }
    if (zipccl_status r = check_rows(x, tokens, row_len, x_stride, ZIPCCL_BF16)) return r;
    if (q_rows > 0 && (!q || !scales)) return ZIPCCL_ERR_INVALID;
    if (q_stride < row_len) return ZIPCCL_ERR_INVALID;
    if (too_far(q_rows, q_stride)) return ZIPCCL_ERR_SIZE;
    if (q_stride % kQuantPad != 0 || !aligned(q, 16) || !aligned(scales, 4)) return ZIPCCL_ERR_ALIGN;
    if (tokens == 0) return ZIPCCL_OK;
    QuantArgs a{};
    a.x = static_cast<const uint16_t*>(x);
    a.slots = slots;
    a.q = static_cast<int8_t*>(q);
    a.scales = scales;
    a.status = status;
    a.x_stride = x_stride;
    a.q_stride = q_stride;
    a.tokens = tokens;
    a.nrows = uint32_t(q_rows);
    a.row_len = uint32_t(row_len);
    a.top_k = slots ? uint32_t(top_k) : 1u;
    return hip_status(launch_quantize_rows(a, static_cast<hipStream_t>(stream)));
}

zipccl_status zipccl_experts_product(const void* q, uint64_t q_stride, const float* scales, uint64_t rows,
                                     const void* w, uint64_t w_stride, const float* w_scales, int num_experts,
                                     uint64_t outputs, uint64_t row_len, const int32_t* offsets, void* out,
                                     uint64_t out_stride, int out_dtype, uint32_t* status, void* stream)
{
    if (!is_dtype(out_dtype) || num_experts < 1 || num_experts > kMaxExperts || row_len < 1 || outputs < 1)
        return ZIPCCL_ERR_INVALID;
    if (!offsets && num_experts != 1) return ZIPCCL_ERR_INVALID;
    if (!w || !w_scales || (rows > 0 && (!q || !scales))) return ZIPCCL_ERR_INVALID;
    if (q_stride < row_len || w_stride < row_len) return ZIPCCL_ERR_INVALID;
    if (rows >= kMaxCount || row_len > kMaxSumLen || outputs >= (1ull << 24) || q_stride > kMaxByteStride ||
        w_stride > kMaxByteStride)
        return ZIPCCL_ERR_SIZE;
    if (q_stride % kQuantPad != 0 || w_stride % kQuantPad != 0 || !aligned(q, 16) || !aligned(w, 16) ||
        !aligned(scales, 4) || !aligned(w_scales, 4) || !aligned(offsets, 4) || (status && !aligned(status, 4)))
        return ZIPCCL_ERR_ALIGN;
    if (zipccl_status r = check_rows(out, rows, outputs, out_stride, out_dtype)) return r;
    if (rows == 0) return ZIPCCL_OK;
    ProductArgs a{};
    a.q = static_cast<const int8_t*>(q);
    a.scales = scales;
    a.w = static_cast<const int8_t*>(w);
    a.w_scales = w_scales;
    a.offsets = offsets;
    a.out = static_cast<uint8_t*>(out);
    a.status = status;
    a.q_stride = q_stride;
    a.w_stride = w_stride;
    a.out_stride = out_stride;
    a.rows = uint32_t(rows);
    a.experts = uint32_t(num_experts);
    a.outputs = uint32_t(outputs);
    a.slabs = uint32_t((row_len + kQuantPad - 1) / kQuantPad);
    a.fp32 = out_dtype == ZIPCCL_FP32;
    if (product_workgroups(a) >= kMaxTiles) return ZIPCCL_ERR_SIZE;
    return hip_status(launch_experts_product(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
