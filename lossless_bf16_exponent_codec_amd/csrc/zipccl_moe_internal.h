// Arguments of the mixture-of-experts kernels, shared by the HIP files and the host layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace zc {

constexpr int kMaxExperts = 1024;      // one thread per expert in the sort's scan
constexpr int kMaxTopK = 64;           // choices of one token
constexpr uint32_t kQuantPad = 128;    // 8-bit rows are padded with zeros to a multiple of this

// ---- sort by expert ----
constexpr uint32_t kSortWaves = 16;
constexpr uint32_t kSortThreads = 64 * kSortWaves;
constexpr uint32_t kSortMaxBlocks = 256;
constexpr uint64_t kSortWorkspace = uint64_t(kSortMaxBlocks) * kMaxExperts * 4;

struct SortArgs {
    const void* ids;       // tokens x top_k, int32 or int64, row stride `stride`
    int32_t* offsets;      // experts + 1
    int32_t* rows;         // tokens * top_k
    int32_t* slots;        // tokens * top_k
    uint32_t* hist;        // workspace: kept choices per block and expert, [block][expert]
    uint32_t* status;      // or null
    uint64_t stride;
    uint32_t n;            // tokens * top_k
    uint32_t top_k;
    uint32_t experts;
    uint32_t per_block;    // choices of one block (a multiple of kSortThreads)
    uint32_t blocks;
    uint32_t wide_ids;     // 1: int64
};
hipError_t launch_moe_sort(const SortArgs& a, hipStream_t s);

// ---- rows by slot: dispatch, combine and their gradients ----
struct RowsArgs {
    const uint8_t* src;      // dispatch: tokens; combine: rows; combine backward: rows (the forward's y)
    const uint8_t* grad;     // combine backward: gradient by token; else null
    uint8_t* dst;            // dispatch: rows; combine: tokens; combine backward: gradient by row
    const int32_t* slots;    // tokens x top_k
    const float* weights;    // tokens x top_k, or null (1)
    float* grad_weights;     // combine backward: tokens x top_k
    uint32_t* status;        // or null
    uint64_t src_stride;     // bytes
    uint64_t grad_stride;
    uint64_t dst_stride;
    uint64_t tokens;
    uint32_t nrows;          // rows by expert (slots must be below)
    uint32_t row_len;        // values
    uint32_t top_k;
    uint32_t fp32;           // 1: fp32 values, 0: BF16
    // filled in by the launches: i / chunks of a row = i * inverse >> shift for i < 2^31, and
    // the tokens of one slice of the grid
    uint32_t inverse, shift, slice;
};
hipError_t launch_moe_dispatch(const RowsArgs& a, hipStream_t s);
hipError_t launch_moe_combine(const RowsArgs& a, hipStream_t s);
hipError_t launch_moe_combine_backward(const RowsArgs& a, hipStream_t s);

// ---- 8-bit rows and the experts' product ----
struct QuantArgs {
    const uint16_t* x;       // BF16
    const int32_t* slots;    // tokens x top_k, or null: row t of q is token t
    int8_t* q;
    float* scales;
    uint32_t* status;
    uint64_t x_stride;       // values
    uint64_t q_stride;       // bytes
    uint64_t tokens;
    uint32_t nrows;          // rows of q
    uint32_t row_len;
    uint32_t top_k;
};
hipError_t launch_quantize_rows(const QuantArgs& a, hipStream_t s);

struct ProductArgs {
    const int8_t* q;
    const float* scales;     // one per row
    const int8_t* w;         // experts x outputs rows
    const float* w_scales;   // experts x outputs
    const int32_t* offsets;  // experts + 1, or null: one expert holds every row
    uint8_t* out;
    uint32_t* status;
    uint64_t q_stride;       // bytes
    uint64_t w_stride;       // bytes
    uint64_t out_stride;     // values
    uint32_t rows;
    uint32_t experts;
    uint32_t outputs;
    uint32_t slabs;          // row_len in slabs of kQuantPad values
    uint32_t fp32;           // out: 1 fp32, 0 BF16
};
// Workgroups of the product's launch.
uint64_t product_workgroups(const ProductArgs& a);
hipError_t launch_experts_product(const ProductArgs& a, hipStream_t s);

}  // namespace zc
