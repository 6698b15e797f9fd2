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

// ---- router: choices and weights from logits, balance loss, gradients ----
constexpr uint32_t kGateBlocks = 256;    // workgroups that leave sums in the workspace
// per workgroup: sums of probabilities and counts of kMaxExperts experts, and the tokens counted
constexpr uint64_t kGateWorkspace = uint64_t(kGateBlocks) * (8 * kMaxExperts + 16);

struct GateArgs {
    const uint8_t* logits;   // tokens x experts
    const uint8_t* mask;     // tokens, 0: the token takes no part; or null
    const void* ids;         // choices that are given (balance, gradient): int32 or int64; or null
    const float* dweights;   // gradient: tokens x top_k, or null
    const float* dloss;      // gradient: one value, or null
    const int32_t* totals;   // gradient: counts of the forward pass (experts + 1), or null
    int32_t* experts;        // choices made: tokens x top_k
    float* weights;          // tokens x top_k
    int32_t* counts;         // experts + 1 (the last: tokens counted), or null: no balance outputs
    float* sums;             // experts
    float* loss;             // one value
    uint8_t* dlogits;        // gradient
    uint8_t* workspace;      // kGateWorkspace bytes, where counts is not null
    uint32_t* status;        // or null
    uint64_t stride;         // of logits, values
    uint64_t dstride;        // of dlogits, values
    uint64_t id_stride;      // of ids, values
    uint64_t tokens;
    uint32_t num_experts;
    uint32_t top_k;
    uint32_t renormalize;    // weights sum to 1 over a token's choices; else they are probabilities
    uint32_t fp32;           // logits and dlogits: 1 fp32, 0 BF16
    uint32_t wide_ids;       // ids: 1 int64
    uint32_t blocks;         // workgroups whose sums the workspace holds
};
hipError_t launch_moe_gate(const GateArgs& a, hipStream_t s);            // makes choices, or counts those given
hipError_t launch_moe_gate_backward(const GateArgs& a, hipStream_t s);

// ---- 4-bit weights and their product ----
constexpr uint32_t kTile4 = 16;          // outputs of a tile of packed weights
constexpr uint32_t kSlab4 = 128;         // inputs of it
constexpr uint32_t kTileBytes4 = kTile4 * kSlab4 / 2;

struct Pack4Args {
    const uint16_t* w;       // BF16, experts * outputs rows
    uint8_t* q;              // tiles
    uint8_t* scales;         // experts x groups x outputs
    uint64_t w_stride;       // values
    uint32_t experts;
    uint32_t outputs;
    uint32_t row_len;
    uint32_t group;
    uint32_t fp32;           // scales: 1 fp32, 0 BF16
};
hipError_t launch_quantize_weights4(const Pack4Args& a, hipStream_t s);

struct Product4Args {
    const uint16_t* x;       // BF16 rows
    const int32_t* index;    // row of x for each row, or null: row s itself
    const uint8_t* q;        // tiles
    const uint8_t* scales;   // experts x groups x outputs
    const int32_t* offsets;  // experts + 1, or null: one expert holds every row
    uint8_t* out;
    uint32_t* status;
    uint64_t x_stride;       // values
    uint64_t out_stride;     // values
    uint32_t x_rows;
    uint32_t rows;
    uint32_t experts;
    uint32_t outputs;
    uint32_t row_len;
    uint32_t slabs;          // row_len in slabs of kSlab4 values
    uint32_t groups;         // row_len in groups
    uint32_t group;          // 32, 64 or a multiple of 128
    uint32_t scales_fp32;    // scales: 1 fp32, 0 BF16
    uint32_t fp32;           // out: 1 fp32, 0 BF16
};
uint64_t product4_workgroups(const Product4Args& a);
hipError_t launch_experts_product4(const Product4Args& a, hipStream_t s);

}  // namespace zc
