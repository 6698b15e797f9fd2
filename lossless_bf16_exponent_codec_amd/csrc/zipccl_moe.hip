// Mixture-of-experts rows for gfx950: the router's choices sorted by expert, tokens
// dispatched to their experts' rows, rows combined back to tokens with weights, and the
// gradients of both.
//
// Every kernel here is bound by memory or, for small calls, by latency: each value is
// read once and written once, sums are fp32 in a fixed order (no atomics on results), so
// a call gives the same bits on every run.
#include <hip/hip_runtime.h>

#include "zipccl.h"
#include "zipccl_moe_internal.h"

namespace zc {

namespace {

template <uint32_t N> struct Constant { static constexpr uint32_t value = N; };

__device__ inline uint32_t lane_id() { return __lane_id(); }

__device__ inline void set_status(uint32_t* status, uint32_t bits)
{
    if (status) atomicOr(status, bits);
}

// ------------------------------------------------------------------------------------
// Sort by expert
//
// A stable counting sort of n = tokens * top_k choices: slot(i) = (choices of smaller
// experts) + (earlier choices of the same expert).  Each workgroup takes a consecutive
// share of the choices and each of its waves a consecutive part of that share, so
// "earlier" splits into earlier workgroups (counts in the workspace), earlier waves and
// earlier groups of 64 of the wave (counts in LDS), and earlier lanes (ballots).  One
// workgroup needs no counts from others: small calls are one launch.
//
// Nothing here is bound by bandwidth (2 MB for 131072 choices); what counts is the chain
// of dependent steps.  A wave therefore ranks its choices once, holds the ranks in
// registers across the scan over experts, and adds the expert's base after it.
// ------------------------------------------------------------------------------------
__device__ inline int32_t load_id(const SortArgs& a, uint32_t i, bool& bad)
{
    const uint64_t at = a.stride == a.top_k ? i : uint64_t(i / a.top_k) * a.stride + i % a.top_k;
    int64_t id = a.wide_ids ? static_cast<const int64_t*>(a.ids)[at] : static_cast<const int32_t*>(a.ids)[at];
    if (id >= int64_t(a.experts)) {
        bad = true;
        id = -1;
    }
    return id < 0 ? -1 : int32_t(id);
}

// Neighbouring shares go to one XCD (workgroups go to the 8 XCDs in turn), where the
// pieces of a line of `rows` that they write meet in one L2.
__device__ inline uint32_t sort_block(const SortArgs& a)
{
    return a.blocks > 1 ? blockIdx.x % 8 * ((a.blocks + 7) / 8) + blockIdx.x / 8 : 0;
}

__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const SortArgs a)
{
    const uint32_t block = sort_block(a);
    if (block >= a.blocks) return;
    __shared__ uint32_t s_count[kMaxExperts];
    for (uint32_t e = threadIdx.x; e < a.experts; e += kSortThreads) s_count[e] = 0;
    __syncthreads();
    const uint32_t first = block * a.per_block, end = min(a.n, first + a.per_block);
    bool bad = false;
    for (uint32_t i = first + threadIdx.x; i < end; i += kSortThreads) {
        const int32_t id = load_id(a, i, bad);
        if (id >= 0) atomicAdd(&s_count[id], 1u);
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < a.experts; e += kSortThreads)
        a.hist[uint64_t(block) * a.experts + e] = s_count[e];
}

// kGroups: groups of 64 choices per wave held in registers; 0: any number, ranked twice.
template <uint32_t kGroups>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const SortArgs a)
{
    const uint32_t block = sort_block(a);
    if (block >= a.blocks) return;
    extern __shared__ uint32_t s_next[];            // [wave][expert]: choices so far, then the expert's base
    __shared__ uint32_t s_wave_sum[kSortWaves];
    __shared__ uint32_t s_before[kSortThreads], s_all[kSortThreads];
    const uint32_t tid = threadIdx.x, lane = lane_id();
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t E = a.experts;
    const uint32_t per_wave = kGroups ? 64 * kGroups : a.per_block / kSortWaves;
    const uint32_t first = block * a.per_block + wave * per_wave, end = min(a.n, first + per_wave);
    uint32_t* next = s_next + wave * E;
    constexpr uint32_t kHeld = kGroups ? kGroups : 1;
    int32_t id[kHeld];
    bool bad = false;
    if constexpr (kGroups > 0) {
#pragma unroll
        for (uint32_t g = 0; g < kGroups; g++) {
            const uint32_t i = first + 64 * g + lane;
            id[g] = i < end ? load_id(a, i, bad) : -1;
        }
    }
    // the other workgroups' counts: threads share an expert's blocks where there are
    // more threads than experts
    if (a.blocks > 1) {
        const uint32_t shares = kSortThreads / E, e = tid % E, share = tid / E;
        uint32_t before = 0, all = 0;
        const auto gather = [&](auto batch) {   // loads in flight
            constexpr uint32_t kBatch = decltype(batch)::value;
            for (uint32_t b0 = 0; b0 < a.blocks; b0 += kBatch * shares) {
                uint32_t c[kBatch];
#pragma unroll
                for (uint32_t j = 0; j < kBatch; j++) c[j] = a.hist[min(b0 + j * shares + share, a.blocks - 1) * E + e];
#pragma unroll
                for (uint32_t j = 0; j < kBatch; j++) {
                    const uint32_t b = b0 + j * shares + share;
                    all += b < a.blocks ? c[j] : 0;
                    before += b < block ? c[j] : 0;
                }
            }
        };
        if (a.blocks > 4 * shares) gather(Constant<16>());
        else gather(Constant<4>());
        if (share >= shares) before = all = 0;   // threads past the last whole share
        s_before[tid] = before;
        s_all[tid] = all;
    }
    for (uint32_t j = tid; j < kSortWaves * E; j += kSortThreads) s_next[j] = 0;
    __syncthreads();

    // Lanes of one expert in a group of 64 find each other by ballots over the bits of
    // its number.  Returns how many earlier choices of the wave have the lane's expert;
    // the first lane of each expert moves the wave's counter on.
    const uint32_t bits = E > 1 ? 32 - __builtin_clz(E - 1) : 0;
    const auto rank = [&](int32_t of) {
        uint64_t same = __ballot(of >= 0);
        for (uint32_t b = 0; b < bits; b++) {
            const bool on = (of >> b) & 1;
            const uint64_t m = __ballot(on);
            same &= on ? m : ~m;
        }
        uint32_t at = 0;
        if (of >= 0) {
            const uint32_t ahead = __popcll(same & ((1ull << lane) - 1));
            at = next[of];
            __builtin_amdgcn_wave_barrier();   // every lane has read before the first one writes
            if (ahead == 0) next[of] = at + __popcll(same);
            at += ahead;
        }
        __builtin_amdgcn_wave_barrier();
        return at;
    };
    uint32_t earlier[kHeld];
    if constexpr (kGroups > 0) {
#pragma unroll
        for (uint32_t g = 0; g < kGroups; g++) earlier[g] = rank(id[g]);
    } else {
        for (uint32_t g = first; g < end; g += 64) rank(g + lane < end ? load_id(a, g + lane, bad) : -1);
    }
    if (bad) set_status(a.status, ZIPCCL_STATUS_BAD_INDEX);
    __syncthreads();

    // thread e: the expert's choices in this block, in the blocks before it, and in all
    uint32_t before = 0, all = 0;
    if (tid < E) {
        if (a.blocks > 1) {
            for (uint32_t share = 0; share < kSortThreads / E; share++) {
                before += s_before[share * E + tid];
                all += s_all[share * E + tid];
            }
        } else {
#pragma unroll
            for (uint32_t w = 0; w < kSortWaves; w++) all += s_next[w * E + tid];
        }
    }
    // exclusive sum of `all` over the experts
    uint32_t scan = all;
    for (uint32_t d = 1; d < 64; d <<= 1) {
        const uint32_t up = __shfl_up(scan, d);
        if (lane >= d) scan += up;
    }
    if (lane == 63) s_wave_sum[wave] = scan;
    __syncthreads();
    uint32_t base = scan - all, total = 0;
#pragma unroll
    for (uint32_t w = 0; w < kSortWaves; w++) {
        const uint32_t v = s_wave_sum[w];
        base += w < wave ? v : 0;
        total += v;
    }
    if (tid < E) {
        if (block == 0) a.offsets[tid] = int32_t(base);
        uint32_t at = base + before, count[kSortWaves];
#pragma unroll
        for (uint32_t w = 0; w < kSortWaves; w++) count[w] = s_next[w * E + tid];
#pragma unroll
        for (uint32_t w = 0; w < kSortWaves; w++) {
            s_next[w * E + tid] = at;
            at += count[w];
        }
    }
    if (block == 0 && tid == 0) a.offsets[E] = int32_t(total);
    // dropped choices leave this many entries at the end of `rows` without a token
    for (uint32_t s = total + block * kSortThreads + tid; s < a.n; s += a.blocks * kSortThreads) a.rows[s] = -1;
    __syncthreads();

    const auto place = [&](uint32_t i, int32_t of, uint32_t slot) {
        if (of >= 0) {
            a.slots[i] = int32_t(slot);
            a.rows[slot] = int32_t(i / a.top_k);
        } else if (i < end) {
            a.slots[i] = -1;
        }
    };
    if constexpr (kGroups > 0) {
#pragma unroll
        for (uint32_t g = 0; g < kGroups; g++)
            place(first + 64 * g + lane, id[g], id[g] >= 0 ? next[id[g]] + earlier[g] : 0);
    } else {
        for (uint32_t g = first; g < end; g += 64) {
            const int32_t of = g + lane < end ? load_id(a, g + lane, bad) : -1;
            place(g + lane, of, rank(of));
        }
    }
}

// ------------------------------------------------------------------------------------
// Rows by slot
//
// Rows are handled in chunks of 16 bytes.  A row whose length is no multiple of 16 bytes
// ends in a chunk that overlaps the one before it (the last 16 bytes of the row): the
// values in the overlap are computed twice and written twice with the same bits.  Rows
// need no alignment beyond their values' own; the hardware takes 16-byte accesses at any
// address of a value.  Rows shorter than 16 bytes go value by value.
// ------------------------------------------------------------------------------------
template <uint32_t BYTES> struct Raw;
template <> struct Raw<16> { typedef uint4 type; };
template <> struct Raw<4> { typedef uint32_t type; };
template <> struct Raw<2> { typedef uint16_t type; };

template <uint32_t BYTES>
__device__ inline typename Raw<BYTES>::type load_raw(const uint8_t* p)
{
    typename Raw<BYTES>::type v;
    __builtin_memcpy(&v, BYTES > 2 ? __builtin_assume_aligned(p, 2) : p, BYTES);
    return v;
}

template <uint32_t BYTES>
__device__ inline void store_raw(uint8_t* p, typename Raw<BYTES>::type v)
{
    __builtin_memcpy(BYTES > 2 ? __builtin_assume_aligned(p, 2) : p, &v, BYTES);
}

__device__ inline uint32_t bf16_rne(float f)
{
    const uint32_t u = __float_as_uint(f);
    return f != f ? 0x7FC0u : (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

// The values of one chunk in fp32.
template <bool FP32, uint32_t BYTES>
struct Chunk {
    static constexpr uint32_t kValues = BYTES / (FP32 ? 4 : 2);
    float v[kValues];

    __device__ inline void unpack(typename Raw<BYTES>::type raw)
    {
        if constexpr (BYTES == 16) {
            const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (uint32_t j = 0; j < kValues; j++) {
                if constexpr (FP32) v[j] = __uint_as_float(w[j]);
                else v[j] = __uint_as_float(j & 1 ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
            }
        } else {
            v[0] = __uint_as_float(FP32 ? uint32_t(raw) : uint32_t(raw) << 16);
        }
    }

    __device__ inline typename Raw<BYTES>::type pack() const
    {
        if constexpr (BYTES == 16) {
            uint32_t w[4];
#pragma unroll
            for (uint32_t j = 0; j < 4; j++) {
                if constexpr (FP32) w[j] = __float_as_uint(v[j]);
                else w[j] = bf16_rne(v[2 * j]) | bf16_rne(v[2 * j + 1]) << 16;
            }
            return make_uint4(w[0], w[1], w[2], w[3]);
        } else if constexpr (FP32) {
            return __float_as_uint(v[0]);
        } else {
            return uint16_t(bf16_rne(v[0]));
        }
    }
};

struct RowShape {
    uint32_t bytes;    // of a row
    uint32_t chunks;   // of `unit` bytes, the last one overlapping where bytes is no multiple

    template <uint32_t BYTES>
    __device__ inline uint32_t at(uint32_t c) const   // byte offset of chunk c
    {
        return min(c * BYTES, bytes - BYTES);
    }
};

template <uint32_t BYTES>
__device__ inline RowShape shape_of(const RowsArgs& a)
{
    const uint32_t bytes = a.row_len * (a.fp32 ? 4u : 2u);
    return {bytes, (bytes + BYTES - 1) / BYTES};
}

constexpr uint32_t kRowThreads = 256;
constexpr uint32_t kRowWaves = kRowThreads / 64;

// The slot of choice k of a token, -1 if it is dropped or out of range.
__device__ inline int32_t slot_of(const RowsArgs& a, uint64_t token, uint32_t k)
{
    const int32_t s = a.slots[token * a.top_k + k];
    if (s >= int32_t(a.nrows)) {
        set_status(a.status, ZIPCCL_STATUS_BAD_INDEX);
        return -1;
    }
    return s < 0 ? -1 : s;
}

// A wave copies kC chunks per lane of one token's row to every slot of the token: the
// row is read once whatever top_k is.
template <uint32_t BYTES, uint32_t kC>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(const RowsArgs a)
{
    const RowShape sh = shape_of<BYTES>(a);
    const uint32_t c0 = blockIdx.x * 64 * kC + lane_id();
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (uint64_t token = uint64_t(blockIdx.y) * kRowWaves + wave; token < a.tokens;
         token += uint64_t(gridDim.y) * kRowWaves) {
        const uint8_t* src = a.src + token * a.src_stride;
        typename Raw<BYTES>::type v[kC];
#pragma unroll
        for (uint32_t j = 0; j < kC; j++)
            if (c0 + 64 * j < sh.chunks) v[j] = load_raw<BYTES>(src + sh.at<BYTES>(c0 + 64 * j));
        for (uint32_t k = 0; k < a.top_k; k++) {
            const int32_t s = slot_of(a, token, k);
            if (s < 0) continue;
            uint8_t* dst = a.dst + uint64_t(uint32_t(s)) * a.dst_stride;
#pragma unroll
            for (uint32_t j = 0; j < kC; j++)
                if (c0 + 64 * j < sh.chunks) store_raw<BYTES>(dst + sh.at<BYTES>(c0 + 64 * j), v[j]);
        }
    }
}

// A wave sums kC chunks per lane of a token's rows, in the order of its choices, and
// rounds once.
template <bool FP32, uint32_t BYTES, uint32_t kC>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(const RowsArgs a)
{
    typedef Chunk<FP32, BYTES> Values;
    const RowShape sh = shape_of<BYTES>(a);
    const uint32_t c0 = blockIdx.x * 64 * kC + lane_id();
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (uint64_t token = uint64_t(blockIdx.y) * kRowWaves + wave; token < a.tokens;
         token += uint64_t(gridDim.y) * kRowWaves) {
        Values acc[kC];
#pragma unroll
        for (uint32_t j = 0; j < kC; j++)
#pragma unroll
            for (uint32_t i = 0; i < Values::kValues; i++) acc[j].v[i] = 0.0f;
        for (uint32_t k = 0; k < a.top_k; k++) {
            const int32_t s = slot_of(a, token, k);
            if (s < 0) continue;
            const float w = a.weights ? a.weights[token * a.top_k + k] : 1.0f;
            const uint8_t* src = a.src + uint64_t(uint32_t(s)) * a.src_stride;
#pragma unroll
            for (uint32_t j = 0; j < kC; j++)
                if (c0 + 64 * j < sh.chunks) {
                    Values x;
                    x.unpack(load_raw<BYTES>(src + sh.at<BYTES>(c0 + 64 * j)));
#pragma unroll
                    for (uint32_t i = 0; i < Values::kValues; i++) acc[j].v[i] = fmaf(w, x.v[i], acc[j].v[i]);
                }
        }
        uint8_t* dst = a.dst + token * a.dst_stride;
#pragma unroll
        for (uint32_t j = 0; j < kC; j++)
            if (c0 + 64 * j < sh.chunks) store_raw<BYTES>(dst + sh.at<BYTES>(c0 + 64 * j), acc[j].pack());
    }
}

__device__ inline float wave_sum(float v)
{
    for (uint32_t d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// One workgroup per token: each choice's row is read for the weight's gradient
// <grad[token], y[slot]> and written with weight * grad[token].  Lane sums are joined by
// a fixed tree over lanes, then waves.
template <bool FP32, uint32_t BYTES>
__global__ __launch_bounds__(kRowThreads) void combine_backward_kernel(const RowsArgs a)
{
    typedef Chunk<FP32, BYTES> Values;
    __shared__ float s_dot[kMaxTopK][kRowWaves];
    const RowShape sh = shape_of<BYTES>(a);
    const uint32_t tid = threadIdx.x, lane = lane_id();
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    for (uint64_t token = blockIdx.x; token < a.tokens; token += gridDim.x) {
        const uint8_t* grad = a.grad + token * a.grad_stride;
        for (uint32_t k = 0; k < a.top_k; k++) {
            const int32_t s = slot_of(a, token, k);
            float dot = 0.0f;
            if (s >= 0) {
                const float w = a.weights ? a.weights[token * a.top_k + k] : 1.0f;
                const uint8_t* src = a.src + uint64_t(uint32_t(s)) * a.src_stride;
                uint8_t* dst = a.dst + uint64_t(uint32_t(s)) * a.dst_stride;
                for (uint32_t c = tid; c < sh.chunks; c += kRowThreads) {
                    const uint32_t at = sh.at<BYTES>(c);
                    Values g, y;
                    g.unpack(load_raw<BYTES>(grad + at));
                    y.unpack(load_raw<BYTES>(src + at));
                    // values of an overlapping last chunk that the chunk before it holds
                    const uint32_t skip = (c * BYTES - at) / (FP32 ? 4 : 2);
#pragma unroll
                    for (uint32_t i = 0; i < Values::kValues; i++) {
                        dot = i >= skip ? fmaf(g.v[i], y.v[i], dot) : dot;
                        g.v[i] *= w;
                    }
                    store_raw<BYTES>(dst + at, g.pack());
                }
            }
            dot = wave_sum(dot);
            if (lane == 0) s_dot[k][wave] = dot;
        }
        __syncthreads();
        if (tid < a.top_k) {
            float dot = 0.0f;
            for (uint32_t w = 0; w < kRowWaves; w++) dot += s_dot[tid][w];
            a.grad_weights[token * a.top_k + tid] = dot;
        }
        __syncthreads();
    }
}

// Parts of a row in x (consecutive workgroups share a token), groups of tokens in y; the
// kernels step over the tokens that a grid does not hold.
dim3 grid_for(const RowsArgs& a, uint32_t unit, uint32_t chunks_per_lane)
{
    const uint64_t bytes = uint64_t(a.row_len) * (a.fp32 ? 4 : 2);
    const uint64_t parts = ((bytes + unit - 1) / unit + 64 * chunks_per_lane - 1) / (64 * chunks_per_lane);
    const uint64_t groups = (a.tokens + kRowWaves - 1) / kRowWaves;
    return dim3(uint32_t(parts), uint32_t(groups < 65535 ? groups : 65535));
}

}  // namespace

hipError_t launch_moe_sort(const SortArgs& a, hipStream_t s)
{
    const dim3 grid(a.blocks > 1 ? (a.blocks + 7) / 8 * 8 : 1), block(kSortThreads);
    if (a.blocks > 1) hipLaunchKernelGGL(sort_count_kernel, grid, block, 0, s, a);
    const auto place = [&](void (*kernel)(SortArgs)) -> hipError_t {
        const uint32_t lds = kSortWaves * a.experts * 4;
        if (lds > 32768) {   // with the kernel's own arrays more than the 64 KB a launch has by default
            if (hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                                   hipFuncAttributeMaxDynamicSharedMemorySize, int(lds)))
                return e;
        }
        hipLaunchKernelGGL(kernel, grid, block, lds, s, a);
        return hipGetLastError();
    };
    switch (a.per_block / kSortThreads) {
        case 1: return place(sort_place_kernel<1>);
        case 2: return place(sort_place_kernel<2>);
        case 4: return place(sort_place_kernel<4>);
        case 8: return place(sort_place_kernel<8>);
        case 16: return place(sort_place_kernel<16>);
        default: return place(sort_place_kernel<0>);
    }
}

hipError_t launch_moe_dispatch(const RowsArgs& a, hipStream_t s)
{
    const uint64_t bytes = uint64_t(a.row_len) * (a.fp32 ? 4 : 2);
    const dim3 block(kRowThreads);
    if (bytes >= 16) hipLaunchKernelGGL((dispatch_kernel<16, 4>), grid_for(a, 16, 4), block, 0, s, a);
    else if (a.fp32) hipLaunchKernelGGL((dispatch_kernel<4, 1>), grid_for(a, 4, 1), block, 0, s, a);
    else hipLaunchKernelGGL((dispatch_kernel<2, 1>), grid_for(a, 2, 1), block, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_moe_combine(const RowsArgs& a, hipStream_t s)
{
    const uint64_t bytes = uint64_t(a.row_len) * (a.fp32 ? 4 : 2);
    const dim3 block(kRowThreads);
    if (bytes >= 16) {
        if (a.fp32) hipLaunchKernelGGL((combine_kernel<true, 16, 2>), grid_for(a, 16, 2), block, 0, s, a);
        else hipLaunchKernelGGL((combine_kernel<false, 16, 2>), grid_for(a, 16, 2), block, 0, s, a);
    } else if (a.fp32) {
        hipLaunchKernelGGL((combine_kernel<true, 4, 1>), grid_for(a, 4, 1), block, 0, s, a);
    } else {
        hipLaunchKernelGGL((combine_kernel<false, 2, 1>), grid_for(a, 2, 1), block, 0, s, a);
    }
    return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const RowsArgs& a, hipStream_t s)
{
    const uint64_t bytes = uint64_t(a.row_len) * (a.fp32 ? 4 : 2);
    const dim3 grid(uint32_t(a.tokens < (1u << 20) ? a.tokens : 1u << 20)), block(kRowThreads);   // the kernel steps on
    if (bytes >= 16) {
        if (a.fp32) hipLaunchKernelGGL((combine_backward_kernel<true, 16>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((combine_backward_kernel<false, 16>), grid, block, 0, s, a);
    } else {
        if (a.fp32) hipLaunchKernelGGL((combine_backward_kernel<true, 4>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((combine_backward_kernel<false, 2>), grid, block, 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace zc
