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

// The rows by expert, 8 times the tokens' bytes at 8 choices, are read and written with
// non-temporal accesses; the tokens' rows, which fit the Infinity Cache where those do not,
// with plain ones (16384 tokens of 7168 to 8 rows each: dispatch 346 us, 385 with plain
// stores, 425 with non-temporal loads; combine 345 us, 400 with plain loads).
typedef uint32_t Quad __attribute__((ext_vector_type(4), aligned(2)));

template <uint32_t BYTES>
__device__ inline typename Raw<BYTES>::type load_raw(const uint8_t* p)
{
    if constexpr (BYTES == 16) {
        const Quad v = __builtin_nontemporal_load(reinterpret_cast<const Quad*>(p));
        return make_uint4(v.x, v.y, v.z, v.w);
    } else {
        return *reinterpret_cast<const typename Raw<BYTES>::type*>(p);
    }
}

template <uint32_t BYTES>
__device__ inline typename Raw<BYTES>::type load_kept(const uint8_t* p)
{
    if constexpr (BYTES == 16) {
        const Quad v = *reinterpret_cast<const Quad*>(p);
        return make_uint4(v.x, v.y, v.z, v.w);
    } else {
        return load_raw<BYTES>(p);
    }
}

template <uint32_t BYTES>
__device__ inline void store_raw(uint8_t* p, typename Raw<BYTES>::type v)
{
    if constexpr (BYTES == 16) __builtin_nontemporal_store(Quad{v.x, v.y, v.z, v.w}, reinterpret_cast<Quad*>(p));
    else *reinterpret_cast<typename Raw<BYTES>::type*>(p) = v;
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

// Slot and weight of the choices of one token: lane k holds choice k (kMaxTopK lanes), -1
// for one that is dropped or out of range.
struct Choices {
    int32_t slot = -1;
    float weight = 1.0f;

    __device__ inline Choices(const RowsArgs& a, uint64_t token)
    {
        const uint32_t k = lane_id();
        if (k >= a.top_k) return;
        slot = a.slots[token * a.top_k + k];
        if (a.weights) weight = a.weights[token * a.top_k + k];
        if (slot >= int32_t(a.nrows)) {
            set_status(a.status, ZIPCCL_STATUS_BAD_INDEX);
            slot = -1;
        }
    }

    __device__ inline int32_t slot_at(uint32_t k) const { return __builtin_amdgcn_readlane(slot, k); }
    __device__ inline float weight_at(uint32_t k) const
    {
        return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(weight), k));
    }
};
static_assert(kMaxTopK <= 64, "a lane per choice");

// Lanes past a row's end repeat its last chunk (one address, one value) rather than leave:
// lane k's choice is read by the others at any place of the row.

// Choices whose rows are in flight together.
constexpr uint32_t kAhead = 4;

// A wave takes one 16-byte chunk per lane of a token's row (1 KB; 2 and 4 KB per wave were
// slower, 350 and 369 us against 347 for the dispatch of 16384 x 7168 to 8 rows each) and
// copies it to every slot of the token: the row is read once whatever top_k is.
template <uint32_t BYTES>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(const RowsArgs a)
{
    const RowShape sh = shape_of<BYTES>(a);
    const uint32_t c = min(blockIdx.x * 64 + lane_id(), sh.chunks - 1);
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (uint64_t token = uint64_t(blockIdx.y) * kRowWaves + wave; token < a.tokens;
         token += uint64_t(gridDim.y) * kRowWaves) {
        const uint32_t at = sh.at<BYTES>(c);
        const auto v = load_kept<BYTES>(a.src + token * a.src_stride + at);   // on its way while the slots are looked up
        const Choices choices(a, token);
        for (uint32_t k = 0; k < a.top_k; k++) {
            const int32_t s = choices.slot_at(k);
            if (s >= 0) store_raw<BYTES>(a.dst + uint64_t(uint32_t(s)) * a.dst_stride + at, v);
        }
    }
}

// A wave sums one chunk per lane of a token's rows, in the order of its choices, and
// rounds once.
template <bool FP32, uint32_t BYTES>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(const RowsArgs a)
{
    typedef Chunk<FP32, BYTES> Values;
    const RowShape sh = shape_of<BYTES>(a);
    const uint32_t c = min(blockIdx.x * 64 + lane_id(), sh.chunks - 1);
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (uint64_t token = uint64_t(blockIdx.y) * kRowWaves + wave; token < a.tokens;
         token += uint64_t(gridDim.y) * kRowWaves) {
        const Choices choices(a, token);
        const uint32_t at = sh.at<BYTES>(c);
        Values acc;
#pragma unroll
        for (uint32_t i = 0; i < Values::kValues; i++) acc.v[i] = 0.0f;
        for (uint32_t k0 = 0; k0 < a.top_k; k0 += kAhead) {
            typename Raw<BYTES>::type raw[kAhead];
            int32_t s[kAhead];
#pragma unroll
            for (uint32_t k = 0; k < kAhead; k++) {
                s[k] = k0 + k < a.top_k ? choices.slot_at(k0 + k) : -1;
                if (s[k] >= 0) raw[k] = load_raw<BYTES>(a.src + uint64_t(uint32_t(s[k])) * a.src_stride + at);
            }
#pragma unroll
            for (uint32_t k = 0; k < kAhead; k++) {
                if (s[k] < 0) continue;
                const float w = choices.weight_at(k0 + k);
                Values x;
                x.unpack(raw[k]);
#pragma unroll
                for (uint32_t i = 0; i < Values::kValues; i++) acc.v[i] = fmaf(w, x.v[i], acc.v[i]);
            }
        }
        store_raw<BYTES>(a.dst + token * a.dst_stride + at, acc.pack());
    }
}

__device__ inline float wave_sum(float v)
{
    for (uint32_t d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// kWaves waves per token: each choice's row is read for the weight's gradient
// <grad[token], y[slot]> and written with weight * grad[token].  Lane sums are joined by
// a fixed tree over lanes, then in the order of the waves.
template <bool FP32, uint32_t BYTES, uint32_t kWaves>
__global__ __launch_bounds__(kRowThreads) void combine_backward_kernel(const RowsArgs a)
{
    typedef Chunk<FP32, BYTES> Values;
    constexpr uint32_t kTokens = kRowWaves / kWaves;   // of a workgroup
    __shared__ float s_dot[kMaxTopK][kRowWaves];
    const RowShape sh = shape_of<BYTES>(a);
    const uint32_t lane = lane_id();
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), part = wave % kWaves;
    for (uint64_t t0 = uint64_t(blockIdx.x) * kTokens; t0 < a.tokens; t0 += uint64_t(gridDim.x) * kTokens) {
        const uint64_t token = t0 + wave / kWaves;
        const bool have = token < a.tokens;
        if (have) {
            const Choices choices(a, token);
            const uint8_t* grad = a.grad + token * a.grad_stride;
            for (uint32_t k0 = 0; k0 < a.top_k; k0 += kAhead) {
                int32_t s[kAhead];
                float w[kAhead], dot[kAhead];
#pragma unroll
                for (uint32_t k = 0; k < kAhead; k++) {
                    s[k] = k0 + k < a.top_k ? choices.slot_at(k0 + k) : -1;
                    w[k] = choices.weight_at((k0 + k) & 63);
                    dot[k] = 0.0f;
                }
                for (uint32_t c = 64 * part + lane; c < sh.chunks; c += 64 * kWaves) {
                    const uint32_t at = sh.at<BYTES>(c);
                    // values of an overlapping last chunk that the chunk before it holds
                    const uint32_t skip = (c * BYTES - at) / (FP32 ? 4 : 2);
                    Values g;
                    typename Raw<BYTES>::type raw[kAhead];
                    g.unpack(load_kept<BYTES>(grad + at));
#pragma unroll
                    for (uint32_t k = 0; k < kAhead; k++)
                        if (s[k] >= 0) raw[k] = load_raw<BYTES>(a.src + uint64_t(uint32_t(s[k])) * a.src_stride + at);
#pragma unroll
                    for (uint32_t k = 0; k < kAhead; k++) {
                        if (s[k] < 0) continue;
                        Values y, d;
                        y.unpack(raw[k]);
#pragma unroll
                        for (uint32_t i = 0; i < Values::kValues; i++) {
                            dot[k] = i >= skip ? fmaf(g.v[i], y.v[i], dot[k]) : dot[k];
                            d.v[i] = g.v[i] * w[k];
                        }
                        store_raw<BYTES>(a.dst + uint64_t(uint32_t(s[k])) * a.dst_stride + at, d.pack());
                    }
                }
#pragma unroll
                for (uint32_t k = 0; k < kAhead; k++) {
                    if (k0 + k >= a.top_k) break;
                    const float sum = wave_sum(dot[k]);
                    if (lane != 0) continue;
                    if constexpr (kWaves == 1) a.grad_weights[token * a.top_k + k0 + k] = sum;
                    else s_dot[k0 + k][wave] = sum;
                }
            }
        }
        if constexpr (kWaves > 1) {
            static_assert(kWaves == kRowWaves, "one token per workgroup");
            __syncthreads();
            if (threadIdx.x < a.top_k) {
                float dot = 0.0f;
#pragma unroll
                for (uint32_t v = 0; v < kWaves; v++) dot += s_dot[threadIdx.x][v];
                a.grad_weights[token * a.top_k + threadIdx.x] = dot;
            }
            __syncthreads();
        }
    }
}

// Parts of a row in x (consecutive workgroups share a token), groups of tokens in y; the
// kernels step over the tokens that a grid does not hold.
dim3 grid_for(const RowsArgs& a, uint32_t unit)
{
    const uint64_t bytes = uint64_t(a.row_len) * (a.fp32 ? 4 : 2);
    const uint64_t parts = ((bytes + unit - 1) / unit + 63) / 64;
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
    const dim3 block(kRowThreads);
    if (a.row_len * (a.fp32 ? 4ull : 2ull) >= 16) hipLaunchKernelGGL(dispatch_kernel<16>, grid_for(a, 16), block, 0, s, a);
    else if (a.fp32) hipLaunchKernelGGL(dispatch_kernel<4>, grid_for(a, 4), block, 0, s, a);
    else hipLaunchKernelGGL(dispatch_kernel<2>, grid_for(a, 2), block, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_moe_combine(const RowsArgs& a, hipStream_t s)
{
    const dim3 block(kRowThreads);
    if (a.row_len * (a.fp32 ? 4ull : 2ull) >= 16) {
        if (a.fp32) hipLaunchKernelGGL((combine_kernel<true, 16>), grid_for(a, 16), block, 0, s, a);
        else hipLaunchKernelGGL((combine_kernel<false, 16>), grid_for(a, 16), block, 0, s, a);
    } else if (a.fp32) {
        hipLaunchKernelGGL((combine_kernel<true, 4>), grid_for(a, 4), block, 0, s, a);
    } else {
        hipLaunchKernelGGL((combine_kernel<false, 2>), grid_for(a, 2), block, 0, s, a);
    }
    return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const RowsArgs& a, hipStream_t s)
{
    const uint64_t bytes = a.row_len * (a.fp32 ? 4ull : 2ull);
    const auto run = [&](auto kernel, uint32_t tokens) {   // tokens of a workgroup
        const uint64_t groups = (a.tokens + tokens - 1) / tokens;
        hipLaunchKernelGGL(kernel, dim3(uint32_t(groups < (1u << 20) ? groups : 1u << 20)), dim3(kRowThreads), 0, s, a);
    };
    // a wave per token up to 2 KB a row (8192 tokens of 4 choices: 28 us against 31 with a
    // workgroup each at 2 KB, 60 and 53 at 4 KB), with enough tokens to fill the GPU (64 of
    // 8 choices, 2 KB: 7.9 and 6.0)
    if (bytes < 16) a.fp32 ? run(combine_backward_kernel<true, 4, 1>, 4) : run(combine_backward_kernel<false, 2, 1>, 4);
    else if (bytes <= 2048 && a.tokens >= 1024) a.fp32 ? run(combine_backward_kernel<true, 16, 1>, 4) : run(combine_backward_kernel<false, 16, 1>, 4);
    else a.fp32 ? run(combine_backward_kernel<true, 16, 4>, 1) : run(combine_backward_kernel<false, 16, 4>, 1);
    return hipGetLastError();
}

}  // namespace zc
