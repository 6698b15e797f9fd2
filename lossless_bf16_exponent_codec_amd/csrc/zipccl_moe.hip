// Mixture-of-experts rows for gfx950: the router's choices sorted by expert, tokens
// dispatched to their experts' rows, rows combined back to tokens with weights, and the
// gradients of both.
//
// Every kernel here is bound by memory or, for small calls, by latency: each value is
// read once and written once, sums are fp32 in a fixed order (no atomics on results), so
// a call gives the same bits on every run.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "zipccl.h"
#include "zipccl_moe_internal.h"

namespace zc {

namespace {

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
// registers across the scan over experts, and adds the expert's base after it.  Over 256
// experts 512 choices take 3.4 us (one launch, near the shortest one).  131072 take 9.0 in a
// row of calls; traced one by one, the count takes 2.8 to 3.0 and the placing 7.0 to 7.2,
// which reads the other workgroups' counts (8 16-byte loads in flight per thread; 16 of 4
// bytes took 0.8 us more, one after another 3 more still).
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

// Counts of a block in the workspace: the experts, padded to whole 16 bytes.
__host__ __device__ inline uint32_t count_row(const SortArgs& a) { return (a.experts + 3) & ~3u; }

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
    const uint32_t wide = count_row(a);
    for (uint32_t e = threadIdx.x; e < wide; e += kSortThreads)
        a.hist[uint64_t(block) * wide + e] = e < a.experts ? s_count[e] : 0;
}

constexpr uint32_t kMostShares = 16;   // of the other workgroups' counts, summed by one thread

// kGroups: groups of 64 choices per wave held in registers; 0: any number, ranked twice.
template <uint32_t kGroups>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const SortArgs a)
{
    const uint32_t block = sort_block(a);
    if (block >= a.blocks) return;
    extern __shared__ __attribute__((aligned(16))) uint32_t s_next[];            // [wave][expert]: choices so far, then the expert's base
    __shared__ uint32_t s_wave_sum[kSortWaves];
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
    // The other workgroups' counts.  A thread takes four experts and every `shares`-th
    // block; the shares meet in LDS, where thread e picks up expert e: its choices in the
    // blocks before this one, and in all.
    uint32_t before = 0, all = 0;
    if (a.blocks > 1) {
        const uint32_t wide = count_row(a), fours = wide / 4, shares = min(kSortThreads / fours, kMostShares);
        const uint32_t four = tid % fours, share = tid / fours;
        uint4 b4 = make_uint4(0, 0, 0, 0), a4 = make_uint4(0, 0, 0, 0);
        const auto gather = [&](auto batch) {   // loads in flight
            constexpr uint32_t kBatch = decltype(batch)::value;
            for (uint32_t b0 = 0; b0 < a.blocks; b0 += kBatch * shares) {
                uint4 c[kBatch];
#pragma unroll
                for (uint32_t j = 0; j < kBatch; j++) {
                    const uint32_t b = min(b0 + j * shares + share, a.blocks - 1);
                    c[j] = *reinterpret_cast<const uint4*>(a.hist + uint64_t(b) * wide + 4 * four);
                }
#pragma unroll
                for (uint32_t j = 0; j < kBatch; j++) {
                    const uint32_t b = b0 + j * shares + share;
                    if (b < a.blocks) a4 = make_uint4(a4.x + c[j].x, a4.y + c[j].y, a4.z + c[j].z, a4.w + c[j].w);
                    if (b < block) b4 = make_uint4(b4.x + c[j].x, b4.y + c[j].y, b4.z + c[j].z, b4.w + c[j].w);
                }
            }
        };
        if (share < shares) {
            if (a.blocks > shares) gather(std::integral_constant<uint32_t, 8>());
            else gather(std::integral_constant<uint32_t, 1>());
        }
        uint32_t* sums = s_next;   // [share][wide] before, then the same of all
        if (share < shares) {
            *reinterpret_cast<uint4*>(sums + share * wide + 4 * four) = b4;
            *reinterpret_cast<uint4*>(sums + (shares + share) * wide + 4 * four) = a4;
        }
        __syncthreads();
        if (tid < E) {
#pragma unroll 8
            for (uint32_t v = 0; v < shares; v++) {
                before += sums[v * wide + tid];
                all += sums[(shares + v) * wide + tid];
            }
        }
        __syncthreads();
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

    // one block: thread e's choices in all are those of the waves
    if (a.blocks == 1 && tid < E) {
#pragma unroll
        for (uint32_t w = 0; w < kSortWaves; w++) all += s_next[w * E + tid];
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

// kStream: non-temporal accesses, for rows that do not fit the Infinity Cache (combine of 16384
// tokens of 7168 from 8 rows each, 1.9 GB: 345 us, 400 with plain loads; the dispatch's stores
// by shared waves are within 3 % either way, 370 and 366).  What fits is left to the caches
// (4096 tokens of 4098 to 4 rows each, 168 MB: dispatch 26.4 us, 36.4 with non-temporal
// stores, whose lines at the ends of rows are written in parts; combine 25.1 and 30.6).
typedef uint32_t Quad __attribute__((ext_vector_type(4), aligned(2)));

template <uint32_t BYTES, bool kStream>
__device__ inline typename Raw<BYTES>::type load_raw(const uint8_t* p)
{
    if constexpr (BYTES == 16) {
        Quad v;
        if constexpr (kStream) v = __builtin_nontemporal_load(reinterpret_cast<const Quad*>(p));
        else v = *reinterpret_cast<const Quad*>(p);
        return make_uint4(v.x, v.y, v.z, v.w);
    } else {
        return *reinterpret_cast<const typename Raw<BYTES>::type*>(p);
    }
}

template <uint32_t BYTES, bool kStream>
__device__ inline void store_raw(uint8_t* p, typename Raw<BYTES>::type v)
{
    if constexpr (BYTES == 16) {
        const Quad q = {v.x, v.y, v.z, v.w};
        if constexpr (kStream) __builtin_nontemporal_store(q, reinterpret_cast<Quad*>(p));
        else *reinterpret_cast<Quad*>(p) = q;
    } else {
        *reinterpret_cast<typename Raw<BYTES>::type*>(p) = v;
    }
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
    uint32_t chunks;   // the last one overlapping where bytes is no multiple of a chunk's

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

// Choices whose rows are in flight together.
constexpr uint32_t kAhead = 4;

// Choices k0 .. k0 + kAhead - 1 of a token: slots (-1 for one that is dropped, out of range,
// or past the last) and weights.
struct Choices {
    int32_t slot[kAhead];
    float weight[kAhead];

    __device__ inline Choices(const RowsArgs& a, uint64_t token, uint32_t k0)
    {
        const uint64_t at = token * a.top_k + k0;
#pragma unroll
        for (uint32_t k = 0; k < kAhead; k++) {
            const bool have = k0 + k < a.top_k;
            slot[k] = have ? a.slots[at + k] : -1;
            weight[k] = have && a.weights ? a.weights[at + k] : 1.0f;
        }
#pragma unroll
        for (uint32_t k = 0; k < kAhead; k++) {
            if (slot[k] < int32_t(a.nrows)) continue;
            set_status(a.status, ZIPCCL_STATUS_BAD_INDEX);
            slot[k] = -1;
        }
    }
};

// One chunk of a token's row to each of its slots: the row is read once whatever top_k is.
template <uint32_t BYTES, bool kStream>
__device__ inline void dispatch_chunk(const RowsArgs& a, uint64_t token, uint32_t at)
{
    const auto v = load_raw<BYTES, false>(a.src + token * a.src_stride + at);
    for (uint32_t k0 = 0; k0 < a.top_k; k0 += kAhead) {
        const Choices c(a, token, k0);
#pragma unroll
        for (uint32_t k = 0; k < kAhead; k++)
            if (c.slot[k] >= 0) store_raw<BYTES, kStream>(a.dst + uint64_t(uint32_t(c.slot[k])) * a.dst_stride + at, v);
    }
}

// One chunk of the weighted sum of a token's rows, in the order of its choices, rounded
// once.
template <bool FP32, uint32_t BYTES, bool kStream>
__device__ inline void combine_chunk(const RowsArgs& a, uint64_t token, uint32_t at)
{
    typedef Chunk<FP32, BYTES> Values;
    Values sum;
#pragma unroll
    for (uint32_t i = 0; i < Values::kValues; i++) sum.v[i] = 0.0f;
    for (uint32_t k0 = 0; k0 < a.top_k; k0 += kAhead) {
        const Choices c(a, token, k0);
        typename Raw<BYTES>::type raw[kAhead];
#pragma unroll
        for (uint32_t k = 0; k < kAhead; k++)
            if (c.slot[k] >= 0) raw[k] = load_raw<BYTES, kStream>(a.src + uint64_t(uint32_t(c.slot[k])) * a.src_stride + at);
#pragma unroll
        for (uint32_t k = 0; k < kAhead; k++) {
            if (c.slot[k] < 0) continue;
            Values x;
            x.unpack(raw[k]);
#pragma unroll
            for (uint32_t i = 0; i < Values::kValues; i++) sum.v[i] = fmaf(c.weight[k], x.v[i], sum.v[i]);
        }
    }
    store_raw<BYTES, kStream>(a.dst + token * a.dst_stride + at, sum.pack());
}

// Two ways of sharing the chunks out.
//
// By waves: a wave takes 64 consecutive chunks (1 KB) of one token, whose slots and
// weights are then scalar values.  Parts of a row in x, so that consecutive workgroups
// share a token, groups of tokens in y.  For rows that fill such parts.
template <class Take>
__device__ inline void by_waves(const RowsArgs& a, const RowShape& sh, Take&& take)
{
    const uint32_t c = blockIdx.x * 64 + lane_id();
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (c >= sh.chunks) return;
    for (uint64_t token = uint64_t(blockIdx.y) * kRowWaves + wave; token < a.tokens;
         token += uint64_t(gridDim.y) * kRowWaves)
        take(token, sh.at<16>(c));
}

// By lanes: lane after lane through the chunks of token after token, for rows of any
// length; each of the 8 XCDs (workgroups go to them in turn) takes a run of tokens, so
// that lines that two rows or two workgroups share meet in one L2.  A slice of the tokens
// in x, slices in y.
template <uint32_t BYTES, class Take>
__device__ inline void by_lanes(const RowsArgs& a, const RowShape& sh, Take&& take)
{
    const uint32_t block = blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8;
    const uint32_t i = block * kRowThreads + threadIdx.x;
    const uint32_t in = uint32_t((uint64_t(i) * a.inverse) >> a.shift);   // token of the slice
    if (in >= a.slice) return;
    for (uint64_t token = uint64_t(blockIdx.y) * a.slice + in; token < a.tokens; token += uint64_t(gridDim.y) * a.slice)
        take(token, sh.at<BYTES>(i - in * sh.chunks));
}

template <uint32_t BYTES, bool kStream>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(const RowsArgs a)
{
    const RowShape sh = shape_of<BYTES>(a);
    by_lanes<BYTES>(a, sh, [&](uint64_t token, uint32_t at) { dispatch_chunk<BYTES, kStream>(a, token, at); });
}

// Dispatch by waves, for rows that stream: kShare waves load the same 1 KB of a token (one
// of them from memory) and write it to every kShare-th of its slots, kParts neighbouring KB
// per workgroup.  16384 tokens of 7168 from HBM to 8 rows of 64 skewed experts: 351 us, 417
// where one wave wrote all 8 rows (4 waves, 1 KB per workgroup 368; 2 waves, 2 KB 374; 1 wave, 4 KB
// 384).  One, two and four waves, to rows of 64 evenly chosen experts, in us:
//   1 row    83   82  130     5 rows  257  244  278     10 rows  477  487  477
//   2 rows  131  125  198     6 rows  301  301  309     12 rows  564  575  576
//   3 rows  170  156  217     7 rows  344  343  332     16 rows  748  755  758
//   4 rows  214  211  240     8 rows  388  397  370     64 rows (4096 tokens)  703  695  679
// so two waves below 7 rows and four from there on, 2 % off at 12 and 16 rows.
constexpr uint32_t kParts = 4;

template <uint32_t kShare>
__global__ __launch_bounds__(64 * kShare * kParts) void dispatch_shared_kernel(const RowsArgs a)
{
    const RowShape sh = shape_of<16>(a);
    const uint32_t parts = (sh.chunks + 63) / 64;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t item = blockIdx.x * kParts + wave / kShare, in = item / parts;
    const uint32_t c = (item - in * parts) * 64 + lane_id();
    if (in >= a.slice || c >= sh.chunks) return;
    const uint32_t at = sh.at<16>(c);
    for (uint64_t token = uint64_t(blockIdx.y) * a.slice + in; token < a.tokens; token += uint64_t(gridDim.y) * a.slice) {
        const auto v = load_raw<16, false>(a.src + token * a.src_stride + at);
        for (uint32_t k = wave % kShare; k < a.top_k; k += kShare) {
            const int32_t s = a.slots[token * a.top_k + k];
            if (s >= int32_t(a.nrows)) set_status(a.status, ZIPCCL_STATUS_BAD_INDEX);
            else if (s >= 0) store_raw<16, true>(a.dst + uint64_t(uint32_t(s)) * a.dst_stride + at, v);
        }
    }
}

template <bool kWaves, bool FP32, uint32_t BYTES, bool kStream>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(const RowsArgs a)
{
    const RowShape sh = shape_of<BYTES>(a);
    const auto take = [&](uint64_t token, uint32_t at) { combine_chunk<FP32, BYTES, kStream>(a, token, at); };
    if constexpr (kWaves) by_waves(a, sh, take);
    else by_lanes<BYTES>(a, sh, take);
}

// Sum over groups of kLanes lanes.
template <uint32_t kLanes>
__device__ inline float lanes_sum(float v)
{
#pragma unroll
    for (uint32_t d = kLanes / 2; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// kLanes lanes per token (a part of a wave, a wave, or all of the workgroup's): each
// choice's row is read for the weight's gradient <grad[token], y[slot]> and written with
// weight * grad[token].  Lane sums are joined by a fixed tree over lanes, then in the order
// of the waves.
template <bool FP32, uint32_t BYTES, uint32_t kLanes, bool kStream>
__global__ __launch_bounds__(kRowThreads) void combine_backward_kernel(const RowsArgs a)
{
    typedef Chunk<FP32, BYTES> Values;
    constexpr bool kWide = kLanes == kRowThreads;
    constexpr uint32_t kTokens = kRowThreads / kLanes;   // of a workgroup
    __shared__ float s_dot[kWide ? kMaxTopK : 1][kRowWaves];
    const RowShape sh = shape_of<BYTES>(a);
    const uint32_t part = threadIdx.x % kLanes;
    for (uint64_t t0 = uint64_t(blockIdx.x) * kTokens; t0 < a.tokens; t0 += uint64_t(gridDim.x) * kTokens) {
        // the last workgroup's groups past the last token repeat it
        const uint64_t mine = t0 + threadIdx.x / kLanes, token = mine < a.tokens ? mine : a.tokens - 1;
        const uint8_t* grad = a.grad + token * a.grad_stride;
        for (uint32_t k0 = 0; k0 < a.top_k; k0 += kAhead) {
            const Choices choice(a, token, k0);
            float dot[kAhead] = {};
            for (uint32_t c = part; c < sh.chunks; c += kLanes) {
                const uint32_t at = sh.at<BYTES>(c);
                // values of an overlapping last chunk that the chunk before it holds
                const uint32_t skip = (c * BYTES - at) / (FP32 ? 4 : 2);
                Values g;
                typename Raw<BYTES>::type raw[kAhead];
                g.unpack(load_raw<BYTES, false>(grad + at));
#pragma unroll
                for (uint32_t k = 0; k < kAhead; k++)
                    if (choice.slot[k] >= 0)
                        raw[k] = load_raw<BYTES, kStream>(a.src + uint64_t(uint32_t(choice.slot[k])) * a.src_stride + at);
#pragma unroll
                for (uint32_t k = 0; k < kAhead; k++) {
                    if (choice.slot[k] < 0) continue;
                    Values y, d;
                    y.unpack(raw[k]);
#pragma unroll
                    for (uint32_t i = 0; i < Values::kValues; i++) {
                        dot[k] = i >= skip ? fmaf(g.v[i], y.v[i], dot[k]) : dot[k];
                        d.v[i] = g.v[i] * choice.weight[k];
                    }
                    store_raw<BYTES, kStream>(a.dst + uint64_t(uint32_t(choice.slot[k])) * a.dst_stride + at, d.pack());
                }
            }
#pragma unroll
            for (uint32_t k = 0; k < kAhead; k++) {
                if (k0 + k >= a.top_k) break;
                const float sum = lanes_sum<kWide ? 64 : kLanes>(dot[k]);
                if constexpr (kWide) {
                    if (lane_id() == 0) s_dot[k0 + k][threadIdx.x >> 6] = sum;
                } else {
                    if (part == 0) a.grad_weights[token * a.top_k + k0 + k] = sum;
                }
            }
        }
        if constexpr (kWide) {
            __syncthreads();
            if (threadIdx.x < a.top_k) {
                float dot = 0.0f;
#pragma unroll
                for (uint32_t v = 0; v < kRowWaves; v++) dot += s_dot[threadIdx.x][v];
                a.grad_weights[token * a.top_k + threadIdx.x] = dot;
            }
            __syncthreads();
        }
    }
}

constexpr uint64_t kInfinityCache = 256ull << 20;

uint64_t row_bytes(const RowsArgs& a) { return uint64_t(a.row_len) * (a.fp32 ? 4 : 2); }

// Whether tokens and rows together pass what the Infinity Cache holds.
bool streams(const RowsArgs& a) { return (a.tokens + a.nrows) * row_bytes(a) > kInfinityCache; }

// Rows that stream go by waves (combine) or by shared waves (dispatch) where they start at lines and fill nine tenths of their
// 64-chunk parts (345 us against 365 by lanes for the combine above; fp32 rows of 4098, 67 us
// by lanes and 82 by waves).  What fits the caches is as fast or faster by lanes (4096 tokens
// of 4096 to 4 rows each, 25.2 us and 28.7).
bool goes_by_waves(const RowsArgs& a)
{
    const uint64_t chunks = (row_bytes(a) + 15) / 16;
    const uint64_t starts = reinterpret_cast<uintptr_t>(a.src) | reinterpret_cast<uintptr_t>(a.dst) | a.src_stride |
                            a.dst_stride;
    return row_bytes(a) >= 16 && streams(a) && starts % 128 == 0 && 10 * chunks >= 9 * ((chunks + 63) / 64 * 64);
}

dim3 wave_grid(const RowsArgs& a)
{
    const uint64_t parts = ((row_bytes(a) + 15) / 16 + 63) / 64, groups = (a.tokens + kRowWaves - 1) / kRowWaves;
    return dim3(uint32_t(parts), uint32_t(groups < 65535 ? groups : 65535));
}

dim3 shared_grid(RowsArgs& a)
{
    const uint64_t parts = ((row_bytes(a) + 15) / 16 + 63) / 64;
    const uint64_t most = (1ull << 22) / parts > 0 ? (1ull << 22) / parts : 1;   // tokens of a slice
    a.slice = uint32_t(a.tokens < most ? a.tokens : most);
    const uint64_t slices = (a.tokens + a.slice - 1) / a.slice;
    return dim3(uint32_t((a.slice * parts + kParts - 1) / kParts), uint32_t(slices < 65535 ? slices : 65535));
}

dim3 lane_grid(RowsArgs& a, uint32_t unit)
{
    const uint64_t chunks = (row_bytes(a) + unit - 1) / unit;
    // slices of at most 2^24 chunks (2^30 bytes of threads' indices stay far below 2^31)
    const uint64_t most = (1ull << 24) / chunks > 0 ? (1ull << 24) / chunks : 1;
    a.slice = uint32_t(a.tokens < most ? a.tokens : most);
    a.shift = 31;
    while ((1ull << (a.shift - 31)) < chunks) a.shift++;
    a.inverse = uint32_t(((1ull << a.shift) + chunks - 1) / chunks);
    const uint64_t blocks = (a.slice * chunks + kRowThreads - 1) / kRowThreads;
    const uint64_t slices = (a.tokens + a.slice - 1) / a.slice;
    return dim3(uint32_t((blocks + 7) / 8 * 8), uint32_t(slices < 65535 ? slices : 65535));
}

// Lanes per token of the combine's gradient: a workgroup above 2 KB a row (4 KB, 10000
// tokens of 4 choices: 61.5 us, 70.3 with a wave each), or where there are few tokens (64 of
// 8 choices at 2 KB: 6.0 and 7.9); else the part of a wave that takes a row at once (11
// chunks: 9.2 us on 16 lanes, 12.8 on 32; 38 chunks: 23.4 on 64, 24.2 on 32).
uint32_t backward_lanes(const RowsArgs& a, uint32_t unit)
{
    const uint64_t chunks = (row_bytes(a) + unit - 1) / unit;
    if (unit == 16 && (row_bytes(a) > 2048 || a.tokens < 1024)) return kRowThreads;
    return chunks <= 8 ? 8 : chunks <= 16 ? 16 : chunks <= 32 ? 32 : 64;
}

}  // namespace

hipError_t launch_moe_sort(const SortArgs& a, hipStream_t s)
{
    const dim3 grid(a.blocks > 1 ? (a.blocks + 7) / 8 * 8 : 1), block(kSortThreads);
    if (a.blocks > 1) hipLaunchKernelGGL(sort_count_kernel, grid, block, 0, s, a);
    const auto place = [&](void (*kernel)(SortArgs)) -> hipError_t {
        // the waves' counters; before them the shares' sums, twice
        uint32_t lds = kSortWaves * a.experts * 4;
        if (a.blocks > 1 && lds < 2 * kSortThreads * 16) lds = 2 * kSortThreads * 16;
        if (lds > 61440) {   // with the kernel's own few bytes close to the 64 KB a launch has by default
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

hipError_t launch_moe_dispatch(const RowsArgs& args, hipStream_t s)
{
    RowsArgs a = args;
    const auto run = [&](auto kernel, dim3 grid, uint32_t threads = kRowThreads) {
        hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, s, a);
    };
    if (goes_by_waves(a)) {
        if (a.top_k >= 7) run(dispatch_shared_kernel<4>, shared_grid(a), 256 * kParts);
        else if (a.top_k >= 2) run(dispatch_shared_kernel<2>, shared_grid(a), 128 * kParts);
        else run(dispatch_shared_kernel<1>, shared_grid(a), 64 * kParts);
    } else if (row_bytes(a) < 16) {
        if (a.fp32) run(dispatch_kernel<4, false>, lane_grid(a, 4));
        else run(dispatch_kernel<2, false>, lane_grid(a, 2));
    } else if (streams(a)) {
        run(dispatch_kernel<16, true>, lane_grid(a, 16));
    } else {
        run(dispatch_kernel<16, false>, lane_grid(a, 16));
    }
    return hipGetLastError();
}

hipError_t launch_moe_combine(const RowsArgs& args, hipStream_t s)
{
    RowsArgs a = args;
    const auto run = [&](auto kernel, dim3 grid) { hipLaunchKernelGGL(kernel, grid, dim3(kRowThreads), 0, s, a); };
    if (row_bytes(a) < 16) {
        if (a.fp32) run(combine_kernel<false, true, 4, false>, lane_grid(a, 4));
        else run(combine_kernel<false, false, 2, false>, lane_grid(a, 2));
    } else if (goes_by_waves(a)) {
        if (a.fp32) run(combine_kernel<true, true, 16, true>, wave_grid(a));
        else run(combine_kernel<true, false, 16, true>, wave_grid(a));
    } else if (streams(a)) {
        if (a.fp32) run(combine_kernel<false, true, 16, true>, lane_grid(a, 16));
        else run(combine_kernel<false, false, 16, true>, lane_grid(a, 16));
    } else {
        if (a.fp32) run(combine_kernel<false, true, 16, false>, lane_grid(a, 16));
        else run(combine_kernel<false, false, 16, false>, lane_grid(a, 16));
    }
    return hipGetLastError();
}

namespace {

template <bool FP32, uint32_t BYTES, bool kStream>
void run_backward(const RowsArgs& a, hipStream_t s)
{
    const uint32_t lanes = backward_lanes(a, BYTES);
    const auto run = [&](auto kernel) {
        const uint64_t per = kRowThreads / lanes, groups = (a.tokens + per - 1) / per;
        hipLaunchKernelGGL(kernel, dim3(uint32_t(groups < (1u << 20) ? groups : 1u << 20)), dim3(kRowThreads), 0, s, a);
    };
    switch (lanes) {
        case 8: run(combine_backward_kernel<FP32, BYTES, 8, kStream>); break;
        case 16: run(combine_backward_kernel<FP32, BYTES, 16, kStream>); break;
        case 32: run(combine_backward_kernel<FP32, BYTES, 32, kStream>); break;
        case 64: run(combine_backward_kernel<FP32, BYTES, 64, kStream>); break;
        default: run(combine_backward_kernel<FP32, BYTES, kRowThreads, kStream>); break;
    }
}

}  // namespace

hipError_t launch_moe_combine_backward(const RowsArgs& a, hipStream_t s)
{
    // tokens' gradients, rows and their gradients
    const bool stream = (a.tokens + 2ull * a.nrows) * row_bytes(a) > kInfinityCache;
    if (row_bytes(a) < 16) {
        if (a.fp32) run_backward<true, 4, false>(a, s);
        else run_backward<false, 2, false>(a, s);
    } else if (stream) {
        if (a.fp32) run_backward<true, 16, true>(a, s);
        else run_backward<false, 16, true>(a, s);
    } else {
        if (a.fp32) run_backward<true, 16, false>(a, s);
        else run_backward<false, 16, false>(a, s);
    }
    return hipGetLastError();
}

}  // namespace zc
