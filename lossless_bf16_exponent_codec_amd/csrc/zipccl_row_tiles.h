// Rows sorted by expert in tiles, shared by the products over them.  Args: rows, experts,
// offsets (or null) and status of a call.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "zipccl.h"

namespace zc {

namespace {

__device__ inline uint32_t lane_id() { return __lane_id(); }

__device__ inline void set_status(uint32_t* status, uint32_t bits)
{
    if (status) atomicOr(status, bits);
}

// Two values rounded to BF16 (to nearest even; a NaN keeps its sign and payload).
__device__ inline uint32_t bf16_pair(float lo, float hi)
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{lo, hi}), b2));
}

// The rows [begin, end) of an expert, from offsets that are kept in range whatever the
// caller's hold.
template <class Args>
__device__ inline void expert_rows(const Args& a, uint32_t e, uint32_t& begin, uint32_t& end)
{
    if (!a.offsets) {
        begin = 0;
        end = a.rows;
        return;
    }
    const int64_t lo = a.offsets[e], hi = a.offsets[e + 1];
    if (lo < 0 || hi < lo || hi > int64_t(a.rows)) set_status(a.status, ZIPCCL_STATUS_BAD_INDEX);
    begin = uint32_t(min(max(lo, int64_t(0)), int64_t(a.rows)));
    end = uint32_t(min(max(hi, int64_t(begin)), int64_t(a.rows)));
}

// Row tiles of kRows rows, counted expert after expert.  Every wave works them out for
// itself from the offsets: lane l looks at experts l, 64 + l, ...
template <uint32_t kRows, class Args>
struct RowTiles {
    uint32_t begin, end, tiles, sum;   // of expert `lane` of the 64 at hand; sum: running, over lanes

    __device__ inline void look(const Args& a, uint32_t e0)
    {
        begin = end = 0;
        if (e0 + lane_id() < a.experts) expert_rows(a, e0 + lane_id(), begin, end);
        sum = tiles = (end - begin + kRows - 1) / kRows;
        for (uint32_t d = 1; d < 64; d <<= 1) {
            const uint32_t up = __shfl_up(sum, d);
            if (lane_id() >= d) sum += up;
        }
    }

    __device__ inline RowTiles(const Args& a) { look(a, 0); }

    __device__ inline uint32_t here() const { return __builtin_amdgcn_readlane(sum, 63); }

    // Tiles of all experts.
    __device__ inline uint32_t count(const Args& a)
    {
        uint32_t n = here();
        for (uint32_t e0 = 64; e0 < a.experts; e0 += 64) {
            look(a, e0);
            n += here();
        }
        if (a.experts > 64) look(a, 0);
        return n;
    }

    // Expert and rows of tile `tile`; false past the last.
    __device__ inline bool find(const Args& a, uint32_t tile, uint32_t& expert, uint32_t& row0, uint32_t& rows)
    {
        uint32_t before = 0;
        for (uint32_t e0 = 0;;) {
            const uint64_t past = __ballot(before + sum > tile);
            if (past) {
                const uint32_t l = uint32_t(__builtin_ctzll(past));
                const uint32_t of = __builtin_amdgcn_readlane(tiles, l);
                const uint32_t at = tile - before - (__builtin_amdgcn_readlane(sum, l) - of);
                if (at >= of) return false;     // offsets that fall made sums pass 32 bits
                expert = e0 + l;
                row0 = __builtin_amdgcn_readlane(begin, l) + at * kRows;
                rows = min(kRows, __builtin_amdgcn_readlane(end, l) - row0);
                return true;
            }
            before += here();
            e0 += 64;
            if (e0 >= a.experts) return false;
            look(a, e0);
        }
    }
};

// Workgroups go to the 8 XCDs in turn; each XCD takes a run of consecutive tiles, and
// tiles run over kBand row tiles, then over the outputs, so that those an XCD works on at
// one time share rows and weights in its L2.
constexpr uint32_t kXcds = 8, kBand = 4;

__device__ inline uint32_t run_of_xcd(uint32_t id, uint32_t total)
{
    const uint32_t per = (total + kXcds - 1) / kXcds;
    return id / kXcds < per ? min(id % kXcds * per + id / kXcds, total) : total;
}

__device__ inline void tile_at(uint32_t t, uint32_t down, uint32_t across, uint32_t& row_tile, uint32_t& column)
{
    const uint32_t band = t / (kBand * across), in = t % (kBand * across);
    const uint32_t high = min(kBand, down - band * kBand);
    row_tile = band * kBand + in % high;
    column = in / high;
}

// Row tiles that any split of `rows` rows over the experts can need.
template <class Args>
uint64_t most_tiles(const Args& a, uint32_t per_tile)
{
    const uint64_t parts = a.experts < a.rows ? a.experts : a.rows;
    return (a.rows + parts * (per_tile - 1)) / per_tile;
}

// Allows a kernel the LDS its launch asks for (past the 64 KB a launch has by default),
// once per device: the call costs as much as the checks of a launch.
template <auto kKernel>
hipError_t allow_lds(uint32_t bytes)
{
    static std::atomic<uint64_t> done{0};   // a bit per device
    if (bytes <= 65536) return hipSuccess;
    int device = 0;
    if (hipError_t e = hipGetDevice(&device)) return e;
    const uint64_t bit = device < 64 ? 1ull << device : 0;
    if (done.load(std::memory_order_acquire) & bit) return hipSuccess;
    if (hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kKernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, int(bytes)))
        return e;
    done.fetch_or(bit, std::memory_order_release);
    return hipSuccess;
}

}  // namespace

}  // namespace zc
