// Experts' weights in 4 bits with a scale per group of inputs, and their product, for gfx950.
//
//   out[s][n] = sum over h of x[index[s]][h] * q[e(s)][n][h] * scale[e(s)][h / group][n]
//
// with q whole numbers from -8 to 7 and e(s) the expert whose rows hold s.  A group's sum is
// taken by matrix instructions in BF16, which hold q exactly, and multiplied by its scale in
// fp32: nothing is rounded to fewer bits before the one rounding of an output.
//
// Weights lie in tiles of 16 outputs x 128 inputs, 1024 bytes in the order in which the 64
// lanes of a wave take them: lane 16 g + o holds, of output o, inputs 32 i + 8 g .. + 7 in its
// dword i, input j of the eight in bits 4 j .. 4 j + 3.  So a wave's 16-byte load is 1 KB in one
// piece, and its dword i is the operand of one 16 x 16 x 32 product.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "zipccl.h"
#include "zipccl_moe_internal.h"
#include "zipccl_row_tiles.h"

namespace zc {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

__device__ inline float bf16_value(uint16_t b) { return __uint_as_float(uint32_t(b) << 16); }

// ------------------------------------------------------------------------------------
// Packing
// ------------------------------------------------------------------------------------

// With s = max |w| / 7 over a group, rounded to the scales' type: q = rint(w / s), within
// -8 .. 7 (0 where s is 0; a group with a NaN or an infinity: q = 0 and scale NaN).  A wave
// per tile of 16 outputs and run of `group` inputs (128 at least).
__global__ __launch_bounds__(64) void quantize_weights4_kernel(const Pack4Args a)
{
    const uint32_t lane = lane_id(), o = lane & 15, g = lane >> 4;
    const uint32_t tiles = (a.outputs + kTile4 - 1) / kTile4, slabs = (a.row_len + kSlab4 - 1) / kSlab4;
    const uint32_t groups = (a.row_len + a.group - 1) / a.group;
    const uint32_t run = a.group < kSlab4 ? 1 : a.group / kSlab4, runs = (slabs + run - 1) / run;
    const uint32_t parts = a.group < kSlab4 ? kSlab4 / a.group : 1;    // groups of a slab
    const uint64_t total = uint64_t(a.experts) * tiles * runs;
    for (uint64_t at = blockIdx.x; at < total; at += gridDim.x) {
        const uint32_t r = uint32_t(at % runs), tile = uint32_t(at / runs % tiles);
        const uint64_t expert = at / runs / tiles;
        const uint32_t n = tile * kTile4 + o;
        const uint16_t* row = a.w + (expert * a.outputs + min(n, a.outputs - 1)) * a.w_stride;
        const auto value = [&](uint32_t h) { return n < a.outputs && h < a.row_len ? row[h] : uint16_t(0); };
        const uint32_t first = r * run, end = min(first + run, slabs);
        uint32_t most[4] = {0, 0, 0, 0};      // of the slab's groups, as bits
        for (uint32_t s = first; s < end; s++)
            for (uint32_t i = 0; i < 4; i++)
                for (uint32_t j = 0; j < 8; j++) {
                    const uint32_t m = value(s * kSlab4 + 32 * i + 8 * g + j) & 0x7FFFu;
                    const uint32_t to = i * parts / 4;
                    for (uint32_t p = 0; p < 4; p++)
                        if (p == to) most[p] = max(most[p], m);
                }
        float scale[4];
        bool bad[4];
        for (uint32_t p = 0; p < 4; p++) {
            most[p] = max(most[p], uint32_t(__shfl_xor(int(most[p]), 16)));
            most[p] = max(most[p], uint32_t(__shfl_xor(int(most[p]), 32)));
            bad[p] = most[p] >= 0x7F80u;
            scale[p] = bad[p] ? __uint_as_float(0x7FC00000u) : bf16_value(uint16_t(most[p])) / 7.0f;
            if (!a.fp32 && !bad[p]) scale[p] = bf16_value(uint16_t(bf16_pair(scale[p], 0.0f)));
            const uint32_t group = a.group < kSlab4 ? first * parts + p : r;
            if (p < parts && g == 0 && n < a.outputs && group < groups) {
                const uint64_t to = (expert * groups + group) * a.outputs + n;
                if (a.fp32) reinterpret_cast<float*>(a.scales)[to] = scale[p];
                else reinterpret_cast<uint16_t*>(a.scales)[to] = bad[p] ? 0x7FC0u : uint16_t(__float_as_uint(scale[p]) >> 16);
            }
        }
        for (uint32_t s = first; s < end; s++) {
            uint32_t w[4];
            for (uint32_t i = 0; i < 4; i++) {
                const uint32_t from = i * parts / 4;
                float sc = scale[0];
                bool b = bad[0];
                for (uint32_t p = 1; p < 4; p++)
                    if (p == from) {
                        sc = scale[p];
                        b = bad[p];
                    }
                w[i] = 0;
                for (uint32_t j = 0; j < 8; j++) {
                    const float v = bf16_value(value(s * kSlab4 + 32 * i + 8 * g + j));
                    const float q = b || sc == 0.0f ? 0.0f : fminf(fmaxf(rintf(v / sc), -8.0f), 7.0f);
                    w[i] |= (uint32_t(int32_t(q)) & 15u) << (4 * j);
                }
            }
            uint8_t* to = a.q + ((expert * tiles + tile) * slabs + s) * kTileBytes4 + 16 * lane;
            *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ------------------------------------------------------------------------------------
// Product
// ------------------------------------------------------------------------------------

// Weights as BF16 divided by 16: the conversion of 4-bit numbers gives q / 16 in fp32, exact in
// 4 significant bits, whose upper half is the BF16.  The conversions are in assembly because the
// compiler shifts bytes that the instruction could select, and waits between single pieces of
// assembly; the halves are joined outside, where the compiler sees what a matrix instruction
// reads and keeps the wait states between.
struct Pair4 {
    uint32_t lo, hi;
    __device__ inline uint32_t joined() const { return __builtin_amdgcn_perm(hi, lo, 0x07060302u); }
};

#define ZC_CVT(d, s) "v_cvt_off_f32_i4 %" #d ", %" #s "\n\t"
#define ZC_CVT_BYTE(b, d, s) "v_cvt_off_f32_i4_sdwa %" #d ", %" #s " dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_" #b "\n\t"

// The two weights of byte kByte of w (u: w >> 4).
template <int kByte>
__device__ inline Pair4 weights2(uint32_t w, uint32_t u)
{
    Pair4 p;
    if constexpr (kByte == 0) asm(ZC_CVT(0, 2) ZC_CVT(1, 3) : "=&v"(p.lo), "=&v"(p.hi) : "v"(w), "v"(u));
    else if constexpr (kByte == 1) asm(ZC_CVT_BYTE(1, 0, 2) ZC_CVT_BYTE(1, 1, 3) : "=&v"(p.lo), "=&v"(p.hi) : "v"(w), "v"(u));
    else if constexpr (kByte == 2) asm(ZC_CVT_BYTE(2, 0, 2) ZC_CVT_BYTE(2, 1, 3) : "=&v"(p.lo), "=&v"(p.hi) : "v"(w), "v"(u));
    else asm(ZC_CVT_BYTE(3, 0, 2) ZC_CVT_BYTE(3, 1, 3) : "=&v"(p.lo), "=&v"(p.hi) : "v"(w), "v"(u));
    return p;
}

// Eight weights of a dword, in the order of a matrix instruction's operand.
__device__ inline v8b weights8(uint32_t w)
{
    Pair4 p[4];
    asm(ZC_CVT(0, 8) ZC_CVT(1, 9) ZC_CVT_BYTE(1, 2, 8) ZC_CVT_BYTE(1, 3, 9) ZC_CVT_BYTE(2, 4, 8) ZC_CVT_BYTE(2, 5, 9)
        ZC_CVT_BYTE(3, 6, 8) ZC_CVT_BYTE(3, 7, 9)
        : "=&v"(p[0].lo), "=&v"(p[0].hi), "=&v"(p[1].lo), "=&v"(p[1].hi), "=&v"(p[2].lo), "=&v"(p[2].hi),
          "=&v"(p[3].lo), "=&v"(p[3].hi)
        : "v"(w), "v"(w >> 4));
    return __builtin_bit_cast(v8b, v4i{int(p[0].joined()), int(p[1].joined()), int(p[2].joined()), int(p[3].joined())});
}

#undef ZC_CVT
#undef ZC_CVT_BYTE

// What lanes of this wave wrote to LDS before can be read by its other lanes after.
__device__ inline void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// 8 values of a row from h on; zeros past its end, which no load passes.  kShort: the row may have
// fewer than 8.
template <bool kShort>
__device__ inline uint4 values8(const uint16_t* row, uint32_t h, uint32_t len)
{
    if (kShort && len < 8) {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (uint32_t j = 0; j < 8; j++) {
            const uint32_t v = row[min(h + j, len - 1)];
            w[j >> 1] |= (h + j < len ? v : 0u) << (16 * (j & 1));
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    const uint32_t from = min(h, len - 8), past = h - from;      // the row's last 8, `past` of them before h
    uint64_t v[2];
    __builtin_memcpy(v, row + from, 16);
    const uint32_t bits = 16 * (past & 3);
    const uint64_t up = past & 3 ? v[1] << (64 - bits) : 0;
    uint64_t lo = v[0] >> bits | up, hi = v[1] >> bits;
    if (past >= 4) {
        lo = hi;
        hi = 0;
    }
    if (past >= 8) lo = 0;
    return make_uint4(uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32));
}

// Row of x for row s of the call.  One out of range is reported (s does not count then) and
// any memory of a row's length taken in its place: the weights'.
__device__ inline const uint16_t* row_of(const Product4Args& a, uint32_t s, bool& counts)
{
    int64_t r = s;
    if (a.index) r = a.index[s];
    counts = r >= 0 && r < int64_t(a.x_rows);
    if (counts) return a.x + uint64_t(r) * a.x_stride;
    set_status(a.status, ZIPCCL_STATUS_BAD_INDEX);
    return reinterpret_cast<const uint16_t*>(a.q);
}

__device__ inline void store_value(const Product4Args& a, uint32_t row, uint32_t n, float v)
{
    const uint64_t at = uint64_t(row) * a.out_stride + n;
    if (a.fp32) reinterpret_cast<float*>(a.out)[at] = v;
    else reinterpret_cast<uint16_t*>(a.out)[at] = v != v ? 0x7FC0u : uint16_t(bf16_pair(v, 0.0f));
}

// Which of a slab's kParts groups lane 16 g + o loads the scale of.
template <uint32_t kParts>
__device__ inline uint32_t part_of(uint32_t g) { return kParts == 4 ? g : kParts == 2 ? g / 2 : 0; }

// The scales of all parts, in every lane, from what the lanes loaded.
template <uint32_t kParts>
__device__ inline void spread_parts(uint32_t v, uint32_t (&to)[kParts])
{
    if constexpr (kParts == 1) {
        to[0] = v;
    } else {
        const auto halves = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        if constexpr (kParts == 2) {
            to[0] = halves[0];
            to[1] = halves[1];
        } else {
            const auto lo = __builtin_amdgcn_permlane16_swap(halves[0], halves[0], false, false);
            const auto hi = __builtin_amdgcn_permlane16_swap(halves[1], halves[1], false, false);
            to[0] = lo[0];
            to[1] = lo[1];
            to[2] = hi[0];
            to[3] = hi[1];
        }
    }
}


// All waves: no LDS access is in flight, and their loads have landed.
__device__ inline void meet_loaded()
{
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// No load moves across.
__device__ inline void load_fence()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Launches for the groups of a slab and the type of the scales.
template <class Run>
hipError_t by_scales(const Product4Args& a, Run run)
{
    const auto with = [&](auto parts) {
        if (a.scales_fp32) run(parts, uint32_t());
        else run(parts, uint16_t());
    };
    if (a.group == 32) with(std::integral_constant<uint32_t, 4>());
    else if (a.group == 64) with(std::integral_constant<uint32_t, 2>());
    else with(std::integral_constant<uint32_t, 1>());
    return hipGetLastError();
}

// ---- few rows for an expert ----
//
// A workgroup multiplies up to 16 rows by kN tiles of 16 outputs.  Its waves share out the row
// length and meet once, to join their sums; until then each streams its part of the weights
// straight into the registers that the matrix instructions take, one slab of 128 inputs ahead.
// Rows are loaded 4 at a time, 256 bytes of each by 16 neighbouring lanes, and change hands in
// the wave's own part of LDS (as the products take them, neighbouring lanes in different
// rows, a load held the CU's address path for 88 cycles, which bounded decode: 66 us for the
// 64 tokens below).
//
// Bound by memory with the conversion close behind: a slab of a wave is 4 KB of weights and 330
// instructions.  64 tokens x 4 of 32 skewed experts, 7168 -> 2048: 55 to 56 us, 4.3 TB/s of weights;
// reading them alone takes 41.  Few calls fill the GPU so; smaller ones take fewer outputs per
// workgroup and more waves along the row.
template <uint32_t kN>
struct Slab4 {
    uint4 q[kN], x[4];
    uint32_t scale[kN];     // as bits, of the lane's part of the slab
};

constexpr uint32_t kStreamRows = 16;

template <uint32_t kN, uint32_t kParts, class Scale, uint32_t kThreads, uint32_t kPerSimd>
__global__ __launch_bounds__(kThreads, kPerSimd) void product4_stream_kernel(const Product4Args a)
{
    constexpr uint32_t kPitch = 16 * kN + 4, kWaves = kThreads / 64;
    constexpr uint32_t kStage = kWaves * 4096, kSums = kWaves * 16 * kPitch * 4;
    constexpr uint32_t shift = sizeof(Scale) == 4 ? 0 : 16;
    __shared__ __attribute__((aligned(16))) uint8_t s_all[kStage > kSums ? kStage : kSums];
    RowTiles<kStreamRows, Product4Args> map(a);
    const uint32_t across = (a.outputs + 16 * kN - 1) / (16 * kN), down = map.count(a);
    const uint32_t t = run_of_xcd(blockIdx.x, down * across);
    if (t >= down * across) return;
    uint32_t row_tile, wide, expert, row0, rows;
    tile_at(t, down, across, row_tile, wide);
    if (!map.find(a, row_tile, expert, row0, rows)) return;
    const uint32_t n0 = wide * 16 * kN;
    const uint32_t lane = lane_id(), o = lane & 15, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t tiles = (a.outputs + kTile4 - 1) / kTile4;
    uint8_t* stage = s_all + wave * 4096;
    const uint16_t* row[4];
    uint32_t good = 0;      // rows that count, as bits
#pragma unroll
    for (uint32_t i = 0; i < 4; i++) {
        bool counts;
        row[i] = row_of(a, row0 + min(4 * i + g, rows - 1), counts);
        const uint64_t all = __ballot(counts);
#pragma unroll
        for (uint32_t j = 0; j < 4; j++) good |= uint32_t((all >> (16 * j)) & 1) << (4 * i + j);
    }
    const uint8_t* w = a.q + uint64_t(expert) * tiles * a.slabs * kTileBytes4;
    const Scale* scales = reinterpret_cast<const Scale*>(a.scales) + uint64_t(expert) * a.groups * a.outputs;
    const uint32_t part = part_of<kParts>(g);
    using S = Slab4<kN>;
    const auto load_weights = [&](S& b, uint32_t s, uint32_t p) {
#pragma unroll
        for (uint32_t j = 0; j < kN; j++)
            b.q[j] = *reinterpret_cast<const uint4*>(w + (uint64_t(min(n0 / kTile4 + j, tiles - 1)) * a.slabs + s) * kTileBytes4 + 16 * lane);
        const uint32_t from = (kParts > 1 ? s * kParts : s * kSlab4 / a.group) * a.outputs;
#pragma unroll
        for (uint32_t j = 0; j < kN; j++) b.scale[j] = (scales + from)[p * a.outputs + min(n0 + 16 * j + o, a.outputs - 1)];
    };
    const auto load_rows = [&](S& b, uint32_t s) {
#pragma unroll
        for (uint32_t i = 0; i < 4; i++) __builtin_memcpy(&b.x[i], row[i] + s * kSlab4 + 8 * o, 16);
    };
    v4f acc[kN] = {};
    const auto multiply = [&](const S& b) {
        // pieces of 16 bytes are swapped by their row, so that 16 lanes reading one piece of 16
        // rows use every bank
        v8b x[4];
#pragma unroll
        for (uint32_t i = 0; i < 4; i++)
            *reinterpret_cast<uint4*>(stage + (4 * i + g) * 256 + (o ^ (4 * i + g)) * 16) = b.x[i];
        wave_order();
#pragma unroll
        for (uint32_t i = 0; i < 4; i++) x[i] = *reinterpret_cast<const v8b*>(stage + o * 256 + ((4 * i + g) ^ o) * 16);
        wave_order();
#pragma unroll
        for (uint32_t j = 0; j < kN; j++) {
            uint32_t bits[kParts];
            spread_parts<kParts>(b.scale[j], bits);
            const uint32_t dwords[4] = {b.q[j].x, b.q[j].y, b.q[j].z, b.q[j].w};
#pragma unroll
            for (uint32_t p = 0; p < kParts; p++) {
                v4f sum = {};
#pragma unroll
                for (uint32_t i = p * 4 / kParts; i < (p + 1) * 4 / kParts; i++)
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i], weights8(dwords[i]), sum, 0, 0, 0);
                const float scale = __uint_as_float(bits[p] << shift);
#pragma unroll
                for (uint32_t r = 0; r < 4; r++) acc[j][r] = fmaf(sum[r], scale, acc[j][r]);
            }
        }
    };
    const uint32_t per = (a.slabs + kWaves - 1) / kWaves;
    const uint32_t first = min(wave * per, a.slabs), end = min(first + per, a.slabs);
    const uint32_t whole = min(end, a.row_len / kSlab4);     // slabs that rows fill
    S b[2];
    if (first < whole) {
        const auto load = [&](S& to, uint32_t s) {
            s = min(s, whole - 1);
            load_weights(to, s, part);
            load_rows(to, s);
        };
        load(b[0], first);
        uint32_t s = first;
        for (; s + 1 < whole; s += 2) {
            load(b[1], s + 1);
            __builtin_amdgcn_sched_barrier(0);
            multiply(b[0]);
            load(b[0], s + 2);
            __builtin_amdgcn_sched_barrier(0);
            multiply(b[1]);
        }
        if (s < whole) multiply(b[0]);
    }
    if (first <= whole && whole < end) {      // the last slab, which rows end in; they may have only some of its parts
        const uint32_t last = kParts > 1 ? a.groups - 1 - whole * kParts : 0;
        load_weights(b[0], whole, min(part, last));
        // the others' sums are 0, and so are their scales: the last group's may be infinite
#pragma unroll
        for (uint32_t j = 0; j < kN; j++) b[0].scale[j] = part > last ? 0 : b[0].scale[j];
#pragma unroll
        for (uint32_t i = 0; i < 4; i++) b[0].x[i] = values8<true>(row[i], whole * kSlab4 + 8 * o, a.row_len);
        multiply(b[0]);
    }
    __syncthreads();    // the stage is free: the sums take its place
    // lane 16 g + o holds rows 4 g .. 4 g + 3 of output o of each 16 x 16 piece
    float* sums = reinterpret_cast<float*>(s_all);
#pragma unroll
    for (uint32_t r = 0; r < 4; r++)
#pragma unroll
        for (uint32_t j = 0; j < kN; j++)
            sums[(wave * 16 + 4 * g + r) * kPitch + 16 * j + o] = (good >> (4 * g + r)) & 1 ? acc[j][r] : 0.0f;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < rows * 16 * kN; i += kThreads) {
        const uint32_t r = i / (16 * kN), n = i % (16 * kN);
        if (n0 + n >= a.outputs) continue;
        float v = 0.0f;
#pragma unroll
        for (uint32_t k = 0; k < kWaves; k++) v += sums[(k * 16 + r) * kPitch + n];
        store_value(a, row0 + r, n0 + n, 16.0f * v);
    }
}

template <uint32_t kN>
uint64_t stream_workgroups(const Product4Args& a)
{
    return (most_tiles(a, kStreamRows) * ((a.outputs + 16 * kN - 1) / (16 * kN)) + kXcds - 1) / kXcds * kXcds;
}

template <uint32_t kN, uint32_t kThreads, uint32_t kPerSimd>
hipError_t launch_stream(const Product4Args& a, hipStream_t s)
{
    const dim3 grid(uint32_t(stream_workgroups<kN>(a))), block(kThreads);
    return by_scales(a, [&](auto parts, auto scale) {
        hipLaunchKernelGGL((product4_stream_kernel<kN, decltype(parts)::value, decltype(scale), kThreads, kPerSimd>), grid, block, 0, s, a);
    });
}

// ---- more rows ----
typedef __attribute__((address_space(1))) const void global_void;
typedef __attribute__((address_space(3))) void lds_void;

// 16 bytes per lane from global memory to LDS: lane l's land at `to` + 16 l.
__device__ inline void load_lds(const void* from, uint8_t* to)
{
    __builtin_amdgcn_global_load_lds((global_void*)from, (lds_void*)to, 16, 0, 0);
}

constexpr uint32_t kTileRows4 = 64;
// LDS of a slab: the rows, and 64 kN outputs' weights.
constexpr uint32_t slot4(uint32_t n) { return kTileRows4 * 256 + 4 * n * kTileBytes4; }

// A tile of 64 rows x 64 kN outputs by 4 waves, each 64 x 16 kN.  Rows and weights go through
// LDS a slab ahead, the rows shared by the waves, the weights each wave's own.  Within a slab
// the conversion of the next 32 inputs' weights stands between the products of this one's.
//
// Per slab and wave (kN 2) 32 products of 16 cycles, 104 instructions of conversion, 32 to scale,
// about 60 for loads and LDS.  8192 rows of 8 experts, 7168 -> 4096: 520 to 545 us, 0.9 PFLOP/s
// (444 without its loads, 342 without its products; the library's product in BF16, weights
// unpacked: 367).  Vector and matrix instructions issue in 57 % of the SIMDs' cycles, the matrix
// units work in 36 %; the rest is waits, for a slab's loads at every slab, which three waves on a
// SIMD do not cover.  Workgroups out of step on a CU do better
// than one of 8 waves that share 128 rows x 256 outputs (601): those convert, and multiply, all
// at the same time.  128 rows for 4 waves convert half as much and leave two waves on a SIMD:
// 515 here, where they fill whole rounds; with half the rows 306 (287).
template <uint32_t kN, uint32_t kParts, class Scale>
__global__ __launch_bounds__(256, kN == 1 ? 4 - (kParts > 2) : 3 - (kParts > 1)) void product4_tile_kernel(const Product4Args a)
{
    constexpr uint32_t shift = sizeof(Scale) == 4 ? 0 : 16, kSlot = slot4(kN);
    __shared__ __attribute__((aligned(1024))) uint8_t s_ring[2 * kSlot];
    RowTiles<kTileRows4, Product4Args> map(a);
    const uint32_t across = (a.outputs + 64 * kN - 1) / (64 * kN), down = map.count(a);
    const uint32_t t = run_of_xcd(blockIdx.x, down * across);
    if (t >= down * across) return;
    uint32_t row_tile, wide, expert, row0, rows;
    tile_at(t, down, across, row_tile, wide);
    if (!map.find(a, row_tile, expert, row0, rows)) return;
    const uint32_t lane = lane_id(), o = lane & 15, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t tiles = (a.outputs + kTile4 - 1) / kTile4;

    // rows 16 wave .. + 15 of the tile are this wave's to load: 4 at a time, 256 bytes of each by
    // 16 neighbouring lanes, pieces of 16 bytes swapped by their row so that 16 lanes reading
    // one piece of 16 rows use every bank
    const uint16_t* row[4];
#pragma unroll
    for (uint32_t i = 0; i < 4; i++) {
        bool counts;
        row[i] = row_of(a, row0 + min(16 * wave + 4 * i + g, rows - 1), counts);
    }
    const bool straight = ((reinterpret_cast<uintptr_t>(a.x) | 2 * a.x_stride) & 15) == 0;
    const uint32_t tile0 = (wide * 4 + wave) * kN;      // this wave's first tile of outputs
    const uint8_t* w = a.q + uint64_t(expert) * tiles * a.slabs * kTileBytes4;
    const auto load = [&](uint32_t s, uint32_t slot) {
        uint8_t* to = s_ring + slot + wave * 4096;
        if (straight && (s + 1) * kSlab4 <= a.row_len) {
#pragma unroll
            for (uint32_t i = 0; i < 4; i++) load_lds(row[i] + s * kSlab4 + 8 * (o ^ (4 * i + g)), to + 1024 * i);
        } else {
#pragma unroll
            for (uint32_t i = 0; i < 4; i++) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (s < a.slabs) x = values8<false>(row[i], s * kSlab4 + 8 * (o ^ (4 * i + g)), a.row_len);
                *reinterpret_cast<uint4*>(to + 1024 * i + 16 * lane) = x;
            }
        }
#pragma unroll
        for (uint32_t n = 0; n < kN; n++)
            load_lds(w + (uint64_t(min(tile0 + n, tiles - 1)) * a.slabs + min(s, a.slabs - 1)) * kTileBytes4 + 16 * lane,
                     s_ring + slot + kTileRows4 * 256 + (wave * kN + n) * 1024);
    };
    const Scale* scales = reinterpret_cast<const Scale*>(a.scales) + uint64_t(expert) * a.groups * a.outputs;
    const uint32_t part = part_of<kParts>(g);
    const auto load_scales = [&](uint32_t (&to)[kN], uint32_t s) {
        s = min(s, a.slabs - 1);
        const uint32_t group = kParts > 1 ? s * kParts : s * kSlab4 / a.group;
        const uint32_t p = kParts > 1 ? min(part, a.groups - 1 - group) : 0;
#pragma unroll
        for (uint32_t n = 0; n < kN; n++) to[n] = (scales + group * a.outputs)[p * a.outputs + min(16 * (tile0 + n) + o, a.outputs - 1)];
    };
    // parts that the last slab lacks have sums of 0; their scales, loaded as the last group's, which
    // may be infinite, become 0 (compared with `step` in the loop instead: 1501 rows each to 2 of
    // 5 experts, 1000 -> 1111, 0.7 us more)
    const bool lacking = kParts > 1 && part > a.groups - 1 - (a.slabs - 1) * kParts;
    v4f acc[4][kN] = {};
    // kMine: tiles of 16 rows that are multiplied
    const auto run = [&](auto of_rows) {
        constexpr uint32_t kMine = decltype(of_rows)::value;
        uint32_t scale[2][kN];
        load(0, 0);
        load_scales(scale[0], 0);
        meet_loaded();
        for (uint32_t step0 = 0; step0 < a.slabs; step0 += 2) {
#pragma unroll
            for (uint32_t u = 0; u < 2; u++) {
                const uint32_t step = step0 + u;
                if (step >= a.slabs) break;
                uint32_t bits[kN][kParts];
#pragma unroll
                for (uint32_t n = 0; n < kN; n++)
                    spread_parts<kParts>(kParts > 1 && (lacking & (step + 1 == a.slabs)) ? 0 : scale[u][n], bits[n]);
                load_fence();
                load(step + 1, (u ^ 1) * kSlot);
                load_fence();
                load_scales(scale[u ^ 1], step + 1);
                load_fence();
                const uint8_t* at = s_ring + u * kSlot + o * 256;
                const uint8_t* at_w = s_ring + u * kSlot + kTileRows4 * 256 + wave * kN * 1024 + 16 * lane;
                // read through vector types: of a struct's load the compiler does not know that it
                // is of another slot than the loads under way write, and waits for those
                v4i packed[kN];
                v8b x[kMine];
                v4i q[2][kN];
                v4f sum[kMine][kN];
#pragma unroll
                for (uint32_t n = 0; n < kN; n++) packed[n] = *reinterpret_cast<const v4i*>(at_w + 1024 * n);
                const auto take_rows = [&](uint32_t i, uint32_t m) {
                    x[m] = *reinterpret_cast<const v8b*>(at + m * 4096 + ((4 * i + g) ^ o) * 16);
                };
#pragma unroll
                for (uint32_t m = 0; m < kMine; m++) take_rows(0, m);
#pragma unroll
                for (uint32_t n = 0; n < kN; n++) q[0][n] = __builtin_bit_cast(v4i, weights8(uint32_t(packed[n][0])));
#pragma unroll
                for (uint32_t i = 0; i < 4; i++) {
                    if (i == 0) __builtin_amdgcn_s_setprio(1);      // before a wave that is not at its products yet
                    __builtin_amdgcn_sched_barrier(0);
                    uint32_t upper[kN];
#pragma unroll
                    for (uint32_t n = 0; n < kN; n++) upper[n] = i < 3 ? uint32_t(packed[n][(i + 1) & 3]) >> 4 : 0;
                    // products, each between the conversion of some of the next weights and its joining
#pragma unroll
                    for (uint32_t m = 0; m < kMine; m++)
#pragma unroll
                        for (uint32_t n = 0; n < kN; n++) {
                            constexpr uint32_t kPieces = 4 / kMine;
                            Pair4 pair[4];
                            const uint32_t w = uint32_t(packed[n][(i + 1) & 3]);
                            const auto piece = [&](uint32_t b) { return i < 3 && m * kPieces <= b && b < (m + 1) * kPieces; };
                            if (piece(0)) pair[0] = weights2<0>(w, upper[n]);
                            if (piece(1)) pair[1] = weights2<1>(w, upper[n]);
                            if (piece(2)) pair[2] = weights2<2>(w, upper[n]);
                            if (piece(3)) pair[3] = weights2<3>(w, upper[n]);
                            __builtin_amdgcn_sched_barrier(0);
                            const v4f c = i % (4 / kParts) == 0 ? v4f{} : sum[m][n];
                            sum[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[m], __builtin_bit_cast(v8b, q[i & 1][n]), c, 0, 0, 0);
                            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                            for (uint32_t b = 0; b < 4; b++)
                                if (piece(b)) q[(i + 1) & 1][n][b] = int(pair[b].joined());
                            if (i < 3 && n == kN - 1) take_rows(i + 1, m);      // the row's last product of these inputs
                        }
                    if ((i + 1) % (4 / kParts) == 0) {
#pragma unroll
                        for (uint32_t n = 0; n < kN; n++) {
                            const float by = __uint_as_float(bits[n][i * kParts / 4] << shift);
#pragma unroll
                            for (uint32_t m = 0; m < kMine; m++)
#pragma unroll
                                for (uint32_t r = 0; r < 4; r++) acc[m][n][r] = fmaf(sum[m][n][r], by, acc[m][n][r]);
                        }
                    }
                }
                __builtin_amdgcn_s_setprio(0);
                meet_loaded();
            }
        }
    };
    if (rows > 32) run(std::integral_constant<uint32_t, 4>());
    else if (rows > 16) run(std::integral_constant<uint32_t, 2>());
    else run(std::integral_constant<uint32_t, 1>());

    // lane 16 g + o holds rows 4 g .. 4 g + 3 of output o of each 16 x 16 piece
#pragma unroll
    for (uint32_t m = 0; m < 4; m++)
#pragma unroll
        for (uint32_t r = 0; r < 4; r++) {
            const uint32_t at = 16 * m + 4 * g + r;
            if (at >= rows) continue;
            bool counts;
            row_of(a, row0 + at, counts);
#pragma unroll
            for (uint32_t n = 0; n < kN; n++) {
                const uint32_t column = 16 * (tile0 + n) + o;
                if (column < a.outputs) store_value(a, row0 + at, column, counts ? 16.0f * acc[m][n][r] : 0.0f);
            }
        }
}

template <uint32_t kN>
uint64_t tile_workgroups(const Product4Args& a)
{
    return (most_tiles(a, kTileRows4) * ((a.outputs + 64 * kN - 1) / (64 * kN)) + kXcds - 1) / kXcds * kXcds;
}

template <uint32_t kN>
hipError_t launch_tiles4(const Product4Args& a, hipStream_t s)
{
    const dim3 grid(uint32_t(tile_workgroups<kN>(a))), block(256);
    return by_scales(a, [&](auto parts, auto scale) {
        hipLaunchKernelGGL((product4_tile_kernel<kN, decltype(parts)::value, decltype(scale)>), grid, block, 0, s, a);
    });
}

// Which kernel, by the tiles that rows spread evenly over the experts would make (the host
// does not know the offsets).  Times in us, outputs x row_len:
//  - from 16 rows for an expert on, tiles of 64 rows, which convert weights once for 64 rows
//    instead of 16, where there is a round of them (32 experts, 2048 x 7168, rows each: 8:
//    53 streamed and 60, 16: 68 and 62, 32: 100 and 74, 64: 162 and 105), or, of rows that
//    fill them, seven tenths of one (1 expert, 4096 x 7168, rows: 320: 45.3 and 48.4, 384:
//    53.5 and 46.5; 5 experts, 240 rows, 1111 x 1000: 16.3 and 14.2; 16 experts, 1400 x 4096,
//    50 rows: 31.2 and 35.7); 128 outputs wide where there are nearly two workgroups for a CU
//    (64 rows of 32 experts: 105, 145 at 64 wide), else 64 (1 expert, 512 rows, 4096 x 4096:
//    32.6 and 30.1; 8 experts, 250 rows, 1024 x 1024: 18.3 and 16.1);
//  - else streamed, with fewer outputs and more waves for a workgroup as there are fewer tiles
//    of 16 x 16 (1 token, 1 expert, 2048 x 7168, 128 tiles: 14.7 at 64 outputs and 4 waves,
//    10.0 at 32 and 8, 8.6 at 16 and 8; 8 experts, 1024 x 2048, 512 tiles: 7.2, 6.4, 7.5;
//    1024 tiles: 16.1, 16.4, 22.3).
enum class Shape4 { narrow, middle, stream, square, wide };

Shape4 choose4(const Product4Args& a)
{
    const uint64_t parts = a.experts < a.rows ? a.experts : a.rows, each = (a.rows + parts - 1) / parts;
    const auto tiles = [&](uint32_t rows, uint32_t outs) {
        return parts * ((each + rows - 1) / rows) * ((a.outputs + outs - 1) / outs);
    };
    constexpr uint32_t kCus = 256;
    const uint64_t large = tiles(kTileRows4, 128);
    // (of rows shorter than a slab the tiles' kernel would read past the end)
    if (a.row_len >= kSlab4 && each >= 16 && large >= (each >= kTileRows4 ? kCus * 11 / 16 : kCus))
        return large < kCus * 7 / 4 ? Shape4::square : Shape4::wide;
    const uint64_t n = tiles(16, 16);
    return n <= kCus ? Shape4::narrow : n < 4 * kCus ? Shape4::middle : Shape4::stream;
}

}  // namespace

hipError_t launch_quantize_weights4(const Pack4Args& a, hipStream_t s)
{
    const uint64_t n = uint64_t(a.experts) * ((a.outputs + kTile4 - 1) / kTile4) * ((a.row_len + kSlab4 - 1) / kSlab4);
    hipLaunchKernelGGL(quantize_weights4_kernel, dim3(uint32_t(n < (1u << 20) ? n : 1u << 20)), dim3(64), 0, s, a);
    return hipGetLastError();
}

uint64_t product4_workgroups(const Product4Args& a)
{
    switch (choose4(a)) {
        case Shape4::narrow: return stream_workgroups<1>(a);
        case Shape4::middle: return stream_workgroups<2>(a);
        case Shape4::stream: return stream_workgroups<4>(a);
        case Shape4::square: return tile_workgroups<1>(a);
        default: return tile_workgroups<2>(a);
    }
}

hipError_t launch_experts_product4(const Product4Args& a, hipStream_t s)
{
    switch (choose4(a)) {
        case Shape4::narrow: return launch_stream<1, 512, 4>(a, s);
        case Shape4::middle: return launch_stream<2, 512, 4>(a, s);
        case Shape4::stream: return launch_stream<4, 256, 3>(a, s);
        case Shape4::square: return launch_tiles4<1>(a, s);
        default: return launch_tiles4<2>(a, s);
    }
}

}  // namespace zc
