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

// Eight weights of a dword as BF16, divided by 16: the conversion of 4-bit numbers gives
// q / 16, exact in 4 significant bits, so that the upper half of its fp32 is the BF16.
__device__ inline v8b weights8(uint32_t w)
{
    const uint32_t u = w >> 4;
    uint32_t b[4];
#pragma unroll
    for (uint32_t j = 0; j < 4; j++)
        b[j] = __builtin_amdgcn_perm(__float_as_uint(__builtin_amdgcn_cvt_off_f32_i4(u >> (8 * j))),
                                     __float_as_uint(__builtin_amdgcn_cvt_off_f32_i4(w >> (8 * j))), 0x07060302u);
    return __builtin_bit_cast(v8b, make_uint4(b[0], b[1], b[2], b[3]));
}

// 8 values of a row from h on; zeros past its end.
__device__ inline uint4 values8(const uint16_t* row, uint32_t h, uint32_t len)
{
    uint4 v = make_uint4(0, 0, 0, 0);
    if (h + 8 <= len) {
        __builtin_memcpy(&v, row + h, 16);
    } else if (h < len) {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (uint32_t j = 0; j < 8; j++)
            if (h + j < len) w[j >> 1] |= uint32_t(row[h + j]) << (16 * (j & 1));
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
}

constexpr uint32_t kThreads4 = 256, kWaves4 = kThreads4 / 64;

// Row of x for row s of the call, or null: a row of zeros in the place of one out of range.
__device__ inline const uint16_t* row_of(const Product4Args& a, uint32_t s)
{
    int64_t r = s;
    if (a.index) r = a.index[s];
    if (r < 0 || r >= int64_t(a.x_rows)) {
        set_status(a.status, ZIPCCL_STATUS_BAD_INDEX);
        return nullptr;
    }
    return a.x + uint64_t(r) * a.x_stride;
}

__device__ inline float scale_at(const Product4Args& a, uint64_t i)
{
    return a.scales_fp32 ? reinterpret_cast<const float*>(a.scales)[i]
                         : bf16_value(reinterpret_cast<const uint16_t*>(a.scales)[i]);
}

__device__ inline void store_value(const Product4Args& a, uint32_t row, uint32_t n, float v)
{
    const uint64_t at = uint64_t(row) * a.out_stride + n;
    if (a.fp32) reinterpret_cast<float*>(a.out)[at] = v;
    else reinterpret_cast<uint16_t*>(a.out)[at] = v != v ? 0x7FC0u : uint16_t(bf16_pair(v, 0.0f));
}

// A tile of 16 kM rows x 16 kN outputs per workgroup, the row length split over its 4 waves,
// which meet once, to join their sums.  kParts: groups of a slab.
template <uint32_t kM, uint32_t kN, uint32_t kParts>
__global__ __launch_bounds__(kThreads4) void product4_kernel(const Product4Args a)
{
    constexpr uint32_t kPitch = 16 * kN + 4;
    __shared__ float s_sums[kWaves4][16 * kM][kPitch];
    const uint32_t across = (a.outputs + 16 * kN - 1) / (16 * kN);
    uint32_t expert, row0, rows;
    RowTiles<16 * kM, Product4Args> map(a);
    if (a.experts > 64 && blockIdx.x == 0) map.count(a);   // one workgroup looks at every offset, for the status
    if (!map.find(a, blockIdx.x / across, expert, row0, rows)) return;
    const uint32_t n0 = blockIdx.x % across * 16 * kN;
    const uint32_t lane = lane_id(), o = lane & 15, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t tiles = (a.outputs + kTile4 - 1) / kTile4;
    const uint16_t* row[kM];
#pragma unroll
    for (uint32_t m = 0; m < kM; m++) row[m] = row_of(a, row0 + min(16 * m + o, rows - 1));
    const uint8_t* w[kN];
    uint32_t column[kN];
#pragma unroll
    for (uint32_t j = 0; j < kN; j++) {
        const uint32_t tile = min(n0 / kTile4 + j, tiles - 1);
        w[j] = a.q + (uint64_t(expert) * tiles + tile) * a.slabs * kTileBytes4 + 16 * lane;
        column[j] = min(n0 + 16 * j + o, a.outputs - 1);
    }
    const uint32_t per = (a.slabs + kWaves4 - 1) / kWaves4;
    const uint32_t first = min(wave * per, a.slabs), end = min(first + per, a.slabs);
    v4f acc[kM][kN] = {};
    for (uint32_t s = first; s < end; s++) {
        uint4 q[kN], x[kM][4];
#pragma unroll
        for (uint32_t j = 0; j < kN; j++) q[j] = *reinterpret_cast<const uint4*>(w[j] + uint64_t(s) * kTileBytes4);
#pragma unroll
        for (uint32_t m = 0; m < kM; m++)
#pragma unroll
            for (uint32_t i = 0; i < 4; i++)
                x[m][i] = row[m] ? values8(row[m], s * kSlab4 + 32 * i + 8 * g, a.row_len) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (uint32_t p = 0; p < kParts; p++) {
            const uint32_t group = kParts > 1 ? min(s * kParts + p, a.groups - 1) : s * kSlab4 / a.group;
            v4f sum[kM][kN] = {};
#pragma unroll
            for (uint32_t i = p * 4 / kParts; i < (p + 1) * 4 / kParts; i++)
#pragma unroll
                for (uint32_t j = 0; j < kN; j++) {
                    const uint32_t dwords[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
                    const v8b b = weights8(dwords[i]);
#pragma unroll
                    for (uint32_t m = 0; m < kM; m++)
                        sum[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, x[m][i]), b, sum[m][j], 0, 0, 0);
                }
#pragma unroll
            for (uint32_t j = 0; j < kN; j++) {
                const float scale = scale_at(a, (uint64_t(expert) * a.groups + group) * a.outputs + column[j]);
#pragma unroll
                for (uint32_t m = 0; m < kM; m++) acc[m][j] += sum[m][j] * scale;
            }
        }
    }
    // lane 16 g + o holds rows 4 g .. 4 g + 3 of output o of each 16 x 16 piece
#pragma unroll
    for (uint32_t m = 0; m < kM; m++)
#pragma unroll
        for (uint32_t j = 0; j < kN; j++)
#pragma unroll
            for (uint32_t r = 0; r < 4; r++) s_sums[wave][16 * m + 4 * g + r][16 * j + o] = acc[m][j][r];
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < rows * 16 * kN; i += kThreads4) {
        const uint32_t r = i / (16 * kN), n = i % (16 * kN);
        if (n0 + n >= a.outputs) continue;
        float v = 0.0f;
#pragma unroll
        for (uint32_t k = 0; k < kWaves4; k++) v += s_sums[k][r][n];
        store_value(a, row0 + r, n0 + n, 16.0f * v);
    }
}

constexpr uint32_t kOuts4 = 4;      // tiles of outputs of a workgroup

// Rows of a workgroup, by an even spread over the experts.
uint32_t row_tiles(const Product4Args& a)
{
    const uint64_t parts = a.experts < a.rows ? a.experts : a.rows, each = (a.rows + parts - 1) / parts;
    return each <= 16 ? 1 : 2;
}

template <uint32_t kM>
hipError_t launch_rows(const Product4Args& a, hipStream_t s)
{
    const dim3 grid(uint32_t(product4_workgroups(a))), block(kThreads4);
    if (a.group == 32) hipLaunchKernelGGL((product4_kernel<kM, kOuts4, 4>), grid, block, 0, s, a);
    else if (a.group == 64) hipLaunchKernelGGL((product4_kernel<kM, kOuts4, 2>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((product4_kernel<kM, kOuts4, 1>), grid, block, 0, s, a);
    return hipGetLastError();
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
    return most_tiles(a, 16 * row_tiles(a)) * ((a.outputs + 16 * kOuts4 - 1) / (16 * kOuts4));
}

hipError_t launch_experts_product4(const Product4Args& a, hipStream_t s)
{
    return row_tiles(a) == 1 ? launch_rows<1>(a, s) : launch_rows<2>(a, s);
}

}  // namespace zc
