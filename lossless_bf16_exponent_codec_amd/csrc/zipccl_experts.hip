// 8-bit rows and the experts' product for gfx950.
//
// quantize_rows: row t of BF16 values x becomes q[h] = rint(127 x[h] / a) and the scale
// a / 127, a = max |x[h]|.  127 x is exact in fp32 (8 + 7 significant bits) and a quotient
// of two such numbers is either a tie or at least 2^-18 away from one, so rounding the
// correctly rounded fp32 quotient gives the integer that exact arithmetic gives.
//
// experts_product: out[s][n] = f32(sum_h q[s][h] w[e(s)][n][h]) * scale[s] * w_scale[e(s)][n],
// e(s) the expert whose rows hold s.  The sums are exact 32-bit integers, so the order in
// which tiles and waves add them does not show.
#include <hip/hip_runtime.h>

#include "zipccl.h"
#include "zipccl_moe_internal.h"

namespace zc {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

__device__ inline uint32_t lane_id() { return __lane_id(); }

__device__ inline void set_status(uint32_t* status, uint32_t bits)
{
    if (status) atomicOr(status, bits);
}

__device__ inline uint32_t bf16_rne(float f)
{
    const uint32_t u = __float_as_uint(f);
    return f != f ? 0x7FC0u : (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

// ------------------------------------------------------------------------------------
// Quantisation of rows
// ------------------------------------------------------------------------------------
constexpr uint32_t kQuantThreads = 256;
constexpr uint32_t kQuantWaves = kQuantThreads / 64;

// 8 values from h on, as bits; zeros past the row's end.
__device__ inline uint4 load8(const uint16_t* row, uint32_t h, uint32_t len)
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

// Largest magnitude of 8 values as BF16 bits without sign (bits order as magnitudes do,
// infinities and NaNs above every finite value).
__device__ inline uint32_t peak_of(uint4 v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) m = max(m, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
    return m;
}

// q of 8 values.  The row is scaled by a power of two that brings its peak into [1, 2)
// (exact; values that underflow on the way quantise to 0 in any case), where the quotient
// needs no care for range: reciprocal, product, and one correction by the remainder.
__device__ inline uint2 quantize8(uint4 v, int exponent, float peak, float inverse)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t q[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const float x = __uint_as_float(j & 1 ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
        const float n = 127.0f * ldexpf(x, exponent);
        const float y = n * inverse;
        const float z = fmaf(fmaf(-y, peak, n), inverse, y);
        q[j >> 2] |= (uint32_t(int(rintf(z))) & 0xFFu) << (8 * (j & 3));
    }
    return make_uint2(q[0], q[1]);
}

__global__ __launch_bounds__(kQuantThreads) void quantize_rows_kernel(const QuantArgs a)
{
    __shared__ uint32_t s_peak[kQuantWaves];
    const uint32_t tid = threadIdx.x, lane = lane_id();
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t padded = (a.row_len + kQuantPad - 1) / kQuantPad * kQuantPad;
    for (uint64_t token = blockIdx.x; token < a.tokens; token += gridDim.x) {
        const uint16_t* row = a.x + token * a.x_stride;
        uint32_t m = 0;
        for (uint32_t h = 8 * tid; h < a.row_len; h += 8 * kQuantThreads) m = max(m, peak_of(load8(row, h, a.row_len)));
        for (uint32_t d = 32; d > 0; d >>= 1) m = max(m, uint32_t(__shfl_xor(int(m), int(d))));
        __syncthreads();
        if (lane == 0) s_peak[wave] = m;
        __syncthreads();
        for (uint32_t w = 0; w < kQuantWaves; w++) m = max(m, s_peak[w]);
        const bool finite = m < 0x7F80u;
        const float most = __uint_as_float(m << 16);
        const float scale = finite ? most / 127.0f : __uint_as_float(0x7FC00000u);
        const bool zero = m == 0 || !finite;
        int e = 0;
        const float peak = zero ? 1.0f : 2.0f * frexpf(most, &e);
        const float inverse = 1.0f / peak;
        for (uint32_t h = 8 * tid; h < padded; h += 8 * kQuantThreads) {
            const uint2 q = zero ? make_uint2(0, 0) : quantize8(load8(row, h, a.row_len), 1 - e, peak, inverse);
            for (uint32_t k = 0; k < a.top_k; k++) {
                const int32_t s = a.slots ? a.slots[token * a.top_k + k] : int32_t(token);
                if (s < 0 || s >= int32_t(a.nrows)) continue;
                *reinterpret_cast<uint2*>(a.q + uint64_t(uint32_t(s)) * a.q_stride + h) = q;
            }
        }
        if (tid < a.top_k) {
            const int32_t s = a.slots ? a.slots[token * a.top_k + tid] : int32_t(token);
            if (s >= int32_t(a.nrows)) set_status(a.status, ZIPCCL_STATUS_BAD_INDEX);
            else if (s >= 0) a.scales[s] = scale;
        }
    }
}

// ------------------------------------------------------------------------------------
// Experts' product
// ------------------------------------------------------------------------------------

// The rows [begin, end) of an expert, from offsets that are kept in range whatever the
// caller's hold.
__device__ inline void expert_rows(const ProductArgs& a, uint32_t e, uint32_t& begin, uint32_t& end)
{
    if (!a.offsets) {
        begin = 0;
        end = a.rows;
        return;
    }
    const int64_t lo = a.offsets[e], hi = a.offsets[e + 1];
    begin = uint32_t(min(max(lo, int64_t(0)), int64_t(a.rows)));
    end = uint32_t(min(max(hi, int64_t(begin)), int64_t(a.rows)));
}

// Row tiles of kRows rows of all experts.
template <uint32_t kRows>
__device__ inline uint32_t count_tiles(const ProductArgs& a)
{
    uint32_t sum = 0;
    for (uint32_t e = lane_id(); e < a.experts; e += 64) {
        uint32_t begin, end;
        expert_rows(a, e, begin, end);
        sum += (end - begin + kRows - 1) / kRows;
    }
    for (uint32_t d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    return __builtin_amdgcn_readfirstlane(sum);
}

// The expert and the rows of row tile `tile`, tiles of kRows rows counted expert after
// expert.  Every wave looks for itself: 64 experts at a time, a running sum over lanes.
// False past the last tile.
template <uint32_t kRows>
__device__ inline bool find_tile(const ProductArgs& a, uint32_t tile, uint32_t& expert, uint32_t& row0, uint32_t& rows)
{
    const uint32_t lane = lane_id();
    uint32_t before = 0;
    for (uint32_t e0 = 0; e0 < a.experts; e0 += 64) {
        uint32_t begin = 0, end = 0;
        if (e0 + lane < a.experts) expert_rows(a, e0 + lane, begin, end);
        const uint32_t tiles = (end - begin + kRows - 1) / kRows;
        uint32_t sum = tiles;
        for (uint32_t d = 1; d < 64; d <<= 1) {
            const uint32_t up = __shfl_up(sum, d);
            if (lane >= d) sum += up;
        }
        const uint64_t past = __ballot(before + sum > tile);
        if (past) {
            const int l = __builtin_ctzll(past);
            const uint32_t at = tile - (before + __shfl(sum, l) - __shfl(tiles, l));
            const uint32_t b = __shfl(begin, l), e = __shfl(end, l);
            expert = __builtin_amdgcn_readfirstlane(e0 + uint32_t(l));
            row0 = __builtin_amdgcn_readfirstlane(b + at * kRows);
            rows = __builtin_amdgcn_readfirstlane(min(kRows, e - row0));
            return true;
        }
        before += __shfl(sum, 63);
    }
    return false;
}

// 8 consecutive outputs from n on: sums of a row scaled, rounded and stored.
struct Outputs {
    float ws[8];
    uint32_t n, count;

    __device__ inline Outputs(const ProductArgs& a, uint32_t expert, uint32_t first)
        : n(first), count(first < a.outputs ? min(8u, a.outputs - first) : 0u)
    {
        const float* from = a.w_scales + uint64_t(expert) * a.outputs + n;
#pragma unroll
        for (uint32_t r = 0; r < 8; r++) ws[r] = r < count ? from[r] : 0.0f;
    }

    __device__ inline void store(const ProductArgs& a, uint32_t row, v4i lo, v4i hi) const
    {
        const float scale = a.scales[row];
        const uint64_t at = uint64_t(row) * a.out_stride + n;
        float f[8];
#pragma unroll
        for (uint32_t r = 0; r < 8; r++) f[r] = float(r < 4 ? lo[r & 3] : hi[r & 3]) * scale * ws[r];
        if (a.fp32) {
            float* o = reinterpret_cast<float*>(a.out) + at;
            if (count == 8) {
                __builtin_memcpy(o, f, 32);
            } else {
#pragma unroll
                for (uint32_t r = 0; r < 7; r++)
                    if (r < count) o[r] = f[r];
            }
        } else {
            uint16_t* o = reinterpret_cast<uint16_t*>(a.out) + at;
            uint32_t b[4];
#pragma unroll
            for (uint32_t r = 0; r < 4; r++) b[r] = bf16_rne(f[2 * r]) | bf16_rne(f[2 * r + 1]) << 16;
            if (count == 8) {
                __builtin_memcpy(o, b, 16);
            } else {
#pragma unroll
                for (uint32_t r = 0; r < 7; r++)
                    if (r < count) o[r] = uint16_t(b[r >> 1] >> (16 * (r & 1)));
            }
        }
    }
};

// All waves: n loads may still be in flight (the oldest have landed), no LDS read is, and
// nothing moves across.
template <uint32_t N>
__device__ inline void wait_loads_and_meet()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

typedef __attribute__((address_space(1))) const void global_void;
typedef __attribute__((address_space(3))) void lds_void;

// 16 bytes per lane from global memory to LDS: lane l's land at `to` + 16 l.
__device__ inline void load_lds(const int8_t* from, uint8_t* to)
{
    __builtin_amdgcn_global_load_lds((global_void*)from, (lds_void*)to, 16, 0, 0);
}

// The share of the tiles this workgroup takes.  Workgroups go to the 8 XCDs in turn; each
// XCD takes a run of consecutive tiles, and tiles run over kBand row tiles, then over the
// outputs, so that those an XCD works on at one time share rows and weights in its L2.
constexpr uint32_t kXcds = 8, kBand = 4;

template <uint32_t kRows>
__device__ inline bool take_tile(const ProductArgs& a, uint32_t across, uint32_t& expert, uint32_t& row0,
                                 uint32_t& rows, uint32_t& column)
{
    const uint32_t down = count_tiles<kRows>(a), total = down * across;
    const uint32_t per = (total + kXcds - 1) / kXcds;
    const uint32_t at = blockIdx.x / kXcds, t = blockIdx.x % kXcds * per + at;
    if (at >= per || t >= total) return false;
    const uint32_t band = t / (kBand * across), in = t % (kBand * across);
    const uint32_t high = min(kBand, down - band * kBand);
    column = in / high;
    return find_tile<kRows>(a, band * kBand + in % high, expert, row0, rows);
}

// A tile of 64 kM rows x 64 kN outputs per workgroup of 4 waves, each 32 kM x 32 kN.  The
// rows go through LDS in steps of 64 values, four steps deep: step h + 4 is requested
// into the place of step h once every wave holds step h in registers, and while a wave
// multiplies step h it reads step h + 1 from LDS.  One barrier per step.
constexpr uint32_t kTileThreads = 256;
constexpr uint32_t kStep = 64, kStages = 4;

template <uint32_t kM, uint32_t kN>
__global__ __launch_bounds__(kTileThreads, kM * kN > 8 ? 1 : 2) void product_tile_kernel(const ProductArgs a)
{
    constexpr uint32_t kRows = 64 * kM, kOuts = 64 * kN;
    constexpr uint32_t kStage = (kRows + kOuts) * kStep, kLoads = kM + kN;   // bytes, loads per thread of a step
    // LDS reads go between the first half of a step's products, loads between the second
    constexpr uint32_t kHalf = kM * kN;
    constexpr uint32_t kReadEach = (2 * kLoads + kHalf - 1) / kHalf, kLoadEach = kHalf > kLoads ? kHalf / kLoads : 1;
    extern __shared__ __attribute__((aligned(1024))) uint8_t s_stage[];
    const uint32_t across = (a.outputs + kOuts - 1) / kOuts;
    uint32_t expert, row0, rows, column;
    if (!take_tile<kRows>(a, across, expert, row0, rows, column)) return;
    const uint32_t n0 = column * kOuts;
    const uint32_t lane = lane_id();
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int8_t* w = a.w + (uint64_t(expert) * a.outputs + n0) * a.w_stride;

    // A load of a wave fills 16 rows of 64 bytes.  The 16-byte pieces of a row are
    // swapped by bits 2-3 of the row so that 16 lanes reading one piece of 16 rows use
    // every bank.  Rows past the tile's end repeat its last one and are not stored.
    const int8_t* from[kLoads];
    const uint32_t r = 16 * wave + lane / 4, piece = (lane & 3) ^ ((lane >> 4) & 3);
#pragma unroll
    for (uint32_t i = 0; i < kLoads; i++)
        from[i] = (i < kM ? a.q + uint64_t(row0 + min(r + 64 * i, rows - 1)) * a.q_stride
                          : w + uint64_t(min(r + 64 * (i - kM), a.outputs - 1 - n0)) * a.w_stride) + 16 * piece;
    const uint32_t steps = 2 * a.slabs;
    const auto load = [&](uint32_t step) {
        const uint32_t at = min(step, steps - 1) * kStep;   // past the end: the last step again, never used
        uint8_t* to = s_stage + (step % kStages) * kStage + 1024 * wave;
#pragma unroll
        for (uint32_t i = 0; i < kLoads; i++) load_lds(from[i] + at, to + 4096 * i);
    };

    const uint32_t wm = (wave >> 1) * 32 * kM, wn = (wave & 1) * 32 * kN;
    const uint32_t half = lane >> 5, turn = (lane >> 2) & 3;
    const uint8_t* read_q = s_stage + (wm + (lane & 31)) * kStep;
    const uint8_t* read_w = s_stage + (kRows + wn + (lane & 31)) * kStep;
    v16i acc[kM][kN] = {};
    v4i fq[2][2][kM], fw[2][2][kN];
    const auto read = [&](uint32_t to, uint32_t step) {
        const uint32_t base = (step % kStages) * kStage;
#pragma unroll
        for (uint32_t k = 0; k < 2; k++) {
            const uint32_t at = base + ((2 * k + half) ^ turn) * 16;
#pragma unroll
            for (uint32_t i = 0; i < kM; i++) fq[to][k][i] = *reinterpret_cast<const v4i*>(read_q + at + 32 * kStep * i);
#pragma unroll
            for (uint32_t j = 0; j < kN; j++) fw[to][k][j] = *reinterpret_cast<const v4i*>(read_w + at + 32 * kStep * j);
        }
    };

    for (uint32_t h = 0; h < kStages; h++) load(h);
    wait_loads_and_meet<(kStages - 1) * kLoads>();
    read(0, 0);
    for (uint32_t h0 = 0; h0 < steps; h0 += 2) {
#pragma unroll
        for (uint32_t u = 0; u < 2; u++) {
            wait_loads_and_meet<(kStages - 2) * kLoads>();
            read(u ^ 1, h0 + u + 1);
            load(h0 + u + kStages);
#pragma unroll
            for (uint32_t k = 0; k < 2; k++)
#pragma unroll
                for (uint32_t i = 0; i < kM; i++)
#pragma unroll
                    for (uint32_t j = 0; j < kN; j++)
                        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[u][k][j], fq[u][k][i], acc[i][j], 0, 0, 0);
#pragma unroll
            for (uint32_t g = 0; g < kHalf; g++) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, kReadEach, 0);
            }
#pragma unroll
            for (uint32_t g = 0; g < kLoads; g++) {
                __builtin_amdgcn_sched_group_barrier(0x008, kLoadEach, 0);
                __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    wait_loads_and_meet<0>();   // the surplus loads have landed: LDS is free

    // Lane l holds, of each 32 x 32 piece, row l % 32 and outputs 8 g + 4 (l / 32) .. + 3.
    // Strips of 32 rows change hands in the wave's own part of LDS so that a lane gets 8
    // outputs in a row and a store covers whole rows of the wave's outputs.
    constexpr uint32_t kPitch = 32 * kN * 4 + 16;       // bytes; the 16 spread rows over the banks
    constexpr uint32_t kPerRow = 4 * kN;                // lanes of a row
    uint8_t* strip = s_stage + wave * (32 * kPitch);
    const uint32_t n = n0 + wn + 8 * (lane % kPerRow);
    const Outputs to(a, expert, n);
#pragma unroll
    for (uint32_t i = 0; i < kM; i++) {
        if (wm + 32 * i >= rows) break;
#pragma unroll
        for (uint32_t j = 0; j < kN; j++)
#pragma unroll
            for (uint32_t g = 0; g < 4; g++) {
                const v4i v = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
                *reinterpret_cast<v4i*>(strip + (lane & 31) * kPitch + (32 * j + 8 * g + 4 * half) * 4) = v;
            }
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (uint32_t at = lane / kPerRow; at < 32; at += 64 / kPerRow) {
            const uint32_t row = wm + 32 * i + at;
            if (row >= rows) break;
            const v4i* v = reinterpret_cast<const v4i*>(strip + at * kPitch + 32 * (lane % kPerRow));
            to.store(a, row0 + row, v[0], v[1]);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Row tiles that any split of `rows` rows over the experts can need.
uint64_t most_tiles(const ProductArgs& a, uint32_t per_tile)
{
    const uint64_t parts = a.experts < a.rows ? a.experts : a.rows;
    return (a.rows + parts * (per_tile - 1)) / per_tile;
}

}  // namespace

hipError_t launch_quantize_rows(const QuantArgs& a, hipStream_t s)
{
    const dim3 grid(uint32_t(a.tokens < (1u << 20) ? a.tokens : 1u << 20));   // the kernel steps on
    hipLaunchKernelGGL(quantize_rows_kernel, grid, dim3(kQuantThreads), 0, s, a);
    return hipGetLastError();
}

namespace {

// Tile shapes (in units of 64 x 64).
constexpr uint32_t kLargeM = 4, kLargeN = 4;
constexpr uint32_t kSmallM = 2, kSmallN = 2;

uint64_t tile_workgroups(const ProductArgs& a, uint32_t m, uint32_t n)
{
    return (most_tiles(a, 64 * m) * ((a.outputs + 64 * n - 1) / (64 * n)) + kXcds - 1) / kXcds * kXcds;
}

template <uint32_t kM, uint32_t kN>
hipError_t launch_tiles(const ProductArgs& a, hipStream_t s)
{
    constexpr uint32_t lds = kStages * 64 * (kM + kN) * kStep;
    const auto kernel = product_tile_kernel<kM, kN>;
    if (lds > 65536) {
        if (hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                               hipFuncAttributeMaxDynamicSharedMemorySize, int(lds)))
            return e;
    }
    hipLaunchKernelGGL(kernel, dim3(uint32_t(tile_workgroups(a, kM, kN))), dim3(kTileThreads), lds, s, a);
    return hipGetLastError();
}

bool use_large(const ProductArgs& a) { return tile_workgroups(a, kLargeM, kLargeN) >= 256; }

}  // namespace

uint64_t product_workgroups(const ProductArgs& a)
{
    return use_large(a) ? tile_workgroups(a, kLargeM, kLargeN) : tile_workgroups(a, kSmallM, kSmallN);
}

hipError_t launch_experts_product(const ProductArgs& a, hipStream_t s)
{
    return use_large(a) ? launch_tiles<kLargeM, kLargeN>(a, s) : launch_tiles<kSmallM, kSmallN>(a, s);
}

}  // namespace zc
