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

// One value's 4 neighbours along the outputs: scaled, rounded and stored.
__device__ inline void store4(const ProductArgs& a, uint32_t row, uint32_t n, v4i acc, float scale, const float* ws)
{
    const uint64_t at = uint64_t(row) * a.out_stride + n;
    float f[4];
#pragma unroll
    for (uint32_t r = 0; r < 4; r++) f[r] = n + r < a.outputs ? float(acc[r]) * scale * ws[n + r] : 0.0f;
    if (a.fp32) {
        float* o = reinterpret_cast<float*>(a.out) + at;
        if (n + 4 <= a.outputs) {
            __builtin_memcpy(o, f, 16);
        } else {
#pragma unroll
            for (uint32_t r = 0; r < 4; r++)
                if (n + r < a.outputs) o[r] = f[r];
        }
    } else {
        uint16_t* o = reinterpret_cast<uint16_t*>(a.out) + at;
        uint32_t b[4];
#pragma unroll
        for (uint32_t r = 0; r < 4; r++) b[r] = bf16_rne(f[r]);
        if (n + 4 <= a.outputs) {
            const uint2 v = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
            __builtin_memcpy(o, &v, 8);
        } else {
#pragma unroll
            for (uint32_t r = 0; r < 4; r++)
                if (n + r < a.outputs) o[r] = uint16_t(b[r]);
        }
    }
}

constexpr uint32_t kTileRows = 128, kTileOuts = 128, kTileThreads = 256;

// 16-byte piece `piece` of row `row` in a slab of 128-byte rows, spread over the banks.
__device__ inline uint32_t lds_at(uint32_t row, uint32_t piece) { return row * 128 + ((piece ^ (row >> 1)) & 7) * 16; }

// A tile of 128 rows x 128 outputs per workgroup, 64 x 64 per wave.  Slabs of 128 values
// along the rows go through registers into LDS.  Rows past the expert's end repeat its
// last row and are not stored.
__global__ __launch_bounds__(kTileThreads) void product_kernel(const ProductArgs a)
{
    __shared__ __attribute__((aligned(16))) uint8_t s_q[kTileRows * 128];
    __shared__ __attribute__((aligned(16))) uint8_t s_w[kTileOuts * 128];
    uint32_t expert, row0, rows;
    const uint32_t across = (a.outputs + kTileOuts - 1) / kTileOuts;
    if (!find_tile<kTileRows>(a, blockIdx.x / across, expert, row0, rows)) return;
    const uint32_t n0 = blockIdx.x % across * kTileOuts;
    const uint32_t tid = threadIdx.x, lane = lane_id();
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
    const int8_t* w = a.w + uint64_t(expert) * a.outputs * a.w_stride;

    const uint32_t piece = tid & 7, r0 = tid >> 3;   // this thread's 16 bytes in rows r0, r0 + 32, ...
    v4i acc[4][4] = {};
    uint4 vq[4], vw[4];
    const auto load = [&](uint32_t slab) {
#pragma unroll
        for (uint32_t i = 0; i < 4; i++) {
            const uint32_t r = min(r0 + 32 * i, rows - 1), n = min(n0 + r0 + 32 * i, a.outputs - 1);
            vq[i] = *reinterpret_cast<const uint4*>(a.q + uint64_t(row0 + r) * a.q_stride + slab * 128 + piece * 16);
            vw[i] = *reinterpret_cast<const uint4*>(w + uint64_t(n) * a.w_stride + slab * 128 + piece * 16);
        }
    };
    load(0);
    for (uint32_t slab = 0; slab < a.slabs; slab++) {
        __syncthreads();
#pragma unroll
        for (uint32_t i = 0; i < 4; i++) {
            *reinterpret_cast<uint4*>(s_q + lds_at(r0 + 32 * i, piece)) = vq[i];
            *reinterpret_cast<uint4*>(s_w + lds_at(r0 + 32 * i, piece)) = vw[i];
        }
        __syncthreads();
        if (slab + 1 < a.slabs) load(slab + 1);
#pragma unroll
        for (uint32_t half = 0; half < 2; half++) {
            v4i fq[4], fw[4];
#pragma unroll
            for (uint32_t i = 0; i < 4; i++) {
                fq[i] = *reinterpret_cast<const v4i*>(s_q + lds_at(wm + 16 * i + (lane & 15), 4 * half + (lane >> 4)));
                fw[i] = *reinterpret_cast<const v4i*>(s_w + lds_at(wn + 16 * i + (lane & 15), 4 * half + (lane >> 4)));
            }
#pragma unroll
            for (uint32_t i = 0; i < 4; i++)
#pragma unroll
                for (uint32_t j = 0; j < 4; j++)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[j], fq[i], acc[i][j], 0, 0, 0);
        }
    }
    // lane l holds outputs 4 (l / 16) .. + 3 of row l % 16 of each 16 x 16 piece
    const float* ws = a.w_scales + uint64_t(expert) * a.outputs;
#pragma unroll
    for (uint32_t i = 0; i < 4; i++) {
        const uint32_t r = wm + 16 * i + (lane & 15);
        if (r >= rows) continue;
        const float scale = a.scales[row0 + r];
#pragma unroll
        for (uint32_t j = 0; j < 4; j++) {
            const uint32_t n = n0 + wn + 16 * j + 4 * (lane >> 4);
            if (n < a.outputs) store4(a, row0 + r, n, acc[i][j], scale, ws);
        }
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

uint64_t product_workgroups(const ProductArgs& a)
{
    return most_tiles(a, kTileRows) * ((a.outputs + kTileOuts - 1) / kTileOuts);
}

hipError_t launch_experts_product(const ProductArgs& a, hipStream_t s)
{
    hipLaunchKernelGGL(product_kernel, dim3(uint32_t(product_workgroups(a))), dim3(kTileThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace zc
