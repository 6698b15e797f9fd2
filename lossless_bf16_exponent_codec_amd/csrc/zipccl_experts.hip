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
#include "zipccl_row_tiles.h"

namespace zc {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));

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

// Running maximum, in both halves, of magnitudes as BF16 bits without sign (bits order as
// magnitudes do, infinities and NaNs above every finite value).
typedef uint16_t Half2 __attribute__((ext_vector_type(2)));

__device__ inline Half2 larger(Half2 m, uint4 v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; j++) m = __builtin_elementwise_max(m, __builtin_bit_cast(Half2, w[j] & 0x7FFF7FFFu));
    return m;
}

// How a row of largest magnitude `most` is scaled.  n = x * up * factor is 127 x times the
// power of two that brings `most` into [1, 2), exact (15 significant bits; values that
// underflow on the way quantise to 0 in any case); `up` is 2^64 for rows so small that
// the factor alone would overflow.
struct RowScale {
    float up = 1.0f, factor = 0.0f, peak = 1.0f, inverse = 0.0f, scale;

    __device__ inline RowScale(uint32_t most_bits)
    {
        const float most = __uint_as_float(most_bits << 16);
        scale = most_bits < 0x7F80u ? most / 127.0f : __uint_as_float(0x7FC00000u);
        if (most_bits == 0 || most_bits >= 0x7F80u) return;   // q = 0
        int e;
        peak = 2.0f * frexpf(most, &e);
        inverse = 1.0f / peak;
        if (e < -100) {
            up = 0x1p64f;
            e += 64;
        }
        factor = ldexpf(127.0f, 1 - e);
    }

    // The quotient n / peak to the nearest fp32 (reciprocal, product, one correction by
    // the remainder), then to the nearest even whole number by adding 1.5 * 2^23, whose
    // low byte is then q's.
    __device__ inline uint32_t quantize(float x) const
    {
        const float n = x * factor, y = n * inverse;
        return __float_as_uint(fmaf(fmaf(-y, peak, n), inverse, y) + 12582912.0f);
    }

    __device__ inline uint2 quantize8(uint4 v) const
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t q[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            float x = __uint_as_float(j & 1 ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
            // a NaN or infinity has no place in a row that is not zeroed; the row's factor is 0 then
            if (up != 1.0f) x *= up;
            q[j] = quantize(x);
        }
        // low bytes of four: pairs, then pairs of pairs
        const auto four = [](const uint32_t* b) {
            return __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400u),
                                         __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), 0x05040100u);
        };
        return make_uint2(four(q), four(q + 4));
    }
};

// Bound by memory: 16384 x 7168 takes 69 us, 5.1 TB/s of the 352 MB it reads and writes (a
// plain copy reaches 5.0), 86 us when each row was read twice (the second time from L2)
// and rounded and packed value by value.
//
// A group of kWaves waves per token.  kHeld: chunks of 8 values per lane that stay in
// registers between the maximum and the quantisation (the row is read once); 0: rows of
// any length, read twice.
template <uint32_t kWaves, uint32_t kHeld>
__global__ __launch_bounds__(kQuantThreads) void quantize_rows_kernel(const QuantArgs a)
{
    constexpr uint32_t kTokens = kQuantWaves / kWaves, kStride = 8 * 64 * kWaves;
    __shared__ uint32_t s_peak[kQuantWaves];
    const uint32_t lane = lane_id();
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t first = 8 * (64 * (wave % kWaves) + lane);
    const uint32_t padded = (a.row_len + kQuantPad - 1) / kQuantPad * kQuantPad;
    for (uint64_t t0 = uint64_t(blockIdx.x) * kTokens; t0 < a.tokens; t0 += uint64_t(gridDim.x) * kTokens) {
        const uint64_t token = t0 + wave / kWaves;
        if (kWaves == 1 && token >= a.tokens) break;
        const uint16_t* row = a.x + token * a.x_stride;
        uint4 held[kHeld > 0 ? kHeld : 1];
        Half2 both = {0, 0};
        if constexpr (kHeld > 0) {
#pragma unroll
            for (uint32_t j = 0; j < kHeld; j++) held[j] = load8(row, first + j * kStride, a.row_len);
        }
        // lane k: slot of choice k (kMaxTopK lanes)
        int32_t slot = a.slots || lane > 0 ? -1 : int32_t(token);
        if (a.slots && lane < a.top_k) slot = a.slots[token * a.top_k + lane];
        if (slot >= int32_t(a.nrows)) {
            set_status(a.status, ZIPCCL_STATUS_BAD_INDEX);
            slot = -1;
        }
        if constexpr (kHeld > 0) {
#pragma unroll
            for (uint32_t j = 0; j < kHeld; j++) both = larger(both, held[j]);
        } else {
            for (uint32_t h = first; h < a.row_len; h += kStride) both = larger(both, load8(row, h, a.row_len));
        }
        uint32_t most = max(both.x, both.y);
        for (uint32_t d = 32; d > 0; d >>= 1) most = max(most, uint32_t(__shfl_xor(int(most), int(d))));
        if constexpr (kWaves > 1) {
            __syncthreads();
            if (lane == 0) s_peak[wave] = most;
            __syncthreads();
#pragma unroll
            for (uint32_t w = 0; w < kQuantWaves; w++) most = max(most, s_peak[w]);
        }
        const bool zero = most == 0 || most >= 0x7F80u;
        const RowScale to(__builtin_amdgcn_readfirstlane(most));
        const auto put = [&](uint32_t h, uint4 v) {
            const uint2 q = zero ? make_uint2(0, 0) : to.quantize8(v);
            for (uint32_t k = 0; k < a.top_k; k++) {
                const int32_t s = __builtin_amdgcn_readlane(slot, k);
                if (s < 0) continue;
                uint8_t* at = reinterpret_cast<uint8_t*>(a.q) + uint64_t(uint32_t(s)) * a.q_stride + h;
                if (h < padded) *reinterpret_cast<uint2*>(at) = q;
            }
        };
        if constexpr (kHeld > 0) {
#pragma unroll
            for (uint32_t j = 0; j < kHeld; j++) put(first + j * kStride, held[j]);
        } else {
            for (uint32_t h0 = 0; h0 < padded; h0 += kStride) put(first + h0, load8(row, first + h0, a.row_len));
        }
        if (wave % kWaves == 0 && slot >= 0) a.scales[slot] = to.scale;
    }
}

// ------------------------------------------------------------------------------------
// Experts' product
// ------------------------------------------------------------------------------------

// Whether sums times a row's scale are finite: no product of 31 bits and a scale below 2^96
// is infinite.
__device__ inline bool tame(float scale) { return fabsf(scale) < 0x1p96f; }

// 8 consecutive outputs from n on: a row's scaled sums times the weights' scales, rounded
// and stored.
struct Outputs {
    float ws[8];
    uint32_t n, count;

    __device__ inline Outputs(const ProductArgs& a, uint32_t expert, uint32_t first)
        : n(first), count(first < a.outputs ? min(8u, a.outputs - first) : 0u)
    {
        const float* from = a.w_scales + uint64_t(expert) * a.outputs;
#pragma unroll
        for (uint32_t r = 0; r < 8; r++) ws[r] = from[min(n + r, a.outputs - 1)];   // no use of a value, so no wait, here
    }

    // v: sum * row scale
    __device__ inline void store(const ProductArgs& a, uint32_t row, v4f lo, v4f hi) const
    {
        const uint64_t at = uint64_t(row) * a.out_stride + n;
        float f[8];
#pragma unroll
        for (uint32_t r = 0; r < 8; r++) f[r] = (r < 4 ? lo[r & 3] : hi[r & 3]) * ws[r];
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
            for (uint32_t r = 0; r < 4; r++) b[r] = bf16_pair(f[2 * r], f[2 * r + 1]);
            if (count == 8) {
                __builtin_memcpy(o, b, 16);
            } else {
#pragma unroll
                for (uint32_t r = 0; r < 7; r++)
                    if (r < count) o[r] = uint16_t(b[r >> 1] >> (16 * (r & 1)));
            }
        }
    }

    // Whether these scales are finite, so that outputs of tame rows are no NaNs.
    __device__ inline bool finite() const
    {
        bool all = true;
#pragma unroll
        for (uint32_t r = 0; r < 8; r++) all &= fabsf(ws[r]) < __builtin_inff();
        return all;
    }

    // After `store` in BF16: NaNs of any sign and payload as the one NaN that every operator
    // writes.  A second look at what was stored keeps the compares out of the loops that store
    // (16384 x 4096: 0.5 to 1.8 % of the product's time there).
    __device__ inline void one_nan(const ProductArgs& a, uint32_t row) const
    {
        uint16_t* o = reinterpret_cast<uint16_t*>(a.out) + uint64_t(row) * a.out_stride + n;
        for (uint32_t r = 0; r < count; r++)
            if ((o[r] & 0x7FFFu) > 0x7F80u) o[r] = 0x7FC0u;
    }
};

// All waves: n loads may still be in flight (the older ones have landed), no LDS read is,
// and nothing moves across.
template <uint32_t N>
__device__ inline void wait_loads_and_meet()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The same for one wave alone.
template <uint32_t N>
__device__ inline void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// All waves: no LDS read is in flight.
__device__ inline void wait_reads_and_meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

typedef __attribute__((address_space(1))) const void global_void;
typedef __attribute__((address_space(3))) void lds_void;

// 16 bytes per lane from global memory to LDS: lane l's land at `to` + 16 l.
__device__ inline void load_lds(const int8_t* from, uint8_t* to)
{
    __builtin_amdgcn_global_load_lds((global_void*)from, (lds_void*)to, 16, 0, 0);
}

// Order of issue: `kProducts` matrix instructions and kOthers of one kind (0x100 LDS
// reads, 0x020 loads) taking turns.
template <int kProducts, int kOthers, int kKind, int kAt = 0>
__device__ inline void take_turns()
{
    if constexpr (kAt < kOthers) {
        constexpr int n = (kAt + 1) * kProducts / kOthers - kAt * kProducts / kOthers;
        if constexpr (n > 0) __builtin_amdgcn_sched_group_barrier(0x008, n, 0);
        __builtin_amdgcn_sched_group_barrier(kKind, 1, 0);
        take_turns<kProducts, kOthers, kKind, kAt + 1>();
    }
}

constexpr uint32_t kTileThreads = 256;
constexpr uint32_t kSlab = kQuantPad;   // values of a row per step

// LDS of a tile of 64 kM rows x 64 kN outputs.
constexpr uint32_t slot_bytes(uint32_t m, uint32_t n) { return 64 * (m + n) * kSlab; }
constexpr uint32_t tile_lds(uint32_t m, uint32_t n, uint32_t slots) { return slots * slot_bytes(m, n); }

// A tile of up to 64 kM rows x 64 kN outputs by 4 waves, each 32 kM x 32 kN.
//
// The rows go through LDS in slabs of 128 values (whole 128-byte lines: requests of 64
// bytes kept the L2's channels busy twice as long), kSlots slabs in a ring.  A wave holds
// the first half of slab s in registers when the step begins.  It reads the second half
// while it multiplies the first; then, slab s being free, it requests slab s + kSlots
// into its place while it multiplies on, and, slab s + 1 having landed, reads that one's
// first half.  Loads are issued one per two matrix instructions: a wave's load keeps the
// CU's address path busy for 16 cycles, a matrix instruction its SIMD for 32, and at one
// load per instruction of each of the four waves the loads held the products up
// (256 x 256 x 7168, zeros: 3540 TOP/s at one per product, 4030 at one per two).
//
// What bounds a large tile is power: 16384 x 4096 x 7168 with quantised Gaussian values
// takes 383-403 us (2.4-2.5 POP/s); the same with zeros, whose bits do not switch, would
// take 240, and the matrix instructions alone with the real values 287.  A library product
// of the same shape without scales takes 408.  A loop with a deeper prefetch (later slabs
// into L2 by small loads) was no faster.  Few rows are bound by the weights' bytes: 256
// choices over 32 skewed experts, 2048 x 7168, take 77 us, 5.6 TB/s.
template <uint32_t kM, uint32_t kN, uint32_t kSlots>
__device__ inline void product_tile(const ProductArgs& a, uint8_t* s_ring, uint32_t expert, uint32_t row0,
                                    uint32_t rows, uint32_t n0)
{
    constexpr uint32_t kRows = 64 * kM, kSlot = slot_bytes(kM, kN);
    constexpr uint32_t kLoads = 2 * (kM + kN), kEarly = kLoads / 2;   // loads of a thread per slab
    constexpr uint32_t kProducts = kM * kN;                           // products of a quarter slab
    constexpr uint32_t kPerRow = 4 * kN;                              // lanes that store a row of a wave
    const uint32_t lane = lane_id();
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int8_t* q = a.q + uint64_t(row0) * a.q_stride;
    const int8_t* w = a.w + (uint64_t(expert) * a.outputs + n0) * a.w_stride;

    // A load of a wave fills 8 rows of 128 bytes.  The 16-byte pieces of a row are swapped
    // by bits 1-3 of the row, so that 16 lanes reading one piece of 16 rows use every
    // bank.  Rows past the tile's end repeat its last one and are not stored.
    uint32_t from[kLoads];
    const uint32_t r = 8 * wave + lane / 8, piece = (lane & 7) ^ ((r >> 1) & 7);
#pragma unroll
    for (uint32_t i = 0; i < kLoads; i++)
        from[i] = (i < 2 * kM ? min(r + 32 * i, rows - 1) * uint32_t(a.q_stride)
                              : min(r + 32 * (i - 2 * kM), a.outputs - 1 - n0) * uint32_t(a.w_stride)) + 16 * piece;
    const auto load = [&](uint32_t slab, uint32_t first, uint32_t end) {
        const uint32_t at = min(slab, a.slabs - 1) * kSlab;   // past the end: the last slab again, never used
        uint8_t* to = s_ring + slab % kSlots * kSlot + 1024 * wave;
#pragma unroll
        for (uint32_t i = first; i < end; i++) load_lds((i < 2 * kM ? q : w) + at + from[i], to + 4096 * i);
    };

    const uint32_t wm = (wave >> 1) * 32 * kM, wn = (wave & 1) * 32 * kN;
    const uint32_t half = lane >> 5, turn = (lane >> 1) & 7;
    const uint8_t* read_q = s_ring + (wm + (lane & 31)) * kSlab;
    const uint8_t* read_w = s_ring + (kRows + wn + (lane & 31)) * kSlab;
    // Quarters of a slab (32 values) that a set of registers holds: two, or all four (one
    // barrier per slab) where the tile is small and the ring deep enough.
    constexpr uint32_t kHeld = kM * kN > 4 || kSlots < 3 ? 2 : 4;
    v16i acc[kM][kN] = {};
    v4i fq[2][kHeld][kM], fw[2][kHeld][kN];
    const auto read = [&](uint32_t to, uint32_t slab, uint32_t first) {   // quarters first .. into registers `to`
        const uint32_t slot = slab % kSlots * kSlot;
#pragma unroll
        for (uint32_t k = 0; k < kHeld; k++) {
            const uint32_t at = slot + ((2 * (first + k) + half) ^ turn) * 16;
#pragma unroll
            for (uint32_t i = 0; i < kM; i++) fq[to][k][i] = *reinterpret_cast<const v4i*>(read_q + at + 32 * kSlab * i);
#pragma unroll
            for (uint32_t j = 0; j < kN; j++) fw[to][k][j] = *reinterpret_cast<const v4i*>(read_w + at + 32 * kSlab * j);
        }
    };
    const auto multiply = [&](uint32_t u, uint32_t k) {
#pragma unroll
        for (uint32_t i = 0; i < kM; i++)
#pragma unroll
            for (uint32_t j = 0; j < kN; j++)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[u][k][j], fq[u][k][i], acc[i][j], 0, 0, 0);
    };
#pragma unroll
    for (uint32_t s = 0; s < kSlots; s++) load(s, 0, kLoads);
    // the scales this lane needs at the end, requested now
    float scale[kM];
#pragma unroll
    for (uint32_t i = 0; i < kM; i++) scale[i] = a.scales[row0 + min(wm + 32 * i + (lane & 31), rows - 1)];
    const uint32_t n = n0 + wn + 8 * (lane % kPerRow);   // the 8 outputs it stores of each row
    const Outputs to(a, expert, n);
    wait_loads_and_meet<(kSlots - 1) * kLoads>();
    read(0, 0, 0);
    if constexpr (kHeld == 4) {
        for (uint32_t s0 = 0; s0 < a.slabs; s0 += 2) {
#pragma unroll
            for (uint32_t u = 0; u < 2; u++) {
                const uint32_t s = s0 + u;
                // slab s is in every wave's registers, slab s + 1 has landed
                wait_loads_and_meet<(kSlots - 2) * kLoads>();
                if (s >= a.slabs) break;
                read(u ^ 1, s + 1, 0);
                load(s + kSlots, 0, kLoads);
#pragma unroll
                for (uint32_t k = 0; k < 4; k++) multiply(u, k);
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                take_turns<2 * kProducts, 4 * (kM + kN), 0x100>();
                take_turns<2 * kProducts, kLoads, 0x020>();
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    } else {
        for (uint32_t s = 0; s < a.slabs; s++) {
            read(1, s, 2);
            multiply(0, 0);
            take_turns<kProducts / 2 + 1, kLoads, 0x100>();
            __builtin_amdgcn_sched_barrier(0);
            wait_reads_and_meet();
            load(s + kSlots, 0, kEarly);
            multiply(0, 1);
            take_turns<kProducts, kEarly, 0x020>();
            __builtin_amdgcn_sched_barrier(0);
            wait_loads_and_meet<(kSlots - 2) * kLoads + kEarly>();
            load(s + kSlots, kEarly, kLoads);
            read(0, s + 1, 0);
            multiply(1, 0);
            multiply(1, 1);
            take_turns<kProducts, kLoads - kEarly, 0x020>();
            take_turns<kProducts / 2 + 1, kLoads, 0x100>();
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // Lane l holds, of each 32 x 32 piece, row l % 32 and outputs 8 g + 4 (l / 32) .. + 3.
    // Strips of 32 rows change hands in the wave's own part of LDS so that a lane gets 8
    // outputs in a row and a store covers whole rows of the wave's outputs.
    constexpr uint32_t kPitch = 32 * kN * 4 + 16;       // bytes; the 16 spread rows over the banks
    static_assert(4 * 32 * kPitch <= kSlots * kSlot, "strips fit the ring");
    wait_loads_and_meet<0>();   // the surplus loads have landed and every wave is done reading: the ring is free
    uint8_t* strip = s_ring + wave * (32 * kPitch);
#pragma unroll
    for (uint32_t i = 0; i < kM; i++) {
        if (wm + 32 * i >= rows) break;
#pragma unroll
        for (uint32_t j = 0; j < kN; j++)
#pragma unroll
            for (uint32_t g = 0; g < 4; g++) {
                const v4f v = {float(acc[i][j][4 * g]) * scale[i], float(acc[i][j][4 * g + 1]) * scale[i],
                               float(acc[i][j][4 * g + 2]) * scale[i], float(acc[i][j][4 * g + 3]) * scale[i]};
                *reinterpret_cast<v4f*>(strip + (lane & 31) * kPitch + (32 * j + 8 * g + 4 * half) * 4) = v;
            }
        __builtin_amdgcn_wave_barrier();
#pragma unroll 4
        for (uint32_t at = lane / kPerRow; at < 32; at += 64 / kPerRow) {
            const uint32_t row = wm + 32 * i + at;
            if (row >= rows) break;
            const v4f* v = reinterpret_cast<const v4f*>(strip + at * kPitch + 32 * (lane % kPerRow));
            to.store(a, row0 + row, v[0], v[1]);
        }
        __builtin_amdgcn_wave_barrier();
    }

    if (a.fp32) return;
    // the lanes of a wave hold the scales of all its rows and outputs
    bool plain = to.finite();
#pragma unroll
    for (uint32_t i = 0; i < kM; i++) plain &= tame(scale[i]);
    if (__all(plain)) return;
#pragma unroll 1
    for (uint32_t at = wm + lane / kPerRow; at < min(wm + 32 * kM, rows); at += 64 / kPerRow) to.one_nan(a, row0 + at);
}

template <uint32_t kM, uint32_t kN, uint32_t kSlots, uint32_t kPerCu>
__global__ __launch_bounds__(kTileThreads, kPerCu) void product_tile_kernel(const ProductArgs a)
{
    extern __shared__ __attribute__((aligned(1024))) uint8_t s_ring[];
    RowTiles<64 * kM, ProductArgs> map(a);
    const uint32_t across = (a.outputs + 64 * kN - 1) / (64 * kN), down = map.count(a);
    const uint32_t t = run_of_xcd(blockIdx.x, down * across);
    if (t >= down * across) return;
    uint32_t row_tile, column, expert, row0, rows;
    tile_at(t, down, across, row_tile, column);
    if (!map.find(a, row_tile, expert, row0, rows)) return;
    product_tile<kM, kN, kSlots>(a, s_ring, expert, row0, rows, 64 * kN * column);
}

// Tiles of 256 x 256, one workgroup per CU.  Where the tiles past the last whole round of
// the 256 CUs are half a round or less, each is cut into four of 128 x 128, so that the
// last round takes a part of a tile's time (1 expert, 4096 x 7168: 352 tiles, 96 over, 167
// us and 184 uncut; 1120 tiles, 96 over, 474 and 494).
constexpr uint32_t kCus = 256, kCutTiles = kCus / 2;

__global__ __launch_bounds__(kTileThreads, 1) void product_large_kernel(const ProductArgs a)
{
    extern __shared__ __attribute__((aligned(1024))) uint8_t s_ring[];
    RowTiles<256, ProductArgs> map(a);
    const uint32_t across = (a.outputs + 255) / 256, down = map.count(a), total = down * across;
    const uint32_t left = total % kCus;
    const uint32_t whole = left <= kCutTiles ? total - left : total;   // the tiles not cut
    const uint32_t first_cut = (whole + kXcds - 1) / kXcds * kXcds;    // the workgroups that share `whole` tiles
    const bool cut = blockIdx.x >= first_cut;
    const uint32_t parts = 4 * (total - whole);
    const uint32_t p = cut ? run_of_xcd(blockIdx.x - first_cut, parts) : run_of_xcd(blockIdx.x, whole);
    if (p >= (cut ? parts : whole)) return;
    uint32_t row_tile, column, expert, row0, rows;
    tile_at(cut ? whole + p / 4 : p, down, across, row_tile, column);
    if (!map.find(a, row_tile, expert, row0, rows)) return;
    if (!cut) {
        product_tile<4, 4, 2>(a, s_ring, expert, row0, rows, 256 * column);
        return;
    }
    const uint32_t r = 128 * (p & 1), n0 = 256 * column + 64 * (p & 2);
    if (r < rows && n0 < a.outputs) product_tile<2, 2, 4>(a, s_ring, expert, row0 + r, min(rows - r, 128u), n0);
}

// A tile of up to 64 rows x 32 outputs per workgroup, the row length split over its 4
// waves: for calls whose tiles do not fill the GPU, where the time is that of one tile's
// chain of steps.  Each wave has a ring of its own and meets no other until the end, when
// the 4 partial sums (whole numbers: in any order) are joined through LDS.  1 to 64 rows of
// one expert, 2048 x 7168: 9.7 us (64 x 64 tiles whose waves share a slab and meet at each
// one: 13.4 to 18); 8 rows of 8 experts, 1024 x 2048: 5.5 us.
constexpr uint32_t kSplitOuts = 32, kSplitSlots = 3;
constexpr uint32_t kSplitSlot = (64 + kSplitOuts) * kSlab, kSplitWaves = kTileThreads / 64;
constexpr uint32_t kSplitLds = kSplitWaves * kSplitSlots * kSplitSlot;

__global__ __launch_bounds__(kTileThreads, 1) void product_split_kernel(const ProductArgs a)
{
    constexpr uint32_t kLoads = kSplitSlot / 1024, kPitch = kSplitOuts + 4;   // pitch: values of a row of sums
    extern __shared__ __attribute__((aligned(1024))) uint8_t s_ring[];
    const uint32_t across = (a.outputs + kSplitOuts - 1) / kSplitOuts;
    uint32_t expert, row0, rows;
    RowTiles<64, ProductArgs> map(a);
    if (a.experts > 64 && blockIdx.x == 0) map.count(a);   // one workgroup looks at every offset, for the status
    if (!map.find(a, blockIdx.x / across, expert, row0, rows)) return;
    const uint32_t n0 = blockIdx.x % across * kSplitOuts;
    const uint32_t tid = threadIdx.x, lane = lane_id();
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int8_t* q = a.q + uint64_t(row0) * a.q_stride;
    const int8_t* w = a.w + (uint64_t(expert) * a.outputs + n0) * a.w_stride;
    uint8_t* ring = s_ring + wave * kSplitSlots * kSplitSlot;

    // what the end needs, requested now: thread t stores outputs 8 (t % 4) .. of row t / 4
    const uint32_t out_row = tid / 4;
    const float scale = a.scales[row0 + min(out_row, rows - 1)];
    const Outputs to(a, expert, n0 + 8 * (tid & 3));

    // the same arrangement of rows and pieces as in product_tile
    uint32_t from[kLoads];
#pragma unroll
    for (uint32_t i = 0; i < kLoads; i++) {
        const uint32_t r = 8 * i + lane / 8, piece = (lane & 7) ^ ((r >> 1) & 7);
        from[i] = (i < 8 ? min(r, rows - 1) * uint32_t(a.q_stride)
                         : min(r - 64, a.outputs - 1 - n0) * uint32_t(a.w_stride)) + 16 * piece;
    }
    const uint32_t per = (a.slabs + kSplitWaves - 1) / kSplitWaves;
    const uint32_t first = min(wave * per, a.slabs), end = min(first + per, a.slabs);
    const auto load = [&](uint32_t s) {
        const uint32_t at = min(s, a.slabs - 1) * kSlab;
        uint8_t* slot = ring + (s - first) % kSplitSlots * kSplitSlot;
#pragma unroll
        for (uint32_t i = 0; i < kLoads; i++) load_lds((i < 8 ? q : w) + at + from[i], slot + 1024 * i);
    };
    v16i acc[2] = {};
    v4i fq[2][4][2], fw[2][4];
    const uint32_t half = lane >> 5, turn = (lane >> 1) & 7;
    const auto read = [&](uint32_t to, uint32_t s) {
        const uint8_t* slot = ring + (s - first) % kSplitSlots * kSplitSlot + (lane & 31) * kSlab;
#pragma unroll
        for (uint32_t k = 0; k < 4; k++) {
            const uint32_t at = ((2 * k + half) ^ turn) * 16;
            fq[to][k][0] = *reinterpret_cast<const v4i*>(slot + at);
            fq[to][k][1] = *reinterpret_cast<const v4i*>(slot + at + 32 * kSlab);
            fw[to][k] = *reinterpret_cast<const v4i*>(slot + at + 64 * kSlab);
        }
    };
    if (first < end) {
#pragma unroll
        for (uint32_t s = 0; s < kSplitSlots; s++) load(first + s);
        wait_loads<(kSplitSlots - 1) * kLoads>();
        read(0, first);
        for (uint32_t s0 = first; s0 < end; s0 += 2) {
#pragma unroll
            for (uint32_t u = 0; u < 2; u++) {
                const uint32_t s = s0 + u;   // a surplus odd step reads a surplus slab and is not added
                wait_loads<(kSplitSlots - 2) * kLoads>();   // slab s is in registers, slab s + 1 has landed
                read(u ^ 1, s + 1);
                load(s + kSplitSlots);
                if (s < end) {
#pragma unroll
                    for (uint32_t k = 0; k < 4; k++) {
                        acc[0] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[u][k], fq[u][k][0], acc[0], 0, 0, 0);
                        acc[1] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[u][k], fq[u][k][1], acc[1], 0, 0, 0);
                    }
                }
            }
        }
    }
    wait_loads_and_meet<0>();
    int32_t* sums = reinterpret_cast<int32_t*>(s_ring);   // [wave][row][kPitch]
#pragma unroll
    for (uint32_t i = 0; i < 2; i++)
#pragma unroll
        for (uint32_t g = 0; g < 4; g++) {
            const v4i v = {acc[i][4 * g], acc[i][4 * g + 1], acc[i][4 * g + 2], acc[i][4 * g + 3]};
            *reinterpret_cast<v4i*>(sums + (wave * 64 + 32 * i + (lane & 31)) * kPitch + 8 * g + 4 * half) = v;
        }
    __syncthreads();
    if (out_row < rows) {
        v4i lo = {}, hi = {};
#pragma unroll
        for (uint32_t v = 0; v < kSplitWaves; v++) {
            const v4i* at = reinterpret_cast<const v4i*>(sums + (v * 64 + out_row) * kPitch + 8 * (tid & 3));
            lo += at[0];
            hi += at[1];
        }
        to.store(a, row0 + out_row, __builtin_convertvector(lo, v4f) * scale, __builtin_convertvector(hi, v4f) * scale);
        if (!a.fp32 && !(to.finite() && tame(scale))) to.one_nan(a, row0 + out_row);
    }
}

}  // namespace

hipError_t launch_quantize_rows(const QuantArgs& a, hipStream_t s)
{
    const auto run = [&](auto kernel, uint32_t tokens) {   // tokens of a workgroup
        const uint64_t groups = (a.tokens + tokens - 1) / tokens;
        hipLaunchKernelGGL(kernel, dim3(uint32_t(groups < (1u << 20) ? groups : 1u << 20)), dim3(kQuantThreads), 0, s, a);
    };
    const uint32_t padded = (a.row_len + kQuantPad - 1) / kQuantPad * kQuantPad;
    if (padded <= 2048 && a.tokens >= 1024) run(quantize_rows_kernel<1, 4>, 4);
    else if (padded <= 4 * 2048) run(quantize_rows_kernel<4, 4>, 1);
    else run(quantize_rows_kernel<4, 0>, 1);
    return hipGetLastError();
}

namespace {

uint64_t columns(const ProductArgs& a, uint32_t outs) { return (a.outputs + outs - 1) / outs; }

template <uint32_t kM, uint32_t kN>
uint64_t tile_workgroups(const ProductArgs& a)
{
    return (most_tiles(a, 64 * kM) * columns(a, 64 * kN) + kXcds - 1) / kXcds * kXcds;
}

template <uint32_t kM, uint32_t kN, uint32_t kSlots, uint32_t kPerCu>
hipError_t launch_tiles(const ProductArgs& a, hipStream_t s)
{
    constexpr uint32_t lds = tile_lds(kM, kN, kSlots);
    if (hipError_t e = allow_lds<product_tile_kernel<kM, kN, kSlots, kPerCu>>(lds)) return e;
    hipLaunchKernelGGL((product_tile_kernel<kM, kN, kSlots, kPerCu>), dim3(uint32_t(tile_workgroups<kM, kN>(a))), dim3(kTileThreads), lds, s, a);
    return hipGetLastError();
}

// most_tiles bounds the whole tiles; cutting the last ones adds 3 workgroups for each
uint64_t large_workgroups(const ProductArgs& a) { return tile_workgroups<4, 4>(a) + 3 * kCutTiles; }

uint64_t split_workgroups(const ProductArgs& a) { return most_tiles(a, 64) * columns(a, kSplitOuts); }

// Which kernel, by the tiles that rows spread evenly over the experts would make (the
// host does not know the offsets).  Times in us, weights outputs x row_len:
//  - one round of split workgroups or less: split (1 expert, 64 rows, 2048 x 7168: 9.7
//    against 13.4 for 64 x 64 tiles; 8 experts, two rounds: 29.9 and 22.3);
//  - up to 64 rows for an expert the weights' reads are what counts.  Few tiles of 64 x 64:
//    four slabs deep while a CU has no second workgroup to run meanwhile (8 experts, 2048 x
//    7168: 20 and 26 at two), else two slabs and four workgroups (16 experts: 35 and 35).
//    Many: 64 x 128, which read the rows half as often (256 choices over 32 skewed
//    experts, 2048 x 7168: 78 against 94 at 64 x 64; 1024 over 128: 279 and 286);
//  - 256 x 256 from 192 rows on when there is a round of it (8 experts, 2048 rows each,
//    2048 x 7168: 212 against 246 at 128 x 128; 512 rows each, half a round: 78 and 62), rows
//    are long enough to make up for one workgroup per CU, which starts and ends alone (1
//    expert, 16384 rows, 2048 outputs: 37.9 against 29.5 at row_len 256, 80.7 and 82.0 at
//    2048, 111 and 120 at 3328), and the last column is not mostly empty (8 experts, 4096
//    rows each, 600 x 4096: 106 and 92);
//  - else 128 x 128 (32 experts, 128 rows each, 2048 x 7168: 105, 148 at 64 x 64), or 64 x
//    128 where those would leave too many CUs idle (1 expert, 512 rows, 4096 x 2048, 128
//    tiles: 12.3 and 10.0; 700 rows, 192 tiles: 12.8 and 14.3).
enum class Shape { split, narrow_deep, narrow, wide, square, large };

Shape choose(const ProductArgs& a)
{
    const uint64_t parts = a.experts < a.rows ? a.experts : a.rows, each = (a.rows + parts - 1) / parts;
    const auto tiles = [&](uint32_t rows, uint32_t outs) { return parts * ((each + rows - 1) / rows) * columns(a, outs); };
    if (tiles(64, kSplitOuts) <= kCus) return Shape::split;
    if (each <= 64) {
        const uint64_t n = tiles(64, 64);
        return n <= kCus + kCus / 2 ? Shape::narrow_deep : n <= 3 * kCus ? Shape::narrow : Shape::wide;
    }
    const bool fits = 9 * 2 * columns(a, 256) <= 10 * columns(a, 128);   // outputs left empty at 256, and at 128
    if (each >= 192 && a.slabs >= 16 && fits && tiles(256, 256) >= kCus) return Shape::large;
    return tiles(128, 128) <= kCus * 5 / 8 ? Shape::wide : Shape::square;
}

}  // namespace

uint64_t product_workgroups(const ProductArgs& a)
{
    switch (choose(a)) {
        case Shape::split: return split_workgroups(a);
        case Shape::large: return large_workgroups(a);
        case Shape::square: return tile_workgroups<2, 2>(a);
        case Shape::wide: return tile_workgroups<1, 2>(a);
        default: return tile_workgroups<1, 1>(a);
    }
}

hipError_t launch_experts_product(const ProductArgs& a, hipStream_t s)
{
    switch (choose(a)) {
        case Shape::narrow_deep: return launch_tiles<1, 1, 4, 2>(a, s);
        case Shape::narrow: return launch_tiles<1, 1, 2, 4>(a, s);
        case Shape::wide: return launch_tiles<1, 2, 2, 3>(a, s);
        case Shape::square: return launch_tiles<2, 2, 2, 2>(a, s);
        case Shape::split: {
            if (hipError_t e = allow_lds<product_split_kernel>(kSplitLds)) return e;
            hipLaunchKernelGGL(product_split_kernel, dim3(uint32_t(split_workgroups(a))), dim3(kTileThreads), kSplitLds,
                               s, a);
            break;
        }
        case Shape::large: {
            constexpr uint32_t lds = tile_lds(4, 4, 2);
            if (hipError_t e = allow_lds<product_large_kernel>(lds)) return e;
            hipLaunchKernelGGL(product_large_kernel, dim3(uint32_t(large_workgroups(a))), dim3(kTileThreads), lds, s, a);
            break;
        }
    }
    return hipGetLastError();
}

}  // namespace zc
