// A router's choices, weights and balance loss for gfx950.
//
// For a token t that takes part and has a logit above minus infinity, p[t] = softmax(z[t]).
//   choices   the top_k largest logits, the lowest expert among equals, minus infinity never
//   weights   p of a choice, or p over the sum of p over the choices
//   balance   counts c[e] of choices, sums s[e] = sum_t p[t][e], n tokens, and the loss
//             L = E / (K n^2) * sum_e c[e] s[e]
//   gradient  dz[e] = sum_{k: id_k = e} w_k (dw_k - sum_j w_j dw_j) for weights over the choices;
//             p_e (g_e - sum_j p_j g_j) for probabilities and the loss, with g_e the choice's dw
//             and dL E / (K n^2) c[e]
//
// Logits are read once, by a group of lanes per token that holds the row in registers.
// Values are fp32; sums over tokens are joined in a fixed order (lanes, waves, workgroups), the
// workgroups' in 64 bits, so a call gives the same bits on every run.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "zipccl.h"
#include "zipccl_moe_internal.h"
#include "zipccl_row_tiles.h"

namespace zc {

namespace {

// exp of x, the distance to the row's largest logit, by the hardware's exp2.  The power of two that
// it takes is rounded, by up to half a place of a number of |x|'s size; d is what that left out of x,
// and exp(d) is 1 + d in fp32.  Off by at most 2^-23 (exp2) and 2^-24 (the sum) of the value, and
// |x| 2^-28 for the constant's rounding.  Without d it was |x| 2^-24, for three instructions less.
// Past x's range d is no number or infinite, and kept from the exponential of 0.
__device__ inline float exp_of(float x)
{
    const float power = x * 1.44269504088896340736f, e = __builtin_amdgcn_exp2f(power);
    const float d = fmaf(power, -0.693147180559945309417f, x);
    return fmaf(e, fminf(d, 1.0f), e);
}

// What lanes of this wave wrote to LDS before can be read by its other lanes after.
__device__ inline void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A lane's partner in the step of a reduction that brings together runs of `kRun` lanes that
// agree already: lanes apart by 1, by 2, then mirrored within 8 and within 16.
template <int kRun>
__device__ inline uint32_t partner(uint32_t v)
{
    constexpr int kControl = kRun == 1 ? 0xB1 : kRun == 2 ? 0x4E : kRun == 4 ? 0x141 : 0x140;
    return uint32_t(__builtin_amdgcn_update_dpp(int(v), int(v), kControl, 0xF, 0xF, false));
}

// ---- keys: unsigned 32 bits in the order of the values, NaNs above all, both zeros alike ----
constexpr uint32_t kClosed = 0x007FFFFFu;    // minus infinity's; 0: a place without a value

__device__ inline uint32_t bits_of(float z)
{
    const uint32_t b = __float_as_uint(z + 0.0f);
    return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}

__device__ inline float value_of(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);   // a NaN's key gives a NaN
}

// A key with its expert, so that the largest is the one to choose and no two are equal.

// Of BF16 logits 16 bits are the key's: the expert (from 1023 down) takes the lower ones.
struct KeyBf16 {
    uint32_t v;
    __device__ inline KeyBf16() : v(0) {}
    __device__ inline KeyBf16(uint32_t key, uint32_t expert) : v((key & 0xFFFF0000u) | (0xFFFFu - expert)) {}
    __device__ inline uint32_t expert() const { return 0xFFFFu - (v & 0xFFFFu); }
    __device__ inline uint32_t key() const { return v & 0x80000000u ? v & 0xFFFF0000u : v | 0xFFFFu; }
    __device__ inline bool open() const { return v > (kClosed | 0xFFFFu); }
    __device__ inline bool same(KeyBf16 o) const { return v == o.v; }
    static __device__ inline KeyBf16 larger(KeyBf16 a, KeyBf16 b) { a.v = max(a.v, b.v); return a; }
    static __device__ inline KeyBf16 smaller(KeyBf16 a, KeyBf16 b) { a.v = min(a.v, b.v); return a; }
    static __device__ inline KeyBf16 either(bool first, KeyBf16 a, KeyBf16 b) { a.v = first ? a.v : b.v; return a; }
    template <int kRun> __device__ inline KeyBf16 turn() const { KeyBf16 k; k.v = partner<kRun>(v); return k; }
    __device__ inline KeyBf16 across(int mask) const { KeyBf16 k; k.v = uint32_t(__shfl_xor(int(v), mask)); return k; }
};

// Of fp32 ones the key and the expert lie in the mantissa of a number from 2 to 4, which the
// 64-bit maximum and minimum order in one instruction each.
struct KeyFp32 {
    double v;
    __device__ inline KeyFp32() : v(0.0) {}
    __device__ inline KeyFp32(uint32_t key, uint32_t expert)
        : v(__hiloint2double(int(0x40000000u | key >> 12), int(key << 20 | (0xFFFFFu - expert)))) {}
    __device__ inline uint32_t lo() const { return uint32_t(__double2loint(v)); }
    __device__ inline uint32_t hi() const { return uint32_t(__double2hiint(v)); }
    __device__ inline uint32_t expert() const { return 0xFFFFFu - (lo() & 0xFFFFFu); }
    __device__ inline uint32_t key() const { return hi() << 12 | lo() >> 20; }
    __device__ inline bool open() const { return hi() >= 0x40000000u && key() > kClosed; }
    __device__ inline bool same(KeyFp32 o) const { return lo() == o.lo(); }     // holds the expert
    static __device__ inline KeyFp32 larger(KeyFp32 a, KeyFp32 b)
    {
        asm("v_max_f64 %0, %1, %2" : "=v"(a.v) : "v"(a.v), "v"(b.v));
        return a;
    }
    static __device__ inline KeyFp32 smaller(KeyFp32 a, KeyFp32 b)
    {
        asm("v_min_f64 %0, %1, %2" : "=v"(a.v) : "v"(a.v), "v"(b.v));
        return a;
    }
    static __device__ inline KeyFp32 either(bool first, KeyFp32 a, KeyFp32 b)
    {
        a.v = __hiloint2double(first ? int(a.hi()) : int(b.hi()), first ? int(a.lo()) : int(b.lo()));
        return a;
    }
    template <int kRun> __device__ inline KeyFp32 turn() const
    {
        KeyFp32 k;
        k.v = __hiloint2double(int(partner<kRun>(hi())), int(partner<kRun>(lo())));
        return k;
    }
    __device__ inline KeyFp32 across(int mask) const
    {
        KeyFp32 k;
        k.v = __hiloint2double(__shfl_xor(int(hi()), mask), __shfl_xor(int(lo()), mask));
        return k;
    }
};

// The largest of a group's kLanes lanes, in every one of them.
template <uint32_t kLanes, class Key>
__device__ inline Key largest(Key k)
{
    k = Key::larger(k, k.template turn<1>());
    k = Key::larger(k, k.template turn<2>());
    if constexpr (kLanes > 4) k = Key::larger(k, k.template turn<4>());
    if constexpr (kLanes > 8) k = Key::larger(k, k.template turn<8>());
    if constexpr (kLanes == 64) {
        k = Key::larger(k, k.across(16));
        k = Key::larger(k, k.across(32));
    }
    return k;
}

// op over the kLanes lanes of a group, the same bits in every one of them.
template <uint32_t kLanes, class Op>
__device__ inline float across(float v, Op op)
{
    const auto with = [&](uint32_t o) { v = op(v, __uint_as_float(o)); };
    with(partner<1>(__float_as_uint(v)));
    with(partner<2>(__float_as_uint(v)));
    if constexpr (kLanes > 4) with(partner<4>(__float_as_uint(v)));
    if constexpr (kLanes > 8) with(partner<8>(__float_as_uint(v)));
    if constexpr (kLanes == 64) {
        with(uint32_t(__shfl_xor(int(__float_as_uint(v)), 16)));
        with(uint32_t(__shfl_xor(int(__float_as_uint(v)), 32)));
    }
    return v;
}

template <uint32_t kLanes>
__device__ inline float total(float v)
{
    return across<kLanes>(v, [](float a, float b) { return a + b; });
}

__device__ inline float larger(float a, float b)    // the one that is a number, if only one is
{
    float m;
    asm("v_max_f32 %0, %1, %2" : "=v"(m) : "v"(a), "v"(b));
    return m;
}

// Keys in descending order, by Batcher's odd-even merge exchange.
template <uint32_t kN, class Key>
__device__ inline void sort(Key* k)
{
#pragma unroll
    for (uint32_t p = 1; p < kN; p *= 2)
#pragma unroll
        for (uint32_t q = p; q > 0; q /= 2)
#pragma unroll
            for (uint32_t j = q % p; j + q < kN; j += 2 * q)
#pragma unroll
                for (uint32_t i = 0; i < q; i++)
                    if (i + j + q < kN && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const Key a = k[i + j], b = k[i + j + q];
                        k[i + j] = Key::larger(a, b);
                        k[i + j + q] = Key::smaller(a, b);
                    }
}

// The first kTop of kN keys in descending order (kTop kN, or 8 of 16).
template <uint32_t kN, uint32_t kTop, class Key>
__device__ inline void sort_top(Key* k)
{
    if constexpr (kTop == kN) {
        sort<kN>(k);
    } else {
        static_assert(kN == 16 && kTop == 8, "two halves");
        sort<8>(k);
        sort<8>(k + 8);
        // of two descending runs, one turned round, the larger ones are the upper half, and rise
        // and fall once: three rounds of exchanges sort them
#pragma unroll
        for (uint32_t i = 0; i < 8; i++) k[i] = Key::larger(k[i], k[15 - i]);
#pragma unroll
        for (uint32_t d = 4; d > 0; d /= 2)
#pragma unroll
            for (uint32_t i = 0; i < 8; i++)
                if ((i & d) == 0) {
                    const Key a = k[i], b = k[i + d];
                    k[i] = Key::larger(a, b);
                    k[i + d] = Key::smaller(a, b);
                }
    }
}

// How a row of up to kLanes * kPer values lies over a group's lanes: chunks of kWide
// neighbours, lane after lane, so that a lane's values are in the order of their experts.
template <uint32_t kLanes, uint32_t kPer>
struct Spread {
    static constexpr uint32_t kWide = kPer < 4 ? kPer : 4;
    static __device__ inline uint32_t first(uint32_t lane, uint32_t i) { return (i / kWide * kLanes + lane) * kWide; }
    static __device__ inline uint32_t expert(uint32_t lane, uint32_t i) { return first(lane, i) + i % kWide; }

    // z of a row: minus infinity past its end, which no load passes.  No lane branches: loads under
    // different lanes' branches wait for one another.
    static __device__ inline void load(float (&z)[kPer], const uint8_t* row, uint32_t lane, uint32_t n, bool fp32)
    {
        if (fp32) load_as<float>(z, reinterpret_cast<const float*>(row), lane, n);
        else load_as<uint16_t>(z, reinterpret_cast<const uint16_t*>(row), lane, n);
    }

    static __device__ inline float as_float(float v) { return v; }
    static __device__ inline float as_float(uint16_t v) { return __uint_as_float(uint32_t(v) << 16); }

    template <class T>
    static __device__ inline void load_as(float (&z)[kPer], const T* row, uint32_t lane, uint32_t n)
    {
        T v[kPer];
        if (n == kLanes * kPer) {
#pragma unroll
            for (uint32_t i = 0; i < kPer; i += kWide) __builtin_memcpy(&v[i], row + first(lane, i), sizeof(T) * kWide);
#pragma unroll
            for (uint32_t i = 0; i < kPer; i++) z[i] = as_float(v[i]);
        } else if (n >= kWide) {
            // a chunk that the row ends in is the row's last kWide values, moved down
#pragma unroll
            for (uint32_t i = 0; i < kPer; i += kWide) __builtin_memcpy(&v[i], row + min(first(lane, i), n - kWide), sizeof(T) * kWide);
#pragma unroll
            for (uint32_t i = 0; i < kPer; i += kWide) {
                const uint32_t e = first(lane, i), moved = e - min(e, n - kWide);
#pragma unroll
                for (uint32_t j = 0; j < kWide; j++) {
                    float x = as_float(v[i + j]);
#pragma unroll
                    for (uint32_t d = 1; d < kWide; d++)
                        if (j + d < kWide) x = moved == d ? as_float(v[i + j + d]) : x;
                    z[i + j] = e + j < n ? x : -__builtin_inff();
                }
            }
        } else {
#pragma unroll
            for (uint32_t i = 0; i < kPer; i++) v[i] = row[min(expert(lane, i), n - 1)];
#pragma unroll
            for (uint32_t i = 0; i < kPer; i++) z[i] = expert(lane, i) < n ? as_float(v[i]) : -__builtin_inff();
        }
    }

    static __device__ inline void store(const float (&v)[kPer], uint8_t* row, uint32_t lane, uint32_t n, bool fp32)
    {
#pragma unroll
        for (uint32_t i = 0; i < kPer; i += kWide) {
            const uint32_t e = first(lane, i);
            if (fp32) {
                float* at = reinterpret_cast<float*>(row) + e;
                if (e + kWide <= n) {
                    __builtin_memcpy(at, &v[i], 4 * kWide);
                } else {
#pragma unroll
                    for (uint32_t j = 0; j < kWide; j++)
                        if (e + j < n) at[j] = v[i + j];
                }
            } else {
                uint16_t* at = reinterpret_cast<uint16_t*>(row) + e;
                uint16_t b[kWide];
#pragma unroll
                for (uint32_t j = 0; j < kWide; j++)
                    b[j] = v[i + j] != v[i + j] ? 0x7FC0u : uint16_t(bf16_pair(v[i + j], 0.0f));
                if (e + kWide <= n) {
                    __builtin_memcpy(at, b, 2 * kWide);
                } else {
#pragma unroll
                    for (uint32_t j = 0; j < kWide; j++)
                        if (e + j < n) at[j] = b[j];
                }
            }
        }
    }
};

__device__ inline const uint8_t* row_of(const uint8_t* base, uint64_t token, uint64_t stride, bool fp32)
{
    return base + token * stride * (fp32 ? 4 : 2);
}

// A choice that the caller made; -1 for one that is dropped, bad where it is out of range.
__device__ inline int32_t given(const GateArgs& a, uint64_t token, uint32_t k, bool& bad)
{
    const uint64_t at = token * a.id_stride + k;
    const int64_t id = a.wide_ids ? static_cast<const int64_t*>(a.ids)[at] : static_cast<const int32_t*>(a.ids)[at];
    bad = id >= int64_t(a.num_experts);
    return id < 0 || bad ? -1 : int32_t(id);
}

// What a workgroup leaves in the workspace; behind it the words of the finish.
__device__ inline float* block_sums(const GateArgs& a) { return reinterpret_cast<float*>(a.workspace); }
__device__ inline uint32_t* block_counts(const GateArgs& a)
{
    return reinterpret_cast<uint32_t*>(a.workspace) + uint64_t(a.blocks) * a.num_experts;
}
__device__ inline uint32_t* block_tokens(const GateArgs& a) { return block_counts(a) + uint64_t(a.blocks) * a.num_experts; }
__device__ inline uint32_t* finish_ticket(const GateArgs& a) { return block_tokens(a) + kGateBlocks; }
__device__ inline double* finish_parts(const GateArgs& a) { return reinterpret_cast<double*>(block_tokens(a) + 2 * kGateBlocks); }
constexpr uint32_t kFinishColumns = 16;
static_assert(uint64_t(kGateBlocks) * 8 * kMaxExperts + 8 * kGateBlocks + 8 * (kMaxExperts / kFinishColumns) <= kGateWorkspace,
              "the workspace holds them");

__device__ inline float loss_of(const GateArgs& a, uint32_t tokens, double sum)
{
    const double n = double(tokens);
    return tokens ? float(double(a.num_experts) / (double(a.top_k) * n * n) * sum) : 0.0f;
}

// exp of z less the row's largest, in place, and their sum: 0 for a row without an open
// expert; a NaN or an infinity makes it a NaN.
template <uint32_t kLanes, uint32_t kPer>
__device__ inline float exps(float (&z)[kPer])
{
    float most = z[0];
#pragma unroll
    for (uint32_t i = 1; i < kPer; i++) most = larger(most, z[i]);
    most = across<kLanes>(most, [](float a, float b) { return larger(a, b); });
    const float base = most == -__builtin_inff() ? 0.0f : most;
    float sum = 0.0f;
#pragma unroll
    for (uint32_t i = 0; i < kPer; i++) {
        z[i] = exp_of(z[i] - base);
        sum += z[i];
    }
    return total<kLanes>(sum);
}

// Forward.  Key: the choices are made here, for logits of its type; void: they are given, and
// counted.  kTop: keys of a lane that can be chosen.
//
// A lane sorts its keys, then the lanes' firsts are compared top_k times and the one chosen
// taken off its lane's list.  Bound by the instructions: 16384 x 256 in fp32, 8 of them with the
// balance outputs, take 4096 waves of 1096, 7.3 of 12.1 us, where memory would need 3.6.  The
// registers of workgroups of 1024, 128 for a lane, are 6 to 8 fewer than 16 fp32 keys for a lane
// would take; those are in scratch memory, 4 MB written in that call, also where smaller
// workgroups run it.
template <uint32_t kLanes, uint32_t kPer, uint32_t kTop, class Key>
__global__ __launch_bounds__(1024) void gate_kernel(const GateArgs a)
{
    using S = Spread<kLanes, kPer>;
    constexpr uint32_t kGroups = 64 / kLanes;
    constexpr bool kMake = !std::is_void_v<Key>;
    extern __shared__ uint32_t s_count[];     // [expert], then [wave][expert] sums
    __shared__ uint32_t s_tokens;
    const uint32_t lane = lane_id() % kLanes, E = a.num_experts, K = a.top_k;
    const uint32_t waves = blockDim.x / 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool fp32 = kMake ? std::is_same_v<Key, KeyFp32> : bool(a.fp32);
    const bool balance = !kMake || a.counts != nullptr;
    if (balance) {
        for (uint32_t e = threadIdx.x; e < E; e += blockDim.x) s_count[e] = 0;
        if (threadIdx.x == 0) {
            s_tokens = 0;
            if (blockIdx.x == 0) *finish_ticket(a) = 0;
        }
        __syncthreads();
    }
    float sums[kPer] = {};
    uint32_t tokens = 0;
    const uint64_t step = uint64_t(gridDim.x) * waves * kGroups;
    for (uint64_t t = uint64_t(blockIdx.x) * waves * kGroups + threadIdx.x / kLanes; t < a.tokens; t += step) {
        float z[kPer];
        S::load(z, row_of(a.logits, t, a.stride, fp32), lane, E, fp32);
        const bool there = !a.mask || a.mask[t] != 0;
        if (!there) {
#pragma unroll
            for (uint32_t i = 0; i < kPer; i++) z[i] = -__builtin_inff();
        }
        int32_t id = -1;       // choice `lane`
        float at_id = 0.0f, top = 0.0f;     // its logit, and the row's largest
        if constexpr (kMake) {
            Key key[kPer];
            bool nan = false;
#pragma unroll
            for (uint32_t i = 0; i < kPer; i++) nan |= z[i] != z[i];
            if (__any(nan)) {   // as one NaN, of one sign and payload
#pragma unroll
                for (uint32_t i = 0; i < kPer; i++) key[i] = Key(z[i] != z[i] ? 0xFFFFFFFFu : bits_of(z[i]), S::expert(lane, i));
            } else {
#pragma unroll
                for (uint32_t i = 0; i < kPer; i++) key[i] = Key(bits_of(z[i]), S::expert(lane, i));
            }
            sort_top<kPer, kTop>(key);
            for (uint32_t k = 0; k < K; k++) {
                const Key best = largest<kLanes>(key[0]);
                if (!best.open()) break;
                const bool mine = key[0].same(best);
#pragma unroll
                for (uint32_t i = 0; i + 1 < kTop; i++) key[i] = Key::either(mine, key[i + 1], key[i]);
                key[kTop - 1] = Key::either(mine, Key(), key[kTop - 1]);
                const float v = value_of(best.key());
                if (k == 0) top = v;
                if (lane == k) {
                    id = int32_t(best.expert());
                    at_id = v;
                }
            }
        }
        float sum = 0.0f;
        if (balance || !a.renormalize) {
            sum = exps<kLanes>(z);
            if (balance && !(sum == 0.0f)) {
                const float over = 1.0f / sum;      // one division for a row: a rounding more for its values
#pragma unroll
                for (uint32_t i = 0; i < kPer; i++) sums[i] += z[i] * over;
                if (lane == 0) tokens++;
            }
        }
        if constexpr (kMake) {
            const float e = id >= 0 ? exp_of(at_id - top) : 0.0f;
            if (a.renormalize) sum = total<kLanes>(e);
            if (lane < K) {
                a.experts[t * K + lane] = id;
                a.weights[t * K + lane] = id >= 0 ? e / sum : 0.0f;
            }
            if (balance && id >= 0) atomicAdd(&s_count[id], 1u);
        } else if (!(sum == 0.0f)) {
            for (uint32_t k = lane; k < K; k += kLanes) {
                bool bad;
                const int32_t g = given(a, t, k, bad);
                if (bad) set_status(a.status, ZIPCCL_STATUS_BAD_INDEX);
                if (g >= 0) atomicAdd(&s_count[g], 1u);
            }
        }
    }
    if (!balance) return;
    // lanes of a wave, then its workgroup's waves in order
    float* s_sums = reinterpret_cast<float*>(s_count + E);
#pragma unroll
    for (uint32_t i = 0; i < kPer; i++) {
#pragma unroll
        for (uint32_t d = kLanes; d < 64; d *= 2) sums[i] += __shfl_xor(sums[i], int(d));
        const uint32_t e = S::expert(lane, i);
        if (lane_id() < kLanes && e < E) s_sums[wave * E + e] = sums[i];
    }
    if (tokens) atomicAdd(&s_tokens, tokens);
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < E; e += blockDim.x) {
        float sum = 0.0f;
        for (uint32_t w = 0; w < waves; w++) sum += s_sums[w * E + e];
        block_sums(a)[uint64_t(blockIdx.x) * E + e] = sum;
        block_counts(a)[uint64_t(blockIdx.x) * E + e] = s_count[e];
    }
    if (threadIdx.x == 0) block_tokens(a)[blockIdx.x] = s_tokens;
}

// The workgroups' sums and counts joined, 16 experts by each workgroup; the last one to be done
// adds up the loss.  What counts is the chain of steps: one batch of loads for each thread.
constexpr uint32_t kFinishThreads = 1024;

__global__ __launch_bounds__(kFinishThreads) void gate_finish_kernel(const GateArgs a)
{
    constexpr uint32_t kShares = kFinishThreads / kFinishColumns, kBatch = kGateBlocks / kShares;
    __shared__ double s_sum[kShares][kFinishColumns];
    __shared__ uint32_t s_number[kShares][kFinishColumns], s_tokens;
    const uint32_t tid = threadIdx.x, E = a.num_experts;
    const uint32_t column = tid % kFinishColumns, share = tid / kFinishColumns;
    const uint32_t e = blockIdx.x * kFinishColumns + column, at = min(e, E - 1);
    if (tid == 0) s_tokens = 0;
    float f[kBatch];
    uint32_t n[kBatch];
#pragma unroll
    for (uint32_t j = 0; j < kBatch; j++) {
        const uint64_t from = uint64_t(min(j * kShares + share, a.blocks - 1)) * E + at;
        f[j] = block_sums(a)[from];
        n[j] = block_counts(a)[from];
    }
    const uint32_t tokens = tid < a.blocks ? block_tokens(a)[tid] : 0;
    static_assert(kGateBlocks <= kFinishThreads && kGateBlocks % kShares == 0, "a thread for each workgroup");
    double sum = 0.0;
    uint32_t number = 0;
#pragma unroll
    for (uint32_t j = 0; j < kBatch; j++)
        if (j * kShares + share < a.blocks) {
            sum += double(f[j]);
            number += n[j];
        }
    s_sum[share][column] = sum;
    s_number[share][column] = number;
    __syncthreads();
    if (tokens) atomicAdd(&s_tokens, tokens);
#pragma unroll
    for (uint32_t d = kShares / 2; d >= 4; d /= 4) {    // four to one
        if (share < d / 2) {
            for (uint32_t s = share + d / 2; s < 2 * d; s += d / 2) {
                sum += s_sum[s][column];
                number += s_number[s][column];
            }
            s_sum[share][column] = sum;
            s_number[share][column] = number;
        }
        __syncthreads();
    }
    if (tid >= 64) return;
    double all = 0.0;
    if (tid < kFinishColumns) {
        for (uint32_t s = 1; s < 4; s++) {
            sum += s_sum[s][tid];
            number += s_number[s][tid];
        }
        if (e < E) {
            a.sums[e] = float(sum);
            a.counts[e] = int32_t(number);
            all = double(number) * sum;
        }
    }
    // lanes, then workgroups, in a fixed tree
    const auto join = [](double v) {
#pragma unroll
        for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
        return v;
    };
    all = join(all);
    if (blockIdx.x == 0 && tid == 0) a.counts[E] = int32_t(s_tokens);
    if (gridDim.x > 1) {
        // Parts are exchanged, not stored and loaded: an exchange always finds the place's last
        // value, and its returned value says that it has been done, for the atomics of every
        // workgroup of the GPU.  The ticket's step is made from what a part's exchange returned,
        // so the ticket cannot be taken before the part is there, and the last workgroup asks for the
        // parts once it has its ticket.  (This order is gfx950's, not the language's: release and
        // acquire would also write back and drop the L2, 2 us.)
        uint32_t before = 0;
        if (tid == 0) {
            const double was = __hip_atomic_exchange(finish_parts(a) + blockIdx.x, all, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            uint32_t step = 1;
            asm volatile("" : "+s"(step) : "v"(was) : "memory");
            before = __hip_atomic_fetch_add(finish_ticket(a), step, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        if (__builtin_amdgcn_readfirstlane(before) + 1 != gridDim.x) return;
        asm volatile("" ::: "memory");
        static_assert(kMaxExperts / kFinishColumns <= 64, "a lane for each workgroup");
        all = tid < gridDim.x ? __hip_atomic_exchange(finish_parts(a) + tid, 0.0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
        all = join(all);
    }
    if (tid == 0) a.loss[0] = loss_of(a, s_tokens, all);
}

// What lane and choice agree on is passed through a row of LDS for each token at hand: the
// probabilities to the choices (their weights), then the choices' gradients to their columns.
// The first row and choices are requested before the counts, which every row needs.
//
// Bound by the chain of its latencies and the instructions: 16384 x 256 in fp32, 8 choices, 11.3 us,
// of which issue (624 for each of 4096 waves) is 4.2 and memory 7.  All waves are resident at once
// there and take one round of tokens, so that their loads, sums and stores stand one behind the other.
template <uint32_t kLanes, uint32_t kPer, bool kFp32>
__global__ __launch_bounds__(256) void gate_backward_kernel(const GateArgs a)
{
    using S = Spread<kLanes, kPer>;
    constexpr uint32_t kGroups = 64 / kLanes;
    __shared__ __attribute__((aligned(16))) float s_rows[256 * kPer];
    const uint32_t lane = lane_id() % kLanes, E = a.num_experts, K = a.top_k;
    float* s_row = s_rows + threadIdx.x / kLanes * (kLanes * kPer);
    const auto put = [&](const float (&v)[kPer]) {
#pragma unroll
        for (uint32_t i = 0; i < kPer; i += S::kWide) __builtin_memcpy(s_row + S::first(lane, i), &v[i], 4 * S::kWide);
    };
    const uint64_t step = uint64_t(gridDim.x) * 4 * kGroups;
    uint64_t t = uint64_t(blockIdx.x) * 4 * kGroups + threadIdx.x / kLanes;
    float z[kPer];
    int32_t id = -1;       // choice `lane`
    float d = 0.0f;        // and its gradient
    bool bad = false, there = false;
    const auto load = [&]() {
        S::load(z, row_of(a.logits, t, a.stride, kFp32), lane, E, kFp32);
        there = !a.mask || a.mask[t] != 0;
        id = -1;
        d = 0.0f;
        bad = false;
        if (a.dweights && lane < K) {
            id = given(a, t, lane, bad);
            d = a.dweights[t * K + lane];
            if (id < 0) d = 0.0f;
        }
    };
    if (t < a.tokens) load();
    float f[kPer] = {};        // gradient of the loss by the probabilities
    if (a.totals) {
        int32_t count[kPer];
#pragma unroll
        for (uint32_t i = 0; i < kPer; i++) count[i] = a.totals[min(S::expert(lane, i), E - 1)];
        const float n = float(a.totals[E]);
        const float per = n > 0.0f ? a.dloss[0] * (float(E) / float(K)) / (n * n) : 0.0f;
#pragma unroll
        for (uint32_t i = 0; i < kPer; i++) f[i] = S::expert(lane, i) < E ? per * float(count[i]) : 0.0f;
    }
    const float none[kPer] = {};
    if (a.dweights) put(none);
    for (; t < a.tokens; t += step, t < a.tokens ? load() : void()) {
        uint8_t* out = const_cast<uint8_t*>(row_of(a.dlogits, t, a.dstride, kFp32));
        if (!there) {
#pragma unroll
            for (uint32_t i = 0; i < kPer; i++) z[i] = -__builtin_inff();
        }
        const float sum = exps<kLanes>(z);
        if (sum == 0.0f) {     // nothing open
            S::store(none, out, lane, E, kFp32);
            continue;
        }
        if (bad) set_status(a.status, ZIPCCL_STATUS_BAD_INDEX);
        float add[kPer] = {};
        if (a.dweights) {
            const bool chosen = id >= 0;
            if (a.renormalize) {
                wave_order();
                put(z);
                wave_order();
                float e = chosen ? s_row[id] : 0.0f, all = total<kLanes>(e);
                if (all < 1e-30f) {     // choices far below the row's largest: from the largest of them
                    const uint8_t* row = row_of(a.logits, t, a.stride, kFp32);
                    float c = -__builtin_inff();
                    if (chosen) c = kFp32 ? reinterpret_cast<const float*>(row)[id]
                                          : __uint_as_float(uint32_t(reinterpret_cast<const uint16_t*>(row)[id]) << 16);
                    const float most = across<kLanes>(c, [](float x, float y) { return larger(x, y); });
                    e = exp_of(c - (most == -__builtin_inff() ? 0.0f : most));
                    all = total<kLanes>(e);
                }
                const float w = all == 0.0f ? 0.0f : e / all;
                d = w * (d - total<kLanes>(w * d));
                wave_order();
                put(none);
            }
            // a lane whose number another one has overwritten shares its expert: then one after the
            // other adds
            wave_order();
            if (chosen) s_row[id] = __uint_as_float(lane + 1);
            wave_order();
            const bool shared = chosen && __float_as_uint(s_row[id]) != lane + 1;
            wave_order();
            if (__any(shared)) {
                if (chosen) s_row[id] = 0.0f;
                for (uint32_t k = 0; k < K; k++) {
                    wave_order();
                    if (chosen && lane == k) s_row[id] += d;
                }
            } else if (chosen) {
                s_row[id] = d;
            }
            wave_order();
#pragma unroll
            for (uint32_t i = 0; i < kPer; i += S::kWide) __builtin_memcpy(&add[i], s_row + S::first(lane, i), 4 * S::kWide);
            wave_order();
            if (chosen) s_row[id] = 0.0f;
        }
        const float over = 1.0f / sum;
        if (a.renormalize) {
            if (a.totals) {
                float dot = 0.0f;
#pragma unroll
                for (uint32_t i = 0; i < kPer; i++) {
                    z[i] *= over;
                    dot += z[i] * f[i];
                }
                dot = total<kLanes>(dot);
#pragma unroll
                for (uint32_t i = 0; i < kPer; i++) add[i] += z[i] * (f[i] - dot);
            }
        } else {
            float dot = 0.0f;
#pragma unroll
            for (uint32_t i = 0; i < kPer; i++) {
                z[i] *= over;
                add[i] += f[i];
                dot += z[i] * add[i];
            }
            dot = total<kLanes>(dot);
#pragma unroll
            for (uint32_t i = 0; i < kPer; i++) add[i] = z[i] * (add[i] - dot);
        }
        S::store(add, out, lane, E, kFp32);
    }
}

// Lanes per token and values per lane.  Lane k holds choice k, so there are at least as many
// lanes as choices.
//
// Gradient: the fewer lanes share a token, the fewer steps join them and the more tokens a wave
// takes at once, up to 16 values for a lane (the loss's of 65536 x 64: 10.3 us with 16 lanes, 8.3
// with 4).  Forward, a lane sorts its values, so more lanes have less to do: 16, or 64 (8191 x
// 61, 3 of them: 4.9 us with 16 lanes, 7.8 with 4; 65536 x 64 without choices to make 9.4 and
// 9.8).
template <bool kGradient, class Run>
hipError_t by_shape(const GateArgs& a, Run run)
{
    using std::integral_constant;
    const uint32_t e = a.num_experts, k = a.top_k;
    integral_constant<uint32_t, 64> wave;
    integral_constant<uint32_t, 16> sixteen;
    integral_constant<uint32_t, 8> eight;
    integral_constant<uint32_t, 4> four;
    if (e > 256 || k > 16) {
        if (e > 512) return run(wave, sixteen);
        if (e > 256) return run(wave, eight);
        return run(wave, four);
    }
    if constexpr (kGradient) {
        if (k <= 4 && e <= 32) return run(four, eight);
        if (k <= 4 && e <= 64) return run(four, sixteen);
        if (k <= 8 && e <= 64) return run(eight, eight);
        if (k <= 8 && e <= 128) return run(eight, sixteen);
    } else {
        if (e <= 16) return run(sixteen, integral_constant<uint32_t, 1>());
        if (e <= 32) return run(sixteen, integral_constant<uint32_t, 2>());
    }
    if (e <= 64) return run(sixteen, four);
    if (e <= 128) return run(sixteen, eight);
    return run(sixteen, sixteen);
}

}  // namespace

hipError_t launch_moe_gate(const GateArgs& args, hipStream_t s)
{
    GateArgs a = args;
    const bool balance = a.counts != nullptr;
    const hipError_t e = by_shape<false>(a, [&](auto lanes, auto per) {
        constexpr uint32_t kLanes = decltype(lanes)::value, kPer = decltype(per)::value;
        constexpr uint32_t kTop = kPer < 8 ? kPer : 8;
        // as many workgroups as the workspace has room for, of as many waves as that leaves
        uint32_t threads = 256;
        while (balance && threads < 1024 && a.tokens * kLanes > uint64_t(kGateBlocks) * threads) threads *= 2;
        if (kLanes == 64) threads = 256;      // their sums in LDS are long
        const uint64_t tokens = threads / kLanes, groups = (a.tokens + tokens - 1) / tokens, most = balance ? kGateBlocks : 1u << 20;
        a.blocks = groups == 0 ? 1 : uint32_t(groups < most ? groups : most);
        const uint32_t lds = balance ? 4 * a.num_experts * (1 + threads / 64) : 0;
        const auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(a.blocks), dim3(threads), lds, s, a); };
        if (a.ids) run(gate_kernel<kLanes, kPer, 1, void>);
        else if (kTop < kPer && a.top_k > kTop) a.fp32 ? run(gate_kernel<kLanes, kPer, kPer, KeyFp32>) : run(gate_kernel<kLanes, kPer, kPer, KeyBf16>);
        else a.fp32 ? run(gate_kernel<kLanes, kPer, kTop, KeyFp32>) : run(gate_kernel<kLanes, kPer, kTop, KeyBf16>);
        return hipGetLastError();
    });
    if (e != hipSuccess || !balance) return e;
    hipLaunchKernelGGL(gate_finish_kernel, dim3((a.num_experts + kFinishColumns - 1) / kFinishColumns), dim3(kFinishThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_moe_gate_backward(const GateArgs& a, hipStream_t s)
{
    return by_shape<true>(a, [&](auto lanes, auto per) {
        constexpr uint32_t kLanes = decltype(lanes)::value, kPer = decltype(per)::value;
        constexpr uint32_t kTokens = 256 / kLanes;
        const uint64_t groups = (a.tokens + kTokens - 1) / kTokens;
        const dim3 grid(uint32_t(groups < (1u << 20) ? groups : 1u << 20));
        if (a.fp32) hipLaunchKernelGGL((gate_backward_kernel<kLanes, kPer, true>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((gate_backward_kernel<kLanes, kPer, false>), grid, dim3(256), 0, s, a);
        return hipGetLastError();
    });
}

}  // namespace zc
