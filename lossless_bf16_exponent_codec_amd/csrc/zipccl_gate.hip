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
// Everything is fp32; sums over tokens are joined in a fixed order (lanes, waves, workgroups),
// the last step in 64 bits, so a call gives the same bits on every run.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "zipccl.h"
#include "zipccl_moe_internal.h"
#include "zipccl_row_tiles.h"

namespace zc {

namespace {

constexpr uint32_t kNoKey = 0;           // of minus infinity: never chosen

// Unsigned keys in the order of the values: 0 for minus infinity, NaNs above all, both zeros
// alike.
__device__ inline uint32_t key_of(float z)
{
    const uint32_t b = __float_as_uint(z + 0.0f);
    if (z != z) return 0xFFFFFFFFu;
    const uint32_t k = b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
    return k == 0x007FFFFFu ? kNoKey : k;
}

__device__ inline float value_of(uint32_t key)
{
    if (key == kNoKey) return -__builtin_inff();
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);   // the NaN's key gives a NaN
}

// exp by the hardware's exp2: off by at most about |x| 2^-24 + 2^-23 of it, for x the distance
// to the row's largest logit.
__device__ inline float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f); }

template <int kTurn>
__device__ inline uint32_t turned(uint32_t v)   // from kTurn lanes on, within 16
{
    return uint32_t(__builtin_amdgcn_update_dpp(int(v), int(v), 0x120 + kTurn, 0xF, 0xF, false));
}

// op over the kLanes lanes of a group, the same bits in every one of them.
template <uint32_t kLanes, class Op>
__device__ inline uint32_t across(uint32_t v, Op op)
{
    v = op(v, turned<8>(v));
    v = op(v, turned<4>(v));
    v = op(v, turned<2>(v));
    v = op(v, turned<1>(v));
    if constexpr (kLanes == 64) {
        v = op(v, uint32_t(__shfl_xor(int(v), 16)));
        v = op(v, uint32_t(__shfl_xor(int(v), 32)));
    }
    return v;
}

template <uint32_t kLanes>
__device__ inline uint32_t largest(uint32_t v)
{
    return across<kLanes>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}

template <uint32_t kLanes>
__device__ inline uint32_t smallest(uint32_t v)
{
    return across<kLanes>(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}

template <uint32_t kLanes>
__device__ inline float total(float v)
{
    return __uint_as_float(across<kLanes>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

// How a row of up to kLanes * kPer values lies over a group's lanes: chunks of kWide
// neighbours, lane after lane, so that a lane's values are in the order of their experts.
template <uint32_t kLanes, uint32_t kPer>
struct Spread {
    static constexpr uint32_t kWide = kPer < 4 ? kPer : 4;
    static __device__ inline uint32_t first(uint32_t lane, uint32_t i) { return (i / kWide * kLanes + lane) * kWide; }
    static __device__ inline uint32_t expert(uint32_t lane, uint32_t i) { return first(lane, i) + i % kWide; }

    // z of a row: minus infinity past its end.
    static __device__ inline void load(float (&z)[kPer], const uint8_t* row, uint32_t lane, uint32_t n, bool fp32)
    {
#pragma unroll
        for (uint32_t i = 0; i < kPer; i += kWide) {
            const uint32_t e = first(lane, i);
            if (fp32) {
                const float* at = reinterpret_cast<const float*>(row) + e;
                if (e + kWide <= n) {
                    __builtin_memcpy(&z[i], at, 4 * kWide);
                } else {
#pragma unroll
                    for (uint32_t j = 0; j < kWide; j++) z[i + j] = e + j < n ? at[j] : -__builtin_inff();
                }
            } else {
                const uint16_t* at = reinterpret_cast<const uint16_t*>(row) + e;
                uint16_t b[kWide];
                if (e + kWide <= n) {
                    __builtin_memcpy(b, at, 2 * kWide);
                } else {
#pragma unroll
                    for (uint32_t j = 0; j < kWide; j++) b[j] = e + j < n ? at[j] : 0xFF80u;
                }
#pragma unroll
                for (uint32_t j = 0; j < kWide; j++) z[i + j] = __uint_as_float(uint32_t(b[j]) << 16);
            }
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

// A choice that the caller made; -1 for one that is dropped.
__device__ inline int32_t given(const GateArgs& a, uint64_t token, uint32_t k)
{
    const uint64_t at = token * a.id_stride + k;
    int64_t id = a.wide_ids ? static_cast<const int64_t*>(a.ids)[at] : static_cast<const int32_t*>(a.ids)[at];
    if (id >= int64_t(a.num_experts)) {
        set_status(a.status, ZIPCCL_STATUS_BAD_INDEX);
        id = -1;
    }
    return id < 0 ? -1 : int32_t(id);
}

// What a workgroup leaves in the workspace.
__device__ inline float* block_sums(const GateArgs& a) { return reinterpret_cast<float*>(a.workspace); }
__device__ inline uint32_t* block_counts(const GateArgs& a)
{
    return reinterpret_cast<uint32_t*>(a.workspace) + uint64_t(a.blocks) * a.num_experts;
}
__device__ inline uint32_t* block_tokens(const GateArgs& a) { return block_counts(a) + uint64_t(a.blocks) * a.num_experts; }

// Forward.  kMake: the choices are made here; else they are given and counted.
template <uint32_t kLanes, uint32_t kPer, bool kMake>
__global__ __launch_bounds__(1024) void gate_kernel(const GateArgs a)
{
    using S = Spread<kLanes, kPer>;
    constexpr uint32_t kGroups = 64 / kLanes;
    extern __shared__ uint32_t s_count[];     // [expert], then [wave][expert] sums
    __shared__ uint32_t s_tokens;
    const uint32_t lane = lane_id() % kLanes, E = a.num_experts, K = a.top_k;
    const uint32_t waves = blockDim.x / 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool balance = !kMake || a.counts != nullptr;
    if (balance) {
        for (uint32_t e = threadIdx.x; e < E; e += blockDim.x) s_count[e] = 0;
        if (threadIdx.x == 0) s_tokens = 0;
        __syncthreads();
    }
    float sums[kPer] = {};
    uint32_t tokens = 0;
    const uint64_t step = uint64_t(gridDim.x) * waves * kGroups;
    for (uint64_t t = uint64_t(blockIdx.x) * waves * kGroups + threadIdx.x / kLanes; t < a.tokens; t += step) {
        const bool there = !a.mask || a.mask[t] != 0;
        float z[kPer];
        uint32_t key[kPer];
        if (there) {
            S::load(z, row_of(a.logits, t, a.stride, a.fp32), lane, E, a.fp32);
        } else {
#pragma unroll
            for (uint32_t i = 0; i < kPer; i++) z[i] = -__builtin_inff();
        }
#pragma unroll
        for (uint32_t i = 0; i < kPer; i++) key[i] = key_of(z[i]);
        uint32_t top;          // key of the row's largest
        int32_t id = -1;       // choice `lane`
        uint32_t id_key = kNoKey;
        if constexpr (kMake) {
            top = kNoKey;
            for (uint32_t k = 0; k < K; k++) {
                uint32_t best = kNoKey, at = 0;
#pragma unroll
                for (uint32_t i = 0; i < kPer; i++)
                    if (key[i] > best) {
                        best = key[i];
                        at = i;
                    }
                const uint32_t most = largest<kLanes>(best);
                if (most == kNoKey) break;
                const uint32_t mine = best == most ? S::expert(lane, at) : 0xFFFFFFFFu;
                const uint32_t winner = smallest<kLanes>(mine);
#pragma unroll
                for (uint32_t i = 0; i < kPer; i++)
                    if (S::expert(lane, i) == winner) key[i] = kNoKey;
                if (k == 0) top = most;
                if (lane == k) {
                    id = int32_t(winner);
                    id_key = most;
                }
            }
        } else {
            uint32_t best = kNoKey;
#pragma unroll
            for (uint32_t i = 0; i < kPer; i++) best = max(best, key[i]);
            top = largest<kLanes>(best);
        }
        const float z0 = value_of(top);
        const bool some = top != kNoKey;
        float over = 1.0f;     // 1 / the sum of exp over the row
        if (balance || !a.renormalize) {
            float sum = 0.0f;
#pragma unroll
            for (uint32_t i = 0; i < kPer; i++) {
                z[i] = some ? exp_of(z[i] - z0) : 0.0f;
                sum += z[i];
            }
            sum = total<kLanes>(sum);
            over = some ? 1.0f / sum : 1.0f;
            if (balance) {
#pragma unroll
                for (uint32_t i = 0; i < kPer; i++) sums[i] += z[i] * over;
                if (some && lane == 0) tokens++;
            }
        }
        if constexpr (kMake) {
            const float e = id >= 0 ? exp_of(value_of(id_key) - z0) : 0.0f;
            float w;
            if (a.renormalize) {
                const float sum = total<kLanes>(e);
                w = some ? e / sum : 0.0f;
            } else {
                w = e * over;
            }
            if (lane < K) {
                a.experts[t * K + lane] = id;
                a.weights[t * K + lane] = w;
            }
            if (balance && id >= 0) atomicAdd(&s_count[id], 1u);
        } else if (some) {
            for (uint32_t k = lane; k < K; k += kLanes) {
                const int32_t g = given(a, t, k);
                if (g >= 0) atomicAdd(&s_count[g], 1u);
            }
        }
    }
    if (!balance) return;
    // lanes of a wave, then its workgroup's waves in order
    float* s_sums = reinterpret_cast<float*>(s_count + E);
#pragma unroll
    for (uint32_t i = 0; i < kPer; i++) {
        if constexpr (kLanes == 16) {
            sums[i] += __shfl_xor(sums[i], 16);
            sums[i] += __shfl_xor(sums[i], 32);
        }
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

// The workgroups' sums and counts joined, and the loss: one workgroup, `shares` threads per
// expert.
__global__ __launch_bounds__(1024) void gate_finish_kernel(const GateArgs a)
{
    __shared__ double s_sum[1024];
    __shared__ uint32_t s_number[1024];
    __shared__ uint32_t s_tokens;
    const uint32_t tid = threadIdx.x, E = a.num_experts, shares = 1024 / E;
    const uint32_t e = tid % E, share = tid / E;
    if (tid == 0) s_tokens = 0;
    double sum = 0.0;
    uint32_t number = 0;
    if (share < shares) {
#pragma unroll 8
        for (uint32_t b = share; b < a.blocks; b += shares) {
            sum += double(block_sums(a)[uint64_t(b) * E + e]);
            number += block_counts(a)[uint64_t(b) * E + e];
        }
    }
    s_sum[tid] = sum;
    s_number[tid] = number;
    __syncthreads();
    uint32_t tokens = 0;
    for (uint32_t b = tid; b < a.blocks; b += 1024) tokens += block_tokens(a)[b];
    if (tokens) atomicAdd(&s_tokens, tokens);
    double part = 0.0;
    if (tid < E) {
        for (uint32_t s = 1; s < shares; s++) {
            sum += s_sum[s * E + tid];
            number += s_number[s * E + tid];
        }
        a.sums[tid] = float(sum);
        a.counts[tid] = int32_t(number);
        part = double(number) * sum;
    }
    __syncthreads();
    s_sum[tid] = part;
    for (uint32_t d = 512; d > 0; d >>= 1) {
        __syncthreads();
        if (tid < d) s_sum[tid] += s_sum[tid + d];
    }
    if (tid == 0) {
        const double n = double(s_tokens);
        a.counts[E] = int32_t(s_tokens);
        a.loss[0] = s_tokens ? float(double(E) / (double(a.top_k) * n * n) * s_sum[0]) : 0.0f;
    }
}

template <uint32_t kLanes, uint32_t kPer>
__global__ __launch_bounds__(256) void gate_backward_kernel(const GateArgs a)
{
    using S = Spread<kLanes, kPer>;
    constexpr uint32_t kGroups = 64 / kLanes;
    const uint32_t lane = lane_id() % kLanes, E = a.num_experts, K = a.top_k;
    float f[kPer] = {};        // gradient of the loss by the probabilities
    if (a.totals) {
        const float n = float(a.totals[E]);
        const float per = n > 0.0f ? a.dloss[0] * (float(E) / float(K)) / (n * n) : 0.0f;
#pragma unroll
        for (uint32_t i = 0; i < kPer; i++) {
            const uint32_t e = S::expert(lane, i);
            if (e < E) f[i] = per * float(a.totals[e]);
        }
    }
    const uint64_t step = uint64_t(gridDim.x) * 4 * kGroups;
    for (uint64_t t = uint64_t(blockIdx.x) * 4 * kGroups + threadIdx.x / kLanes; t < a.tokens; t += step) {
        uint8_t* out = const_cast<uint8_t*>(row_of(a.dlogits, t, a.dstride, a.fp32));
        const uint8_t* row = row_of(a.logits, t, a.stride, a.fp32);
        float z[kPer], add[kPer] = {};
        uint32_t top = kNoKey;
        if (!a.mask || a.mask[t] != 0) {
            S::load(z, row, lane, E, a.fp32);
#pragma unroll
            for (uint32_t i = 0; i < kPer; i++) top = max(top, key_of(z[i]));
            top = largest<kLanes>(top);
        }
        if (top == kNoKey) {
            S::store(add, out, lane, E, a.fp32);
            continue;
        }
        const float z0 = value_of(top);
        float sum = 0.0f;
#pragma unroll
        for (uint32_t i = 0; i < kPer; i++) {
            z[i] = exp_of(z[i] - z0);
            sum += z[i];
        }
        const float over = 1.0f / total<kLanes>(sum);
        float g[kPer];
#pragma unroll
        for (uint32_t i = 0; i < kPer; i++) {
            z[i] *= over;
            g[i] = f[i];
        }
        if (a.dweights) {
            int32_t id = lane < K ? given(a, t, lane) : -1;
            float d = id >= 0 ? a.dweights[t * K + lane] : 0.0f;
            if (a.renormalize) {
                float c = -__builtin_inff();
                if (id >= 0) c = a.fp32 ? reinterpret_cast<const float*>(row)[id]
                                        : __uint_as_float(uint32_t(reinterpret_cast<const uint16_t*>(row)[id]) << 16);
                const uint32_t most = largest<kLanes>(key_of(c));
                const float e = id >= 0 && most != kNoKey ? exp_of(c - value_of(most)) : 0.0f;
                const float all = total<kLanes>(e);
                const float w = most != kNoKey ? e / all : 0.0f;
                const float dot = total<kLanes>(w * d);
                d = w * (d - dot);
            }
            for (uint32_t k = 0; k < K; k++) {
                const int32_t at = __shfl(id, int(k), int(kLanes));
                const float v = __shfl(d, int(k), int(kLanes));
                if (at < 0) continue;
#pragma unroll
                for (uint32_t i = 0; i < kPer; i++)
                    if (S::expert(lane, i) == uint32_t(at)) add[i] += v;
            }
            if (!a.renormalize) {
#pragma unroll
                for (uint32_t i = 0; i < kPer; i++) {
                    g[i] += add[i];
                    add[i] = 0.0f;
                }
            }
        }
        if (a.totals || !a.renormalize) {
            float dot = 0.0f;
#pragma unroll
            for (uint32_t i = 0; i < kPer; i++) dot += z[i] * g[i];
            dot = total<kLanes>(dot);
#pragma unroll
            for (uint32_t i = 0; i < kPer; i++) add[i] += z[i] * (g[i] - dot);
        }
        S::store(add, out, lane, E, a.fp32);
    }
}

// Lanes per token and values per lane.  A lane holds a token's choice `lane`, so 16 lanes do
// up to 16 choices.
template <class Run>
hipError_t by_shape(const GateArgs& a, Run run)
{
    const auto with = [&](auto lanes, auto per) { return run(lanes, per); };
    using std::integral_constant;
    integral_constant<uint32_t, 16> few;
    integral_constant<uint32_t, 64> wave;
    if (a.num_experts > 256 || a.top_k > 16) {
        if (a.num_experts > 512) return with(wave, integral_constant<uint32_t, 16>());
        if (a.num_experts > 256) return with(wave, integral_constant<uint32_t, 8>());
        return with(wave, integral_constant<uint32_t, 4>());
    }
    if (a.num_experts > 128) return with(few, integral_constant<uint32_t, 16>());
    if (a.num_experts > 64) return with(few, integral_constant<uint32_t, 8>());
    if (a.num_experts > 32) return with(few, integral_constant<uint32_t, 4>());
    if (a.num_experts > 16) return with(few, integral_constant<uint32_t, 2>());
    return with(few, integral_constant<uint32_t, 1>());
}

}  // namespace

hipError_t launch_moe_gate(const GateArgs& args, hipStream_t s)
{
    GateArgs a = args;
    const bool balance = a.counts != nullptr;
    a.blocks = 0;
    hipError_t e = by_shape(a, [&](auto lanes, auto per) {
        constexpr uint32_t kLanes = decltype(lanes)::value, kPer = decltype(per)::value;
        if (a.tokens == 0) return hipSuccess;
        const uint32_t threads = 256, tokens = threads / kLanes;
        const uint64_t groups = (a.tokens + tokens - 1) / tokens, most = balance ? kGateBlocks : 1u << 20;
        const uint32_t blocks = uint32_t(groups < most ? groups : most);
        const uint32_t lds = balance ? 4 * a.num_experts * (1 + threads / 64) : 0;
        a.blocks = blocks;
        if (a.ids) hipLaunchKernelGGL((gate_kernel<kLanes, kPer, false>), dim3(blocks), dim3(threads), lds, s, a);
        else hipLaunchKernelGGL((gate_kernel<kLanes, kPer, true>), dim3(blocks), dim3(threads), lds, s, a);
        return hipGetLastError();
    });
    if (e != hipSuccess || !balance) return e;
    hipLaunchKernelGGL(gate_finish_kernel, dim3(1), dim3(1024), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_moe_gate_backward(const GateArgs& a, hipStream_t s)
{
    return by_shape(a, [&](auto lanes, auto per) {
        constexpr uint32_t kLanes = decltype(lanes)::value, kPer = decltype(per)::value;
        constexpr uint32_t kTokens = 256 / kLanes;
        const uint64_t groups = (a.tokens + kTokens - 1) / kTokens;
        hipLaunchKernelGGL((gate_backward_kernel<kLanes, kPer>), dim3(uint32_t(groups < (1u << 20) ? groups : 1u << 20)),
                           dim3(256), 0, s, a);
        return hipGetLastError();
    });
}

}  // namespace zc
