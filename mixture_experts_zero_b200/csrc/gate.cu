// gate.cu -- general routing gates of a mixture-of-experts layer, and their gradient.
//
//   forward   s_i = softmax(z)_i or 1 / (1 + e^-z_i)              (fp32 logits z, or bf16)
//             key_i = s_i + b_i                                   (b: balance bias, choice only)
//             groups: E / G consecutive experts each; a group's score is the sum of its group_rank
//             (1 or 2) largest keys; the top_groups best groups stay (equal scores: lower group)
//             picks: the K largest keys of the groups that stay, in descending order (equal keys:
//             lower expert)
//             gate_r = scale * s_r, or scale * s_r / (sum of the K chosen s) when renormalised
//   backward  p = s_chosen / Q, Q = sum of the chosen s:
//             renormalised:  dz_r = scale * p_r * f_r * (dg_r - sum_q p_q dg_q), f = 1 for softmax
//                            (the gates are then a softmax over the chosen logits alone),
//                            f_r = 1 - s_r for sigmoid; every other logit's gradient is 0
//             sigmoid:       dz_r = scale * dg_r * s_r (1 - s_r), 0 elsewhere
//             softmax:       dz_i = s_i (ds_i - D), ds_r = scale * dg_r (0 where not chosen),
//                            D = sum_r ds_r s_r
//
// The picks are integers, so they are decided in 64 bits: two programs that evaluate the formula
// in 64 bits agree on them unless two keys lie within about 1e-16 of each other.
#include <cuda_bf16.h>

#include "common.cuh"

namespace lcmoe {

namespace {

constexpr int GATE_THREADS = 256;
constexpr uint32_t FULL = 0xffffffffu;

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) {
    return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p))) << 16);
}
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
    return v;
}

// order-preserving integer of a double that is not NaN (never 0: 0 stands for "taken")
__device__ __forceinline__ unsigned long long ordered(double v) {
    const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(v + 0.0));
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// the lane-wise maximum of k, and the smallest i among the lanes that hold it
__device__ __forceinline__ int arg_max(unsigned long long k, int i) {
    const uint32_t hi = static_cast<uint32_t>(k >> 32);
    const uint32_t mh = __reduce_max_sync(FULL, hi);
    const uint32_t lo = hi == mh ? static_cast<uint32_t>(k) : 0u;
    const uint32_t ml = __reduce_max_sync(FULL, lo);
    const bool mine = hi == mh && static_cast<uint32_t>(k) == ml;
    return static_cast<int>(__reduce_min_sync(FULL, mine ? static_cast<uint32_t>(i) : 0x7fffffffu));
}

__device__ __forceinline__ double sigmoid64(double z) { return 1.0 / (1.0 + exp(-z)); }
__device__ __forceinline__ float sigmoid32(float z) { return 1.0f / (1.0f + expf(-z)); }

// p_r of the chosen logits (lane r < K; other lanes pass z = -inf and get 0): s_r / sum of the
// chosen s. Where the largest chosen logit of a sigmoid is below -40, 1 + e^z is 1 in fp32 and the
// quotient is the softmax of the chosen logits, which cannot underflow. All -inf: 0.
__device__ __forceinline__ float chosen_share(float z, bool sigmoid) {
    const float m = warp_max(z);
    if (m == __int_as_float(0xff800000)) return z != z ? z : 0.0f;
    const float s = (sigmoid && !(m < -40.0f)) ? sigmoid32(z) : expf(z - m);
    return s / warp_sum(s);
}

// One warp per token; the token's keys lie in the warp's shared-memory row (doubles).
template <class LT>
__global__ void __launch_bounds__(GATE_THREADS)
    gate_kernel(const LT* __restrict__ logits, const float* __restrict__ bias, int T, int E, int K,
                lc_moe_gate_opts o, int32_t* __restrict__ idx, float* __restrict__ gate,
                int32_t* __restrict__ counts, uint32_t* __restrict__ status) {
    extern __shared__ double s_dyn[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    double* key = s_dyn + static_cast<size_t>(warp) * E;
    int32_t* s_hist = reinterpret_cast<int32_t*>(s_dyn + static_cast<size_t>(warps) * E);
    if (counts) {
        for (int i = threadIdx.x; i < E; i += blockDim.x) s_hist[i] = 0;
        __syncthreads();
    }
    const bool sigmoid = o.score == LC_MOE_SCORE_SIGMOID;
    const int size = E / o.groups;
    for (int t = blockIdx.x * warps + warp; t < T; t += gridDim.x * warps) {
        const LT* zt = logits + static_cast<int64_t>(t) * E;
        __syncwarp();
        float m = __int_as_float(0xff800000);
        double S = 1.0;
        if (!sigmoid) {
            for (int i = lane; i < E; i += 32) m = fmaxf(m, load_logit(zt + i));
            m = warp_max(m);
            double part = 0.0;
            for (int i = lane; i < E; i += 32) {
                const float z = load_logit(zt + i);
                part += z == m && m < 0.0f && isinf(m) ? 0.0 : exp(static_cast<double>(z) - m);
            }
            S = warp_sum(part);
            if (S == 0.0) S = 1.0;  // every logit is -inf: all scores are 0
        }
        bool nan = false;
        for (int i = lane; i < E; i += 32) {
            const float z = load_logit(zt + i);
            double s;
            if (sigmoid) s = sigmoid64(z);
            else s = (z == m && m < 0.0f && isinf(m)) ? 0.0 : exp(static_cast<double>(z) - m) / S;
            const double k = bias ? s + static_cast<double>(bias[i]) : s;
            nan |= k != k;
            key[i] = k;
        }
        __syncwarp();
        uint32_t kept = FULL;  // bit g: group g stays
        if (o.top_groups < o.groups) {
            unsigned long long mine = 0;  // lane g: the ordered score of group g
            for (int g = 0; g < o.groups; ++g) {
                double a = -INFINITY, b = -INFINITY;
                for (int i = lane; i < size; i += 32) {
                    const double k = key[g * size + i];
                    if (k > a) { b = a; a = k; }
                    else if (k > b) b = k;
                }
#pragma unroll
                for (int w = 16; w; w >>= 1) {
                    const double a2 = __shfl_xor_sync(FULL, a, w), b2 = __shfl_xor_sync(FULL, b, w);
                    b = fmax(fmin(a, a2), fmax(b, b2));
                    a = fmax(a, a2);
                }
                const double score = o.group_rank == 2 && size > 1 ? a + b : a;
                nan |= score != score;
                if (lane == g) mine = ordered(score);
            }
            kept = 0;
            for (int r = 0; r < o.top_groups; ++r) {
                const int g = arg_max(mine, lane);
                kept |= 1u << g;
                if (lane == g) mine = 0;
            }
        }
        int my_idx = 0;
        const bool bad = __any_sync(FULL, nan);
        if (bad) {
            my_idx = lane;
            if (lane == 0) set_status(status, LC_MOE_DEV_NAN_KEY);
        } else {
            // K rounds of warp arg-max; each lane offers its best untaken key
            unsigned long long taken = 0, best = 0;
            int at = 0x7fffffff;
            auto offer = [&]() {
                best = 0;
                at = 0x7fffffff;
                for (int i = lane, j = 0; i < E; i += 32, ++j) {
                    if ((taken >> j) & 1) continue;
                    if (!((kept >> (i / size)) & 1u) && o.top_groups < o.groups) continue;
                    const unsigned long long k = ordered(key[i]);
                    if (k > best) {
                        best = k;
                        at = i;
                    }
                }
            };
            offer();
            for (int r = 0; r < K; ++r) {
                const int w = arg_max(best, at);
                if (lane == r) my_idx = w;
                if ((w & 31) == lane) {
                    taken |= 1ull << (w >> 5);
                    offer();
                }
            }
        }
        // gates, from the chosen logits
        const float z = lane < K ? load_logit(zt + my_idx) : __int_as_float(0xff800000);
        float g;
        if (o.renorm) g = chosen_share(z, sigmoid);
        else if (sigmoid) g = sigmoid32(z);
        else g = static_cast<float>(isinf(z) ? 0.0 : exp(static_cast<double>(z) - m) / S);
        if (lane < K) {
            const int64_t at = static_cast<int64_t>(t) * K + lane;
            idx[at] = my_idx;
            gate[at] = bad ? __int_as_float(0x7fc00000) : o.scale * g;
            if (counts) atomicAdd(&s_hist[my_idx], 1);
        }
    }
    if (counts) {
        __syncthreads();
        for (int i = threadIdx.x; i < E; i += blockDim.x) {
            const int c = s_hist[i];
            if (c) atomicAdd(&counts[i], c);
        }
    }
}

// One warp per token. The row is written in full first, then the chosen entries over it.
template <class LT>
__global__ void __launch_bounds__(GATE_THREADS)
    gate_backward_kernel(const LT* __restrict__ logits, const int32_t* __restrict__ idx,
                         const float* __restrict__ dgate, int T, int E, int K, lc_moe_gate_opts o,
                         LT* __restrict__ dlogits, uint32_t* __restrict__ status) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const bool sigmoid = o.score == LC_MOE_SCORE_SIGMOID;
    const float NEG_INF = __int_as_float(0xff800000);
    for (int t = blockIdx.x * warps + warp; t < T; t += gridDim.x * warps) {
        const LT* zt = logits + static_cast<int64_t>(t) * E;
        LT* out = dlogits + static_cast<int64_t>(t) * E;
        int i = -1;
        float z = NEG_INF, dg = 0.0f;
        if (lane < K) {
            i = idx[static_cast<int64_t>(t) * K + lane];
            if (i < 0 || i >= E) {
                set_status(status, LC_MOE_DEV_IDX_RANGE);
                i = -1;
            } else {
                z = load_logit(zt + i);
                dg = o.scale * dgate[static_cast<int64_t>(t) * K + lane];
            }
        }
        float mine, D = 0.0f;  // dz of the chosen logit through its own score
        float inv_S = 0.0f, m = 0.0f;
        const bool dense = !sigmoid && !o.renorm;
        if (o.renorm) {
            const float p = chosen_share(z, sigmoid);
            const float mean = warp_sum(p * dg);
            const float f = sigmoid ? 1.0f / (1.0f + expf(z)) : 1.0f;
            mine = p * f * (dg - mean);
        } else if (sigmoid) {
            const float e = expf(-fabsf(z));
            mine = dg * e / ((1.0f + e) * (1.0f + e));
        } else {
            m = NEG_INF;
            for (int j = lane; j < E; j += 32) m = fmaxf(m, load_logit(zt + j));
            m = warp_max(m);
            if (m == NEG_INF) m = 0.0f;  // every logit is -inf: all scores are 0
            float part = 0.0f;
            for (int j = lane; j < E; j += 32) part += expf(load_logit(zt + j) - m);
            const float S = warp_sum(part);
            inv_S = S > 0.0f || S != S ? 1.0f / S : 0.0f;
            const float s = i >= 0 ? expf(z - m) * inv_S : 0.0f;
            D = warp_sum(s * dg);
            mine = s * dg;
        }
        // picks of the same expert add up, in rank order, at the first of them
        const uint32_t same = __match_any_sync(FULL, i);
        float total = 0.0f;
        for (int r = 0; r < K; ++r) {
            const float v = __shfl_sync(FULL, mine, r);
            if ((same >> r) & 1u) total += v;
        }
        const bool first = i >= 0 && lane == __ffs(same) - 1;
        if (dense) {
            for (int j = lane; j < E; j += 32) store_logit(out + j, -expf(load_logit(zt + j) - m) * inv_S * D);
            if (i >= 0) total -= expf(z - m) * inv_S * D;
        } else {
            for (int j = lane; j < E; j += 32) store_logit(out + j, 0.0f);
        }
        __syncwarp();
        if (first) store_logit(out + i, total);
    }
}

}  // namespace

cudaError_t launch_gate(const void* logits, int bf16, const float* bias, int T, int E, int K,
                        const lc_moe_gate_opts& o, int32_t* idx, float* gate, int32_t* counts,
                        uint32_t* status, cudaStream_t st) {
    const DevInfo* di = current_device_info();
    if (!di) return cudaErrorUnknown;
    const int warps = E <= 1024 ? 8 : 4;
    const size_t smem = static_cast<size_t>(warps) * E * 8 + (counts ? static_cast<size_t>(E) * 4 : 0);
    static PerDeviceOnce setup;
    const cudaError_t e = setup.run([](int) {
        cudaError_t r = cudaFuncSetAttribute(gate_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize, 80 * 1024);
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(gate_kernel<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize, 80 * 1024);
        return r;
    });
    if (e != cudaSuccess) return e;
    int blocks = (T + warps - 1) / warps;
    if (blocks > di->sm_count * 4) blocks = di->sm_count * 4;
    if (bf16)
        gate_kernel<__nv_bfloat16><<<blocks, warps * 32, smem, st>>>(
            static_cast<const __nv_bfloat16*>(logits), bias, T, E, K, o, idx, gate, counts, status);
    else
        gate_kernel<float><<<blocks, warps * 32, smem, st>>>(static_cast<const float*>(logits), bias, T, E, K, o,
                                                              idx, gate, counts, status);
    return cudaGetLastError();
}

cudaError_t launch_gate_backward(const void* logits, int bf16, const int32_t* idx, const float* dgate, int T,
                                 int E, int K, const lc_moe_gate_opts& o, void* dlogits, uint32_t* status,
                                 cudaStream_t st) {
    const DevInfo* di = current_device_info();
    if (!di) return cudaErrorUnknown;
    int blocks = (T + 7) / 8;
    if (blocks > di->sm_count * 8) blocks = di->sm_count * 8;
    if (bf16)
        gate_backward_kernel<__nv_bfloat16><<<blocks, GATE_THREADS, 0, st>>>(
            static_cast<const __nv_bfloat16*>(logits), idx, dgate, T, E, K, o, static_cast<__nv_bfloat16*>(dlogits),
            status);
    else
        gate_backward_kernel<float><<<blocks, GATE_THREADS, 0, st>>>(static_cast<const float*>(logits), idx, dgate, T,
                                                                      E, K, o, static_cast<float*>(dlogits), status);
    return cudaGetLastError();
}

}  // namespace lcmoe
