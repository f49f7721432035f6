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
// in 64 bits agree on them unless two keys lie within about 1e-16 of each other. The kernel gets
// there from fp32 keys with a bound on their error: it collects the keys within the bounds of the
// K-th largest, sorts them, and evaluates them again in 64 bits where two neighbours among the first K
// or the K-th and one behind it are not apart by their bounds (a few tokens in a thousand). More than
// 32 candidates, or fewer than K lanes with a key of the groups that stay, send the token to K rounds
// over all its keys in 64 bits.
//
// One warp per token, E / 32 logits a lane, each read once. What bounds it is instructions and their
// latency: per logit a load, an exponential, a key and three comparisons, then some hundreds a token
// for the choice (about 1050 in all at E = 768). Measured on a B200 with inputs that are not in L2:
// 16384 x 768 softmax with a bias, K = 12, in 39 us (1.3 TB/s), with 8 groups of sigmoid scores 53 us; from L2
// 33 and 49 us; one token in 5 us. Rows of equal logits take the K rounds: a batch of nothing else 198 and
// 243 us from L2, one with a quarter of them 151 and 197, with one in a hundred 60 and 82. 128 experts in 16
// groups of which 2 stay share lanes, so that a token in five takes them: 42 us, without groups 18.
#include <cuda_bf16.h>

#include <type_traits>

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
// from e^-|z|, which does not overflow
__device__ __forceinline__ float sigmoid32(float z) {
    const float e = expf(-fabsf(z));
    return (z < 0.0f ? e : 1.0f) / (1.0f + e);
}

// p_r of the chosen logits (lane r < K; other lanes pass z = -inf and get 0): s_r / sum of the chosen
// s. Sigmoids of negative logits are e^z / (1 + e^z), all of them times the same e^-m where the largest
// chosen logit m is negative, so that no quotient underflows before its share does. All -inf: 0.
__device__ __forceinline__ float chosen_share(float z, bool sigmoid) {
    const float m = warp_max(z);
    if (m == __int_as_float(0xff800000)) return z != z ? z : 0.0f;
    float s;
    if (!sigmoid) s = expf(z - m);
    else s = z < 0.0f ? expf(z - fminf(m, 0.0f)) / (1.0f + expf(z)) : sigmoid32(z);
    return s / warp_sum(s);
}

__device__ __forceinline__ float redux_max(float v) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float redux_min(float v) {
    float r;
    asm("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// Which lanes keep the larger value in the 15 steps of a bitonic network that sorts in descending
// order: bit s for step s.
__device__ __forceinline__ uint32_t sort_directions() {
    const uint32_t lane = threadIdx.x & 31;
    uint32_t dir = 0, s = 0;
#pragma unroll
    for (uint32_t k = 2; k <= 32; k *= 2)
#pragma unroll
        for (uint32_t j = k / 2; j; j /= 2) dir |= (~(lane / j ^ lane / k) & 1u) << s++;
    return dir;
}
// The 32 lanes' values in descending order over the lanes.
__device__ __forceinline__ float sort_descending(float v, uint32_t dir) {
    int s = 0;
#pragma unroll
    for (int k = 2; k <= 32; k *= 2)
#pragma unroll
        for (int j = k / 2; j; j /= 2, ++s) {
            const float w = __shfl_xor_sync(FULL, v, j);
            v = dir & (1u << s) ? fmaxf(v, w) : fminf(v, w);
        }
    return v;
}

// largest of a lane's values (three operands an instruction)
template <int N>
__device__ __forceinline__ float largest(const float (&v)[N]) {
    float m = v[0];
#pragma unroll
    for (int j = 1; j < N; j += 2) {
        if (j + 1 < N) asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(v[j]), "f"(v[j + 1 < N ? j + 1 : j]));
        else m = fmaxf(m, v[j]);
    }
    return m;
}

// a >= b, a > b as 1 or 0: sums and bit patterns of such tests then run on the floating-point pipe,
// which has room where the comparisons fill the other
__device__ __forceinline__ float is_ge(float a, float b) {
    float r;
    asm("set.ge.f32.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float is_gt(float a, float b) {
    float r;
    asm("set.gt.f32.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// 64-bit softmax denominator of a row with maximum m (1 for a row of -inf, whose scores are 0).
template <class LT>
__device__ __noinline__ double softmax_sum64(const LT* zt, int E, float m) {
    double part = 0.0;
    const bool none = m < 0.0f && isinf(m);
    for (int i = threadIdx.x & 31; i < E && !none; i += 32) part += exp(static_cast<double>(load_logit(zt + i)) - m);
    const double S = warp_sum(part);
    return S == 0.0 ? 1.0 : S;
}

__device__ __forceinline__ double score64(float z, float m, double S, bool sigmoid) {
    if (sigmoid) return sigmoid64(z);
    return z == m && m < 0.0f && isinf(m) ? 0.0 : exp(static_cast<double>(z) - m) / S;
}

// A row's keys in 64 bits into the warp's shared-memory row; returns whether one is NaN (in any lane).
template <class LT>
__device__ __noinline__ bool keys64(const LT* zt, const float* bias, int E, bool sigmoid, float m, double* key) {
    const int lane = threadIdx.x & 31;
    const double S = sigmoid ? 1.0 : softmax_sum64(zt, E, m);
    bool nan = false;
    __syncwarp();
    for (int base = lane; base < E; base += 128) {
        double k[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int i = min(base + 32 * q, E - 1);
            k[q] = score64(load_logit(zt + i), m, S, sigmoid) + (bias ? static_cast<double>(__ldg(bias + i)) : 0.0);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (base + 32 * q < E) {
                nan |= k[q] != k[q];
                key[base + 32 * q] = k[q];
            }
    }
    __syncwarp();
    return __any_sync(FULL, nan);
}

// The groups that stay, decided in 64 bits from the keys in shared memory: bit g for group g (0
// where a group's score is NaN).
__device__ __noinline__ uint32_t groups64(const double* key, const lc_moe_gate_opts& o, int size, int team) {
    const int lane = threadIdx.x & 31, g = lane / team;
    double a = -INFINITY, b = -INFINITY;
    if (g < o.groups)
        for (int i = lane % team; i < size; i += team) {
            const double k = key[g * size + i];
            b = fmax(b, fmin(a, k));
            a = fmax(a, k);
        }
    for (int w = 1; w < team; w <<= 1) {
        const double a2 = __shfl_xor_sync(FULL, a, w), b2 = __shfl_xor_sync(FULL, b, w);
        b = fmax(fmin(a, a2), fmax(b, b2));
        a = fmax(a, a2);
    }
    double score = o.group_rank == 2 && size > 1 ? a + b : a;
    score = __shfl_sync(FULL, score, (lane * team) & 31);  // lane g: group g
    if (__any_sync(FULL, lane < o.groups && score != score)) return 0;
    int rank = 0;
    for (int q = 0; q < o.groups; ++q) {
        const double other = __shfl_sync(FULL, score, q);
        rank += other > score || (other == score && q < lane);
    }
    return __ballot_sync(FULL, lane < o.groups && rank < o.top_groups);
}

// K picks from the 64-bit keys in shared memory, for any row: K rounds of a warp-wide maximum over
// each lane's largest key that is left. Lane r < K returns its pick. The keys are overwritten.
__device__ __noinline__ int pick64(double* key, int E, int K, uint32_t kept, int size) {
    const int lane = threadIdx.x & 31;
    unsigned long long* left = reinterpret_cast<unsigned long long*>(key);
    for (int i = lane; i < E; i += 32) left[i] = (kept >> (i / size)) & 1u ? ordered(key[i]) : 0ull;
    unsigned long long best = 0;
    int at = 0x7fffffff, my_idx = 0;
    auto offer = [&]() {
        best = 0;
        at = 0x7fffffff;
        for (int i = lane; i < E; i += 32) {
            const unsigned long long k = left[i];
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
            left[w] = 0;
            offer();
        }
    }
    return my_idx;
}

// Error bounds of the fp32 keys. u = 2^-23.
//   softmax: __expf is within 2 + 1.2 x steps at -x = z - m, whose rounding adds x / 2; the sum of E
//   terms averages that over the softmax (x is ln E <= 7.7 on average at most: 15 u), its additions
//   (up to 16 in sequence in each of four chains, 2 to join them, 5 over the lanes) add 12 u, quotient,
//   product and key 4 u: s is within (33 + 1.7 x) u s, which is at most 33 u / S for any x >= 0, and
//   2^-15 s for every x <= 88.
//   sigmoid: __expf(-z) is within 2 + 1.2 |z| steps and counts for 1 - s of the quotient, whose sum and
//   quotient add 3 u: (3.5 + (1 - s) (2 + 1.2 |z|)) u s, at most 7 u for any z, and 2^-16 s for z >= -88.
//   Scores below e^-87 count as 0 (1e-37 covers them); key = s + b adds u |key|.
constexpr float U23 = 1.1920929e-07f;

// team: lanes to a group when group scores are taken (a power of two, so that all groups run at once);
// a group's keys start size + pad words apart in the warp's row of row_len doubles, so that the
// teams' reads fall on different banks.
// CTAs to an SM: 64 registers a thread hold up to 12 keys a lane without spills, up to 32 keys want 128
// (16384 x 768 from L2: 32.9 us with 2 CTAs, 34.8 with 3, 35.0 with 4). 64 keys a lane take blocks of 128
// threads, which 2 CTAs leave up to 255 registers each.
constexpr int gate_ctas(int vpl) { return vpl <= 12 ? 4 : 2; }

// FILLED: E is 32 VPL.
template <class LT, int VPL, bool FILLED>
__global__ void __launch_bounds__(VPL <= 32 ? 256 : 128, gate_ctas(VPL))
    gate_kernel(const LT* __restrict__ logits, const float* __restrict__ bias, int T, int E, int K,
                lc_moe_gate_opts o, int team, int pad, int row_len, int32_t* __restrict__ idx,
                float* __restrict__ gate, int32_t* __restrict__ counts, uint32_t* __restrict__ status) {
    extern __shared__ double s_dyn[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    double* row64 = s_dyn + static_cast<size_t>(warp) * row_len;  // this warp's keys, or its candidates
    float* row32 = reinterpret_cast<float*>(row64);
    int32_t* cand = reinterpret_cast<int32_t*>(row64);
    int32_t* s_hist = reinterpret_cast<int32_t*>(s_dyn + static_cast<size_t>(warps) * row_len);
    if (counts) {
        for (int i = threadIdx.x; i < E; i += blockDim.x) s_hist[i] = 0;
        __syncthreads();
    }
    const float NEG_INF = __int_as_float(0xff800000);
    const bool sigmoid = o.score == LC_MOE_SCORE_SIGMOID;
    const bool grouped = o.top_groups < o.groups;
    // without a bias and without sums of scores the logits themselves are in the keys' order
    const bool by_z = !bias && (!grouped || o.group_rank == 1);
    const int size = E / o.groups;
    // i / size for i < E <= 32 size (E <= 2048): the error of the quotient stays below 1 / size
    const uint32_t inv_size = ((1u << 22) + size - 1) / size;
    auto group_of = [&](int i) { return static_cast<int>((static_cast<uint32_t>(i) * inv_size) >> 22); };
    bool bias_nan = false;
    float bmin = 0.0f;  // the smallest finite bias: score = key - b <= key - bmin
    if (bias) {
        bmin = __int_as_float(0x7f800000);
        for (int i = lane; i < E; i += 32) {
            const float b = __ldg(bias + i);
            if (b > NEG_INF) bmin = fminf(bmin, b);
            bias_nan |= b != b;
        }
        bmin = redux_min(bmin);
    }
    const int stride = gridDim.x * warps;
    const uint32_t dir = sort_directions();
    auto in = [&](int j) { return FILLED || lane + 32 * j < E; };  // whether place j of this lane is an expert
    for (int64_t t = blockIdx.x * warps + warp; t < T; t += stride) {
        const LT* zt = logits + t * E;
        float v[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) v[j] = in(j) ? load_logit(zt + lane + 32 * j) : NEG_INF;
        float m = NEG_INF, S = 1.0f, inv_S = 1.0f;
        bool nan = false;
        if (!sigmoid) {
            m = redux_max(largest(v));
        }
        const float m0 = m == NEG_INF ? 0.0f : m;
        if (by_z) {
#pragma unroll
            for (int j = 0; j < VPL; ++j) nan |= v[j] != v[j];
            nan |= !sigmoid && m == __int_as_float(0x7f800000);
            if (!sigmoid && !o.renorm) {
                float part[4] = {};
#pragma unroll
                for (int j = 0; j < VPL; ++j) part[j % 4] += __expf(v[j] - m0);
                S = warp_sum((part[0] + part[1]) + (part[2] + part[3]));
                inv_S = S > 0.0f ? __fdividef(1.0f, S) : 0.0f;
            }
        } else {
            float part[4] = {};  // NaN where a logit is
            if (sigmoid) {
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    v[j] = __fdividef(1.0f, 1.0f + __expf(-v[j]));
                    part[0] += v[j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    v[j] = __expf(v[j] - m0);
                    part[j % 4] += v[j];
                }
                S = warp_sum((part[0] + part[1]) + (part[2] + part[3]));
                inv_S = S > 0.0f || S != S ? __fdividef(1.0f, S) : 0.0f;
            }
            const float any = (part[0] + part[1]) + (part[2] + part[3]);
            nan = bias_nan || any != any;
            // a place past E has score 0 and key -inf
            if (bias) {
#pragma unroll
                for (int j = 0; j < VPL; ++j)
                    v[j] = fmaf(v[j], inv_S, in(j) ? __ldg(bias + lane + 32 * j) : NEG_INF);
            } else {
#pragma unroll
                for (int j = 0; j < VPL; ++j) v[j] = fmaf(v[j], inv_S, in(j) ? 0.0f : NEG_INF);
            }
        }
        // bound on the error of a key k, whose score is at most k - bmin
        auto error_of = [&](float k) {
            if (by_z) {
                // logits are exact; where the 64-bit score hardly depends on them they decide nothing: next to
                // 0, and sigmoids that are 1 in 64 bits (from 37 on, and by the line below up to 80)
                if (sigmoid ? k < -700.0f || k > 80.0f : m0 - k > 700.0f) return __int_as_float(0x7f800000);
                return 1e-13f + (sigmoid ? 1e-15f * __expf(k) : 0.0f);
            }
            const float rel = (sigmoid ? 0x1p-16f : 0x1p-15f) * (k - bmin), all = (sigmoid ? 7.0f : 33.0f * inv_S) * U23;
            return fminf(rel, all) + U23 * fabsf(k) + 1e-37f;
        };
        // kept: the groups that stay (0: a key or a group's score is NaN)
        uint32_t kept = __any_sync(FULL, nan) ? 0u : FULL;
        if (grouped && kept) {
            // group scores: teams of lanes over the keys in shared memory
            __syncwarp();
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (in(j)) row32[lane + 32 * j + group_of(lane + 32 * j) * pad] = v[j];
            __syncwarp();
            const int g = lane / team, part = lane % team;
            float a = NEG_INF, b = NEG_INF;
            if (g < o.groups)
                for (int i = part; i < size; i += team) {
                    const float k = row32[g * (size + pad) + i];
                    b = fmaxf(b, fminf(a, k));
                    a = fmaxf(a, k);
                }
            for (int w = 1; w < team; w <<= 1) {
                const float a2 = __shfl_xor_sync(FULL, a, w), b2 = __shfl_xor_sync(FULL, b, w);
                b = fmaxf(fminf(a, a2), fmaxf(b, b2));
                a = fmaxf(a, a2);
            }
            const bool two = o.group_rank == 2 && size > 1;
            float score = two ? a + b : a;
            // two finite keys whose sum fp32 cannot hold: left to 64 bits, as a NaN
            if (two && isinf(score) && !isinf(a) && !isinf(b)) score = __int_as_float(0x7fc00000);
            float err = two ? error_of(a) + error_of(b) + U23 * fabsf(score) : error_of(a);
            // lane g: group g
            score = __shfl_sync(FULL, score, (lane * team) & 31);
            err = __shfl_sync(FULL, err, (lane * team) & 31);
            if (lane >= o.groups) score = NEG_INF;
            int rank = 0;
            for (int q = 0; q < o.groups; ++q) {
                const float other = __shfl_sync(FULL, score, q);
                rank += other > score || (other == score && q < lane);
            }
            kept = __ballot_sync(FULL, lane < o.groups && rank < o.top_groups);
            // The groups that stay and those that leave are apart by their bounds. Where keys have a bias, an
            // infinite score is what it is in 64 bits, and one of -inf that leaves is never above one that stays.
            const bool sure = !by_z && isinf(score);
            float low = __int_as_float(0x7f800000), high = NEG_INF;
            if ((kept >> lane) & 1u) {
                if (!sure) low = isinf(err) ? NEG_INF : score - err;
            } else if (lane < o.groups && score != NEG_INF) {
                high = score + err;
            }
            low = redux_min(low);
            high = redux_max(high);
            if (!(low > high) || __any_sync(FULL, score != score)) {
                keys64(zt, bias, E, sigmoid, m, row64);
                kept = groups64(row64, o, size, team);
            }
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int i = lane + 32 * j;
                if (in(j) && !((kept >> group_of(i)) & 1u)) v[j] = NEG_INF;
            }
        }
        int total = 0;
        if (kept) {
            // the K-th largest of the lanes' largest keys is at most the K-th largest key
            const float tau = __shfl_sync(FULL, sort_descending(largest(v), dir), K - 1);
            const float least = tau - 2.0f * error_of(tau) - U23 * fabsf(tau);
            if (least > NEG_INF) {
                // the places that hold candidates, as bits of numbers below 2^16
                constexpr int WORDS = (VPL + 15) / 16;
                uint32_t bits[WORDS];
                int mine = 0;
#pragma unroll
                for (int h = 0; h < WORDS; ++h) {
                    float sum = 0.0f;
#pragma unroll
                    for (int j = (16 * h + 15 < VPL ? 16 * h + 15 : VPL - 1); j >= 16 * h; --j)
                        sum = fmaf(sum, 2.0f, is_ge(v[j], least));
                    bits[h] = static_cast<uint32_t>(sum);
                    mine += __popc(bits[h]);
                }
                int before = mine;
#pragma unroll
                for (int w = 1; w < 32; w <<= 1) {
                    const int n = __shfl_up_sync(FULL, before, w);
                    if (lane >= w) before += n;
                }
                total = __shfl_sync(FULL, before, 31);
                __syncwarp();
                if (total <= 32) {
                    before -= mine;
#pragma unroll
                    for (int h = 0; h < WORDS; ++h)
                        while (bits[h]) {
                            cand[before++] = lane + 32 * (16 * h + __ffs(bits[h]) - 1);
                            bits[h] &= bits[h] - 1;
                        }
                }
            }
        }
        int my_idx;
        float z = NEG_INF;
        if (total && total <= 32) {
            __syncwarp();
            // one candidate a lane: key and bound again, then its rank among them
            int i = lane < total ? cand[lane] : 0x7fffffff;
            float k = NEG_INF, err = 0.0f, b = 0.0f;
            if (lane < total) {
                z = load_logit(zt + i);
                b = bias ? __ldg(bias + i) : 0.0f;
                if (by_z) {
                    k = z;
                    err = error_of(z);
                } else if (sigmoid) {
                    const float s = __fdividef(1.0f, 1.0f + __expf(-z));
                    k = s + b;
                    err = s * (3.5f + (1.0f - s) * (2.0f + 1.2f * fminf(fabsf(z), 88.0f))) * U23 + U23 * fabsf(k) + 1e-37f;
                } else {
                    const float s = __expf(z - m0) * inv_S;
                    k = s + b;
                    err = s * (33.0f + 1.7f * fminf(m0 - z, 88.0f)) * U23 + U23 * fabsf(k) + 1e-37f;
                }
            }
            float above = 0.0f, level = 0.0f;  // candidates with a larger key, and with a key as large or larger
#pragma unroll 4
            for (int q = 0; q < total; ++q) {
                const float kq = __shfl_sync(FULL, k, q);
                above += is_gt(kq, k);
                level += is_ge(kq, k);
            }
            int rank = static_cast<int>(above);
            if (__any_sync(FULL, lane < total && level - above > 1.0f)) {  // equal keys: lower expert first
                rank = 0;
                for (int q = 0; q < total; ++q) {
                    const float kq = __shfl_sync(FULL, k, q);
                    const int iq = __shfl_sync(FULL, i, q);
                    rank += kq > k || (kq == k && iq < i);
                }
            }
            // The first K in the order: neighbours apart by their bounds, or equal in logit and bias. Every
            // candidate behind them: the same against the K-th (neighbours that are apart say nothing about
            // a third with a wider bound).
            __syncwarp();
            if (lane < total) cand[rank] = lane;
            __syncwarp();
            const int from = lane < total ? cand[lane] : lane;
            const int i_s = __shfl_sync(FULL, i, from);
            const float k_s = __shfl_sync(FULL, k, from), e_s = __shfl_sync(FULL, err, from);
            const float z_s = __shfl_sync(FULL, z, from), b_s = __shfl_sync(FULL, b, from);
            const int other = lane < K - 1 ? lane + 1 : K - 1;
            const float k_n = __shfl_sync(FULL, k_s, other), e_n = __shfl_sync(FULL, e_s, other);
            const float z_n = __shfl_sync(FULL, z_s, other), b_n = __shfl_sync(FULL, b_s, other);
            const bool same = z_s == z_n && b_s == b_n;
            const bool close = lane < total && !(fabsf(k_s - k_n) > e_s + e_n) && !same;
            my_idx = i_s;
            z = z_s;
            if (__any_sync(FULL, close)) {
                const double S64 = sigmoid ? 1.0 : softmax_sum64(zt, E, m);
                z = lane < total ? load_logit(zt + i) : NEG_INF;
                const double k64 = lane < total ? score64(z, m, S64, sigmoid) + static_cast<double>(b) : -INFINITY;
                rank = 0;
                for (int q = 0; q < total; ++q) {
                    const double kq = __shfl_sync(FULL, k64, q);
                    const int iq = __shfl_sync(FULL, i, q);
                    rank += kq > k64 || (kq == k64 && iq < i);
                }
                __syncwarp();
                if (lane < total) cand[rank] = i;
                __syncwarp();
                my_idx = lane < total ? cand[lane] : 0;
                z = load_logit(zt + my_idx);
            }
        } else {
            const bool nan64 = keys64(zt, bias, E, sigmoid, m, row64);
            if (nan64) kept = 0;
            else if (grouped && !kept) kept = groups64(row64, o, size, team);
            else if (!kept) kept = FULL;
            my_idx = kept ? pick64(row64, E, K, kept, grouped ? size : E) : lane;
            if (lane < K) z = load_logit(zt + my_idx);
        }
        __syncwarp();
        const bool bad = !kept;
        if (bad && lane == 0) set_status(status, LC_MOE_DEV_NAN_KEY);
        // gates, from the chosen logits
        if (lane >= K) z = NEG_INF;
        float g;
        if (o.renorm) g = chosen_share(z, sigmoid);
        else if (sigmoid) g = sigmoid32(z);
        else g = expf(z - m0) * inv_S;
        if (lane < K) {
            const int64_t at = t * K + lane;
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

// W consecutive values of a row, as one 16-byte access where W allows.
template <class LT, int W>
struct Vec;
template <class LT>
struct Vec<LT, 1> {
    static __device__ __forceinline__ void load(const LT* p, float* v) { v[0] = load_logit(p); }
    static __device__ __forceinline__ void store(LT* p, const float* v) { store_logit(p, v[0]); }
};
template <>
struct Vec<float, 4> {
    static __device__ __forceinline__ void load(const float* p, float* v) {
        const float4 q = __ldcs(reinterpret_cast<const float4*>(p));
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    }
    static __device__ __forceinline__ void store(float* p, const float* v) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    }
};
template <>
struct Vec<__nv_bfloat16, 8> {
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* v) {
        const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) v[2 * j] = bf16lo(w[j]), v[2 * j + 1] = bf16hi(w[j]);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) {
        __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                       pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
    }
};

// One warp per token. The row is written in full first, then the chosen entries over it. V: values
// a lane holds of the row (0: nothing of it is needed, every entry that is not chosen is 0). Rows
// are read and written once, in 16-byte pieces (W values) where E and the pointers allow; what
// bounds it is memory: 16384 x 768 fp32 in 20.4 us (5.0 TB/s) with inputs that are not in L2. Up to 24
// values a lane 40 registers do with 20 bytes of spills: 6 CTAs an SM take 21.3 us where 64 registers and 4
// CTAs take 21.6 (six sets of tensors in turn).
template <class LT, int W, int V>
__global__ void __launch_bounds__(GATE_THREADS, V <= 24 ? 6 : 1)
    gate_backward_kernel(const LT* __restrict__ logits, const int32_t* __restrict__ idx,
                         const float* __restrict__ dgate, int T, int E, int K, lc_moe_gate_opts o,
                         LT* __restrict__ dlogits, uint32_t* __restrict__ status) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (GATE_THREADS / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (t >= T) return;
    const bool sigmoid = o.score == LC_MOE_SCORE_SIGMOID;
    const float NEG_INF = __int_as_float(0xff800000);
    const LT* zt = logits + t * E;
    LT* out = dlogits + t * E;
    constexpr int NV = V / W;
    float e[V > 0 ? V : 1];
    if (V > 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int at = (lane + 32 * j) * W;
#pragma unroll
            for (int w = 0; w < W; ++w) e[j * W + w] = NEG_INF;
            if (at < E) Vec<LT, W>::load(zt + at, e + j * W);
        }
    }
    int i = -1;
    float z = NEG_INF, dg = 0.0f;
    if (lane < K) {
        i = idx[t * K + lane];
        if (i < 0 || i >= E) {
            set_status(status, LC_MOE_DEV_IDX_RANGE);
            i = -1;
        } else {
            z = load_logit(zt + i);
            dg = dgate[t * K + lane];
        }
    }
    // every logit is reached (V > 0): dgate itself; else dz of the chosen logit, before the factor
    float mine = dg;
    float inv_S = 0.0f, m = 0.0f, D = 0.0f, share = 0.0f;
    if (V > 0) {
        m = NEG_INF;
#pragma unroll
        for (int j = 0; j < V; ++j) m = fmaxf(m, e[j]);
        m = redux_max(m);
        if (m == NEG_INF) m = 0.0f;  // every logit is -inf: all scores are 0
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            e[j] = __expf(e[j] - m);
            part += e[j];
        }
        const float S = warp_sum(part);
        inv_S = S > 0.0f || S != S ? 1.0f / S : 0.0f;
        share = i >= 0 ? __expf(z - m) * inv_S : 0.0f;
        D = warp_sum(share * dg);
    } else if (o.renorm) {
        const float p = chosen_share(z, sigmoid);
        const float f = sigmoid ? 1.0f / (1.0f + expf(z)) : 1.0f;
        // dg_r - sum_q p_q dg_q as sum_q p_q (dg_r - dg_q): a pick that has nearly all of the share does
        // not lose its small gradient in the difference
        float apart = 0.0f;
        for (int q = 0; q < K; ++q) apart = fmaf(__shfl_sync(FULL, p, q), dg - __shfl_sync(FULL, dg, q), apart);
        mine = p * f * apart;
    } else {
        const float q = expf(-fabsf(z));
        mine = dg * q / ((1.0f + q) * (1.0f + q));
    }
    // picks of the same expert add up, in rank order, at the first of them
    const uint32_t same = __match_any_sync(FULL, i);
    float total = mine;
    const bool repeated = __any_sync(FULL, i >= 0 && __popc(same) > 1);
    if (repeated) {
        total = 0.0f;
        for (int r = 0; r < K; ++r) {
            const float v = __shfl_sync(FULL, mine, r);
            if ((same >> r) & 1u) total += v;
        }
    }
    const bool first = i >= 0 && lane == __ffs(same) - 1;
    if (V > 0) {
        const float c = -inv_S * (o.scale * D), ds = total;
        if (warp_sum(first ? share : 0.0f) > 0.75f) {
            // The picks hold most of the share: ds - D may be a small difference of nearly equal numbers. With 1
            // as the sum of all shares it is sum_q s_q (ds - ds_q) over the picked experts plus ds times the
            // shares of the others, which are summed by themselves. Where the others hold a quarter or more, so
            // does their part ds * rest, and ds - D keeps within some tens of half steps of the sizes added
            // (from 0.5 on 16.0 us from L2 at 16384 x 768, from 0.75 on 14.8, from 0.9 on 14.4).
            const uint32_t firsts = __ballot_sync(FULL, first);
            using Bits = typename std::conditional<(V > 32), unsigned long long, uint32_t>::type;
            Bits chosen = 0;  // of this lane's places
            float apart = 0.0f;
            for (int q = 0; q < K; ++q) {
                const int iq = __shfl_sync(FULL, i, q);
                const float s_q = __shfl_sync(FULL, share, q), apart_q = ds - __shfl_sync(FULL, ds, q);
                if (!((firsts >> q) & 1u)) continue;  // no pick, or an expert that an earlier pick has named
                const int place = iq / W;
                if (place % 32 == lane) chosen |= Bits(1) << (place / 32 * W + iq % W);
                apart = fmaf(s_q, apart_q, apart);
            }
            float rest = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) rest += (chosen >> j) & 1u ? 0.0f : e[j];
            total = share * fmaf(ds, warp_sum(rest) * inv_S, apart);
        } else {
            total = share * (ds - D);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int at = (lane + 32 * j) * W;
#pragma unroll
            for (int w = 0; w < W; ++w) e[j * W + w] *= c;
            if (at < E) Vec<LT, W>::store(out + at, e + j * W);
        }
    } else {
        const float zero[W] = {};
        for (int at = lane * W; at < E; at += 32 * W) Vec<LT, W>::store(out + at, zero);
    }
    __syncwarp();  // the row's entries are written before the chosen ones
    if (first) store_logit(out + i, o.scale * total);
}

}  // namespace

namespace {

template <class LT, int VPL, bool FILLED>
cudaError_t launch_gate_f(const LT* logits, const float* bias, int T, int E, int K, const lc_moe_gate_opts& o,
                          int32_t* idx, float* gate, int32_t* counts, uint32_t* status, cudaStream_t st) {
    const DevInfo* di = current_device_info();
    if (!di) return cudaErrorUnknown;
    constexpr int MAX_WARPS = VPL <= 32 ? 8 : 4;
    constexpr int MAX_SMEM = MAX_WARPS * (32 * VPL * 8 + 32 * 31 * 4) + 32 * VPL * 4;
    static PerDeviceOnce setup;
    const cudaError_t e = setup.run([](int) {
        return cudaFuncSetAttribute(gate_kernel<LT, VPL, FILLED>, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM);
    });
    if (e != cudaSuccess) return e;
    // few tokens: spread them over the SMs
    const int warps = T <= di->sm_count ? 1 : T <= 4 * di->sm_count ? 2 : MAX_WARPS;
    int team = 32;
    while (team * o.groups > 32) team >>= 1;
    const int pad = (team - E / o.groups) & 31;
    int row_len = E > 32 ? E : 32;
    if (o.top_groups < o.groups && (E + o.groups * pad + 1) / 2 > row_len) row_len = (E + o.groups * pad + 1) / 2;
    const size_t smem = static_cast<size_t>(warps) * row_len * 8 + (counts ? static_cast<size_t>(E) * 4 : 0);
    int blocks = (T - 1) / warps + 1;
    if (blocks > di->sm_count * gate_ctas(VPL)) blocks = di->sm_count * gate_ctas(VPL);  // one wave
    gate_kernel<LT, VPL, FILLED><<<blocks, warps * 32, smem, st>>>(logits, bias, T, E, K, o, team, pad, row_len, idx, gate,
                                                                 counts, status);
    return cudaGetLastError();
}

template <class LT, int VPL>
cudaError_t launch_gate_t(const LT* logits, const float* bias, int T, int E, int K, const lc_moe_gate_opts& o,
                          int32_t* idx, float* gate, int32_t* counts, uint32_t* status, cudaStream_t st) {
    if (E == 32 * VPL) return launch_gate_f<LT, VPL, true>(logits, bias, T, E, K, o, idx, gate, counts, status, st);
    return launch_gate_f<LT, VPL, false>(logits, bias, T, E, K, o, idx, gate, counts, status, st);
}

template <class LT>
cudaError_t launch_gate_l(const LT* logits, const float* bias, int T, int E, int K, const lc_moe_gate_opts& o,
                          int32_t* idx, float* gate, int32_t* counts, uint32_t* status, cudaStream_t st) {
    const int vpl = (E + 31) / 32;
    if (vpl <= 1) return launch_gate_t<LT, 1>(logits, bias, T, E, K, o, idx, gate, counts, status, st);
    if (vpl <= 4) return launch_gate_t<LT, 4>(logits, bias, T, E, K, o, idx, gate, counts, status, st);
    if (vpl <= 8) return launch_gate_t<LT, 8>(logits, bias, T, E, K, o, idx, gate, counts, status, st);
    if (vpl <= 12) return launch_gate_t<LT, 12>(logits, bias, T, E, K, o, idx, gate, counts, status, st);
    if (vpl <= 16) return launch_gate_t<LT, 16>(logits, bias, T, E, K, o, idx, gate, counts, status, st);
    if (vpl <= 24) return launch_gate_t<LT, 24>(logits, bias, T, E, K, o, idx, gate, counts, status, st);
    if (vpl <= 32) return launch_gate_t<LT, 32>(logits, bias, T, E, K, o, idx, gate, counts, status, st);
    return launch_gate_t<LT, 64>(logits, bias, T, E, K, o, idx, gate, counts, status, st);
}

}  // namespace

cudaError_t launch_gate(const void* logits, int bf16, const float* bias, int T, int E, int K,
                        const lc_moe_gate_opts& o, int32_t* idx, float* gate, int32_t* counts,
                        uint32_t* status, cudaStream_t st) {
    if (bf16)
        return launch_gate_l(static_cast<const __nv_bfloat16*>(logits), bias, T, E, K, o, idx, gate, counts, status, st);
    return launch_gate_l(static_cast<const float*>(logits), bias, T, E, K, o, idx, gate, counts, status, st);
}

namespace {

template <class LT, int W>
void launch_gate_backward_w(const LT* logits, const int32_t* idx, const float* dgate, int T, int E, int K,
                            const lc_moe_gate_opts& o, LT* dlogits, uint32_t* status, cudaStream_t st) {
    constexpr int WARPS = GATE_THREADS / 32;
    const int blocks = (T - 1) / WARPS + 1;
    const int vpl = o.score == LC_MOE_SCORE_SOFTMAX && !o.renorm ? ((E + W - 1) / W + 31) / 32 * W : 0;
#define LC_GATE_BWD(V) \
    gate_backward_kernel<LT, W, V><<<blocks, GATE_THREADS, 0, st>>>(logits, idx, dgate, T, E, K, o, dlogits, status)
    if (vpl == 0) LC_GATE_BWD(0);
    else if (vpl <= 8) LC_GATE_BWD(8);
    else if (vpl <= 16) LC_GATE_BWD(16);
    else if (vpl <= 24) LC_GATE_BWD(24);
    else if (vpl <= 32) LC_GATE_BWD(32);
    else LC_GATE_BWD(64);
#undef LC_GATE_BWD
}

}  // namespace

cudaError_t launch_gate_backward(const void* logits, int bf16, const int32_t* idx, const float* dgate, int T,
                                 int E, int K, const lc_moe_gate_opts& o, void* dlogits, uint32_t* status,
                                 cudaStream_t st) {
    const bool aligned = ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(dlogits)) & 15u) == 0;
    if (bf16) {
        const __nv_bfloat16* z = static_cast<const __nv_bfloat16*>(logits);
        __nv_bfloat16* dz = static_cast<__nv_bfloat16*>(dlogits);
        if (aligned && E % 8 == 0) launch_gate_backward_w<__nv_bfloat16, 8>(z, idx, dgate, T, E, K, o, dz, status, st);
        else launch_gate_backward_w<__nv_bfloat16, 1>(z, idx, dgate, T, E, K, o, dz, status, st);
    } else {
        const float* z = static_cast<const float*>(logits);
        float* dz = static_cast<float*>(dlogits);
        if (aligned && E % 4 == 0) launch_gate_backward_w<float, 4>(z, idx, dgate, T, E, K, o, dz, status, st);
        else launch_gate_backward_w<float, 1>(z, idx, dgate, T, E, K, o, dz, status, st);
    }
    return cudaGetLastError();
}

}  // namespace lcmoe
