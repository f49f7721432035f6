// combine.cu -- the weighted sum of the MoE equation, with the zero-computation experts fused.
//
//   out_t = sum_{r < K} g_{t,r} * v_{t,r},   v = Y[pair_row] for an FFN pick,
//                                            v = x_t          for a zero-computation pick
// (LongCat-Flash llm-wiki entity page, section 2.1: E_i(x_t) = x_t for the Z zero experts).
// One warp per token; each lane owns 8-element (16-byte) column chunks and accumulates in fp32,
// in rank order, with one fused multiply-add per pick: the zero-expert term costs one read of
// x_t per token (shared by all its zero picks) and no extra pass.
//
// Its gradient, for the same picks:
//   dgate_{t,r} = sum_c dout_{t,c} v_{t,r,c}
//   dY[pair_row] = g_{t,r} dout_t                (rows of Y are in one pick each, so none adds up)
//   dx_t = (sum of the gates of t's zero picks) dout_t
// with the products and sums in fp32 and one rounding to bf16 at dY and dx.
#include "common.cuh"

namespace lcmoe {

namespace {

constexpr int COMBINE_THREADS = 256;

// Loads in flight per lane: two 16-byte column chunks (c and c + 32) of PB picks at a time.
constexpr int PB = 4;

__device__ __forceinline__ void fma_row(float (&acc)[8], float g, const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        acc[2 * j] = __fmaf_rn(g, bf16lo(w[j]), acc[2 * j]);
        acc[2 * j + 1] = __fmaf_rn(g, bf16hi(w[j]), acc[2 * j + 1]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&acc)[8]) {
    return make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                      pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
}

// Work item: one token's row (SPLIT = false), or a (token, column block) of `span` 16-byte chunks
// (SPLIT = true, when T is too small for one warp per token to fill the GPU).
template <bool SPLIT>
__global__ void __launch_bounds__(COMBINE_THREADS)
    combine_kernel(const uint4* __restrict__ x, const uint4* __restrict__ y,
                   const float* __restrict__ gate, const int32_t* __restrict__ pair_row, int T,
                   int d8, int K, int cb, int span, uint4* __restrict__ out) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int warps_total = gridDim.x * (COMBINE_THREADS / 32);
    const int items = SPLIT ? T * cb : T;  // T * cb stays near the warp count of one wave
    for (int it = blockIdx.x * (COMBINE_THREADS / 32) + warp; it < items; it += warps_total) {
        const int t = SPLIT ? it / cb : it;
        const int c_begin = SPLIT ? (it - t * cb) * span : 0;
        const int c_end = SPLIT ? min(d8, c_begin + span) : d8;
        float my_g = 0.0f;
        int my_row = -1;
        if (lane < K) {
            my_g = gate[static_cast<int64_t>(t) * K + lane];
            my_row = pair_row[static_cast<int64_t>(t) * K + lane];
        }
        const bool any_zero = __any_sync(0xffffffffu, lane < K && my_row < 0);
        const uint4* xt = x + static_cast<int64_t>(t) * d8;
        for (int c0 = c_begin; c0 < c_end; c0 += 64) {  // warp-uniform trip count
            const int ca = c0 + lane, cb2 = c0 + 32 + lane;
            const bool ina = ca < c_end, inb = cb2 < c_end;
            uint4 xa = make_uint4(0, 0, 0, 0), xb = xa;
            if (any_zero) {
                if (ina) xa = __ldg(xt + ca);
                if (inb) xb = __ldg(xt + cb2);
            }
            float acc_a[8], acc_b[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) acc_a[j] = acc_b[j] = 0.0f;
            for (int r0 = 0; r0 < K; r0 += PB) {
                float g[PB];
                int row[PB];
                uint4 va[PB], vb[PB];
#pragma unroll
                for (int u = 0; u < PB; ++u) {
                    g[u] = __shfl_sync(0xffffffffu, my_g, (r0 + u) & 31);
                    row[u] = __shfl_sync(0xffffffffu, my_row, (r0 + u) & 31);
                }
#pragma unroll
                for (int u = 0; u < PB; ++u) {
                    const bool pick = r0 + u < K;
                    const uint4* yr = y + static_cast<int64_t>(row[u] < 0 ? 0 : row[u]) * d8;
                    va[u] = (pick && row[u] >= 0 && ina) ? __ldg(yr + ca) : xa;
                    vb[u] = (pick && row[u] >= 0 && inb) ? __ldg(yr + cb2) : xb;
                }
                // rank order: pick r0, r0 + 1, ... each one fused multiply-add per element
#pragma unroll
                for (int u = 0; u < PB; ++u) {
                    if (r0 + u < K) {
                        fma_row(acc_a, g[u], va[u]);
                        fma_row(acc_b, g[u], vb[u]);
                    }
                }
            }
            if (ina) out[static_cast<int64_t>(t) * d8 + ca] = pack8(acc_a);
            if (inb) out[static_cast<int64_t>(t) * d8 + cb2] = pack8(acc_b);
        }
    }
}

__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float s) {
    const uint32_t p[4] = {a.x, a.y, a.z, a.w}, q[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        s = __fmaf_rn(bf16lo(p[j]), bf16lo(q[j]), s);
        s = __fmaf_rn(bf16hi(p[j]), bf16hi(q[j]), s);
    }
    return s;
}

__device__ __forceinline__ uint4 times8(float g, const uint4& v) {
    float acc[8];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        acc[2 * j] = g * bf16lo(w[j]);
        acc[2 * j + 1] = g * bf16hi(w[j]);
    }
    return pack8(acc);
}

__device__ __forceinline__ float warp_total(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A team of wpt warps per token holds the token's row of dout in registers (NC 16-byte chunks a
// lane) and passes over its picks, two at a time: every row of Y is read once and its gradient
// written once, dout and x are read once. Lane r keeps the sum of pick r; the warps' sums join in
// shared memory in warp order. With few tokens blockIdx.y deals the picks out to `splits` CTAs.
// Memory bounds it; loads in flight decide: T = 16384, d = 6144, 8 FFN picks a token on average (3.8 GB)
// in 727 us with 2 CTAs an SM, 630 with 3, 625 with 4 (6.1 TB/s).
template <int NC>
__global__ void __launch_bounds__(COMBINE_THREADS, NC <= 3 ? 4 : 3)
    combine_backward_kernel(const uint4* __restrict__ dout, const uint4* __restrict__ x,
                            const uint4* __restrict__ y, int64_t y_rows, const float* __restrict__ gate,
                            const int32_t* __restrict__ pair_row, int T, int d8, int K, int wpt, int splits,
                            uint4* __restrict__ dy, float* __restrict__ dgate, uint4* __restrict__ dx,
                            uint32_t* __restrict__ status) {
    __shared__ float s_sum[COMBINE_THREADS / 32][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int teams = (COMBINE_THREADS / 32) / wpt, tw = warp % wpt;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * teams + warp / wpt;
    const bool live = t < T;
    float g = 0.0f, sum = 0.0f;
    int row = -1;
    if (live && lane < K) {
        g = gate[t * K + lane];
        row = pair_row[t * K + lane];
    }
    const bool mine = live && lane < K && lane % splits == static_cast<int>(blockIdx.y);
    if (live) {
        const bool bad = row >= y_rows;
        if (mine && bad && tw == 0) set_status(status, LC_MOE_DEV_IDX_RANGE);
        const uint32_t zeros = __ballot_sync(0xffffffffu, mine && row < 0);
        const uint32_t rows = __ballot_sync(0xffffffffu, mine && row >= 0 && !bad);
        const float g_zero = warp_total(row < 0 ? g : 0.0f);
        for (int c0 = tw * 32 * NC + lane; c0 - lane < d8; c0 += wpt * 32 * NC) {
            uint4 o[NC];
#pragma unroll
            for (int i = 0; i < NC; ++i) o[i] = c0 + 32 * i < d8 ? __ldg(dout + t * d8 + c0 + 32 * i) : make_uint4(0, 0, 0, 0);
            if (blockIdx.y == 0) {
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (c0 + 32 * i < d8) __stcs(dx + t * d8 + c0 + 32 * i, times8(g_zero, o[i]));
            }
            if (zeros) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (c0 + 32 * i < d8) s = dot8(o[i], __ldcs(x + t * d8 + c0 + 32 * i), s);
                s = warp_total(s);
                if ((zeros >> lane) & 1u) sum += s;
            }
            for (uint32_t left = rows; left;) {
                const int ra = __ffs(left) - 1;
                left &= left - 1;
                const int rb = left ? __ffs(left) - 1 : -1;  // the second pick of the pair, if there is one
                left &= left ? left - 1 : 0;
                const int64_t ya = static_cast<int64_t>(__shfl_sync(0xffffffffu, row, ra)) * d8;
                const int64_t yb = static_cast<int64_t>(__shfl_sync(0xffffffffu, row, rb & 31)) * d8;
                const float ga = __shfl_sync(0xffffffffu, g, ra), gb = __shfl_sync(0xffffffffu, g, rb & 31);
                uint4 va[NC], vb[NC];
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    va[i] = vb[i] = make_uint4(0, 0, 0, 0);
                    if (c0 + 32 * i < d8) {
                        va[i] = __ldcs(y + ya + c0 + 32 * i);
                        if (rb >= 0) vb[i] = __ldcs(y + yb + c0 + 32 * i);
                    }
                }
                float sa = 0.0f, sb = 0.0f;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    if (c0 + 32 * i < d8) {
                        __stcs(dy + ya + c0 + 32 * i, times8(ga, o[i]));
                        if (rb >= 0) __stcs(dy + yb + c0 + 32 * i, times8(gb, o[i]));
                    }
                    sa = dot8(o[i], va[i], sa);
                    sb = dot8(o[i], vb[i], sb);
                }
                sa = warp_total(sa);
                sb = warp_total(sb);
                if (lane == ra) sum += sa;
                if (lane == rb) sum += sb;
            }
        }
        if (bad) sum = 0.0f;
    }
    if (wpt == 1) {
        if (mine) dgate[t * K + lane] = sum;
        return;
    }
    s_sum[warp][lane] = sum;
    __syncthreads();
    if (mine && tw == 0) {
        float all = 0.0f;
        for (int w = 0; w < wpt; ++w) all += s_sum[warp + w][lane];
        dgate[t * K + lane] = all;
    }
}

}  // namespace

cudaError_t launch_combine_backward(const void* dout, const void* x, const void* y, int64_t y_rows,
                                    const float* gate, const int32_t* pair_row, int T, int d, int K, void* dy,
                                    float* dgate, void* dx, uint32_t* status, cudaStream_t st) {
    const DevInfo* di = current_device_info();
    if (!di) return cudaErrorUnknown;
    if (T == 0) return cudaSuccess;
    const int warps = COMBINE_THREADS / 32, d8 = d / 8;
    // as many warps to a token as leave a lane at most 4 chunks of its row (or all 8)
    int wpt = 1;
    while (wpt < warps && d8 > wpt * 32 * 4) wpt *= 2;
    const int teams = warps / wpt;
    const int blocks = (T - 1) / teams + 1;
    // few tokens: deal a token's picks out until there are 2 CTAs an SM
    int splits = 1;
    while (splits < K && blocks * splits < 2 * di->sm_count) splits *= 2;
    if (splits > K) splits = K;
    const int nc = (d8 + wpt * 32 - 1) / (wpt * 32);
    const dim3 grid(blocks, splits);
    const auto launch = [&](auto kernel) {
        kernel<<<grid, COMBINE_THREADS, 0, st>>>(static_cast<const uint4*>(dout), static_cast<const uint4*>(x),
                                                 static_cast<const uint4*>(y), y_rows, gate, pair_row, T, d8, K, wpt, splits,
                                                 static_cast<uint4*>(dy), dgate, static_cast<uint4*>(dx), status);
    };
    if (nc == 1) launch(combine_backward_kernel<1>);
    else if (nc == 2) launch(combine_backward_kernel<2>);
    else if (nc == 3) launch(combine_backward_kernel<3>);
    else launch(combine_backward_kernel<4>);
    return cudaGetLastError();
}

cudaError_t launch_combine(const void* x, const void* y, const float* gate,
                           const int32_t* pair_row, int T, int d, int K, void* out,
                           cudaStream_t st) {
    const DevInfo* di = current_device_info();
    if (!di) return cudaErrorUnknown;
    if (T == 0) return cudaSuccess;
    const int warps = COMBINE_THREADS / 32;
    const int d8 = d / 8;
    // column blocks per token: enough (token, block) items for 8 blocks of 8 warps per SM
    const int max_cb = (d8 + 63) / 64;
    int cb = (di->sm_count * 8 * warps + T - 1) / T;
    if (cb > max_cb) cb = max_cb;
    if (cb < 1) cb = 1;
    const int span = ((d8 + cb - 1) / cb + 63) / 64 * 64;
    cb = (d8 + span - 1) / span;
    const int64_t items = static_cast<int64_t>(T) * cb;
    int64_t blocks = (items + warps - 1) / warps;
    if (blocks > di->sm_count * 8) blocks = di->sm_count * 8;
    if (cb > 1)
        combine_kernel<true><<<static_cast<int>(blocks), COMBINE_THREADS, 0, st>>>(
            static_cast<const uint4*>(x), static_cast<const uint4*>(y), gate, pair_row, T, d8, K, cb, span,
            static_cast<uint4*>(out));
    else
        combine_kernel<false><<<static_cast<int>(blocks), COMBINE_THREADS, 0, st>>>(
            static_cast<const uint4*>(x), static_cast<const uint4*>(y), gate, pair_row, T, d8, K, 1, d8,
            static_cast<uint4*>(out));
    return cudaGetLastError();
}

}  // namespace lcmoe
