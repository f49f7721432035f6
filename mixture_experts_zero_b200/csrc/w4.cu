// w4.cu -- SwiGLU experts with 4-bit weights and a bf16 scale per group of input columns.
//
//   w[r, c] = (code[r, c] - 8) * scale[r, c / group],  code in 0..15, group 32, 64 or 128
//   H[rows_e, I] (bf16) = silu(X_e Wg[e]^T) * (X_e Wu[e]^T)
//   Y[rows_e, d] (bf16) = H_e Wd[e]^T
// for rows grouped by expert. A decode batch gives an expert a few rows, so the products are a
// stream of the weights: what bounds them is the 0.5 + 2 / group bytes a weight takes from HBM and
// the integer work that turns codes into operands.
//
// Layout. Codes are stored in tiles of 16 rows x 64 columns (512 bytes, tile rows then tile
// columns in order) whose lane (4 (r % 8) + (c % 32) / 8) owns 16 bytes: word 2 (c % 64 / 32) +
// r % 16 / 8 holds 8 consecutive columns of a row, nibble p the column 2 (p % 4) + p / 4 of them.
// A warp's 16-byte loads of a tile are then contiguous, and a lane gets exactly the codes of its
// places in the A operand of mma.m16n8k16: the order of the reduction's columns is free as long
// as both operands share it, so columns 8 t .. 8 t + 7 of a 32-column group are given to lane t of
// each quad (two k-steps of 4 columns a lane), which lets the lane read the 8 activations as 16
// contiguous bytes as well. Scales are [rows / 16][cols / group][8][2]: the two rows (r, r + 8)
// that a lane accumulates come as one 32-bit word.
//
// The legacy mma.sync path is used on purpose: with at most 8 rows an expert the 256 multiply-adds
// per weight code of an MMA are already mostly padding, and operands in registers spare the trip
// of the unpacked weights through shared memory that tcgen05 would need.
//
// Codes become bf16 exactly: 0x4300 | n is 128 + n in bf16, minus 136 gives n - 8. A group's sum is
// accumulated in fp32 on its own and then times its scale, so a scale is never rounded into a
// weight.
#include "common.cuh"

namespace lcmoe {

namespace {

constexpr uint32_t FULL = 0xffffffffu;

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
}

// nibbles p and p + 4 of a word as two bf16 values n - 8
template <int P>
__device__ __forceinline__ uint32_t codes_bf16x2(uint32_t w) {
    return sub_bf16x2(((w >> (4 * P)) & 0x000f000fu) | 0x43004300u, 0x43084308u);
}

// D += A B, m16n8k16, bf16 operands, fp32 accumulators
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float silu_mul(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

// ------------------------------------------------------------------------------- quantiser --

// One warp per 16 rows x (64 columns, or 128 when the group is 128). scale = bf16(amax / 7) (1 for
// a group whose scale would be 0), code = 8 + round(w / scale), a division in fp32, to nearest
// even, within -7..7.
__global__ void __launch_bounds__(256)
    quantize_w4_kernel(const __nv_bfloat16* __restrict__ src, int64_t tile_rows, int cols, int group,
                       uint4* __restrict__ codes, uint32_t* __restrict__ scale) {
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int span = group == 128 ? 128 : 64;
    const int units = cols / span;
    const int64_t total = tile_rows * units;
    const int64_t warps_total = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); it < total;
         it += warps_total) {
        const int64_t tr = it / units;
        const int c0 = static_cast<int>(it - tr * units) * span;
        for (int h = 0; h < 2; ++h) {
            const __nv_bfloat16* row = src + (tr * 16 + g + 8 * h) * cols + c0 + 8 * t;
            uint4 v[4];
            float amax[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                amax[q] = 0.0f;
                if (32 * q >= span) continue;
                v[q] = *reinterpret_cast<const uint4*>(row + 32 * q);
                const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    amax[q] = fmaxf(amax[q], fmaxf(fabsf(bf16lo(w[j])), fabsf(bf16hi(w[j]))));
                amax[q] = fmaxf(amax[q], __shfl_xor_sync(FULL, amax[q], 1));
                amax[q] = fmaxf(amax[q], __shfl_xor_sync(FULL, amax[q], 2));
            }
            if (group >= 64) {
                amax[0] = amax[1] = fmaxf(amax[0], amax[1]);
                amax[2] = amax[3] = fmaxf(amax[2], amax[3]);
            }
            if (group == 128) {
                const float m = fmaxf(amax[0], amax[2]);
                amax[0] = amax[1] = amax[2] = amax[3] = m;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (32 * q >= span) continue;
                __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(amax[q], 7.0f));
                float s = __bfloat162float(sb);
                if (s == 0.0f) {
                    s = 1.0f;
                    sb = __float2bfloat16_rn(1.0f);
                }
                const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
                uint32_t word = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float x = (j & 1) ? bf16hi(w[j >> 1]) : bf16lo(w[j >> 1]);
                    const float n = fminf(fmaxf(rintf(__fdiv_rn(x, s)), -7.0f), 7.0f);
                    word |= static_cast<uint32_t>(static_cast<int>(n) + 8) << (4 * ((j >> 1) + 4 * (j & 1)));
                }
                const int c = c0 + 32 * q;
                uint32_t* tile = reinterpret_cast<uint32_t*>(codes + (tr * (cols / 64) + c / 64) * 32 + lane);
                tile[2 * (q & 1) + h] = word;
                if (t == 0 && c % group == 0)
                    reinterpret_cast<__nv_bfloat16*>(scale)[(tr * (cols / group) + c / group) * 16 + 2 * g + h] = sb;
            }
        }
    }
}

// --------------------------------------------------------------------------------- products --

struct W4Args {
    const int32_t* offsets;      // [N + 1] row offsets of the experts
    const __nv_bfloat16* x;      // [rows_cap, k] grouped rows
    const uint8_t* codes;        // [N][m / 16][k / 64][512]
    const uint32_t* scale;       // [N][m / 16][k / group][8] row pairs
    __nv_bfloat16* out;          // [rows_cap, n_out]
    uint32_t* status;
    int64_t rows_cap;
    int N, k, m, n_out, group;   // m: weight rows of an expert (2I or d)
};

constexpr int W4_THREADS = 256;
constexpr int RED = 68;  // padded feature stride of the partial sums

// Item: 64 weight rows of one expert (32 gate and 32 up rows, or 64 output features) times up to 8
// of its rows. A CTA's 8 warps split the reduction and join their sums in shared memory.
template <bool SWIGLU>
__global__ void __launch_bounds__(W4_THREADS) w4_kernel(const W4Args a) {
    extern __shared__ uint8_t s_raw[];
    float* red = reinterpret_cast<float*>(s_raw);                          // [8][8][RED]
    int64_t* pre = reinterpret_cast<int64_t*>(s_raw + 8 * 8 * RED * 4);    // [N + 1] item prefix sums
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int tiles = a.m / 64;
    if (warp == 0) {
        int64_t run = 0;
        if (lane == 0) pre[0] = 0;
        for (int base = 0; base < a.N; base += 32) {
            const int e = base + lane;
            int64_t n = 0;
            if (e < a.N) {
                int cnt = a.offsets[e + 1] - a.offsets[e];
                if (a.offsets[e] < 0 || cnt < 0 || a.offsets[e + 1] > a.rows_cap) {
                    cnt = 0;
                    set_status(a.status, LC_MOE_DEV_IDX_RANGE);
                }
                n = static_cast<int64_t>((cnt + 7) / 8) * tiles;
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(FULL, n, o);
                if (lane >= o) n += v;
            }
            if (e < a.N) pre[e + 1] = run + n;
            run += __shfl_sync(FULL, n, 31);
        }
    }
    __syncthreads();
    const int64_t total = pre[a.N];
    const int nk = a.k / 64, ngrp = a.k / a.group;
    for (int64_t item = blockIdx.x; item < total; item += gridDim.x) {
        int lo = 0, hi = a.N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] <= item) lo = mid;
            else hi = mid - 1;
        }
        const int e = lo;
        const int64_t local = item - pre[e];
        const int tile = static_cast<int>(local % tiles);
        const int64_t row0 = a.offsets[e] + (local / tiles) * 8;
        const int rows = static_cast<int>(min(static_cast<int64_t>(8), a.offsets[e + 1] - row0));
        // weight row blocks (16 rows) of this item: SwiGLU takes two of the gate and two of the up rows
        const int64_t mblk = a.m / 16;
        int blk[4];
#pragma unroll
        for (int b = 0; b < 4; ++b)
            blk[b] = SWIGLU ? (b >> 1) * (a.m / 32) + tile * 2 + (b & 1) : tile * 4 + b;
        const __nv_bfloat16* xr = a.x + (row0 + g) * a.k + 8 * t;
        float acc[4][4] = {};
        for (int ks = warp; ks < nk; ks += 8) {
            uint4 xv[2];
#pragma unroll
            for (int G = 0; G < 2; ++G)
                xv[G] = g < rows ? *reinterpret_cast<const uint4*>(xr + ks * 64 + 32 * G) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int64_t bb = e * mblk + blk[b];
                const uint4 w = *reinterpret_cast<const uint4*>(a.codes + ((bb * nk + ks) * 32 + lane) * 16);
                const uint32_t wr[2][2] = {{w.x, w.y}, {w.z, w.w}};
#pragma unroll
                for (int G = 0; G < 2; ++G) {
                    float s4[4] = {};
                    mma16816(s4, codes_bf16x2<0>(wr[G][0]), codes_bf16x2<0>(wr[G][1]), codes_bf16x2<1>(wr[G][0]),
                             codes_bf16x2<1>(wr[G][1]), xv[G].x, xv[G].y);
                    mma16816(s4, codes_bf16x2<2>(wr[G][0]), codes_bf16x2<2>(wr[G][1]), codes_bf16x2<3>(wr[G][0]),
                             codes_bf16x2<3>(wr[G][1]), xv[G].z, xv[G].w);
                    const uint32_t sc = a.scale[(bb * ngrp + (ks * 64 + 32 * G) / a.group) * 8 + g];
                    acc[b][0] += bf16lo(sc) * s4[0];
                    acc[b][1] += bf16lo(sc) * s4[1];
                    acc[b][2] += bf16hi(sc) * s4[2];
                    acc[b][3] += bf16hi(sc) * s4[3];
                }
            }
        }
        float* mine = red + warp * 8 * RED;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            mine[(2 * t) * RED + 16 * b + g] = acc[b][0];
            mine[(2 * t + 1) * RED + 16 * b + g] = acc[b][1];
            mine[(2 * t) * RED + 16 * b + g + 8] = acc[b][2];
            mine[(2 * t + 1) * RED + 16 * b + g + 8] = acc[b][3];
        }
        __syncthreads();
        constexpr int FEAT = SWIGLU ? 32 : 64;
        for (int i = threadIdx.x; i < 8 * FEAT; i += W4_THREADS) {
            const int n = i / FEAT, f = i % FEAT;
            if (n < rows) {
                float p = 0.0f, q = 0.0f;
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    p += red[(w * 8 + n) * RED + f];
                    if (SWIGLU) q += red[(w * 8 + n) * RED + 32 + f];
                }
                a.out[(row0 + n) * a.n_out + tile * FEAT + f] = __float2bfloat16_rn(SWIGLU ? silu_mul(p, q) : p);
            }
        }
        __syncthreads();
    }
}

template <bool SWIGLU>
cudaError_t launch_w4(const W4Args& a, cudaStream_t st) {
    const DevInfo* di = current_device_info();
    if (!di) return cudaErrorUnknown;
    const size_t smem = 8 * 8 * RED * 4 + (static_cast<size_t>(a.N) + 1) * 8;
    w4_kernel<SWIGLU><<<di->sm_count * 4, W4_THREADS, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_w4(const void* src, int64_t rows, int cols, int group, void* codes, void* scale,
                               cudaStream_t st) {
    const DevInfo* di = current_device_info();
    if (!di) return cudaErrorUnknown;
    const int64_t units = rows / 16 * (cols / (group == 128 ? 128 : 64));
    int64_t blocks = (units + 7) / 8;
    if (blocks > di->sm_count * 16) blocks = di->sm_count * 16;
    quantize_w4_kernel<<<static_cast<int>(blocks), 256, 0, st>>>(static_cast<const __nv_bfloat16*>(src), rows / 16, cols,
                                                                 group, static_cast<uint4*>(codes),
                                                                 static_cast<uint32_t*>(scale));
    return cudaGetLastError();
}

cudaError_t launch_swiglu_w4(const void* x_perm, int64_t rows_cap, const int32_t* offsets, int N, const void* w13q,
                             const void* w13_scale, int group, int d, int I, void* h, uint32_t* status,
                             cudaStream_t st) {
    W4Args a{offsets, static_cast<const __nv_bfloat16*>(x_perm), static_cast<const uint8_t*>(w13q),
             static_cast<const uint32_t*>(w13_scale), static_cast<__nv_bfloat16*>(h), status, rows_cap,
             N, d, 2 * I, I, group};
    return launch_w4<true>(a, st);
}

cudaError_t launch_down_w4(const void* h, int64_t rows_cap, const int32_t* offsets, int N, const void* w2q,
                           const void* w2_scale, int group, int d, int I, void* y, uint32_t* status,
                           cudaStream_t st) {
    W4Args a{offsets, static_cast<const __nv_bfloat16*>(h), static_cast<const uint8_t*>(w2q),
             static_cast<const uint32_t*>(w2_scale), static_cast<__nv_bfloat16*>(y), status, rows_cap,
             N, I, d, d, group};
    return launch_w4<false>(a, st);
}

}  // namespace lcmoe
