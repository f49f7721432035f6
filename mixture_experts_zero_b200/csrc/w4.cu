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
    asm(
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
    const uint8_t* scale;        // [N][m / 16][k / group][32]
    __nv_bfloat16* out;          // [rows_cap, n_out]
    uint32_t* status;
    int64_t rows_cap;
    int N, k, m, n_out, group;   // m: weight rows of an expert (2I or d)
    int split;                   // warps that share a tile's reduction (1, 2, 4 or 8)
};

constexpr int W4_WARPS = 8;
constexpr int W4_THREADS = 32 * W4_WARPS;
constexpr int TOK = 16;                       // rows of an expert per item
constexpr int STAGES = 4;                     // ring depth of each warp
constexpr int STAGE_BYTES = 4 * 512 + 2 * 128;  // codes of 4 blocks of 16 rows x 64 columns, their scales
constexpr int RED = 68;                       // padded feature stride of the partial sums
constexpr int RED_WARP = 8 * RED;             // floats of one warp's partial sums (8 rows x 64 features)
constexpr size_t RING_BYTES = static_cast<size_t>(W4_WARPS) * STAGES * STAGE_BYTES;
constexpr size_t RED_BYTES = 2ull * W4_WARPS * RED_WARP * 4;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One step of 64 columns of a warp: 64 weight rows from the ring times NT tiles of 8 rows.
template <int NT, bool G32>
__device__ __forceinline__ void w4_step(const uint8_t* stage, int lane, const uint4 (&xv)[2][2], float (&acc)[4][2][4]) {
    const int g = lane >> 2;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const uint4 w = *reinterpret_cast<const uint4*>(stage + b * 512 + lane * 16);
        const uint32_t wr[2][2] = {{w.x, w.y}, {w.z, w.w}};
        float s4[NT][4];
#pragma unroll
        for (int G = 0; G < 2; ++G) {
            const uint32_t a0 = codes_bf16x2<0>(wr[G][0]), a1 = codes_bf16x2<0>(wr[G][1]);
            const uint32_t a2 = codes_bf16x2<1>(wr[G][0]), a3 = codes_bf16x2<1>(wr[G][1]);
            const uint32_t a4 = codes_bf16x2<2>(wr[G][0]), a5 = codes_bf16x2<2>(wr[G][1]);
            const uint32_t a6 = codes_bf16x2<3>(wr[G][0]), a7 = codes_bf16x2<3>(wr[G][1]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (G == 0 || G32) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) s4[n][i] = 0.0f;
                }
                mma16816(s4[n], a0, a1, a2, a3, xv[n][G].x, xv[n][G].y);
                mma16816(s4[n], a4, a5, a6, a7, xv[n][G].z, xv[n][G].w);
            }
            if (G == 1 || G32) {
                const uint32_t sc = *reinterpret_cast<const uint32_t*>(stage + 2048 + (G32 ? G * 128 : 0) + b * 32 + g * 4);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[b][n][0] = fmaf(bf16lo(sc), s4[n][0], acc[b][n][0]);
                    acc[b][n][1] = fmaf(bf16lo(sc), s4[n][1], acc[b][n][1]);
                    acc[b][n][2] = fmaf(bf16hi(sc), s4[n][2], acc[b][n][2]);
                    acc[b][n][3] = fmaf(bf16hi(sc), s4[n][3], acc[b][n][3]);
                }
            }
        }
    }
}

// Item: `8 / split` tiles of 64 weight rows of one expert (32 gate and 32 up rows, or 64 output
// features) times up to 16 of its rows. The CTA's warps form 8 / split teams, one for each tile; a
// team's warps take every split-th step of 64 columns and join their sums in shared memory. Each
// warp streams its codes and scales through a ring of its own (cp.async, no barriers), which runs
// on across items; the activations of the next step are loaded into registers a step ahead.
template <bool SWIGLU, bool G32>
__global__ void __launch_bounds__(W4_THREADS, 2) w4_kernel(const W4Args a) {
    extern __shared__ __align__(128) uint8_t s_raw[];
    float* red = reinterpret_cast<float*>(s_raw + RING_BYTES);
    int32_t* pre = reinterpret_cast<int32_t*>(s_raw + RING_BYTES + RED_BYTES);  // [N + 1] row-tile prefix sums
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    if (warp == 0) {
        int run = 0;
        if (lane == 0) pre[0] = 0;
        for (int base = 0; base < a.N; base += 32) {
            const int e = base + lane;
            int n = 0;
            if (e < a.N) {
                const int lo = a.offsets[e], hi = a.offsets[e + 1];
                if (lo < 0 || hi < lo || hi > a.rows_cap) set_status(a.status, LC_MOE_DEV_IDX_RANGE);
                else n = (hi - lo + TOK - 1) / TOK;
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(FULL, n, o);
                if (lane >= o) n += v;
            }
            if (e < a.N) pre[e + 1] = run + n;
            run += __shfl_sync(FULL, n, 31);
        }
    }
    __syncthreads();
    const int tiles = a.m / 64, teams = W4_WARPS / a.split;
    const int team = warp / a.split, kw = warp % a.split;
    const int super = (tiles + teams - 1) / teams;  // items per 16 rows of an expert
    const int64_t total = static_cast<int64_t>(pre[a.N]) * super;
    const int nk = a.k / 64, ngrp = a.k / a.group;
    const int64_t blk_codes = static_cast<int64_t>(nk) * 512, blk_scale = static_cast<int64_t>(ngrp) * 32;
    const int64_t mblk = a.m / 16;

    struct Item {
        int64_t row0;  // first row
        int rows;      // 1..16
        int e, tile;
    };
    auto locate = [&](int64_t item) {
        const int rt = static_cast<int>(item / super);
        int lo = 0, hi = a.N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] <= rt) lo = mid;
            else hi = mid - 1;
        }
        Item it;
        it.e = lo;
        it.tile = static_cast<int>(item - static_cast<int64_t>(rt) * super) * teams + team;
        it.row0 = __ldg(a.offsets + lo) + static_cast<int64_t>(rt - pre[lo]) * TOK;
        it.rows = static_cast<int>(min(static_cast<int64_t>(TOK), __ldg(a.offsets + lo + 1) - it.row0));
        return it;
    };
    // 16-row weight blocks of a tile: SwiGLU takes two of the gate rows and two of the up rows
    auto block_of = [&](int tile, int b) {
        return SWIGLU ? (b >> 1) * static_cast<int>(mblk / 2) + tile * 2 + (b & 1) : tile * 4 + b;
    };

    // ---- ring: the producer runs STAGES - 1 steps ahead of the consumer
    const uint32_t ring = smem_u32(s_raw) + warp * STAGES * STAGE_BYTES;
    int64_t p_item = blockIdx.x;
    int p_ks = nk, p_slot = 0;
    const uint8_t *p_codes = nullptr, *p_scale = nullptr;
    int64_t p_up = 0;
    auto produce = [&]() {
        while (p_ks >= nk && p_item < total) {  // next item in which this warp's team has a tile
            const Item it = locate(p_item);
            p_item += gridDim.x;
            if (it.tile >= tiles) continue;
            p_ks = kw;
            const int64_t first = it.e * mblk + block_of(it.tile, 0);
            p_codes = a.codes + first * blk_codes + static_cast<int64_t>(kw) * 512 + lane * 16;
            p_up = SWIGLU ? (mblk / 2) * blk_codes : 2 * blk_codes;
            // lane (g, t) fetches block t's scales of rows g and g + 8
            p_scale = a.scale + (it.e * mblk + block_of(it.tile, t)) * blk_scale + g * 4;
        }
        if (p_ks < nk) {
            const uint32_t dst = ring + p_slot * STAGE_BYTES;
            cp_async16(dst + lane * 16, p_codes);
            cp_async16(dst + 512 + lane * 16, p_codes + blk_codes);
            cp_async16(dst + 1024 + lane * 16, p_codes + p_up);
            cp_async16(dst + 1536 + lane * 16, p_codes + p_up + blk_codes);
            const uint8_t* sc = p_scale + static_cast<int64_t>(p_ks * 64 / a.group) * 32;
            cp_async4(dst + 2048 + t * 32 + g * 4, sc);
            if (G32) cp_async4(dst + 2176 + t * 32 + g * 4, sc + 32);
            p_codes += a.split * 512;
            p_ks += a.split;
            p_slot = p_slot + 1 == STAGES ? 0 : p_slot + 1;
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) produce();

    uint4 xn[2][2];
    auto load_x = [&](const Item& it, int ks) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int G = 0; G < 2; ++G)
                xn[n][G] = g + 8 * n < it.rows
                               ? __ldg(reinterpret_cast<const uint4*>(a.x + (it.row0 + g + 8 * n) * a.k + ks * 64 + 32 * G + 8 * t))
                               : make_uint4(0, 0, 0, 0);
    };
    Item it{}, nx{};
    if (static_cast<int64_t>(blockIdx.x) < total) {
        nx = locate(blockIdx.x);
        load_x(nx, kw);
    }
    int slot = 0, buf = 0;
    for (int64_t item = blockIdx.x; item < total; item += gridDim.x) {
        it = nx;
        const bool more = item + gridDim.x < total;
        if (more) nx = locate(item + gridDim.x);
        const bool mine = it.tile < tiles;
        float acc[4][2][4];
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[b][n][i] = 0.0f;
        if (mine) {
            for (int ks = kw; ks < nk; ks += a.split) {
                uint4 xv[2][2];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int G = 0; G < 2; ++G) xv[n][G] = xn[n][G];
                if (ks + a.split < nk) load_x(it, ks + a.split);
                else if (more) load_x(nx, kw);
                cp_async_wait<STAGES - 2>();
                __syncwarp();  // the stage is visible, and the slot before it has been read by every lane
                const uint8_t* stage = s_raw + (warp * STAGES + slot) * STAGE_BYTES;
                produce();
                if (it.rows > 8) w4_step<2, G32>(stage, lane, xv, acc);
                else w4_step<1, G32>(stage, lane, xv, acc);
                slot = slot + 1 == STAGES ? 0 : slot + 1;
            }
        } else if (more) {
            load_x(nx, kw);
        }
        // join the team's partial sums, 8 rows at a time (two buffers: one barrier each)
        const int parts = it.rows > 8 ? 2 : 1;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            if (n >= parts) break;
            float* r = red + buf * W4_WARPS * RED_WARP;
            float* w = r + warp * RED_WARP;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                w[(2 * t) * RED + 16 * b + g] = acc[b][n][0];
                w[(2 * t + 1) * RED + 16 * b + g] = acc[b][n][1];
                w[(2 * t) * RED + 16 * b + g + 8] = acc[b][n][2];
                w[(2 * t + 1) * RED + 16 * b + g + 8] = acc[b][n][3];
            }
            __syncthreads();
            if (mine) {
                constexpr int FEAT = SWIGLU ? 32 : 64;
                const float* s = r + team * a.split * RED_WARP;
                for (int i = kw * 32 + lane; i < 8 * FEAT; i += a.split * 32) {
                    const int row = i / FEAT, f = i % FEAT;
                    if (8 * n + row < it.rows) {
                        float p = 0.0f, q = 0.0f;
                        for (int k = 0; k < a.split; ++k) {
                            p += s[k * RED_WARP + row * RED + f];
                            if (SWIGLU) q += s[k * RED_WARP + row * RED + 32 + f];
                        }
                        a.out[(it.row0 + 8 * n + row) * a.n_out + it.tile * FEAT + f] =
                            __float2bfloat16_rn(SWIGLU ? silu_mul(p, q) : p);
                    }
                }
            }
            buf ^= 1;
        }
    }
    cp_async_wait<0>();
}

template <bool SWIGLU, bool G32>
cudaError_t launch_w4_t(const W4Args& a, cudaStream_t st) {
    const DevInfo* di = current_device_info();
    if (!di) return cudaErrorUnknown;
    static PerDeviceOnce setup;
    const cudaError_t e = setup.run([](int) {
        return cudaFuncSetAttribute(w4_kernel<SWIGLU, G32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(RING_BYTES + RED_BYTES + 2049 * 4));
    });
    if (e != cudaSuccess) return e;
    const size_t smem = RING_BYTES + RED_BYTES + (static_cast<size_t>(a.N) + 1) * 4;
    w4_kernel<SWIGLU, G32><<<di->sm_count * 2, W4_THREADS, smem, st>>>(a);
    return cudaGetLastError();
}

template <bool SWIGLU>
cudaError_t launch_w4(W4Args a, cudaStream_t st) {
    // as many warps on a tile's reduction as leave each of them 8 steps of 64 columns
    a.split = W4_WARPS;
    while (a.split > 1 && a.k / 64 / a.split < 8) a.split /= 2;
    return a.group == 32 ? launch_w4_t<SWIGLU, true>(a, st) : launch_w4_t<SWIGLU, false>(a, st);
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
             static_cast<const uint8_t*>(w13_scale), static_cast<__nv_bfloat16*>(h), status, rows_cap,
             N, d, 2 * I, I, group, 0};
    return launch_w4<true>(a, st);
}

cudaError_t launch_down_w4(const void* h, int64_t rows_cap, const int32_t* offsets, int N, const void* w2q,
                           const void* w2_scale, int group, int d, int I, void* y, uint32_t* status,
                           cudaStream_t st) {
    W4Args a{offsets, static_cast<const __nv_bfloat16*>(h), static_cast<const uint8_t*>(w2q),
             static_cast<const uint8_t*>(w2_scale), static_cast<__nv_bfloat16*>(y), status, rows_cap,
             N, I, d, d, group, 0};
    return launch_w4<false>(a, st);
}

}  // namespace lcmoe
