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
// mma.sync with the weights as its 16-row operand and 8 token rows as the other is used on purpose:
// with a few rows an expert the matrix products are mostly padding on any unit, and operands that
// are unpacked into registers spare the unpacked weights the trip through shared memory that
// tcgen05 would need (8 KB written and read again for every 2 KB of codes).
//
// Codes become bf16 exactly: 0x4300 | n is 128 + n in bf16, minus 136 gives n - 8. A group's sum is
// accumulated in fp32 on its own and then times its scale, so a scale is never rounded into a
// weight.
//
// Measured on a B200 (copy rate 6.5 TB/s): 32 tokens over 115 experts of 6144 x 2048, group 64, 2.3 GB
// in 450 us (5.1 TB/s); 128 tokens over 512 experts, 9.0 GB in 1.69 ms at 1965 MHz and, call after call, in
// 1.95 ms at the 1.70 GHz that the 1000 W limit leaves; one token over 8 experts, 156 MB in 47 us. The
// time goes with the SM clock, not with HBM. 7 integer operations for 8 weights on a half-rate pipe and
// the mma.sync next to them make up most of it (the stream without the products takes 345 us, without
// unpacking 374; these instructions alone would take three quarters of the cycles).
// No gain came from byte permutes or multiplications in place of shifts, from more logic operations
// for fewer shifts, from products of 16 + n or 128 + n that start at -24 or -136 times the sum of the
// activations (which drops the subtraction), from ring stages of one block by 256 columns, or from
// 24 warps an SM. With many rows an expert it reaches 0.13 to 0.22 PFLOP/s: the weights are unpacked
// again for every 16 of them.
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
    uint32_t v;  // (w >> 4 P) & 0x000f000f | 0x43004300 in one logic operation
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w >> (4 * P)), "r"(0x000f000fu), "r"(0x43004300u));
    return sub_bf16x2(v, 0x43084308u);
}

// D = A B + C, m16n8k16, bf16 operands, fp32 accumulators
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

__device__ __forceinline__ float silu_mul(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

// ------------------------------------------------------------------------------- quantiser --

// One warp per 16 rows x (64 columns, or 128 when the group is 128). scale = bf16(amax / 7) (1 for
// a group whose scale would be 0), code = 8 + round(w / scale), a division in fp32, to nearest
// even, within -7..7. Run once for a model's weights: 64 matrices of 4096 x 6144 in 1.96 to 2.29 ms (2.07 to
// 1.79 TB/s, groups of 128 to 32), bound by the pipe of reciprocals, roundings and conversions (73 to 76 %).
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
    // byte distances between 16-row blocks of the codes and of the scales: to the next block, and from
    // a block of gate rows to the up rows of the same features (down product: two blocks on)
    int64_t code_blk, scale_blk, code_up;
};

constexpr int W4_WARPS = 8;
constexpr int W4_THREADS = 32 * W4_WARPS;
constexpr int STAGES = 4;                       // ring depth of each warp (even)
constexpr int STAGE_BYTES = 4 * 512 + 2 * 128;  // codes of 4 blocks of 16 rows x 64 columns, their scales
constexpr int RED = 68;                         // padded feature stride of the partial sums
constexpr int RED_WARP = 8 * RED;               // floats of one warp's partial sums (8 rows x 64 features)
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

// A ring stage (64 weight rows x 64 columns) times NT tiles of 8 rows.
template <int NT, int MAXNT, bool G32>
__device__ __forceinline__ void w4_stage(const uint8_t* stage, int lane, const uint4 (&xv)[MAXNT][2],
                                         float (*acc)[MAXNT][4]) {
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
                if (G == 0 || G32) mma16816(s4[n], a0, a1, a2, a3, xv[n][G].x, xv[n][G].y, 0.0f, 0.0f, 0.0f, 0.0f);
                else mma16816(s4[n], a0, a1, a2, a3, xv[n][G].x, xv[n][G].y, s4[n][0], s4[n][1], s4[n][2], s4[n][3]);
                mma16816(s4[n], a4, a5, a6, a7, xv[n][G].z, xv[n][G].w, s4[n][0], s4[n][1], s4[n][2], s4[n][3]);
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

template <int V>
struct Int {
    static constexpr int value = V;
};

constexpr int W4_CTAS = 2;  // to an SM
// ring, partial sums, prefix sums and numbers of the live experts
constexpr size_t w4_smem(int n) { return RING_BYTES + RED_BYTES + (n + 1) * 4 + n * 2; }
// CTAs that an SM's 228 KB hold (1 KB of it goes to each): 2 up to 1194 experts, 1 above. The tables are
// not cut to the rows of the call: offsets that are out of order may name more experts than it has rows.
constexpr int w4_ctas(int n) { return W4_CTAS * (w4_smem(n) + 1024) <= 228 * 1024 ? W4_CTAS : 1; }
static_assert(w4_ctas(1194) == 2 && w4_ctas(1195) == 1 && w4_smem(2048) <= 227 * 1024, "shared memory");

// Item: `8 / split` tiles of 64 HALVES weight rows of one expert (as many gate as up rows, or output
// features) times up to 8 MAXNT of its rows. The CTA's warps form 8 / split teams, one for each
// tile; a team's warps take every split-th step of 64 columns and join their sums in shared memory.
// Each warp streams its codes and scales through a ring of its own (cp.async, no barriers), which
// runs on across items; the activations of the next step are loaded into registers a step ahead.
template <bool SWIGLU, bool G32, int HALVES, int MAXNT>
__global__ void __launch_bounds__(W4_THREADS, W4_CTAS) w4_kernel(const W4Args a) {
    constexpr int TOK = 8 * MAXNT;
    extern __shared__ __align__(128) uint8_t s_raw[];
    float* red = reinterpret_cast<float*>(s_raw + RING_BYTES);
    // the experts that have rows: [live + 1] prefix sums of their row tiles, [live] their numbers
    int32_t* pre = reinterpret_cast<int32_t*>(s_raw + RING_BYTES + RED_BYTES);
    uint16_t* ids = reinterpret_cast<uint16_t*>(pre + a.N + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    int live, row_tiles;
    {
        // each thread counts up to 8 consecutive experts, then a scan over the CTA (N <= 2048)
        int32_t* part = reinterpret_cast<int32_t*>(red);  // [2][W4_WARPS]
        const int per = (a.N + W4_THREADS - 1) / W4_THREADS, first = threadIdx.x * per;
        int rt[8], sum = 0, some = 0;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            rt[i] = 0;
            if (i < per && first + i < a.N) {
                const int lo = __ldg(a.offsets + first + i), hi = __ldg(a.offsets + first + i + 1);
                if (lo < 0 || hi < lo || hi > a.rows_cap) bad = true;
                else rt[i] = (hi - lo + TOK - 1) / TOK;
            }
            sum += rt[i];
            some += rt[i] > 0;
        }
        int sum_to = sum, some_to = some;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(FULL, sum_to, o), v = __shfl_up_sync(FULL, some_to, o);
            if (lane >= o) {
                sum_to += u;
                some_to += v;
            }
        }
        if (lane == 31) {
            part[warp] = sum_to;
            part[W4_WARPS + warp] = some_to;
        }
        if (__syncthreads_or(bad)) {
            // Offsets that fall somewhere or leave [0, rows_cap]: experts may then share rows, and their tiles
            // may add up to more than 32 bits hold. One thread takes the experts that are within bounds and
            // begin where the last one taken ends, or behind it; these have rows of their own.
            if (threadIdx.x == 0) {
                set_status(a.status, LC_MOE_DEV_IDX_RANGE);
                int end = 0, before = 0, taken = 0;
                for (int e = 0; e < a.N; ++e) {
                    const int lo = __ldg(a.offsets + e), hi = __ldg(a.offsets + e + 1);
                    if (lo < end || hi <= lo || hi > a.rows_cap) continue;
                    pre[taken] = before;
                    ids[taken++] = static_cast<uint16_t>(e);
                    before += (hi - lo + TOK - 1) / TOK;
                    end = hi;
                }
                pre[taken] = before;
                part[0] = taken;
            }
            __syncthreads();
            live = part[0];
            row_tiles = pre[live];
        } else {
            row_tiles = live = 0;
#pragma unroll
            for (int w = 0; w < W4_WARPS; ++w) {
                if (w == warp) {
                    sum_to += row_tiles;
                    some_to += live;
                }
                row_tiles += part[w];
                live += part[W4_WARPS + w];
            }
            int at = some_to - some, before = sum_to - sum;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (rt[i] > 0) {
                    pre[at] = before;
                    ids[at++] = static_cast<uint16_t>(first + i);
                    before += rt[i];
                }
            if (threadIdx.x == 0) pre[live] = row_tiles;
        }
    }
    __syncthreads();
    const int tiles = a.m / (64 * HALVES), teams = W4_WARPS / a.split;
    const int team = warp / a.split, kw = warp % a.split;
    const int super = (tiles + teams - 1) / teams;  // items per row tile of an expert
    const int nk = a.k / 64;
    const int64_t mblk = a.m / 16;

    // This CTA's items are blockIdx.x, blockIdx.x + gridDim.x, ... of row_tiles * super: (row tile,
    // place among its `super`), and the live expert of the row tile.
    struct Cursor {
        int rt, place, e;
    };
    const int step_rt = gridDim.x / super, step_place = gridDim.x % super;
    auto settle = [&](Cursor& c) {
        while (c.e + 1 < live && pre[c.e + 1] <= c.rt) ++c.e;
    };
    auto advance = [&](Cursor& c) {
        c.rt += step_rt;
        c.place += step_place;
        if (c.place >= super) {
            c.place -= super;
            ++c.rt;
        }
        settle(c);
    };
    auto begin = [&]() {
        Cursor c{static_cast<int>(blockIdx.x) / super, static_cast<int>(blockIdx.x) % super, 0};
        settle(c);
        return c;
    };
    struct Item {
        int row0, rows;  // first row, 1..TOK rows
        int e, tile;
    };
    auto item_at = [&](const Cursor& c) {
        Item it;
        it.e = ids[c.e];
        it.tile = c.place * teams + team;
        it.row0 = __ldg(a.offsets + it.e) + (c.rt - pre[c.e]) * TOK;
        it.rows = min(TOK, __ldg(a.offsets + it.e + 1) - it.row0);
        return it;
    };
    // block b (16 weight rows) of the first half of a tile: SwiGLU takes two of the gate rows and two
    // of the up rows; the second half's blocks follow at a distance of 2 (SwiGLU) or 4 blocks
    auto block_of = [&](int tile, int b) {
        return SWIGLU ? (b >> 1) * static_cast<int>(mblk / 2) + tile * 2 * HALVES + (b & 1) : tile * 4 * HALVES + b;
    };

    // ---- ring: the producer runs STAGES - 1 stages ahead of the consumer
    const uint32_t ring = smem_u32(s_raw) + warp * STAGES * STAGE_BYTES + lane * 16;
    const uint32_t ring_sc = smem_u32(s_raw) + warp * STAGES * STAGE_BYTES + 2048 + t * 32 + g * 4;
    const uint32_t sc_step = 2048u / static_cast<uint32_t>(a.group);  // scale bytes per 64 columns
    Cursor pc = begin();
    int p_ks = nk;
    const uint8_t *p_codes = nullptr, *p_scale = nullptr;
    auto produce = [&](auto half, uint32_t slot) {  // slot: byte offset in the ring
        constexpr int H = decltype(half)::value;
        if (H == 0) {
            while (p_ks >= nk && pc.rt < row_tiles) {  // next item in which this warp's team has a tile
                const int tile = pc.place * teams + team;
                if (tile < tiles) {
                    const int64_t e = ids[pc.e];
                    p_ks = kw;
                    p_codes = a.codes + (e * mblk + block_of(tile, 0)) * a.code_blk + kw * 512 + lane * 16;
                    // lane (g, t) fetches block t's scales of rows g and g + 8
                    p_scale = a.scale + (e * mblk + block_of(tile, t)) * a.scale_blk + g * 4;
                }
                advance(pc);
            }
        }
        if (p_ks < nk) {
            const uint32_t dst = ring + slot;
            const uint8_t* c = H ? p_codes + (SWIGLU ? 2 : 4) * a.code_blk : p_codes;
            const uint8_t* up = c + a.code_up;
            cp_async16(dst, c);
            cp_async16(dst + 512, c + a.code_blk);
            cp_async16(dst + 1024, up);
            cp_async16(dst + 1536, up + a.code_blk);
            const uint8_t* sc = (H ? p_scale + (SWIGLU ? 2 : 4) * a.scale_blk : p_scale) + (p_ks * sc_step & ~31u);
            cp_async4(ring_sc + slot, sc);
            if (G32) cp_async4(ring_sc + slot + 128, sc + 32);
            if (H == HALVES - 1) {
                p_codes += a.split * 512;
                p_ks += a.split;
            }
        }
        cp_async_commit();
    };
    static_assert(STAGES == 4 && HALVES <= 2, "the halves alternate through the ring's prologue");
    produce(Int<0>(), 0);
    produce(Int<HALVES - 1>(), STAGE_BYTES);
    produce(Int<0>(), 2 * STAGE_BYTES);

    // the gate/up product lets the down product start; the down product waits for it before it reads
    // H (weights and offsets are older than both kernels)
    if (SWIGLU) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    else asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- activations of the next step, in registers: rows g and g + 8 of the item. A row past the
    // item's last repeats the last (its column of the product is not stored).
    struct Rows {
        const __nv_bfloat16* p;  // row g of the item, this lane's columns
        int64_t off[MAXNT];      // from there to rows g + 8 n, in elements
    };
    auto rows_of = [&](const Item& it) {
        Rows r;
        const int first = min(g, it.rows - 1);
        r.p = a.x + static_cast<int64_t>(it.row0 + first) * a.k + (kw * 64 + 8 * t);
#pragma unroll
        for (int n = 0; n < MAXNT; ++n) r.off[n] = static_cast<int64_t>(min(g + 8 * n, it.rows - 1) - first) * a.k;
        return r;
    };
    // H is written while the down product is already running: no read-only loads there
    auto load16 = [](const __nv_bfloat16* p) {
        return SWIGLU ? __ldg(reinterpret_cast<const uint4*>(p)) : *reinterpret_cast<const uint4*>(p);
    };
    auto load_x = [&](uint4 (&v)[MAXNT][2], const Rows& r, int rows) {
#pragma unroll
        for (int n = 0; n < MAXNT; ++n)
            if (n == 0 || rows > 8 * n) {
                v[n][0] = load16(r.p + r.off[n]);
                v[n][1] = load16(r.p + r.off[n] + 32);
            }
    };
    Item it{}, nx{};
    Rows xr{}, xn{};
    uint4 xa[MAXNT][2], xb[MAXNT][2];
#pragma unroll
    for (int n = 0; n < MAXNT; ++n) xa[n][0] = xa[n][1] = xb[n][0] = xb[n][1] = make_uint4(0, 0, 0, 0);
    Cursor c = begin();
    if (c.rt < row_tiles) {
        nx = item_at(c);
        xn = rows_of(nx);
        load_x(xa, xn, nx.rows);
    }
    // Steps take turns on xa and xb; which is next carries over from item to item, and with two halves
    // a step so do the ring's slots, which are then constants (0 and 1 go with xa). With one half they
    // are counted: the next one to read and the one before it, which the producer fills.
    int turn = 0, buf = 0;
    uint32_t slot = 0, last = (STAGES - 1) * STAGE_BYTES;
    const uint8_t* my_ring = s_raw + warp * STAGES * STAGE_BYTES;
    const int steps = (nk - kw + a.split - 1) / a.split;
    const int x_step = a.split * 64;
    while (c.rt < row_tiles) {
        it = nx;
        xr = xn;
        advance(c);
        const bool more = c.rt < row_tiles;
        if (more) {
            nx = item_at(c);
            xn = rows_of(nx);
        }
        const bool mine = it.tile < tiles;
        float acc[4 * HALVES][MAXNT][4];
#pragma unroll
        for (int b = 0; b < 4 * HALVES; ++b)
#pragma unroll
            for (int n = 0; n < MAXNT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[b][n][i] = 0.0f;
        if (mine) {
            int left = steps;
            // one step on the activations `v`, while those of the next step (of this item or the next) load into `w`
            auto step = [&](auto nt, auto odd, uint4 (&v)[MAXNT][2], uint4 (&w)[MAXNT][2]) {
                constexpr int NT = decltype(nt)::value;
                xr.p += x_step;
                if (--left) load_x(w, xr, it.rows);
                else if (more) load_x(w, xn, nx.rows);
                auto half = [&](auto h, auto ahead) {
                    constexpr int H = decltype(h)::value, S = 2 * decltype(odd)::value + H;
                    cp_async_wait<STAGES - 2>();
                    __syncwarp();  // the stage is visible, and the slot before it has been read by every lane
                    if (HALVES > 1) {
                        produce(ahead, (S + STAGES - 1) % STAGES * STAGE_BYTES);
                        w4_stage<NT, MAXNT, G32>(my_ring + S * STAGE_BYTES, lane, v, acc + 4 * H);
                    } else {
                        produce(ahead, last);
                        w4_stage<NT, MAXNT, G32>(my_ring + slot, lane, v, acc);
                        last = slot;
                        slot = slot == (STAGES - 1) * STAGE_BYTES ? 0u : slot + STAGE_BYTES;
                    }
                };
                half(Int<0>(), Int<HALVES - 1>());
                if (HALVES > 1) half(Int<HALVES - 1>(), Int<0>());
            };
            auto run = [&](auto nt) {
                while (left) {
                    if (turn == 0) {
                        step(nt, Int<0>(), xa, xb);
                        turn = 1;
                        if (!left) break;
                    }
                    step(nt, Int<1>(), xb, xa);
                    turn = 0;
                }
            };
            if (MAXNT > 1 && it.rows > 8) run(Int<MAXNT>());
            else run(Int<1>());
        } else if (more) {
            if (turn == 0) load_x(xa, xn, nx.rows);
            else load_x(xb, xn, nx.rows);
        }
        // join the team's partial sums, 8 rows x 64 weight rows at a time (two buffers: one barrier each)
#pragma unroll
        for (int ph = 0; ph < MAXNT * HALVES; ++ph) {
            const int n = ph / HALVES, hf = ph % HALVES;
            if (8 * n >= it.rows) break;
            float* r = red + buf * W4_WARPS * RED_WARP;
            float* w = r + warp * RED_WARP;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                w[(2 * t) * RED + 16 * b + g] = acc[4 * hf + b][n][0];
                w[(2 * t + 1) * RED + 16 * b + g] = acc[4 * hf + b][n][1];
                w[(2 * t) * RED + 16 * b + g + 8] = acc[4 * hf + b][n][2];
                w[(2 * t + 1) * RED + 16 * b + g + 8] = acc[4 * hf + b][n][3];
            }
            __syncthreads();
            if (mine) {
                // two neighbouring features a thread
                constexpr int PAIRS = SWIGLU ? 16 : 32;
                const float* s = r + team * a.split * RED_WARP;
                __nv_bfloat16* dst = a.out + static_cast<int64_t>(it.row0 + 8 * n) * a.n_out + (it.tile * HALVES + hf) * (2 * PAIRS);
                const int rows = min(8, it.rows - 8 * n);
                for (int i = kw * 32 + lane; i < rows * PAIRS; i += a.split * 32) {
                    const int row = i / PAIRS, f = 2 * (i % PAIRS);
                    float2 p = make_float2(0.0f, 0.0f), q = p;
                    for (int k = 0; k < a.split; ++k) {
                        const float2 u = *reinterpret_cast<const float2*>(s + k * RED_WARP + row * RED + f);
                        p.x += u.x, p.y += u.y;
                        if (SWIGLU) {
                            const float2 v = *reinterpret_cast<const float2*>(s + k * RED_WARP + row * RED + 32 + f);
                            q.x += v.x, q.y += v.y;
                        }
                    }
                    if (SWIGLU) p = make_float2(silu_mul(p.x, q.x), silu_mul(p.y, q.y));
                    *reinterpret_cast<uint32_t*>(dst + static_cast<int64_t>(row) * a.n_out + f) = pack_bf16x2(p.x, p.y);
                }
            }
            buf ^= 1;
        }
    }
    cp_async_wait<0>();
}

template <bool SWIGLU, bool G32, int HALVES, int MAXNT>
cudaError_t launch_w4_t(const W4Args& a, cudaStream_t st) {
    const DevInfo* di = current_device_info();
    if (!di) return cudaErrorUnknown;
    static PerDeviceOnce setup;
    const cudaError_t e = setup.run([](int) {
        return cudaFuncSetAttribute(w4_kernel<SWIGLU, G32, HALVES, MAXNT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(w4_smem(2048)));
    });
    if (e != cudaSuccess) return e;
    const size_t smem = w4_smem(a.N);
    // The down product is launched while the gate/up product still runs: its CTAs fetch their first
    // weights as SMs become free and wait for the other kernel before they read H.
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(di->sm_count * w4_ctas(a.N));  // one wave
    cfg.blockDim = dim3(W4_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = SWIGLU ? 0 : 1;
    const cudaError_t launched = cudaLaunchKernelEx(&cfg, w4_kernel<SWIGLU, G32, HALVES, MAXNT>, a);
    if (launched != cudaSuccess) cudaGetLastError();
    return launched;
}

// Warps on a tile's reduction. Fewer warps mean fewer sums to join, but also fewer and longer items:
// a split that leaves a warp 16 steps of 64 columns, raised while there are fewer than 8 items an SM
// (one token over 8 experts, down product: 22 us with 4 warps on a tile, 20 with 8).
int split_of(const W4Args& a, int tile_rows, int tok, int sm_count) {
    const int64_t tiles = a.m / tile_rows, row_tiles = (a.rows_cap < a.N ? a.rows_cap : a.N) + a.rows_cap / tok;
    const int steps = a.k / 64;
    int split = 1;
    while (split < W4_WARPS && split * 2 <= steps &&
           (steps / split >= 32 || row_tiles * ((tiles * split + W4_WARPS - 1) / W4_WARPS) < 8 * sm_count))
        split *= 2;
    return split;
}

template <bool SWIGLU, int HALVES, int MAXNT>
cudaError_t launch_w4_n(W4Args a, cudaStream_t st) {
    a.code_blk = static_cast<int64_t>(a.k / 64) * 512;
    a.scale_blk = static_cast<int64_t>(a.k / a.group) * 32;
    a.code_up = SWIGLU ? a.m / 32 * a.code_blk : 2 * a.code_blk;
    const DevInfo* di = current_device_info();
    if (!di) return cudaErrorUnknown;
    a.split = split_of(a, 64 * HALVES, 8 * MAXNT, di->sm_count);
    return a.group == 32 ? launch_w4_t<SWIGLU, true, HALVES, MAXNT>(a, st) : launch_w4_t<SWIGLU, false, HALVES, MAXNT>(a, st);
}

// The tile by the rows an expert can have on average (rows_cap / N; zero experts take some of them):
// 128 weight rows by 8 rows, or 64 by 16. Measured, in that order: 8 picks an expert (5.6 rows), 120 and
// 143 us; 12 picks (8.3 rows), 160 and 154 us; 32 picks (21 rows), 155 and 131 us.
template <bool SWIGLU>
cudaError_t launch_w4(const W4Args& a, cudaStream_t st) {
    if (a.rows_cap < static_cast<int64_t>(10) * a.N && a.m % 128 == 0) return launch_w4_n<SWIGLU, 2, 1>(a, st);
    return launch_w4_n<SWIGLU, 1, 2>(a, st);
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
             N, d, 2 * I, I, group, 0, 0, 0, 0};
    return launch_w4<true>(a, st);
}

cudaError_t launch_down_w4(const void* h, int64_t rows_cap, const int32_t* offsets, int N, const void* w2q,
                           const void* w2_scale, int group, int d, int I, void* y, uint32_t* status,
                           cudaStream_t st) {
    W4Args a{offsets, static_cast<const __nv_bfloat16*>(h), static_cast<const uint8_t*>(w2q),
             static_cast<const uint8_t*>(w2_scale), static_cast<__nv_bfloat16*>(y), status, rows_cap,
             N, I, d, d, group, 0, 0, 0, 0};
    return launch_w4<false>(a, st);
}

}  // namespace lcmoe
