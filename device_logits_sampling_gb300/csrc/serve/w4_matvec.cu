// arc_w4_matvec: a few rows times a matrix of 4-bit weights with group scales.
#include <atomic>
#include <climits>
#include <cstdint>
#include <cstring>

#include "launch_util.cuh"
#include "serve/arc_w4.h"
#include "serve_util.cuh"
#include "w4_many.cuh"

namespace {

using namespace arcs;

struct W4Args {
    arc_w4_weight w;
    const void* x;
    void* y;
    int64_t x_stride, y_stride;
    int32_t rows;
    int32_t y_f32;
    int32_t x_bf16;
};

// ------------------------------------------------------------------ few rows
// 1 .. 8 rows of x: fp16 matrix instructions with 16 weight rows on the long
// side and the rows of x on the short one.
//
// Mathematics.  A row of x is scaled by a power of two to [2^14, 2^15) and
// taken as fp16: exact for values above 2^-25 of its largest.  A 4-bit code q,
// masked out of its word, IS the fp16 subnormal q * 2^-24 (or, one nibble up,
// 16 q * 2^-24, with x divided by 16 beforehand), so a word of eight weights
// becomes four operand registers with one shift and four ANDs and no
// conversion.  The zero point and the scale of a group act on its fp32 sum:
//     y += s (sum q x - z sum x),
// with the group's sum of x computed once a block.
//
// Layout.  A block's 16 warps are `parts` slices of the inner dimension (at
// most 512 values each) times 16 / parts groups of 16 weight rows; blocks walk
// over tiles of the outer dimension.  Each warp streams its own slice of its
// own rows through a private ring of stages with 16-byte asynchronous copies;
// the only barrier is the one that joins the slices' sums.  Weights are read
// once, in their natural layout: the order of the inner dimension inside a
// product is free, x is laid out to match what one shared load of a lane
// gives.  Inner dimensions over one block's reach are split over a cluster,
// whose first block adds the others' sums.
//
// Bounds and figures.  Instruction issue: about 150 warp instructions for each
// KB of weights (groups of 64) of the 174 that its share of memory time leaves
// an SM.  One row by 129,280 x 4,096, groups of 64: 61 us, 4.6 TB/s, 68% of the
// measured copy rate; 4,096 x 4,096: 5.9 us, most of it a launch and one round
// trip to memory. Measured and left: 16 rows in two tiles (163 us, shared-memory
// bound: w4_many.cu takes 82), joining every tile (69 us against 64), a rolled
// staging loop (19,500 clocks for 7 rows against 10,700).
constexpr int kFewThreads = 512;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kXVecs = 8;               // 16-byte vectors of x a thread stages
constexpr int kPart = 512;              // inner values of a warp's stage

struct FewArgs {
    W4Args a;
    int32_t slice;    // inner values of a block, a multiple of 128
    int32_t part;     // inner values of a warp, a multiple of 128, at most kPart
    int32_t parts;    // 1, 2, 4, 8 or 16
    int32_t stages;   // 2, 3 or 4
    int32_t cluster;  // blocks that share a tile
    int32_t tiles;
    int32_t period;   // tiles between joins
    int32_t x_vec;
    // shared-memory layout, bytes
    int32_t x_off, xs_off, scale_off, red_off, join_off, up_off;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 16-byte chunk c of weight row r (0 .. 15) in a stage: the chunks of a
// 128-byte line are permuted by the row's bit-reversed low bits, so that lanes
// reading 4, 8 or 16 bytes of one chunk in 8, 4 or 2 rows meet in no bank.
__device__ __forceinline__ constexpr int row_bits(int r) { return ((r & 1) << 2) | (r & 2) | ((r >> 2) & 1); }
template <int PITCH>
__device__ __forceinline__ int weight_at(int r, int c) {
    return r * PITCH + ((c & 8) | ((c & 7) ^ row_bits(r))) * 16;
}

// Eight 16-bit values as they lie.
__device__ __forceinline__ uint4 raw8(const void* p, bool vec) {
    if (vec) return *static_cast<const uint4*>(p);
    const uint16_t* e = static_cast<const uint16_t*>(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = e[2 * i] | (static_cast<uint32_t>(e[2 * i + 1]) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// x of the block's slice to shared memory: fp16, scaled row by row, in the
// order of the products, and the sums of each group.  All of it is loaded at
// once (64 KB at most: eight vectors a thread), so the block waits for memory
// once before its first product.
template <int DT, int G, bool Z>
__device__ __forceinline__ void stage_x(const FewArgs& f, uint8_t* dyn, int k0, int ks) {
    const int tid = threadIdx.x;
    const int rows = f.a.rows, units = ks >> 3, groups = ks / G, all = units * rows;
    uint32_t* top = reinterpret_cast<uint32_t*>(dyn + f.up_off);  // then the rows' factors
    uint4 raw[kXVecs];
    int row[kXVecs], unit[kXVecs];  // the vectors tid, tid + 512, ..., without a division each
    {
        const int rows_on = kFewThreads / units, units_on = kFewThreads - rows_on * units;
        int m = tid / units, u = tid - m * units;
#pragma unroll
        for (int j = 0; j < kXVecs; ++j) {
            row[j] = m;
            unit[j] = u;
            raw[j] = m < rows ? raw8(static_cast<const char*>(f.a.x) + (m * f.a.x_stride + k0 + u * 8) * 2, f.x_vec)
                              : make_uint4(0u, 0u, 0u, 0u);
            m += rows_on;
            u += units_on;
            if (u >= units) {
                u -= units;
                ++m;
            }
        }
    }
    if (tid < 8) top[tid] = 0;
    __syncthreads();
    float v[8];
    auto unpack = [&](const uint4& r) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = Half<DT>::unpack(w[i]);
            v[2 * i] = p.x;
            v[2 * i + 1] = p.y;
        }
    };
#pragma unroll
    for (int j = 0; j < kXVecs; ++j) {
        if (j * kFewThreads >= all) break;
        // magnitudes of 16-bit floats order as their bits do; a row with an infinite or NaN value comes out as
        // such whatever its factor
        const uint4 r = raw[j];
        const uint32_t w = __vmaxu2(__vmaxu2(r.x & 0x7FFF7FFFu, r.y & 0x7FFF7FFFu), __vmaxu2(r.z & 0x7FFF7FFFu, r.w & 0x7FFF7FFFu));
        const uint32_t most = max(w & 0xFFFFu, w >> 16);
        if ((units & 31) == 0) {  // a warp's vectors are of one row
            const uint32_t largest = __reduce_max_sync(0xFFFFFFFFu, most);
            if ((tid & 31) == 0 && row[j] < rows) atomicMax(top + row[j], largest);
        } else if (row[j] < rows) {
            atomicMax(top + row[j], most);
        }
    }
    __syncthreads();
    if (tid < 8) {
        const float largest = Half<DT>::unpack(top[tid]).x;
        const int ex = static_cast<int>(__float_as_uint(largest) >> 23) - 127;
        const int e = largest == 0.0f ? 0 : (14 - ex > 120 ? 120 : 14 - ex);
        reinterpret_cast<float*>(top)[tid] = exp2i(e);
    }
    __syncthreads();
    const float* up = reinterpret_cast<const float*>(top);
    float* xs = reinterpret_cast<float*>(dyn + f.xs_off);
    for (int i = tid; i < groups * 8; i += kFewThreads)
        if (i % 8 >= rows) xs[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < kXVecs; ++j) {
        if (j * kFewThreads >= all) break;
        // vectors of a group are neighbouring lanes: units is a multiple of G / 8
        const int m = row[j], u = unit[j], k = u * 8;
        const bool on = m < rows;
        unpack(raw[j]);
        const float s = on ? up[m] : 0.0f;
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] *= s;
            sum += v[e];
        }
        const int gi = k / G, in = k % G, t = in / (G / 4), w = (in % (G / 4)) >> 3;
        alignas(16) const __half2 h[4] = {__floats2half2_rn(v[0], v[4]), __floats2half2_rn(v[2], v[6]),
                                          __floats2half2_rn(v[1] * 0.0625f, v[5] * 0.0625f),
                                          __floats2half2_rn(v[3] * 0.0625f, v[7] * 0.0625f)};
        if (on)
            *reinterpret_cast<uint4*>(dyn + f.x_off + (((gi * (G / 32) + w) * rows + m) * 4 + t) * 16) =
                *reinterpret_cast<const uint4*>(h);
#pragma unroll
        for (int x = 1; x < G / 8; x <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
        // without zero points the sum comes times the common one, 8 * 2^-24
        if (on && (u & (G / 8 - 1)) == 0) xs[gi * 8 + m] = Z ? sum : sum * 0x1p-21f;
    }
}

template <int N>
struct alignas(4 * N) Words {
    uint32_t w[N];
};
// G: group. P: inner values of a part at most (512 or
// 256). Z: zero points are given.
template <int G, int P, bool Z>
__global__ void __launch_bounds__(kFewThreads, 1) few_kernel(const __grid_constant__ FewArgs f) {
    extern __shared__ __align__(1024) uint8_t dyn[];
    const W4Args& a = f.a;
    constexpr int WG = G / 32;            // weight words of a group that a lane takes
    constexpr int PG = P / G;             // groups of a full part
    constexpr int PITCH = P / 2;          // bytes of a weight row in a stage
    constexpr int STAGE = 16 * PITCH;
    constexpr int SC = 16 * PG / 32;      // scales of a part that a lane loads
    constexpr int CPY = PITCH / 32;       // 16-byte copies of a lane a stage
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int part = warp % f.parts, sub = warp / f.parts;  // slice of the inner dimension, group of 16 rows
    const int per_tile = kFewWarps / f.parts * 16;
    const int rank = f.cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int first_tile = static_cast<int>(blockIdx.x) / f.cluster, tile_step = static_cast<int>(gridDim.x) / f.cluster;
    const int k0 = rank * f.slice;                                              // the block's slice
    const int ks = a.w.ins - k0 < f.slice ? a.w.ins - k0 : f.slice;
    const int p0 = part * f.part;                                               // the warp's, within it
    const int pk = ks - p0 < f.part ? (ks - p0 > 0 ? ks - p0 : 0) : f.part;
    const int pg = pk / G;                                                      // its groups
    const int groups = a.w.ins / G;

    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(dyn)) + warp * f.stages * STAGE;
    // [group][row]: the scale, and with Z the zero point times 2^-24
    constexpr int SW = Z ? 2 : 1;
    float* scales = reinterpret_cast<float*>(dyn + f.scale_off) + warp * (16 * PG * SW);
    const float* xs = reinterpret_cast<const float*>(dyn + f.xs_off) + (p0 / G) * 8 + 2 * t;
    const uint8_t* xf = dyn + f.x_off + (static_cast<size_t>(p0 / 32) * a.rows * 4 + g * 4 + t) * 16;

    // A lane copies chunk cc of the rows ch, ch + step, ...; the rows' permutation (weight_at) is an
    // exclusive or with a constant of the unrolled copy.
    constexpr int kRowsAtOnce = P == 512 ? 2 : 4;
    const int cc = lane % (32 / kRowsAtOnce), ch = lane / (32 / kRowsAtOnce);
    const uint32_t copy_to = ring + weight_at<PITCH>(ch, cc);
    const bool whole_part = pk == P;
    const char* const q_from = static_cast<const char*>(a.w.q) + (k0 + p0) / 2 + cc * 16;
    auto issue = [&](int tile, int stage) {
        if (tile < f.tiles) {
            const int64_t n0 = static_cast<int64_t>(tile) * per_tile + sub * 16 + ch;
            const char* q = q_from + n0 * a.w.row_bytes;
            const uint32_t dst = copy_to + stage * STAGE;
            const bool full = whole_part && n0 - ch + 16 <= a.w.outs;
#pragma unroll
            for (int i = 0; i < CPY; ++i) {
                const int r = kRowsAtOnce * i;
                const uint32_t to = (dst ^ (row_bits(r) * 16)) + r * PITCH;
                if (full) {
                    copy16(to, q, true);
                } else {
                    const bool on = n0 + r < a.w.outs && cc * 32 < pk;
                    copy16(to, on ? q : a.w.q, on);
                }
                q += kRowsAtOnce * a.w.row_bytes;
            }
        }
        copies_end();
    };
    // scales and zero points of a tile, loaded a tile ahead: row lane % 16, every other group
    uint16_t sv[SC];
    uint8_t zv[SC];
    const int64_t s_from = (k0 + p0) / G + (lane >> 4);
    auto fetch = [&](int tile) {
        const int64_t n = static_cast<int64_t>(tile) * per_tile + sub * 16 + (lane & 15);
        const bool row = tile < f.tiles && n < a.w.outs;
        const uint16_t* s = static_cast<const uint16_t*>(a.w.scales) + n * groups + s_from;
        const uint8_t* z = a.w.zeros + n * groups + s_from;
#pragma unroll
        for (int i = 0; i < SC; ++i) {
            const bool on = row && 2 * i + (lane >> 4) < pg;
            sv[i] = on ? __ldg(s + 2 * i) : 0;
            if (Z) zv[i] = on ? __ldg(z + 2 * i) : 0;
        }
    };
    int next = first_tile, fill = 0;
    for (int i = 0; i < f.stages - 1; ++i) {
        issue(next, fill++);
        next += tile_step;
    }
    fetch(first_tile);

    if (a.x_bf16)
        stage_x<ARC_BF16, G, Z>(f, dyn, k0, ks);
    else
        stage_x<ARC_F16, G, Z>(f, dyn, k0, ks);
    __syncthreads();
    if (f.cluster > 1) cluster_sync_all();  // every block runs before its memory is written to

    const uint32_t read_at = g * PITCH;
    const uint32_t gbits = row_bits(g) * 16;  // those of row g + 8 too
    int stage = 0, turn = 0, count = 0;
    for (int tile = first_tile; tile < f.tiles; tile += tile_step) {
        if (f.stages == 2)
            copies_wait<0>();
        else if (f.stages == 3)
            copies_wait<1>();
        else
            copies_wait<2>();
        __syncwarp();  // every lane has read the scales of the tile before
#pragma unroll
        for (int i = 0; i < SC; ++i) {
            const int e = (lane + 32 * i) * SW;
            scales[e] = a.x_bf16 ? __uint_as_float(static_cast<uint32_t>(sv[i]) << 16) : __half2float(__ushort_as_half(sv[i]));
            if (Z) scales[e + 1] = __half2float(__ushort_as_half(zv[i]));  // the code's bits as fp16: z * 2^-24
        }
        __syncwarp();  // every lane's copies and scales are in; the stage before is free
        issue(next, fill);
        next += tile_step;
        fill = fill + 1 == f.stages ? 0 : fill + 1;
        fetch(tile + tile_step);

        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = 0.0f;
        const uint8_t* st = dyn + (warp * f.stages + stage) * STAGE + read_at;
        stage = stage + 1 == f.stages ? 0 : stage + 1;
        auto one_group = [&](int gi) {
            // chunk of the lane's words and the byte within it
            const int c = WG == 4 ? gi * 4 + t : WG == 2 ? gi * 2 + (t >> 1) : gi;
            const int o = WG == 4 ? 0 : WG == 2 ? (t & 1) * 8 : t * 4;
            const uint8_t* at = st + ((c * 16) ^ gbits) + o;
            const Words<WG> w0 = *reinterpret_cast<const Words<WG>*>(at);
            const Words<WG> w1 = *reinterpret_cast<const Words<WG>*>(at + 8 * PITCH);
            float acc[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = 0.0f;
#pragma unroll
            for (int w = 0; w < WG; ++w) {
                constexpr uint32_t lo = 0x000F000Fu, hi = 0x00F000F0u;
                const uint32_t u0 = w0.w[w] >> 8, u1 = w1.w[w] >> 8;
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (g < a.rows) x = *reinterpret_cast<const uint4*>(xf + (gi * WG + w) * a.rows * 64);
                mma16816(acc, w0.w[w] & lo, w1.w[w] & lo, u0 & lo, u1 & lo, x.x, x.y);
                mma16816(acc, w0.w[w] & hi, w1.w[w] & hi, u0 & hi, u1 & hi, x.z, x.w);
            }
            float s0, s1, z0 = 1.0f, z1 = 1.0f;
            if constexpr (Z) {
                const float2 b0 = *reinterpret_cast<const float2*>(scales + (gi * 16 + g) * 2);
                const float2 b1 = *reinterpret_cast<const float2*>(scales + (gi * 16 + g + 8) * 2);
                s0 = b0.x, z0 = b0.y, s1 = b1.x, z1 = b1.y;
            } else {
                s0 = scales[gi * 16 + g];
                s1 = scales[gi * 16 + g + 8];
            }
            const float2 sx = *reinterpret_cast<const float2*>(xs + gi * 8);
            y[0] = fmaf(s0, fmaf(-z0, sx.x, acc[0]), y[0]);
            y[1] = fmaf(s0, fmaf(-z0, sx.y, acc[1]), y[1]);
            y[2] = fmaf(s1, fmaf(-z1, sx.x, acc[2]), y[2]);
            y[3] = fmaf(s1, fmaf(-z1, sx.y, acc[3]), y[3]);
        };
        if (whole_part) {
#pragma unroll
            for (int gi = 0; gi < PG; ++gi) one_group(gi);
        } else {
            for (int gi = 0; gi < pg; ++gi) one_group(gi);
        }

        // Join the parts (and the cluster's slices): each warp leaves its sums, [row of x][weight row], in the
        // tile's slot; after f.period tiles the warps of a row group meet and add them. Two sets of slots in
        // turn: one barrier a period.
        const int vals = 16 * a.rows;
        float* mine = reinterpret_cast<float*>(dyn + f.red_off) + ((turn * f.period + count) * kFewWarps + warp) * vals;
        if (2 * t < a.rows) {
            mine[2 * t * 16 + g] = y[0];
            mine[2 * t * 16 + g + 8] = y[2];
        }
        if (2 * t + 1 < a.rows) {
            mine[2 * t * 16 + 16 + g] = y[1];
            mine[2 * t * 16 + 16 + g + 8] = y[3];
        }
        ++count;
        if (count < f.period && tile + tile_step < f.tiles) continue;
        if (f.parts == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + sub), "r"(f.parts * 32) : "memory");
        const float* red = reinterpret_cast<const float*>(dyn + f.red_off) + (turn * f.period * kFewWarps + sub * f.parts) * vals;
        const float* up = reinterpret_cast<const float*>(dyn + f.up_off);
        const int64_t n0 = static_cast<int64_t>(tile) * per_tile + sub * 16;  // the last tile's
        auto finish = [&](int i, float v) {
            const int c = i / vals, m = (i - c * vals) >> 4, r = i & 15;
            const int64_t n = n0 + r - static_cast<int64_t>(count - 1 - c) * tile_step * per_tile;
            if (n >= a.w.outs) return;
            const int64_t at = m * a.y_stride + n;
            if (a.y_f32)
                static_cast<float*>(a.y)[at] = v;
            else if (a.x_bf16)
                static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
            else
                static_cast<__half*>(a.y)[at] = __float2half_rn(v);
        };
        const int join_at = (turn * f.cluster * (kFewWarps / f.parts) + sub) * f.period * vals;  // of rank 0
        const int join_rank = (kFewWarps / f.parts) * f.period * vals;
        for (int i = part * 32 + lane; i < count * vals; i += f.parts * 32) {
            const int c = i / vals, e = i - c * vals;
            const float* p = red + c * kFewWarps * vals + e;
            float v = 0.0f;
            for (int q = 0; q < f.parts; ++q) v += p[q * vals];
            // the products' unit first: a row of tiny values has a large factor, and dividing by it would leave
            // fp32's normal range
            v = v * 0x1p24f / up[e >> 4];  // powers of two
            if (f.cluster == 1) {
                finish(i, v);
            } else {
                // into the first block's memory, a place for each rank
                const uint32_t local = static_cast<uint32_t>(__cvta_generic_to_shared(
                    dyn + f.join_off + (join_at + rank * join_rank + i) * 4));
                uint32_t remote;
                asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(local));
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote), "f"(v) : "memory");
            }
        }
        if (f.cluster > 1) {
            __syncwarp();
            cluster_sync_all();
            if (rank == 0)
                for (int i = part * 32 + lane; i < count * vals; i += f.parts * 32) {
                    const float* p = reinterpret_cast<const float*>(dyn + f.join_off) + join_at + i;
                    float v = 0.0f;
                    for (int c = 0; c < f.cluster; ++c) v += p[c * join_rank];
                    finish(i, v);
                }
        }
        turn ^= 1;
        count = 0;
    }
    copies_wait<0>();
}

template <int G, int P, bool Z>
int start_few(const FewArgs& f, int smem, int dev, int sms, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    if (arc::prepare(few_kernel<G, P, Z>, dev, done, 100) != cudaSuccess) return ARC_E_CUDA;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.blockDim = dim3(kFewThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(f.cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = f.cluster > 1 ? 1 : 0;
    // As many clusters as run at once, found out once for each size: a cluster's blocks share a part of the GPU
    // whose SMs they need not divide evenly, and the 38 clusters of four that 152 SMs would hold took two rounds
    // (16,384 x 16,384: 60 us)
    static std::atomic<int> at_once[64][9];
    int clusters = sms;
    if (f.cluster > 1) {
        std::atomic<int>& known = at_once[dev & 63][f.cluster];
        clusters = known.load(std::memory_order_relaxed);
        if (clusters == 0) {
            cfg.gridDim = dim3(static_cast<unsigned>(f.cluster), 1, 1);
            if (cudaOccupancyMaxActiveClusters(&clusters, few_kernel<G, P, Z>, &cfg) != cudaSuccess || clusters < 1) {
                (void)cudaGetLastError();
                clusters = sms / f.cluster;
            }
            known.store(clusters, std::memory_order_relaxed);
        }
    }
    cfg.gridDim = dim3(static_cast<unsigned>((clusters < f.tiles ? clusters : f.tiles) * f.cluster), 1, 1);
    if (cudaLaunchKernelEx(&cfg, few_kernel<G, P, Z>, f) != cudaSuccess) {
        (void)cudaGetLastError();
        return ARC_E_CUDA;
    }
    return ARC_OK;
}

template <int G>
int launch_few(const W4Args& a, int dev, int sms, cudaStream_t st) {
    FewArgs f;
    f.a = a;
    // a block's x stays within 64 KB: 4,096 inner values of 8 rows
    constexpr int reach = kXVecs * kFewThreads;
    int c = 1;
    while (c * reach < a.w.ins) c *= 2;
    f.cluster = c;
    f.slice = ((a.w.ins + c - 1) / c + 127) / 128 * 128;
    while (f.cluster > 1 && (f.cluster - 1) * f.slice >= a.w.ins) --f.cluster;  // no empty slice
    int parts = 1;
    while (parts * kPart < f.slice) parts *= 2;
    // More parts of the inner dimension make smaller tiles: the parts whose rounds over the blocks cost least,
    // counted in weight rows (a cost of 4 or 12 rows for a tile's join changed nothing: 18.7 to 19.0 us at 11,007)
    auto tiles_of = [&](int p) { return (a.w.outs + kFewWarps / p * 16 - 1) / (kFewWarps / p * 16); };
    auto cost_of = [&](int p) {
        const int64_t at_once = sms / f.cluster;
        return (tiles_of(p) + at_once - 1) / at_once * (kFewWarps / p * 16);
    };
    const int groups = f.slice / G;
    // shared memory of `p` parts and `n` stages
    auto layout = [&](int p, int n) {
        f.parts = p;
        f.part = ((f.slice + p - 1) / p + 127) / 128 * 128;
        const int most = f.part > 256 ? 512 : 256;  // the kernel's P
        f.stages = n;
        int off = n * kFewWarps * 16 * most / 2;
        auto take = [&](int bytes) {
            const int at = off;
            off += (bytes + 127) / 128 * 128;
            return at;
        };
        f.x_off = take(a.rows * f.slice * 2);
        f.xs_off = take(groups * 8 * 4);
        f.scale_off = take(kFewWarps * 16 * (most / G) * (a.w.zeros ? 8 : 4));
        f.red_off = take(2 * f.period * kFewWarps * 16 * a.rows * 4);
        f.join_off = take(f.cluster > 1 ? 2 * f.cluster * (kFewWarps / p) * f.period * 16 * a.rows * 4 : 0);
        f.up_off = take(8 * 4);
        return off;
    };
    f.period = 1;
    int best = 0;
    for (int p = parts; p <= kFewWarps && (p == parts || f.slice / p >= 128); p *= 2)
        if (layout(p, 2) <= arc::kSmemPerBlock && (best == 0 || cost_of(p) < cost_of(best))) best = p;
    if (best == 0) return ARC_E_UNSUPPORTED;
    int stages = 4;
    while (stages > 2 && layout(best, stages) > arc::kSmemPerBlock) --stages;
    // what is left goes to rarer joins
    for (f.period = 8; f.period > 1 && layout(best, stages) > arc::kSmemPerBlock;) f.period /= 2;
    const int off = layout(best, stages);
    parts = best;
    f.tiles = static_cast<int32_t>(tiles_of(parts));
    f.x_vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.x_stride % 8 == 0;
    if (f.part > 256)
        return a.w.zeros ? start_few<G, 512, true>(f, off, dev, sms, st) : start_few<G, 512, false>(f, off, dev, sms, st);
    return a.w.zeros ? start_few<G, 256, true>(f, off, dev, sms, st) : start_few<G, 256, false>(f, off, dev, sms, st);
}

int launch_few_group(const W4Args& a, int dev, int sms, cudaStream_t st) {
    if (a.w.group == 128) return launch_few<128>(a, dev, sms, st);
    if (a.w.group == 64) return launch_few<64>(a, dev, sms, st);
    return launch_few<32>(a, dev, sms, st);
}

// More rows take the 5th-generation tensor cores (w4_many.cu).  129,280 x 4,096, groups of 128: 8 rows 65 us here
// and 82 to 88 there; 9 rows, which do not fit one tile here, 84 there.
constexpr int kFewRows = 8;

int check_weight(const arc_w4_weight* w) {
    if (w == nullptr || w->q == nullptr || w->scales == nullptr) return ARC_E_NULL;
    if (w->group != 32 && w->group != 64 && w->group != 128) return ARC_E_UNSUPPORTED;
    if (w->outs <= 0 || w->outs > INT_MAX || w->ins <= 0 || w->ins > ARC_W4_MAX_INS || w->ins % w->group != 0 ||
        w->row_bytes < w->ins / 2)
        return ARC_E_SHAPE;
    if (reinterpret_cast<uintptr_t>(w->q) % 16 != 0 || w->row_bytes % 16 != 0 ||
        reinterpret_cast<uintptr_t>(w->scales) % 2 != 0)
        return ARC_E_ALIGN;
    return ARC_OK;
}

}  // namespace

extern "C" {

size_t arc_w4_workspace_bytes(const arc_w4_weight* weight, int64_t rows) {
    if (check_weight(weight) != ARC_OK || rows <= kFewRows || rows > ARC_W4_MAX_ROWS) return 0;
    return many_workspace(weight->ins, rows);
}

int arc_w4_matvec(const arc_w4_weight* weight, const void* x, int64_t rows, int64_t x_stride, int32_t x_dtype, void* y,
                  int64_t y_stride, int32_t y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = check_weight(weight);
    if (rc != ARC_OK) return rc;
    if (x == nullptr || y == nullptr) return ARC_E_NULL;
    if (x_dtype != ARC_BF16 && x_dtype != ARC_F16) return ARC_E_DTYPE;
    if (y_dtype != x_dtype && y_dtype != ARC_F32) return ARC_E_DTYPE;
    if (rows <= 0 || rows > ARC_W4_MAX_ROWS || x_stride < weight->ins || y_stride < weight->outs) return ARC_E_SHAPE;
    if (reinterpret_cast<uintptr_t>(x) % 2 != 0 || reinterpret_cast<uintptr_t>(y) % (y_dtype == ARC_F32 ? 4 : 2) != 0)
        return ARC_E_ALIGN;
    if (const size_t need = arc_w4_workspace_bytes(weight, rows)) {
        if (workspace == nullptr || workspace_bytes < need) return ARC_E_WORKSPACE;
        if (reinterpret_cast<uintptr_t>(workspace) % 16 != 0) return ARC_E_ALIGN;
    }
    W4Args a{*weight, x, y, x_stride, y_stride, static_cast<int32_t>(rows), y_dtype == ARC_F32,
             x_dtype == ARC_BF16};
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return ARC_E_CUDA;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (rows <= kFewRows) return launch_few_group(a, dev, sms, st);
    ManyArgs m{};
    m.q = weight->q;
    m.scales = weight->scales;
    m.zeros = weight->zeros;
    m.x = x;
    m.y = y;
    m.row_bytes = weight->row_bytes;
    m.outs = weight->outs;
    m.x_stride = x_stride;
    m.y_stride = y_stride;
    m.ins = weight->ins;
    m.group = weight->group;
    m.rows = static_cast<int32_t>(rows);
    m.y_f32 = a.y_f32;
    m.x_bf16 = a.x_bf16;
    return launch_many(m, workspace, dev, sms, st);
}

}  // extern "C"
