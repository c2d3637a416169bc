// arc_kv_attend: attention of a step's new tokens over the paged 8-bit cache.
//
// Work.  An item is (sequence, tile of up to R query rows, cached head); the
// rows of an item are the new tokens' query heads that share the cached head.
// An item is a run of steps of 16 cached tokens (32 for heads of 64).  All items' steps lie one
// after another on a line (their counts come from the lengths in device
// memory), the line is cut into equal pieces, one for each warp of the grid,
// so that ragged lengths, one long sequence and many short ones all fill the
// GPU alike.  A piece that begins or ends inside an item leaves a partial
// (maximum, sum, output); the block joins its warps' partials in shared memory
// and, where an item spans blocks, the last block to arrive joins the blocks'
// in the order of the line, so results do not depend on timing.
//
// A step.  Each warp streams its steps through its own ring of shared-memory
// stages with asynchronous 16-byte copies; no block barrier is met on the way.
// S^T = K Q^T and O^T = V^T P^T run on fp16 matrix instructions: 16 tokens (or
// 16 values of the head) are the long side of a tile and the R = 8 or 16 query
// rows the short one, so that one token's grouped heads waste little.  The
// order of head values inside the products is free: a lane takes the bytes
// that one 16-byte shared load gives it, and the query is laid out to match;
// e4m3 codes become fp16 pairs by one conversion each, and the two scales
// enter outside the products.
//
// Softmax.  A step's weights are taken relative to the step's own largest score
// of the row, times 2^14, as fp16: half a step of fp16 off where they are
// within 2^-28 of that, and lost below 2^-39 of it, whatever other steps and
// their value scales are.  The step's product with the values goes into the
// running fp32 sums with one factor a row: the page's value scale times
// 2^(step's largest - running largest); for heads of 64 a factor a half, which
// may lie in two pages.  Measured and replaced:
// weights relative to the running maximum of score plus scale exponent, at most
// 1 and summed up across steps by the matrix instruction, lost what lay below
// 2^-25 of the largest, which a page of a far larger scale made of all others.
//
// Bounds and figures.  64 sequences of 4,096 to 32,768 tokens (1.85 GB): 282 us,
// 6.6 TB/s, 97% of the measured copy rate (278 us with the products summed up by
// the matrix instruction): the 12 warps of an SM need some 2,000 clocks a step,
// which is what memory gives them 4 KB in.  One sequence of 200,003: 74 us (81%);
// 256 of 1 to 4,096: 65 us (67%): the line's ends, about 12,000 clocks to the first
// step and as many for the joins.  Short calls are those: 14 us.  48 sequences of 1
// to 5 drafted tokens, heads of 64, a window: 36 us.  Measured and left: a block for
// each (sequence, head) and one token at a time a warp (157 ms for the 200,003),
// more warps with fewer registers and stages (95 us for it), joins row by row in
// every thread (84 us).
#include <atomic>

#include "kv_device.cuh"
#include "kv_host.cuh"
#include "launch_util.cuh"
#include "serve_util.cuh"

namespace {

using namespace arcs;

constexpr int kMaxBlocks = 256;  // blocks of a launch: at most one for each SM
constexpr float kNothing = -3.0e38f;  // maximum of no score: finite, so that differences need no special case
// An item's fixed cost in steps (query load, output store), for the cut.  With 1, 2, 3 and 4: 256 ragged sequences
// 82, 68, 65 and 65 us, heads of 64 50, 46, 48 and 49, heads of 256 69, 62, 60 and 60; 500 short ones 37, 35, 36 and 37;
// drafts 37, 36, 36 and 35; sequences of one length 69 to 70 with any.
constexpr int kItemCost = 3;
constexpr float kLift = 16384.0f;  // of the weights as fp16: 2^14 of its 2^15.99
constexpr int kStatusBytes = kMaxBlocks * 4;

struct AttendArgs {
    arc_kv_cache c;
    arc_kv_step s;
    arc_kv_query q;
    uint32_t* err;
    uint32_t* arrived;  // one counter a block, 0 between calls
    float* partial;     // two slots a block
    int32_t group;      // query heads for each cached one
    int32_t bf16;
    int32_t vec;        // bit 0: q, 1: out allow 16-byte accesses
};

// Warps of a block and stages of a warp's ring, for one block an SM.
template <int D, int NT>
struct Shape;
template <>
struct Shape<64, 1> {
    static constexpr int kWarps = 16, kStages = 2;
};
template <>
struct Shape<64, 2> {
    static constexpr int kWarps = 12, kStages = 3;
};
template <>
struct Shape<128, 1> {
    static constexpr int kWarps = 12, kStages = 3;
};
template <>
struct Shape<128, 2> {
    static constexpr int kWarps = 8, kStages = 4;
};
template <>
struct Shape<256, 1> {
    static constexpr int kWarps = 8, kStages = 2;
};

// A step is 16 tokens; for heads of 64, whose 16 tokens are 2 KB, 32: the work
// that a step costs whatever its size is shared by two halves, which may lie in
// different pages.
template <int D>
struct Step {
    static constexpr int kShift = D == 64 ? 5 : 4;
    static constexpr int kHalves = 1 << (kShift - 4);
};

struct Part {        // a partial's item
    int64_t from, to;  // the item's units on the line
    int64_t first;     // its sequence's first row
    int32_t rows;      // query rows of its sequence and head (tokens * group)
    int32_t row0;      // first row of its tile
    int32_t head;
    int32_t tokens;    // new tokens of the sequence
};

template <int D, int NT>
struct Smem {
    static constexpr int kW = Shape<D, NT>::kWarps, kS = Shape<D, NT>::kStages, kR = 8 * NT;
    static constexpr int kH = Step<D>::kHalves;
    static constexpr int kHalf = 32 * D;   // 16 keys and 16 values
    static constexpr int kStage = kH * kHalf;
    static constexpr int kRing = kS * kStage, kHead = kR * D * 4;
    static constexpr int kPerWarp = kRing + kHead;
    static constexpr int kThreads = kW * 32;
    static_assert(kRing >= kHead, "the last partial goes where the ring was");
    float scales[kW][kS][kH][2];
    float m[2 * kW][kR], l[2 * kW][kR];
    Part part[2 * kW];
    uint32_t run[32];  // partials of the same item, as a mask
    int64_t before[kThreads + 1];
    int64_t wsum[kW];
    uint32_t last;
    float weight[kMaxBlocks][kR];  // of the blocks' partials in their join
    static constexpr int kBytes = kW * kPerWarp;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ uint2 lds8(const uint8_t* p) { return *reinterpret_cast<const uint2*>(p); }
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The product alone.
__device__ __forceinline__ void mma16816_only(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Byte offset of 16-byte chunk `c` of token row `r` in a stage's half: the
// chunks of each 128-byte line are permuted so that the lanes of a fragment
// load, which read one chunk of 2 to 8 rows, meet in no bank.
template <int D>
__device__ __forceinline__ int chunk_at(int r, int c) {
    const int lin = r * (D / 16) + c, line = lin >> 3;
    int f;
    if constexpr (D == 64)
        f = 2 * (line & 3);
    else if constexpr (D == 128)
        f = line & 7;
    else
        f = (line & 3) ^ ((line >> 2) & 1) ^ (((line >> 3) & 1) << 2);
    return (line * 8 + ((lin & 7) ^ f)) * 16;
}

// A sequence of the step: its rows, and its steps on the line.
struct Seq {
    int64_t first;   // first row
    int32_t pos, n;  // tokens held before, new tokens
    int32_t step0;   // first step that any row sees
    int32_t cost;    // units of an item: steps + kItemCost; 0: nothing to do
    int32_t tiles;   // of R rows
    bool bad, late;  // offsets are wrong; past the page table
};

template <int R, int TS>
__device__ __forceinline__ Seq load_seq(const AttendArgs& a, int64_t b) {
    Seq q;
    q.late = false;
    q.cost = 0;
    q.tiles = 0;
    q.step0 = 0;
    q.pos = __ldg(a.s.positions + b);
    int64_t n;
    q.bad = !rows_of(a.s, b, q.first, n);
    q.n = static_cast<int32_t>(n);
    if (n == 0 || q.pos < 0) return q;
    if (q.pos + n > int64_t{a.s.max_pages} * a.c.page_size) {
        q.late = true;
        return q;
    }
    const int end = q.pos + q.n;
    q.step0 = a.q.window > 0 && q.pos + 1 > a.q.window ? (q.pos + 1 - a.q.window) >> TS : 0;
    q.cost = ((end + (1 << TS) - 1) >> TS) - q.step0 + kItemCost;
    q.tiles = static_cast<int32_t>((n * a.group + R - 1) / R);
    return q;
}

__device__ __forceinline__ int64_t units_of(const AttendArgs& a, const Seq& q) {
    return int64_t{q.tiles} * a.c.heads * q.cost;
}

// A place on the line: an item, and a unit of it.
template <int R, int TS>
struct Cursor {
    Seq q;
    int64_t b;
    int64_t left;  // units of the warp's piece from here on
    int32_t tile, head, unit;

    // The line promises one while `left` is positive; should the lengths change
    // under the call, the piece ends at the last sequence.
    __device__ __forceinline__ void next_item(const AttendArgs& a) {
        unit = 0;
        if (++head < a.c.heads) return;
        head = 0;
        if (++tile < q.tiles) return;
        tile = 0;
        do {
            if (++b >= a.s.B) {
                left = 0;
                return;
            }
            q = load_seq<R, TS>(a, b);
        } while (q.cost == 0);
    }
};

// Offsets that do not ascend: the sequences before the first wrong pair; the rows from there on, which are nobody's,
// become NaN. Called by whole blocks.
__device__ __forceinline__ int64_t wrong_offsets(const AttendArgs& a) {
    const int64_t sound = sound_sequences(a.s), row0 = unclaimed_rows(a.s, sound);
    const int64_t dim = a.c.head_dim, per_row = a.q.q_heads * dim, vals = (a.s.T - row0) * per_row;
    const int64_t step = int64_t{gridDim.x} * blockDim.x;
    for (int64_t i = int64_t{blockIdx.x} * blockDim.x + threadIdx.x; i < vals; i += step)
        static_cast<uint16_t*>(a.q.out)[(row0 + i / per_row) * a.q.out_token_stride + i % per_row / dim * a.q.out_head_stride +
                                        i % dim] = a.bf16 ? 0x7FC0u : 0x7E00u;
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.err) atomicOr(a.err, ARC_KV_ERR_OFFSETS);
    return sound;
}

template <int D, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::kWarps * 32, 1) attend_kernel(const __grid_constant__ AttendArgs a) {
    using S = Smem<D, NT>;
    constexpr int R = S::kR, W = S::kW, ST = S::kS, kThreads = S::kThreads;
    constexpr int TS = Step<D>::kShift, HV = Step<D>::kHalves;
    constexpr int KS = D / 16;   // 16-value slices of a head
    constexpr int KC = D / 64;   // 16-byte chunks of a key that a lane takes
    constexpr int LB = D / 8;    // values of a head that a lane holds of the output
    extern __shared__ __align__(128) uint8_t dyn[];
    __shared__ S sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;

    // ---- the line: units before each thread's run of sequences
    const int64_t run = (a.s.B + kThreads - 1) / kThreads;
    int64_t mine, incl;
    uint32_t seen;
    int64_t sound = a.s.B;
    for (;; sound = wrong_offsets(a)) {  // (twice where offsets are wrong)
        mine = 0;
        seen = 0;
        for (int64_t b = run * tid; b < run * (tid + 1) && b < sound; ++b) {
            const Seq q = load_seq<R, TS>(a, b);
            mine += units_of(a, q);
            if (q.bad) seen |= ARC_KV_ERR_OFFSETS;
            if (q.late) seen |= ARC_KV_ERR_POSITION;
        }
        incl = mine;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int64_t o = __shfl_up_sync(0xFFFFFFFFu, incl, m);
            if (lane >= m) incl += o;
        }
        if (lane == 31) sm.wsum[warp] = incl;
        if (tid < 2 * W) sm.part[tid].from = -1;
        if (!__syncthreads_or(seen & ARC_KV_ERR_OFFSETS)) break;
    }
    if (seen && a.err && blockIdx.x == 0) atomicOr(a.err, seen);
    int64_t off = 0, total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const int64_t s = sm.wsum[w];
        if (w < warp) off += s;
        total += s;
    }
    sm.before[tid] = off + incl - mine;
    if (tid == 0) sm.before[kThreads] = total;

    // rows without work: parked sequences give 0, those past their page table NaN
    for (int64_t b = blockIdx.x; b < sound; b += gridDim.x) {
        const Seq q = load_seq<R, TS>(a, b);
        if (q.cost != 0 || q.n == 0) continue;
        const uint32_t fill = q.late ? (a.bf16 ? 0x7FC0u : 0x7E00u) : 0u;
        const int64_t vals = int64_t{q.n} * a.q.q_heads * D;
        for (int64_t i = tid; i < vals; i += kThreads) {
            const int64_t th = i / D;
            static_cast<uint16_t*>(a.q.out)[(q.first + th / a.q.q_heads) * a.q.out_token_stride +
                                            (th % a.q.q_heads) * a.q.out_head_stride + i % D] = static_cast<uint16_t>(fill);
        }
    }
    __syncthreads();
    if (total == 0) return;

    // ---- this block's and this warp's piece; short lines take fewer blocks
    const int64_t want = (total + W - 1) / W;
    const int64_t blocks = want < gridDim.x ? want : gridDim.x;
    if (blockIdx.x >= blocks) return;
    const int64_t pieces = blocks * W, piece = static_cast<int64_t>(blockIdx.x) * W + warp;
    // floor(total * i / of), without the product; four lanes find the four cuts
    auto cut = [total](int64_t i, int64_t of) { return total / of * i + total % of * i / of; };
    const int64_t cuts = cut(lane < 2 ? piece + lane : int64_t{blockIdx.x} + (lane & 1), lane < 2 ? pieces : blocks);
    const int64_t from = __shfl_sync(0xFFFFFFFFu, cuts, 0), to = __shfl_sync(0xFFFFFFFFu, cuts, 1);
    const int64_t block_from = __shfl_sync(0xFFFFFFFFu, cuts, 2), block_to = __shfl_sync(0xFFFFFFFFu, cuts, 3);

    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(dyn)) + warp * S::kPerWarp;
    float* const head_store = reinterpret_cast<float*>(dyn + warp * S::kPerWarp + S::kRing);
    float* const tail_store = reinterpret_cast<float*>(dyn + warp * S::kPerWarp);

    if (from < to) {
        Cursor<R, TS> at;  // of the arithmetic; `ahead` of the copies
        {
            int lo = 0, hi = kThreads;  // the run of sequences that holds `from`
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (sm.before[mid] <= from)
                    lo = mid;
                else
                    hi = mid;
            }
            int64_t rest = from - sm.before[lo];
            at.b = run * lo;
            at.q = load_seq<R, TS>(a, at.b);
            while (rest >= units_of(a, at.q) && at.b + 1 < a.s.B) {
                rest -= units_of(a, at.q);
                at.q = load_seq<R, TS>(a, ++at.b);
            }
            const int64_t item = at.q.cost <= 0     ? 0
                                 : rest >> 31 == 0 ? static_cast<uint32_t>(rest) / static_cast<uint32_t>(at.q.cost)
                                                   : rest / at.q.cost;
            at.unit = static_cast<int32_t>(rest - item * at.q.cost);
            at.tile = static_cast<int32_t>(item >> 31 == 0 ? static_cast<uint32_t>(item) / static_cast<uint32_t>(a.c.heads)
                                                           : item / a.c.heads);
            at.head = static_cast<int32_t>(item - int64_t{at.tile} * a.c.heads);
            at.left = at.q.cost > 0 ? to - from : 0;
        }
        Cursor<R, TS> ahead = at;

        // ---- copies
        int issued = 0;                 // stage of the next copy
        int step = 0, step_end = 0;     // of the item that is being copied
        int first = 0, last = 0;        // tokens that its rows see; the others are filled with zeros
        const int32_t* table = nullptr;
        const char *k_head = nullptr, *v_head = nullptr;  // its head, this lane's 16 bytes
        const float *k_scale = nullptr, *v_scale = nullptr;
        int page = 0, page_of = -1, page_next = 0, page_ahead = -1;  // page id, its index, the id after it, that one's
        int64_t page_at = 0;
        bool ok = true;
        const int ps_shift = 31 - __clz(a.c.page_size), ps_mask = a.c.page_size - 1;
        auto enter = [&]() {  // the next item that has a step
            while (step == step_end && ahead.left > 0) {
                if (ahead.unit == ahead.q.cost) ahead.next_item(a);
                if (ahead.left <= 0) return;
                const int n = ahead.q.cost - ahead.unit < ahead.left ? ahead.q.cost - ahead.unit : static_cast<int>(ahead.left);
                step = ahead.q.step0 + (ahead.unit > kItemCost ? ahead.unit - kItemCost : 0);
                ahead.unit += n;
                ahead.left -= n;
                step_end = ahead.q.step0 + (ahead.unit > kItemCost ? ahead.unit - kItemCost : 0);
            }
            const int row0 = ahead.tile * R, rows = ahead.q.n * a.group;
            const bool one = ahead.q.n == 1;
            last = ahead.q.pos + (one ? 0 : ((row0 + R < rows ? row0 + R : rows) - 1) / a.group);
            first = a.q.window > 0 ? ahead.q.pos + (one ? 0 : row0 / a.group) - a.q.window + 1 : 0;
            table = a.s.page_table + ahead.b * a.s.table_stride;
            const int64_t head = ahead.head * a.c.head_stride + lane * 16;
            k_head = static_cast<const char*>(a.c.k) + head;
            v_head = static_cast<const char*>(a.c.v) + head;
            k_scale = a.c.k_scale + ahead.head;
            v_scale = a.c.v_scale + ahead.head;
            page_of = page_ahead = -1;
        };
        uint32_t to[2];  // a lane's copies alternate between two places of a pattern that moves on by rows
        to[0] = ring + chunk_at<D>(lane / (D / 16), lane % (D / 16));
        to[1] = ring + chunk_at<D>((lane + 32) / (D / 16), (lane + 32) % (D / 16));
        auto issue = [&]() {
            if (step == step_end) enter();
            if (step < step_end) {
#pragma unroll
                for (int hv = 0; hv < HV; ++hv) {
                    const int tok0 = (step << TS) + 16 * hv, pi = tok0 >> ps_shift;
                    // (a half that no row sees takes no page)
                    const bool none = HV > 1 && (tok0 > last || tok0 + 15 < first);
                    if (!none && pi != page_of) {
                        page = pi == page_ahead ? page_next : __ldg(table + pi);
                        page_of = pi;
                        page_ahead = -1;
                        if (((pi + 1) << ps_shift) <= last && ((pi + 1) << ps_shift) >> TS < step_end) {
                            page_next = __ldg(table + pi + 1);
                            page_ahead = pi + 1;
                        }
                        ok = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.c.pages);
                        page_at = ok ? page * a.c.page_stride : 0;
                        if (!ok && lane == 0 && a.err) atomicOr(a.err, ARC_KV_ERR_PAGE);
                    }
                    const bool here = ok && !none;
                    const int64_t at = here ? page_at + (tok0 & ps_mask) * D : 0;
                    const char *kp = k_head + at, *vp = v_head + at;
                    const uint32_t move = issued * S::kStage + hv * S::kHalf;
                    const bool whole = here && tok0 >= first && tok0 + 15 <= last;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        // D = 256: the pattern of chunk_at has a period of 16 rows, eight copies
                        const uint32_t dst = (D == 256 ? ring + chunk_at<D>((lane + 32 * i) / 16, (lane + 32 * i) % 16)
                                                       : to[i & 1] + (i >> 1) * 1024) + move;
                        const int tok = tok0 + (lane + 32 * i) / (D / 16);
                        const bool on = whole || (here && tok <= last && tok >= first);
                        copy16(dst, kp + i * 512, on);
                        copy16(dst + 16 * D, vp + i * 512, on);
                    }
                    if (here) {
                        if (lane < 2)
                            copy4(static_cast<uint32_t>(__cvta_generic_to_shared(&sm.scales[warp][issued][hv][lane])),
                                  (lane ? v_scale : k_scale) + static_cast<int64_t>(page) * a.c.heads);
                    } else if (lane < 2) {
                        // (a bad page spoils the rows that see its tokens, through their scores)
                        sm.scales[warp][issued][hv][lane] = none || lane ? 1.0f : __int_as_float(0x7FC00000);
                    }
                }
                ++step;
            }
            copies_end();
            issued = issued + 1 == ST ? 0 : issued + 1;
        };
#pragma unroll
        for (int i = 0; i < ST - 1; ++i) issue();

        // ---- the piece, item by item
        int stage = 0;
        int64_t here = from;  // unit of the line
        while (at.left > 0) {
            if (at.unit == at.q.cost) at.next_item(a);
            if (at.left <= 0) break;
            const int64_t item_from = here - at.unit;
            const int32_t unit0 = at.unit;
            const int32_t unit1 = at.q.cost - unit0 < at.left ? at.q.cost : unit0 + static_cast<int32_t>(at.left);
            const int row0 = at.tile * R, rows = at.q.n * a.group;

            const bool one = at.q.n == 1;  // a row's token, without the division where there is one
            auto token_of = [&](int r) { return one ? 0 : r / a.group; };

            // queries: fp16, each row scaled by a power of two to [2^14, 2^15)
            uint32_t qf[NT][KS][2];
            float rf[NT][2];
            int hi[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float x[D / 4];
                const int r = row0 + 8 * nt + g;
                const int tok = token_of(r < rows ? r : rows - 1);
                if (r < rows) {
                    const char* p = static_cast<const char*>(a.q.q) +
                                    ((at.q.first + tok) * a.q.q_token_stride +
                                     (at.head * a.group + r - tok * a.group) * a.q.q_head_stride + t * (D / 4)) * 2;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        float e[8];
                        if (a.bf16)
                            load8<ARC_BF16>(p + 16 * i, a.vec & 1, e);
                        else
                            load8<ARC_F16>(p + 16 * i, a.vec & 1, e);
#pragma unroll
                        for (int k = 0; k < 8; ++k) x[8 * i + k] = e[k];
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < D / 4; ++k) x[k] = 0.0f;
                }
                float top = 0.0f;
#pragma unroll
                for (int k = 0; k < D / 4; ++k) top = fmaxf(top, fabsf(x[k]));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                // 2^(14 - exponent), kept inside fp32's normal range
                const int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
                const int up = top == 0.0f ? 0 : (14 - ex > 126 ? 126 : (14 - ex < -113 ? -113 : 14 - ex));
                const float f = exp2i(up);
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    qf[nt][j][0] = pack_f16(x[4 * j] * f, x[4 * j + 1] * f);
                    qf[nt][j][1] = pack_f16(x[4 * j + 2] * f, x[4 * j + 3] * f);
                }
                const float back = exp2i(-up) * (a.q.scale * 1.4426950408889634f);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    rf[nt][e] = __shfl_sync(0xFFFFFFFFu, back, (2 * t + e) * 4);
                    const int rr = row0 + 8 * nt + 2 * t + e;
                    hi[nt][e] = at.q.pos + token_of(rr < rows ? rr : rows - 1);
                }
            }
            const int hi_first = at.q.pos + token_of(row0);
            const int hi_last = at.q.pos + token_of((row0 + R < rows ? row0 + R : rows) - 1);

            float o[NT][KS][4], m[NT][2], l[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < KS; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.0f;
                m[nt][0] = m[nt][1] = kNothing;
                l[nt][0] = l[nt][1] = 0.0f;
            }

            for (int u = unit0 < kItemCost ? kItemCost : unit0; u < unit1; ++u) {
                copies_wait<ST - 2>();
                __syncwarp();  // every lane's copies are in, and every lane is done with the stage before
                issue();
                const uint8_t* const st = dyn + warp * S::kPerWarp + stage * S::kStage;
                float ks[HV], vs[HV];
#pragma unroll
                for (int hv = 0; hv < HV; ++hv) {
                    ks[hv] = sm.scales[warp][stage][hv][0];
                    vs[hv] = sm.scales[warp][stage][hv][1];
                }
                stage = stage + 1 == ST ? 0 : stage + 1;
                const int tok0 = (at.q.step0 + u - kItemCost) << TS;

                float s[HV][NT][4];
#pragma unroll
                for (int hv = 0; hv < HV; ++hv) {
                    const uint8_t* kst = st + hv * S::kHalf;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[hv][nt][e] = 0.0f;
#pragma unroll
                    for (int i = 0; i < KC; ++i) {
                        const uint4 k0 = lds16(kst + chunk_at<D>(g, KC * t + i));
                        const uint4 k1 = lds16(kst + chunk_at<D>(g + 8, KC * t + i));
                        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            uint32_t a0, a1, a2, a3;
                            e4m3x4_to_half2(w0[w], a0, a2);
                            e4m3x4_to_half2(w1[w], a1, a3);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816(s[hv][nt], a0, a1, a2, a3, qf[nt][4 * i + w][0], qf[nt][4 * i + w][1]);
                        }
                    }
                }
                const bool edge = tok0 + 16 * HV - 1 > hi_first || (a.q.window > 0 && tok0 <= hi_last - a.q.window);
                float top[NT][2];  // each row's largest score of the step
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = kNothing;
#pragma unroll
                for (int hv = 0; hv < HV; ++hv) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s[hv][nt][e] *= ks[hv] * rf[nt][e & 1];
                            if (edge) {
                                const int tok = tok0 + 16 * hv + g + (e >> 1) * 8, h = hi[nt][e & 1];
                                if (tok > h || (a.q.window > 0 && tok <= h - a.q.window)) s[hv][nt][e] = -INFINITY;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) top[nt][e] = fmaxf(top[nt][e], fmaxf(s[hv][nt][e], s[hv][nt][e + 2]));
                    }
                }
#pragma unroll
                for (int x = 4; x < 32; x <<= 1)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            top[nt][e] = fmaxf(top[nt][e], __shfl_xor_sync(0xFFFFFFFFu, top[nt][e], x));
                bool up = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) up = up || top[nt][e] > m[nt][e];
                if (__any_sync(0xFFFFFFFFu, up)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float f[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float mn = fmaxf(m[nt][e], top[nt][e]);
                            f[e] = ex2(m[nt][e] - mn);
                            m[nt][e] = mn;
                            l[nt][e] *= f[e];
                        }
#pragma unroll
                        for (int i = 0; i < KS; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[nt][i][e] *= f[e & 1];
                    }
                }
                float f[NT][2];  // what the step's weights count in the running sums
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) f[nt][e] = ex2(top[nt][e] - m[nt][e]);
#pragma unroll
                for (int hv = 0; hv < HV; ++hv) {
                    const uint8_t* vst = st + hv * S::kHalf + 16 * D;
                    uint32_t pf[NT][2];
                    float fv[NT][2];  // and its products, half by half
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float p[4];
#pragma unroll
                        for (int e = 0; e < 2; ++e) fv[nt][e] = f[nt][e] * (vs[hv] * (1.0f / kLift));
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            p[e] = ex2(s[hv][nt][e] - top[nt][e & 1]);
                            l[nt][e & 1] = fmaf(p[e], f[nt][e & 1], l[nt][e & 1]);
                        }
                        // token-major to row-major: what the products take
                        pf[nt][0] = transpose8x8(pack_f16(p[0] * kLift, p[1] * kLift));
                        pf[nt][1] = transpose8x8(pack_f16(p[2] * kLift, p[3] * kLift));
                    }

                    // values: tokens 2t, 2t+1, 2t+8, 2t+9, D / 8 bytes from g * D / 8
                    uint32_t v[4][LB / 4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 2 * t + (i & 1) + (i >> 1) * 8;
                        if constexpr (D == 64) {
                            const uint2 x = lds8(vst + chunk_at<D>(r, g >> 1) + (g & 1) * 8);
                            v[i][0] = x.x;
                            v[i][1] = x.y;
                        } else {
#pragma unroll
                            for (int c = 0; c < D / 128; ++c) {
                                const uint4 x = lds16(vst + chunk_at<D>(r, (D / 128) * g + c));
                                v[i][4 * c] = x.x;
                                v[i][4 * c + 1] = x.y;
                                v[i][4 * c + 2] = x.z;
                                v[i][4 * c + 3] = x.w;
                            }
                        }
                    }
                    if (edge && hi_first != hi_last) {
                        // a token that some rows see and others do not: its NaN values must not
                        // reach the others through 0 * NaN
                        uint32_t any = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int w = 0; w < LB / 4; ++w) any |= ((v[i][w] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                        if (__any_sync(0xFFFFFFFFu, any != 0)) {
                            for (int r = 0; r < R; ++r) {
                                const int rr = row0 + r, h = at.q.pos + (rr < rows ? rr : rows - 1) / a.group;
                                uint32_t hit = 0;  // values of this lane's that are NaN in a token row r sees
                                for (int i = 0; i < 4; ++i) {
                                    const int tok = tok0 + 16 * hv + 2 * t + (i & 1) + (i >> 1) * 8;
                                    if (tok > h || (a.q.window > 0 && tok <= h - a.q.window)) continue;
#pragma unroll
                                    for (int k = 0; k < LB; ++k)
                                        if (((v[i][k >> 2] >> (8 * (k & 3))) & 0x7Fu) == 0x7Fu) hit |= 1u << k;
                                }
                                hit |= __shfl_xor_sync(0xFFFFFFFFu, hit, 1);
                                hit |= __shfl_xor_sync(0xFFFFFFFFu, hit, 2);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                    for (int e = 0; e < 2; ++e)
                                        if (8 * nt + 2 * t + e == r)
#pragma unroll
                                            for (int k = 0; k < LB; ++k)
                                                if ((hit >> k) & 1) o[nt][k >> 1][2 * (k & 1) + e] = __int_as_float(0x7FC00000);
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int w = 0; w < LB / 4; ++w) {
                                    const uint32_t bad = ((v[i][w] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                                    v[i][w] &= ~((bad >> 7) * 0xFFu);
                                }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        const int w = i >> 1;
                        const uint32_t x = __byte_perm(v[0][w], v[1][w], (i & 1) ? 0x7362 : 0x5140);
                        const uint32_t y = __byte_perm(v[2][w], v[3][w], (i & 1) ? 0x7362 : 0x5140);
                        uint32_t a0, a1, a2, a3;
                        e4m3x4_to_half2(x, a0, a1);
                        e4m3x4_to_half2(y, a2, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float d[4];
                            mma16816_only(d, a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[nt][i][e] = fmaf(d[e], fv[nt][e & 1], o[nt][i][e]);
                        }
                    }
                }
            }

            // ---- the part is done: lanes' sums, then the output or a partial
#pragma unroll
            for (int x = 4; x < 32; x <<= 1)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) l[nt][e] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][e], x);
            const int32_t units = unit1 - unit0;
            at.unit = unit1;
            at.left -= units;
            here += units;
            if (units == at.q.cost) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int rr = row0 + 8 * nt + 2 * t + e;
                        if (rr >= rows) continue;
                        const int tok = token_of(rr);
                        const float inv = 1.0f / l[nt][e];
                        char* p = static_cast<char*>(a.q.out) +
                                  ((at.q.first + tok) * a.q.out_token_stride +
                                   (at.head * a.group + rr - tok * a.group) * a.q.out_head_stride + g * LB) * 2;
#pragma unroll
                        for (int c = 0; c < LB / 8; ++c) {
                            float x[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) x[k] = o[nt][4 * c + (k >> 1)][2 * (k & 1) + e] * inv;
                            if (a.bf16)
                                store8<ARC_BF16>(p + 16 * c, a.vec & 2, x);
                            else
                                store8<ARC_F16>(p + 16 * c, a.vec & 2, x);
                        }
                    }
            } else {
                // the piece's first item goes to its own store (the ring is in use), the last one over the ring
                const bool tail = at.left == 0;
                const int slot = 2 * warp + (tail ? 1 : 0);
                float* store = tail ? tail_store : head_store;
                if (tail) {
                    copies_wait<0>();
                    __syncwarp();
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = 8 * nt + 2 * t + e;
                        float* p = store + r * D + g * LB;
#pragma unroll
                        for (int c = 0; c < LB / 4; ++c)
                            *reinterpret_cast<float4*>(p + 4 * c) =
                                make_float4(o[nt][2 * c][e], o[nt][2 * c][2 + e], o[nt][2 * c + 1][e], o[nt][2 * c + 1][2 + e]);
                        if (g == 0) {
                            sm.m[slot][r] = m[nt][e];
                            sm.l[slot][r] = l[nt][e];
                        }
                    }
                if (lane == 0)
                    sm.part[slot] = Part{item_from, item_from + at.q.cost, at.q.first, rows, row0, at.head, at.q.n};
            }
        }
        copies_wait<0>();
    }
    __syncthreads();

    // ---- join the block's partials.  Those of one item are a run; a warp takes a row of a run.
    static_assert(2 * W <= 32, "a lane for each partial");
    constexpr int DV = D / 32;                // values of a lane
    constexpr int kSlot = R * D + 2 * R;      // floats of a block's partial: output, maxima, sums
    auto write = [&](const Part& p, int r, const float (&x)[DV]) {
        const int rr = p.row0 + r, tok = p.tokens == 1 ? 0 : rr / a.group;
        uint16_t* out = static_cast<uint16_t*>(a.q.out) + (p.first + tok) * a.q.out_token_stride +
                        (p.head * a.group + rr - tok * a.group) * a.q.out_head_stride + lane * DV;
        uint32_t w[DV / 2];
#pragma unroll
        for (int i = 0; i < DV / 2; ++i)
            w[i] = a.bf16 ? Half<ARC_BF16>::pack(x[2 * i], x[2 * i + 1]) : Half<ARC_F16>::pack(x[2 * i], x[2 * i + 1]);
        if (a.vec & 2) {
            if constexpr (DV == 2)
                *reinterpret_cast<uint32_t*>(out) = w[0];
            else if constexpr (DV == 4)
                *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
            else
                *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < DV / 2; ++i) {
                out[2 * i] = static_cast<uint16_t>(w[i]);
                out[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
            }
        }
    };
    const int64_t my_from = lane < 2 * W ? sm.part[lane].from : -1;
    const uint32_t run_of = __match_any_sync(0xFFFFFFFFu, my_from);
    const uint32_t leaders = __ballot_sync(0xFFFFFFFFu, my_from >= 0 && lane == __ffs(run_of) - 1);
    const int runs = __popc(leaders);
    if (warp == 0) sm.run[lane] = my_from >= 0 ? run_of : 0;
    __syncthreads();
    // a thread for each partial and row: its weight in its run, from the run's maximum
    for (int i = tid; i < 2 * W * R; i += kThreads) {
        const int e = i / R, r = i % R;
        const uint32_t run = sm.run[e];
        float mm = kNothing, l = 0.0f;
        for (uint32_t left = run; left; left &= left - 1) mm = fmaxf(mm, sm.m[__ffs(left) - 1][r]);
        for (uint32_t left = run; left; left &= left - 1) {
            const int k = __ffs(left) - 1;
            l = fmaf(sm.l[k][r], ex2(sm.m[k][r] - mm), l);
        }
        if (run) {
            const Part& p = sm.part[e];
            const bool whole = p.from >= block_from && p.to <= block_to;
            const float f = ex2(sm.m[e][r] - mm);
            sm.weight[e][r] = whole ? f / l : f;
            if (!whole && e == __ffs(run) - 1 && p.row0 + r < p.rows) {
                float* slot = a.partial + (static_cast<int64_t>(blockIdx.x) * 2 + (p.from >= block_from ? 1 : 0)) * kSlot;
                __stcg(slot + R * D + r, mm);
                __stcg(slot + R * D + R + r, l);
            }
        }
    }
    __syncthreads();
    for (int task = warp; task < runs * R; task += W) {
        const int r = task % R;
        const int lead = __fns(leaders, 0, task / R + 1);
        const Part p = sm.part[lead];
        if (p.row0 + r >= p.rows) continue;
        float x[DV];
#pragma unroll
        for (int i = 0; i < DV; ++i) x[i] = 0.0f;
        for (uint32_t left = sm.run[lead]; left; left &= left - 1) {
            const int e = __ffs(left) - 1;
            const float fe = sm.weight[e][r];
            const float* v = reinterpret_cast<const float*>(dyn + (e >> 1) * S::kPerWarp + ((e & 1) ? 0 : S::kRing)) + r * D + lane * DV;
#pragma unroll
            for (int i = 0; i < DV; i += 2) {
                const float2 y = *reinterpret_cast<const float2*>(v + i);
                x[i] = fmaf(y.x, fe, x[i]);
                x[i + 1] = fmaf(y.y, fe, x[i + 1]);
            }
        }
        if (p.from >= block_from && p.to <= block_to) {
            write(p, r, x);
        } else {
            float* slot = a.partial + (static_cast<int64_t>(blockIdx.x) * 2 + (p.from >= block_from ? 1 : 0)) * kSlot;
#pragma unroll
            for (int i = 0; i < DV; i += 2) __stcg(reinterpret_cast<float2*>(slot + r * D + lane * DV + i), make_float2(x[i], x[i + 1]));
        }
    }
    if (leaders == 0) return;  // the same in every warp

    // ---- items over several blocks (this block's first, and its last): the last block to arrive joins all,
    // in their order
    const int ends[2] = {__ffs(leaders) - 1, 31 - __clz(leaders)};
    bool any = false;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const Part p = sm.part[ends[k]];
        any = any || p.from < block_from || p.to > block_to;
    }
    if (!any) return;
    __threadfence();
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        if (k == 1 && ends[1] == ends[0]) break;
        const Part p = sm.part[ends[k]];
        if (p.from >= block_from && p.to <= block_to) continue;
        // (the block of unit f is floor(((f + 1) * blocks - 1) / total))
        const int64_t at = (((lane ? p.to - 1 : p.from) + 1) * blocks - 1) / total;
        const int64_t c0 = __shfl_sync(0xFFFFFFFFu, at, 0), c1 = __shfl_sync(0xFFFFFFFFu, at, 1);
        if (tid == 0) sm.last = atomicInc(a.arrived + c0, static_cast<uint32_t>(c1 - c0)) == static_cast<uint32_t>(c1 - c0);
        __syncthreads();
        if (sm.last) {
            __threadfence();
            const int n = static_cast<int>(c1 - c0) + 1;
            const float* first = a.partial + (c0 * 2 + 1) * kSlot;  // the item starts in c0's second slot,
            auto slot_of = [&](int c) { return first + (c == 0 ? 0 : (2 * c - 1) * kSlot); };  // then the first ones
            for (int r = warp; r < R; r += W) {
                if (p.row0 + r >= p.rows) break;
                float mc[kMaxBlocks / 32], lc[kMaxBlocks / 32];
                float mm = kNothing, l = 0.0f;
#pragma unroll
                for (int i = 0; i < kMaxBlocks / 32; ++i) {
                    const int c = lane + 32 * i;
                    mc[i] = c < n ? __ldcg(slot_of(c) + R * D + r) : kNothing;
                    lc[i] = c < n ? __ldcg(slot_of(c) + R * D + R + r) : 0.0f;
                }
#pragma unroll
                for (int i = 0; i < kMaxBlocks / 32; ++i) mm = fmaxf(mm, mc[i]);
#pragma unroll
                for (int x = 16; x; x >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, x));
#pragma unroll
                for (int i = 0; i < kMaxBlocks / 32; ++i) {
                    mc[i] = ex2(mc[i] - mm);
                    l = fmaf(lc[i], mc[i], l);
                }
#pragma unroll
                for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
#pragma unroll
                for (int i = 0; i < kMaxBlocks / 32; ++i) {
                    const int c = lane + 32 * i;
                    if (c < n) sm.weight[c][r] = mc[i] / l;
                }
            }
            __syncthreads();
            for (int r = warp; r < R; r += W) {
                if (p.row0 + r >= p.rows) break;
                float x[DV];
#pragma unroll
                for (int i = 0; i < DV; ++i) x[i] = 0.0f;
#pragma unroll 8
                for (int c = 0; c < n; ++c) {
                    const float f = sm.weight[c][r];
                    const float* q = slot_of(c) + r * D + lane * DV;
#pragma unroll
                    for (int i = 0; i < DV; i += 2) {
                        const float2 v = __ldcg(reinterpret_cast<const float2*>(q + i));
                        x[i] = fmaf(v.x, f, x[i]);
                        x[i + 1] = fmaf(v.y, f, x[i + 1]);
                    }
                }
                write(p, r, x);
            }
        }
        __syncthreads();
    }
}

template <int D, int NT>
int launch(const AttendArgs& a, int dev, int sms, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    using S = Smem<D, NT>;
    static_assert(S::kBytes + sizeof(S) <= arc::kSmemPerBlock, "shared memory");
    if (arc::prepare(attend_kernel<D, NT>, dev, done, 100) != cudaSuccess) return ARC_E_CUDA;
    const int grid = sms < kMaxBlocks ? sms : kMaxBlocks;
    attend_kernel<D, NT><<<grid, S::kThreads, S::kBytes, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? ARC_OK : ARC_E_CUDA;
}

}  // namespace

extern "C" {

size_t arc_kv_attend_workspace_bytes(const arc_kv_cache* cache) {
    if (check_cache(cache) != ARC_OK) return 0;
    const size_t rows = cache->head_dim == 256 ? 8 : 16;
    return kStatusBytes + size_t{kMaxBlocks} * 2 * (rows * cache->head_dim + 2 * rows) * 4;
}

int arc_kv_attend(const arc_kv_cache* cache, const arc_kv_step* step, const arc_kv_query* query, uint32_t* err_word,
                  void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_cache(cache);
    if (rc == ARC_OK) rc = check_step(cache, step);
    if (rc != ARC_OK) return rc;
    if (query == nullptr || query->q == nullptr || query->out == nullptr) return ARC_E_NULL;
    if (query->dtype != ARC_BF16 && query->dtype != ARC_F16) return ARC_E_DTYPE;
    if (query->q_heads <= 0 || query->q_heads > (1 << 16) || query->q_heads % cache->heads != 0) return ARC_E_SHAPE;
    // rows of a (sequence, cached head) are counted in 32 bits
    if (step->T * (query->q_heads / cache->heads) > (int64_t{1} << 30)) return ARC_E_SHAPE;
    if (query->window < 0 || !(query->scale >= -3.0e38f && query->scale <= 3.0e38f)) return ARC_E_OPTION;
    if (!aligned(query->q, 2) || !aligned(query->out, 2) || !aligned(err_word, 4)) return ARC_E_ALIGN;
    if (workspace == nullptr || workspace_bytes < arc_kv_attend_workspace_bytes(cache)) return ARC_E_WORKSPACE;
    if (!aligned(workspace, 16)) return ARC_E_ALIGN;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return ARC_E_CUDA;
    }
    AttendArgs a;
    a.c = *cache;
    a.s = *step;
    a.q = *query;
    a.err = err_word;
    a.arrived = static_cast<uint32_t*>(workspace);
    a.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + kStatusBytes);
    a.group = query->q_heads / cache->heads;
    a.bf16 = query->dtype == ARC_BF16;
    a.vec = (vectors(query->q, query->q_token_stride, query->q_head_stride) ? 1 : 0) |
            (vectors(query->out, query->out_token_stride, query->out_head_stride) ? 2 : 0);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // Rows of a (sequence, cached head) on average.  Tiles of 16 read the cache half as often and pay when they are
    // full: groups of 10 to 16 heads, one token each, heads of 128: 136 us against 168 with tiles of 8; of 64: 88 to
    // 91 against 100; pieces of 30 to 90 tokens 449 against 566 and 266 against 317.  Ragged drafts leave many of them
    // half empty: 1 to 5 tokens at 9 rows on average 64 us against 72, at 15 87 against 93, at 18 to 24 still 91 to 103
    // against 100 to 110; sequences of one length, at 16 rows 132 against 139, at 20 163 against 155 (heads of 64: 45
    // against 50, 57 against 62, 60 to 67 against 67 to 73, 83 against 93, 99 against 102).  The lengths are on the
    // device, so the border lies between the ragged and the even ones.
    const int64_t small = step->row_offsets != nullptr && a.group <= 8 ? 18 : 8;
    const bool wide = step->T * a.group > step->B * small;
    if (cache->head_dim == 64) return wide ? launch<64, 2>(a, dev, sms, st) : launch<64, 1>(a, dev, sms, st);
    if (cache->head_dim == 128) return wide ? launch<128, 2>(a, dev, sms, st) : launch<128, 1>(a, dev, sms, st);
    return launch<256, 1>(a, dev, sms, st);
}

}  // extern "C"
