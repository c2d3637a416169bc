// arc_kv_attend_shared: attention of a step's new tokens behind a prefix that all sequences share.
//
// Three kernels, the first two side by side where the first leaves SMs free, else one after the other.  The prefix: all
// rows of a cached head (new tokens times its query heads) against the prefix's pages, which are read once for them.  The
// sequences' own tokens: kv_attend.cuh's kernel, with its results in fp32.  And the join of a row's parts, each an output
// with the base-2 logarithm of its sum of weights:
//     out = sum_i 2^(log_i - max) out_i / sum_i 2^(log_i - max).
//
// The prefix.  A unit is a cached head and up to 256 rows (128 for heads of 256).  A chunk is 128 tokens (64 for heads
// of 256) of the prefix; all units' chunks lie on a line that is cut into one piece a block.  A block runs through its
// piece tile by tile, and leaves a partial for each unit that it has met.
//
// Products.  Codes are loaded a tile ahead into registers and become fp16 in shared memory, exactly.  S = Q K^T and O
// += P V run on the 5th-generation tensor cores, M = 128 rows: Q and K from shared memory, P from tensor memory, where
// the softmax has put it over S, V as it lies, tokens as rows, read across.
//
// Softmax.  P holds the weights relative to a reference of the row and the value scales relative to a reference of the
// tiles, 2^12 times, as fp16, and O is summed up in tensor memory in their units.  The references stay while the
// largest score of a step's 64 tokens lies at most 3 above the row's (as a power of two) or 10 below, and its pages'
// value scales within 1/16 of theirs; a tile is a chunk, or the part of one whose pages agree.  Else the row's becomes
// the step's own largest score and 4, room for larger ones, and the sums so far are multiplied by what that changes, in
// fp32: a weight keeps its bits beside those of its own step, whatever scores and scales came before.  (A reference
// lies at most 2^60 below the largest weight times scale so far, so that the sums stay in fp32's range.)  The sum of
// the weights is kept apart, relative to the largest score.
//
// Roles of a block: two groups of four warps take the softmax, a thread a row (two groups of 128 rows, or for heads of
// 256 one, half of the output each), a group makes fp16 of codes, a thread for each group of rows issues its products
// and a warp looks up pages and scales.  While one group of rows is at its softmax the products of the other run.
//
// Every wait has a limit; a block whose wait runs out leaves NaN.
//
// Bounds and figures.  256 sequences behind 16,384 tokens, 64 + 8 heads of 128 (137 GFLOP): the prefix about 147 us, 930
// TFLOP/s, 49% of the measured bf16 rate; a step of 64 tokens takes some 2,500 clocks, the products alone 1,262: what
// is left are the latencies of the softmax's steps (barrier, scores, maximum, exponentials, barrier), which two warps a
// scheduler do not hide.  64 behind 32,768, 32 + 8 heads: 45 us of 76 in all.  Few rows: latency, 20 us for the three
// kernels, 28 one after another.  Value scales between 2^-12 and 2^-4 on pages of 32, where references move and chunks
// are split: 360 us for the first case's 196 in all.  Measured and left, the prefix of the first case: output read back
// and added up in registers each tile 252 us; steps of 128 tokens, one ahead 169; weights made before the maximum is known
// and again where the reference moves 186 to 255; one thread for all products 161; loops over a step's scores unrolled
// further 10% to 30% slower each time.
#include "kv_shared.cuh"

#include <atomic>
#include <climits>
#include <cstring>

#include "kv_attend.cuh"
#include "launch_util.cuh"
#include "tensor_core.cuh"

namespace arcs {
namespace {

constexpr float kSpread = 16.0f;  // of the value scales that share a reference
constexpr int kInfos = 8;         // ring of tiles' descriptions
// Scales are at most kMost.  Value scales below kLeast count as 0: references of pages that lie further apart than that
// would take each other's weights to 0 as fp16, and with them the sum of the weights.
constexpr float kMost = 4294967296.0f, kLeast = 1.0f / (1ull << 60);
// A new reference lies kRoom above the step's largest score; it stays while that is at most kAbove above it (2^(12 + 3)
// is the largest weight as fp16) and kBelow below.
constexpr float kLift = 12.0f, kRoom = 4.0f, kAbove = 3.0f, kBelow = 10.0f;
constexpr float kSpan = 60.0f;
// References up to here: a score's and a reference's half steps of fp32 are then 1/4, so that the largest weight stays below
// 2^15.75.  Past it a weight as fp16 may be infinite or lost: the row becomes NaN.  Measured and left: scores rounded before
// the reference is taken away, as the largest is, which would hold for any; 1 to 4% of each call.
constexpr float kFar = 4194304.0f;

template <int D>
struct Prefix {
    static constexpr int kStep = 64;                     // tokens of a step
    static constexpr int kSteps = D == 256 ? 1 : 2;      // of a tile
    static constexpr int kTokens = kStep * kSteps;       // of a tile
    static constexpr int kTiles = D == 256 ? 1 : 2;      // tiles of 128 rows
    static constexpr int kRows = 128 * kTiles;
    static constexpr int kOut = D == 256 ? 128 : D;      // values of the output that a thread adds up
    static constexpr int kGranules = kTokens / 16;
    static constexpr int kThreads = 512;
    static constexpr int kQ = 128 * D * 2;
    static constexpr int kOp = kTokens * D * 2, kOps = D == 64 ? 8 : 5;  // ring of fp16 tiles, K and V in turn
    static constexpr int kSmem = kTiles * kQ + kOps * kOp + 1024;
    static constexpr int kEach = kTokens * D / 16 / 128;  // 16 codes each, of K or V, that a converting thread has
    // columns of tensor memory: two steps' scores of each tile of rows, weights over them (heads of 256: beside), output
    static constexpr int kS = 0, kP = D == 256 ? 128 : 0, kPStep = D == 256 ? 32 : 64, kO = 256;
    // registers of a thread once the roles part, of 128 at the launch of 512 threads (4 * 128 = 512)
    static constexpr int kSoftmaxRegs = 176, kConvertRegs = 104, kIssueRegs = 56;
    static_assert(2 * kSoftmaxRegs + kConvertRegs + kIssueRegs <= 512, "registers of the launch");
    static_assert(kO + kTiles * D <= 512, "tensor memory");
};

struct PrefixArgs {
    arc_kv_cache c;
    const void* q;
    int64_t q_token_stride, q_head_stride;
    const int32_t* pages;
    uint32_t* err;
    float* slots;      // [slot][tile of 128 rows][D / 4][128][4]
    float* slot_logs;  // [slot][rows of a unit]
    int64_t rows;      // of a cached head
    int64_t row_groups;
    int64_t total;     // chunks on the line
    int32_t chunks;    // of the prefix
    int32_t prefix_pages;
    int32_t pieces;
    int32_t group;
    int32_t bf16, vec;
    float scale;       // times log2(e)
};

__host__ __device__ inline int64_t cut_of(int64_t total, int64_t i, int64_t of) { return total / of * i + total % of * i / of; }

struct __align__(16) Info {  // a tile
    int32_t tokens;
    int32_t flags;    // 1: the last of its unit's, 2: the last of all, 4: another reference than the tile before's, 8: its
                      // values count as zeros
    float value;      // the reference of the value scales,
    float value_log;  // its logarithm
    float key[8];     // of each 16 tokens: key scale,
    float lift[8];    // 12 + the logarithm of the value scale over the reference,
    float back[8];    // 2^-lift; where there are no tokens key and back are 0 and the lift takes every weight to 0
    int64_t at[8];    // bytes from the cache's beginning to each page's part; -1: a bad page
};

struct PrefixBars {
    uint64_t q_full[2], s_full[2][2], p_full[2][2], o_full[2][2];  // [tile of rows][step's parity]
    uint64_t op_full[8], op_empty[8];
    uint64_t info_full[kInfos], info_empty[kInfos];
    uint64_t drained[2];
    uint32_t tmem, failed;
    Info info[kInfos];
};

// One thread issues the products of tile w of the rows.  The scores are two steps ahead of the output, whose weights the
// softmax makes meanwhile: where a step's output is issued its scores' place is free, and the step after next's follow at
// once.  At a unit's end they wait for the next unit's queries.
template <int D>
__device__ __forceinline__ bool issue_prefix(PrefixBars& bars, uint32_t q_at, uint32_t ops, uint32_t tmem, int w) {
    using X = Prefix<D>;
    constexpr uint32_t s_desc = (1u << 4) | (static_cast<uint32_t>(X::kStep / 8) << 17) | (8u << 24);
    constexpr uint32_t o_desc = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(D / 8) << 17) | (8u << 24);
    constexpr uint32_t kBlock = X::kTokens * 128;  // 64 values of all tokens
    auto op_of = [](uint32_t u) { return u % X::kOps; };
    auto op_phase = [](uint32_t u) { return (u / X::kOps) & 1; };
    const uint64_t queries = operand_at(q_at + w * X::kQ);
    uint32_t q_phase = 0;
    uint32_t ahead = 0;  // the next step whose scores are to be issued, of tile ahead / kSteps
    int ahead_flags = 0;
    bool unit_done = false;  // the scores of this unit's last step are out
    auto scores = [&]() {
        const uint32_t t = ahead / X::kSteps, half = ahead % X::kSteps;
        const uint64_t b = operand_at(ops + op_of(2 * t) * X::kOp + half * (X::kStep * 128));
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
            mma_f16_shared(tmem + X::kS + w * 128 + (ahead & 1) * 64, queries + (k >> 2) * (128 * 128 / 16) + (k & 3) * 2,
                           b + (k >> 2) * (kBlock / 16) + (k & 3) * 2, s_desc, k != 0);
        commit_to(&bars.s_full[w][ahead & 1]);
        if (half == X::kSteps - 1) {
            commit_to(&bars.op_empty[op_of(2 * t)]);
            unit_done = ahead_flags & 1;
        }
        ++ahead;
    };
    // What the coming steps wait for but their weights: keys of the step `ahead` where it begins a tile, values of step n
    // where it does.  It is looked at while the softmax is at work, and together: a look at a barrier takes 150 clocks even
    // at a finished phase, 400 beside the other warps.
    auto look = [&](bool keys, bool values, uint32_t n) {
        keys = keys && ahead % X::kSteps == 0;
        values = values && n % X::kSteps == 0;
        const uint32_t t = ahead / X::kSteps, u = 2 * (n / X::kSteps) + 1;
        uint64_t* const info_bar = &bars.info_full[t % kInfos];
        uint64_t* const k_bar = &bars.op_full[op_of(2 * t)];
        uint64_t* const v_bar = &bars.op_full[op_of(u)];
        uint32_t info_done = 1, k_done = 1, v_done = 1;
        if (keys) {
            info_done = bar_done(info_bar, (t / kInfos) & 1);
            k_done = bar_done(k_bar, op_phase(2 * t));
        }
        if (values) v_done = bar_done(v_bar, op_phase(u));
        if (!info_done && !bar_wait(info_bar, (t / kInfos) & 1, &bars.failed)) return false;
        if (keys) ahead_flags = bars.info[t % kInfos].flags;
        if (!k_done && !bar_wait(k_bar, op_phase(2 * t), &bars.failed)) return false;
        return v_done || bar_wait(v_bar, op_phase(u), &bars.failed);
    };
    uint32_t n = 0;  // the step whose output comes next
    for (bool all = false; !all;) {
        // ---- a unit: its first two steps' scores
        unit_done = false;
        if (!look(true, true, n) || !bar_wait(&bars.q_full[w], q_phase, &bars.failed)) return false;
        q_phase ^= 1;
        fence_after();
        scores();
        if (!unit_done) {
            if (!look(true, false, n)) return false;
            fence_after();
            scores();
        }
        const uint32_t first = n;
        bool more = !unit_done;
        if (more && !look(true, false, n)) return false;
        for (;;) {
            const uint32_t u = 2 * (n / X::kSteps) + 1, half = n % X::kSteps;
            if (!bar_wait(&bars.p_full[w][n & 1], (n >> 1) & 1, &bars.failed)) return false;
            fence_after();
            const uint64_t b = operand_across(ops + op_of(u) * X::kOp + half * (X::kStep * 128), kBlock);
#pragma unroll
            for (int k = 0; k < X::kStep / 16; ++k)
                mma_f16(tmem + X::kO + w * D, tmem + X::kP + w * 128 + (n & 1) * X::kPStep + k * 8, b + k * (2048 / 16), o_desc,
                        k != 0 || n != first);
            commit_to(&bars.o_full[w][n & 1]);
            if (half == X::kSteps - 1) commit_to(&bars.op_empty[op_of(u)]);
            if (more) scores();
            if (++n == ahead) break;
            more = !unit_done;
            if (!look(more, true, n)) return false;
        }
        all = ahead_flags & 2;
    }
    return true;
}

template <int D>
__global__ void __launch_bounds__(512, 1) prefix_kernel(const __grid_constant__ PrefixArgs a) {
    using X = Prefix<D>;
    extern __shared__ uint8_t raw_smem[];
    __shared__ PrefixBars bars;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the own tokens' kernel needs nothing of this one
    uint8_t* const dyn = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t{1023});
    uint8_t* const q_tiles = dyn;
    uint8_t* const ops = dyn + X::kTiles * X::kQ;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t from = cut_of(a.total, blockIdx.x, a.pieces), to = cut_of(a.total, blockIdx.x + 1, a.pieces);
    const int tiles = X::kTiles == 2 && a.rows > 128 ? 2 : 1;  // of rows

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            bar_init(&bars.q_full[i], D == 256 ? 8 : 4);
            for (int b = 0; b < 2; ++b) {
                bar_init(&bars.s_full[i][b], 1);
                bar_init(&bars.o_full[i][b], 1);
                bar_init(&bars.p_full[i][b], D == 256 ? 8 : 4);
            }
        }
        for (int i = 0; i < 8; ++i) {
            bar_init(&bars.op_full[i], 4);
            bar_init(&bars.op_empty[i], tiles);
        }
        for (int i = 0; i < kInfos; ++i) {
            bar_init(&bars.info_full[i], 1);
            bar_init(&bars.info_empty[i], D == 256 ? 8 : 4 * tiles);
        }
        for (int i = 0; i < 2; ++i) bar_init(&bars.drained[i], 1);
        bars.failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_operands();
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(shared_of(&bars.tmem)), "n"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = bars.tmem;

    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(X::kIssueRegs));
        if (warp - 12 < tiles && elect_one()) {
            // ---- products: a thread for each tile of rows, in warps that wait for nobody
            if (!issue_prefix<D>(bars, shared_of(q_tiles), shared_of(ops), tmem, warp - 12)) {
                commit_to(&bars.drained[warp - 12]);
                uint32_t quiet = 0;
                bar_wait(&bars.drained[warp - 12], 0, &quiet);
            }
        }
        if (warp == 14) {
            // ---- tiles: a lane for each page of a chunk, whose number and scales are loaded ahead
            const int ps = a.c.page_size, span = ps < X::kTokens ? ps : X::kTokens, per = X::kTokens / span;
            const int ps_shift = 31 - __clz(ps), span_shift = 31 - __clz(span);
            struct Place {  // of a chunk; stepped on, since its divisions take longer than a tile
                int64_t c;
                int head, group, chunk;
            };
            Place now;
            now.c = from;
            now.chunk = static_cast<int>(from % a.chunks);
            now.head = static_cast<int>(from / a.chunks / a.row_groups);
            now.group = static_cast<int>(from / a.chunks % a.row_groups);
            auto step = [&](Place p) {
                ++p.c;
                if (++p.chunk == a.chunks) {
                    p.chunk = 0;
                    if (++p.group == a.row_groups) {
                        p.group = 0;
                        ++p.head;
                    }
                }
                return p;
            };
            auto first_of = [&](const Place& p) { return static_cast<int>((int64_t{p.chunk} * X::kTokens) >> ps_shift); };
            auto count_of = [&](int first) { return a.prefix_pages - first < per ? a.prefix_pages - first : per; };
            auto load_id = [&](const Place& p) {
                const int first = first_of(p);
                return p.c < to && lane < count_of(first) ? __ldg(a.pages + first + lane) : -1;
            };
            auto load_scales = [&](const Place& p, int page, float& k, float& v) {
                k = __int_as_float(0x7FC00000);  // a bad page spoils every row, through its scores
                v = 1.0f;
                if (p.c >= to || static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.c.pages)) return;
                const int64_t at = static_cast<int64_t>(page) * a.c.heads + p.head;
                k = __ldg(a.c.k_scale + at);
                v = __ldg(a.c.v_scale + at);
            };
            // the page of this chunk, of the next and of the one after it; this one's scales
            Place next = step(now), after = step(next);
            int id = load_id(now), id_next = load_id(next);
            float key = 0.0f, val = 0.0f;
            load_scales(now, id, key, val);
            uint32_t t = 0;
            bool ok = true;
            float value = 0.0f;  // the reference of the value scales; 0: none yet
            while (ok && now.c < to) {
                if (now.chunk == 0) value = 0.0f;
                float key_next, val_next;
                load_scales(next, id_next, key_next, val_next);
                const int id_after = load_id(after);
                const int first = first_of(now), n = count_of(first);
                const int offset = ((now.chunk & 3) * X::kTokens) & (ps - 1);  // where pages are larger than a tile (at most four)
                const bool good = lane < n && static_cast<uint32_t>(id) < static_cast<uint32_t>(a.c.pages);
                if (lane < n && !good && a.err) atomicOr(a.err, ARC_KV_ERR_PAGE);
                if (good && !(key >= 0.0f && key <= kMost && val >= 0.0f && val <= kMost)) {
                    if (a.err) atomicOr(a.err, ARC_KV_ERR_SCALE);
                    key = __int_as_float(0x7FC00000);
                    val = 1.0f;
                }
                const bool none = val < kLeast;  // pages of zeros, a tile of their own, go with any reference
                const uint32_t nones = __ballot_sync(0xFFFFFFFFu, none);
                const int64_t at = (good ? id : 0) * a.c.page_stride + now.head * a.c.head_stride + int64_t{offset} * D;
                const bool ends_all = next.c == to, unit_ends = next.chunk == 0 || ends_all;
                for (int start = 0; ok && start < n; ++t) {
                    // the pages from `start` on whose scales go with the reference, or with one another
                    bool apart = lane > start && lane < n;
                    const bool none0 = nones >> start & 1;
                    const float v0 = __shfl_sync(0xFFFFFFFFu, val, start);
                    const bool stays = none0 ? value > 0.0f : v0 <= value && v0 * kSpread >= value;
                    if (stays) {
                        apart = apart && (none != none0 || (!none0 && !(val <= value && val * kSpread >= value)));
                    } else {
                        float hi = lane >= start && lane < n ? val : 0.0f, lo = hi;
#pragma unroll
                        for (int m = 1; m < 8; m <<= 1) {
                            const float h = __shfl_up_sync(0xFFFFFFFFu, hi, m), l = __shfl_up_sync(0xFFFFFFFFu, lo, m);
                            if (lane - m >= start) {
                                hi = fmaxf(hi, h);
                                lo = fminf(lo, l);
                            }
                        }
                        apart = apart && (none != none0 || (!none0 && hi > kSpread * lo));
                        const uint32_t ends = __ballot_sync(0xFFFFFFFFu, apart);
                        value = __shfl_sync(0xFFFFFFFFu, hi, ends ? __ffs(ends) - 2 : n - 1);
                        if (none0) value = 1.0f;
                    }
                    const uint32_t ends = __ballot_sync(0xFFFFFFFFu, apart);
                    const int end = ends ? __ffs(ends) - 1 : n;
                    ok = warp_wait(&bars.info_empty[t % kInfos], (t / kInfos & 1) ^ 1, &bars.failed);
                    if (!ok) break;
                    Info& info = bars.info[t % kInfos];
                    const int page = start + (lane * 16 >> span_shift);  // of the lane's 16 tokens
                    const float k16 = __shfl_sync(0xFFFFFFFFu, key, page & 31), v16 = __shfl_sync(0xFFFFFFFFu, val, page & 31);
                    if (lane < X::kGranules) {
                        const bool there = page < end;
                        const float lift = kLift + (v16 == value || none0 ? 0.0f : __log2f(v16 / value));
                        info.key[lane] = there ? k16 : 0.0f;
                        info.lift[lane] = there ? lift : -kAlone;
                        info.back[lane] = there ? ex2(-lift) : 0.0f;
                    }
                    if (lane == 0) {
                        info.tokens = (end - start) << span_shift;
                        info.flags = (end == n && unit_ends ? (ends_all ? 3 : 1) : 0) | (stays ? 0 : 4) | (none0 ? 8 : 0);
                        info.value = value;
                        info.value_log = __log2f(value);
                    }
                    if (lane >= start && lane < end) info.at[lane - start] = good ? at : -1;
                    __syncwarp();
                    if (lane == 0) bar_arrive(&bars.info_full[t % kInfos]);
                    start = end;
                }
                id = id_next;
                id_next = id_after;
                key = key_next;
                val = val_next;
                now = next;
                next = after;
                after = step(after);
            }
        }
        __syncwarp();
    } else if (warp >= 8) {
        // ---- codes to fp16: 64 values a row of 128 bytes, its 16-byte chunks permuted by the token
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(X::kConvertRegs));
        const int me = tid - 256;
        constexpr int N = X::kEach;
        // Four lanes take 64 values of a token and a warp eight tokens at a time, so that eight lanes' stores, of an even
        // and an odd token, meet in no bank; the blocks of 64 values one after another.
        constexpr int kTurns = X::kTokens / 32;  // of the 128 threads through a block's tokens
        auto token_of = [&](int j) { return (j % kTurns) * 32 + (me >> 2); };
        auto chunk_of = [&](int j) { return (j / kTurns) * 4 + (me & 3); };
        const int ps = a.c.page_size, span = ps < X::kTokens ? ps : X::kTokens, shift = 31 - __clz(span);
        uint4 k[N], v[N];
        auto load = [&](uint32_t t, const void* from, bool values, uint4 (&x)[N]) {
            const Info& info = bars.info[t % kInfos];
            const int tokens = values && (info.flags & 8) ? 0 : info.tokens;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int token = token_of(j), chunk = chunk_of(j);
                const int64_t at = token < tokens ? info.at[token >> shift] : -1;
                x[j] = at < 0 ? make_uint4(0, 0, 0, 0)
                              : load_past_l1(static_cast<const char*>(from) + at + (token & (span - 1)) * D + chunk * 16);
            }
        };
        uint32_t os = 0, phase = 1;
        auto convert = [&](const uint4 (&x)[N]) {
            if (!warp_wait(&bars.op_empty[os], phase, &bars.failed)) return false;
            uint8_t* dst = ops + os * X::kOp;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int token = token_of(j), chunk = chunk_of(j);
                uint32_t h[8];
                e4m3x4_to_half2(x[j].x, h[0], h[1]);
                e4m3x4_to_half2(x[j].y, h[2], h[3]);
                e4m3x4_to_half2(x[j].z, h[4], h[5]);
                e4m3x4_to_half2(x[j].w, h[6], h[7]);
                uint8_t* row = dst + (chunk >> 2) * (X::kTokens * 128) + token * 128;
                const int at = (((chunk & 3) * 2) ^ (token & 7)) * 16;
                *reinterpret_cast<uint4*>(row + at) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(row + (at ^ 16)) = make_uint4(h[4], h[5], h[6], h[7]);
            }
            fence_operands();
            __syncwarp();
            if (lane == 0) bar_arrive(&bars.op_full[os]);
            if (++os == X::kOps) {
                os = 0;
                phase ^= 1;
            }
            return true;
        };
        bool ok = warp_wait(&bars.info_full[0], 0, &bars.failed), last = !ok;
        if (ok) {
            load(0, a.c.k, false, k);
            load(0, a.c.v, true, v);
            last = bars.info[0].flags & 2;
        }
#pragma unroll 1
        for (uint32_t t = 1; ok; ++t) {  // tile t - 1 is converted while tile t is loaded
            const bool more = !last;
            if (more) {
                ok = warp_wait(&bars.info_full[t % kInfos], (t / kInfos) & 1, &bars.failed);
                if (!ok) break;
                last = bars.info[t % kInfos].flags & 2;
            }
            ok = convert(k);
            if (ok && more) load(t, a.c.k, false, k);
            if (ok) ok = convert(v);
            if (!more) break;
            if (ok) load(t, a.c.v, true, v);
        }
    } else {
        // ---- softmax and sums: a thread a row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(X::kSoftmaxRegs));
        const int who = warp >> 2, r = tid & 127;
        const int w = D == 256 ? 0 : who;         // its tile of rows
        const int o0 = D == 256 ? who * 128 : 0;  // its first value of the output
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + X::kS + w * 128, p_at = tmem + lanes + X::kP + w * 128;
        const uint32_t o_at = tmem + lanes + X::kO + w * D + o0;
        constexpr int C = X::kOut;
        bool ok = true;
        uint32_t t = 0;
        for (int64_t c = from; w < tiles && c < to;) {
            const int64_t unit = c / a.chunks;
            const int64_t head = unit / a.row_groups;
            const int64_t row = (unit - head * a.row_groups) * X::kRows + w * 128 + r;
            const int64_t slot = blockIdx.x + unit;
            c = (unit + 1) * a.chunks;
            float back;
            {  // (where a wait has run out too: the groups meet here)
                // queries: fp16, each row scaled by a power of two to [2^14, 2^15)
                uint32_t x[C / 2];
                float top = 0.0f;
                const bool real = row < a.rows;
                const int64_t tok = real ? row / a.group : 0;
                const uint16_t* p = static_cast<const uint16_t*>(a.q) + tok * a.q_token_stride +
                                    (head * a.group + (real ? row - tok * a.group : 0)) * a.q_head_stride + o0;
#pragma unroll
                for (int i = 0; i < C / 8; ++i) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (real) {
                        if (a.vec) {
                            v = *reinterpret_cast<const uint4*>(p + 8 * i);
                        } else {
                            v = make_uint4(p[8 * i] | p[8 * i + 1] << 16, p[8 * i + 2] | p[8 * i + 3] << 16,
                                           p[8 * i + 4] | p[8 * i + 5] << 16, p[8 * i + 6] | p[8 * i + 7] << 16);
                        }
                    }
                    x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
                }
                auto both = [&](uint32_t v) { return a.bf16 ? Half<ARC_BF16>::unpack(v) : Half<ARC_F16>::unpack(v); };
#pragma unroll
                for (int i = 0; i < C / 2; ++i) {
                    const float2 f = both(x[i]);
                    top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
                if constexpr (D == 256) {
                    // (the halves of a row meet where the last unit's queries were)
                    float* const tops = reinterpret_cast<float*>(q_tiles);
                    tops[who * 128 + r] = top;
                    asm volatile("bar.sync 1, 256;" ::: "memory");
                    top = fmaxf(top, tops[(who ^ 1) * 128 + r]);
                    asm volatile("bar.sync 1, 256;" ::: "memory");
                }
                // 2^(14 - exponent), kept inside fp32's normal range
                const int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
                const int up = top == 0.0f ? 0 : (14 - ex > 126 ? 126 : (14 - ex < -113 ? -113 : 14 - ex));
                const float f = a.scale < 0.0f ? -exp2i(up) : exp2i(up);  // the scale's sign goes with the queries
                back = exp2i(-up) * fabsf(a.scale);
#pragma unroll
                for (int i = 0; i < C / 8; ++i) {
                    uint32_t h[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 v = both(x[4 * i + k]);
                        h[k] = Half<ARC_F16>::pack(v.x * f, v.y * f);
                    }
                    const int chunk = o0 / 8 + i;  // 8 values
                    uint8_t* at = q_tiles + w * X::kQ + (chunk >> 3) * (128 * 128) + r * 128 + (((chunk & 7) ^ (r & 7)) * 16);
                    *reinterpret_cast<uint4*>(at) = make_uint4(h[0], h[1], h[2], h[3]);
                }
                fence_operands();
                __syncwarp();
                if (lane == 0) bar_arrive(&bars.q_full[w]);
            }
            // the row's reference, its largest score, the largest of score and value scale, the sum relative to m
            float ref = 0.0f, m = kNothing, peak = kNothing, l = 0.0f, value = 1.0f, value_log = 0.0f;
            bool fresh = true;
            ok = ok && warp_wait(&bars.info_full[t % kInfos], (t / kInfos) & 1, &bars.failed);
            while (ok) {
                const Info& info = bars.info[t % kInfos];
                const int granules = info.tokens >> 4, flags = info.flags;
#pragma unroll 1
                for (int half = 0; half < X::kSteps; ++half) {
                    const uint32_t n = t * X::kSteps + half;
                    const uint32_t s_now = s_at + (n & 1) * 64, p_now = p_at + (n & 1) * X::kPStep;
                    const float4 key = *reinterpret_cast<const float4*>(&info.key[4 * half]);
                    const float4 lift = *reinterpret_cast<const float4*>(&info.lift[4 * half]);
                    const float keys[4] = {key.x * back, key.y * back, key.z * back, key.w * back};
                    const float4 unlift = *reinterpret_cast<const float4*>(&info.back[4 * half]);
                    const float lifts[4] = {lift.x, lift.y, lift.z, lift.w};
                    const float unlifts[4] = {unlift.x, unlift.y, unlift.z, unlift.w};
                    const int left = granules - 4 * half;  // groups of 16 tokens that there are
                    ok = warp_wait(&bars.s_full[w][n & 1], (n >> 1) & 1, &bars.failed);
                    if (!ok) break;
                    fence_after();
                    uint32_t s[2][32];
                    tmem_load32(s_now, s[0]);
                    tmem_load32(s_now + 32, s[1]);
                    tmem_wait_load32(s[0]);
                    tmem_wait_load32(s[1]);
                    float hi[4] = {kNothing, kNothing, kNothing, kNothing}, top = kNothing;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            hi[g] = max3(hi[g], __uint_as_float(s[g >> 1][16 * (g & 1) + 2 * i]),
                                         __uint_as_float(s[g >> 1][16 * (g & 1) + 2 * i + 1]));
#pragma unroll
                    for (int g = 0; g < 4; ++g) top = fmaxf(top, g < left ? hi[g] * keys[g] : kNothing);
                    const bool move = left > 0 && (((flags & 4) && half == 0) || top > ref + kAbove || top < ref - kBelow);
                    if (__any_sync(0xFFFFFFFFu, move)) {
                        const float old = ref, old_value = value_log;
                        value = info.value;
                        value_log = info.value_log;
                        if (fresh) {
                            ref = top + kRoom;
                        } else {
                            if (move) ref = fmaxf(top + kRoom, peak - kSpan - value_log);
                            ok = warp_wait(&bars.o_full[w][(n - 1) & 1], ((n - 1) >> 1) & 1, &bars.failed);
                            if (!ok) break;
                            fence_after();
                            const float f = ex2((old - ref) + (old_value - value_log));
                            const uint64_t f2 = pack2(f, f);
#pragma unroll 1
                            for (int b = 0; b < C / 16; ++b) {
                                uint32_t y[16];
                                tmem_load16(o_at + 16 * b, y);
                                tmem_wait_load16(y);
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const uint64_t z = mul2(pack2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1])), f2);
                                    y[2 * i] = static_cast<uint32_t>(z);
                                    y[2 * i + 1] = static_cast<uint32_t>(z >> 32);
                                }
                                tmem_store16(o_at + 16 * b, y);
                            }
                        }
                        if (fabsf(ref) > kFar) l = __int_as_float(0x7FC00000);
                    }
                    fresh = false;
                    if (left > 0) peak = fmaxf(peak, top + value_log);
                    const float now = fmaxf(m, top);
                    float sum = 0.0f;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        uint32_t p[16];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int g = 2 * b + h;
                            const float add = lifts[g] - ref;
                            const uint64_t f2 = pack2(keys[g], keys[g]), add2 = pack2(add, add);
                            float part[2] = {0.0f, 0.0f};
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const uint64_t z = fma2(pack2(__uint_as_float(s[b][16 * h + 2 * i]),
                                                              __uint_as_float(s[b][16 * h + 2 * i + 1])), f2, add2);
                                const float e0 = ex2(half_of(z, 0)), e1 = ex2(half_of(z, 1));
                                p[8 * h + i] = Half<ARC_F16>::pack(e0, e1);
                                // (the weights as they enter the product: their roundings cancel in the quotient)
                                const float2 w2 = Half<ARC_F16>::unpack(p[8 * h + i]);
                                part[0] += w2.x;
                                part[1] += w2.y;
                            }
                            sum = fmaf(part[0] + part[1], unlifts[g], sum);
                        }
                        if (D != 256 || b == who) tmem_store16(p_now + 16 * b, p);
                    }
                    tmem_wait_store();
                    fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        bar_arrive(&bars.p_full[w][n & 1]);
                        if (half + 1 == X::kSteps) bar_arrive(&bars.info_empty[t % kInfos]);
                    }
                    l = fmaf(l, ex2(m - now), sum * ex2(ref - now));
                    m = now;
                }
                if (!ok) break;
                ++t;
                if (flags & 1) break;
                ok = warp_wait(&bars.info_full[t % kInfos], (t / kInfos) & 1, &bars.failed);
            }
            // ---- the unit's partial
            const uint32_t last = t * X::kSteps - 1;
            if (ok) ok = warp_wait(&bars.o_full[w][last & 1], (last >> 1) & 1, &bars.failed);
            if (ok) {
                fence_after();
                const float f = ex2(ref - m) * (value * (1.0f / 4096.0f)) / l;  // (the weights have 2^kLift)
                float4* out = reinterpret_cast<float4*>(a.slots) + ((slot * X::kTiles + w) * (D / 4) + o0 / 4) * 128 + r;
#pragma unroll
                for (int b = 0; b < C / 32; ++b) {
                    uint32_t y[32];
                    tmem_load32(o_at + 32 * b, y);
                    tmem_wait_load32(y);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        out[(8 * b + i) * 128] = make_float4(__uint_as_float(y[4 * i]) * f, __uint_as_float(y[4 * i + 1]) * f,
                                                             __uint_as_float(y[4 * i + 2]) * f, __uint_as_float(y[4 * i + 3]) * f);
                }
                fence_before();
            }
            if (D != 256 || who == 0)
                a.slot_logs[slot * X::kRows + w * 128 + r] = ok ? m + __log2f(l) : __int_as_float(0x7FC00000);
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 12)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
}

// ------------------------------------------------------------------ the join
struct JoinArgs {
    const float* rows;
    const float* logs;
    const float* slots;
    const float* slot_logs;
    void* out;
    int64_t out_token_stride, out_head_stride;
    int64_t head_rows, row_groups, total;
    int32_t chunks, pieces, group, q_heads, bf16, vec;
};

// 32 rows of a cached head, a lane each, and 32 of the output's values, four a warp.
template <int D>
__global__ void __launch_bounds__(256) shared_join_kernel(const __grid_constant__ JoinArgs a) {
    using X = Prefix<D>;
    __shared__ float weight[kMaxBlocks + 1][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t head = blockIdx.y, row = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    const bool real = row < a.head_rows;
    // 32 rows lie in one tile
    const int64_t group = static_cast<int64_t>(blockIdx.x) * 32 / X::kRows, unit = head * a.row_groups + group;
    const int in = static_cast<int>(row - group * X::kRows);
    const int64_t c0 = ((unit * a.chunks + 1) * a.pieces - 1) / a.total;
    const int n = static_cast<int>((((unit + 1) * a.chunks) * a.pieces - 1) / a.total - c0) + 1;
    const int64_t slot0 = c0 + unit;
    const int64_t tok = real ? row / a.group : 0, own = tok * a.q_heads + head * a.group + (real ? row - tok * a.group : 0);
    for (int i = warp; i <= n; i += 8)
        weight[i][lane] = i < n ? __ldg(a.slot_logs + (slot0 + i) * X::kRows + in) : __ldg(a.logs + own);
    __syncthreads();
    // (a row that nothing is joined to: what the prefix gave it, NaN included, counts nothing)
    const bool alone = weight[n][lane] == kAlone;
    float top = kNothing, total = 0.0f;
    for (int i = 0; i <= n; ++i) top = fmaxf(top, weight[i][lane]);
    for (int i = 0; i <= n; ++i) total += ex2(weight[i][lane] - top);
    __syncthreads();
    for (int i = warp; i <= n; i += 8)
        weight[i][lane] = alone ? (i == n ? 1.0f : 0.0f) : ex2(weight[i][lane] - top) / total;
    __syncthreads();
    const int quad = blockIdx.z * 8 + warp;  // the warp's four values
    const float f0 = weight[n][lane];
    float4 x = reinterpret_cast<const float4*>(a.rows)[own * (D / 4) + quad];
    x = make_float4(x.x * f0, x.y * f0, x.z * f0, x.w * f0);
    const float4* part = reinterpret_cast<const float4*>(a.slots) + ((slot0 * X::kTiles + in / 128) * (D / 4) + quad) * 128 + in % 128;
#pragma unroll 8
    for (int s = 0; s < n; ++s) {
        const float f = weight[s][lane];
        const float4 v = part[static_cast<int64_t>(s) * X::kTiles * (D / 4) * 128];
        if (f != 0.0f)  // (rows that nothing is joined to)
            x = make_float4(fmaf(v.x, f, x.x), fmaf(v.y, f, x.y), fmaf(v.z, f, x.z), fmaf(v.w, f, x.w));
    }
    if (!real) return;
    uint16_t* out = static_cast<uint16_t*>(a.out) + tok * a.out_token_stride +
                    (head * a.group + row - tok * a.group) * a.out_head_stride + quad * 4;
    const uint32_t lo = a.bf16 ? Half<ARC_BF16>::pack(x.x, x.y) : Half<ARC_F16>::pack(x.x, x.y);
    const uint32_t hi = a.bf16 ? Half<ARC_BF16>::pack(x.z, x.w) : Half<ARC_F16>::pack(x.z, x.w);
    if (a.vec) {
        *reinterpret_cast<uint2*>(out) = make_uint2(lo, hi);
    } else {
        out[0] = static_cast<uint16_t>(lo);
        out[1] = static_cast<uint16_t>(lo >> 16);
        out[2] = static_cast<uint16_t>(hi);
        out[3] = static_cast<uint16_t>(hi >> 16);
    }
}

template <int D>
int launch_prefix(const PrefixArgs& p, const JoinArgs& j, const arc_kv_cache& cache, const arc_kv_step& step,
                  const arc_kv_query& query, uint32_t* err_word, void* workspace, const SharedLayout& at,
                  int64_t prefix_tokens, int dev, int sms, cudaStream_t st) {
    using X = Prefix<D>;
    static std::atomic<uint64_t> done{0};
    static_assert(X::kSmem + sizeof(PrefixBars) <= arc::kSmemPerBlock, "shared memory");
    if (arc::prepare(prefix_kernel<D>, dev, done, 100) != cudaSuccess) return ARC_E_CUDA;
    prefix_kernel<D><<<static_cast<unsigned>(p.pieces), X::kThreads, X::kSmem, st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return ARC_E_CUDA;
    const int rc = launch_behind(cache, step, query, err_word, workspace, at, prefix_tokens, dev, sms, st);
    if (rc != ARC_OK) return rc;
    const dim3 grid(static_cast<unsigned>((p.rows + 31) / 32), static_cast<unsigned>(cache.heads), D / 32);
    shared_join_kernel<D><<<grid, 256, 0, st>>>(j);
    return cudaGetLastError() == cudaSuccess ? ARC_OK : ARC_E_CUDA;
}

int64_t tokens_of_tile(int dim) { return dim == 256 ? 64 : 128; }

}  // namespace

SharedLayout shared_layout(const arc_kv_cache& cache, int64_t T, int64_t q_heads) {
    SharedLayout s;
    const int64_t dim = cache.head_dim, head_rows = T * (q_heads / cache.heads);
    s.group_rows = dim == 256 ? 128 : 256;
    s.row_groups = (head_rows + s.group_rows - 1) / s.group_rows;
    s.units = s.row_groups * cache.heads;
    const int64_t slots = s.units + kMaxBlocks;
    auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    s.rows = up(attend_workspace(cache));
    s.logs = s.rows + up(static_cast<size_t>(T) * q_heads * dim * 4);
    s.slots = s.logs + up(static_cast<size_t>(T) * q_heads * 4);
    s.slot_logs = s.slots + up(static_cast<size_t>(slots) * s.group_rows * dim * 4);
    s.bytes = s.slot_logs + up(static_cast<size_t>(slots) * s.group_rows * 4);
    return s;
}

namespace {

bool shared_rows_fit(const arc_kv_cache& cache, int64_t T, int64_t q_heads) {
    return T > 0 && T <= (int64_t{1} << 24) && q_heads > 0 && q_heads <= (1 << 16) && q_heads % cache.heads == 0 &&
           T * q_heads <= ARC_KV_SHARED_MAX_ROWS;
}

}  // namespace
}  // namespace arcs

extern "C" {

size_t arc_kv_attend_shared_workspace_bytes(const arc_kv_cache* cache, int64_t T, int32_t q_heads) {
    if (arcs::check_cache(cache) != ARC_OK || !arcs::shared_rows_fit(*cache, T, q_heads)) return 0;
    return arcs::shared_layout(*cache, T, q_heads).bytes;
}

int arc_kv_attend_shared(const arc_kv_cache* cache, const arc_kv_step* step, const arc_kv_query* query,
                         const int32_t* prefix, int32_t prefix_pages, uint32_t* err_word, void* workspace,
                         size_t workspace_bytes, void* stream) {
    using namespace arcs;
    int rc = check_attend(cache, step, query, err_word);
    if (rc != ARC_OK) return rc;
    if (prefix == nullptr) return ARC_E_NULL;
    if (prefix_pages <= 0 || prefix_pages > step->max_pages) return ARC_E_SHAPE;
    if (!shared_rows_fit(*cache, step->T, query->q_heads)) return ARC_E_SHAPE;
    if (query->window != 0) return ARC_E_OPTION;
    if (!aligned(prefix, 4)) return ARC_E_ALIGN;
    const SharedLayout at = shared_layout(*cache, step->T, query->q_heads);
    if (workspace == nullptr || workspace_bytes < at.bytes) return ARC_E_WORKSPACE;
    if (!aligned(workspace, 16)) return ARC_E_ALIGN;
    int dev = 0, sms = 0;
    rc = device_of(dev, sms);
    if (rc != ARC_OK) return rc;
    char* const ws = static_cast<char*>(workspace);
    const int64_t tokens = int64_t{prefix_pages} * cache->page_size, tile = tokens_of_tile(cache->head_dim);
    PrefixArgs p;
    p.c = *cache;
    p.q = query->q;
    p.q_token_stride = query->q_token_stride;
    p.q_head_stride = query->q_head_stride;
    p.pages = prefix;
    p.err = err_word;
    p.slots = reinterpret_cast<float*>(ws + at.slots);
    p.slot_logs = reinterpret_cast<float*>(ws + at.slot_logs);
    p.group = query->q_heads / cache->heads;
    p.rows = step->T * p.group;
    p.row_groups = at.row_groups;
    p.chunks = static_cast<int32_t>((tokens + tile - 1) / tile);
    p.total = at.units * p.chunks;
    p.prefix_pages = prefix_pages;
    const int most = sms < kMaxBlocks ? sms : kMaxBlocks;
    p.pieces = static_cast<int32_t>(p.total < most ? p.total : most);
    p.bf16 = query->dtype == ARC_BF16;
    p.vec = vectors(query->q, query->q_token_stride, query->q_head_stride);
    p.scale = query->scale * 1.4426950408889634f;
    JoinArgs j;
    j.rows = reinterpret_cast<const float*>(ws + at.rows);
    j.logs = reinterpret_cast<const float*>(ws + at.logs);
    j.slots = p.slots;
    j.slot_logs = p.slot_logs;
    j.out = query->out;
    j.out_token_stride = query->out_token_stride;
    j.out_head_stride = query->out_head_stride;
    j.head_rows = p.rows;
    j.row_groups = p.row_groups;
    j.total = p.total;
    j.chunks = p.chunks;
    j.pieces = p.pieces;
    j.group = p.group;
    j.q_heads = query->q_heads;
    j.bf16 = p.bf16;
    j.vec = vectors(query->out, query->out_token_stride, query->out_head_stride);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cache->head_dim == 64)
        return launch_prefix<64>(p, j, *cache, *step, *query, err_word, workspace, at, tokens, dev, sms, st);
    if (cache->head_dim == 128)
        return launch_prefix<128>(p, j, *cache, *step, *query, err_word, workspace, at, tokens, dev, sms, st);
    return launch_prefix<256>(p, j, *cache, *step, *query, err_word, workspace, at, tokens, dev, sms, st);
}

}  // extern "C"
