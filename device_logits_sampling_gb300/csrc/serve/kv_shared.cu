// arc_kv_attend_shared: attention of a step's new tokens behind a prefix that all sequences share.
//
// Three kernels.  The prefix: all rows of a cached head (new tokens times its query heads) against the prefix's pages,
// which are read once for them.  The sequences' own tokens: kv_attend.cuh's kernel, with its results in fp32.  And the
// join of a row's parts, each an output with the base-2 logarithm of its sum of weights:
//     out = sum_i 2^(log_i - max) out_i / sum_i 2^(log_i - max).
//
// The prefix.  A unit is a cached head and up to 256 rows (128 for heads of 256).  A chunk is 128 tokens (64 for heads
// of 256) of the prefix; all units' chunks lie on a line that is cut into one piece a block.  A block runs through its
// piece tile by tile, and leaves a partial for each unit that it has met.
//
// A tile is a chunk, or the part of one whose pages' value scales lie within a factor of 64: the weights enter the
// second product as fp16, 2^14 times themselves relative to the tile's largest and times their page's scale over the
// tile's largest scale, so no page's own scale pushes its weights out of fp16.
//
// Products.  Codes come in by bulk copies, page by page, and become fp16 in shared memory, exactly.  S = Q K^T and
// O = P V run on the 5th-generation tensor cores, M = 128 rows: Q and K from shared memory, P from tensor memory, where
// the softmax has put it over S, V as it lies, tokens as rows, read across.  A tile's O is read back and added up in
// registers with a factor a row, so weights are relative to their own tile's largest score, whatever came before.
//
// Roles of a block: two groups of four warps take softmax and sums, a thread a row (two groups of 128 rows, or for heads
// of 256 one, half of the output each), one group makes fp16 of codes, a warp issues the products and a warp the copies.
// While one group of rows is at its softmax the products of the other run.
//
// Every wait has a limit; a block whose wait runs out leaves NaN.
#include "kv_shared.cuh"

#include <atomic>
#include <climits>
#include <cstring>

#include "kv_attend.cuh"
#include "launch_util.cuh"
#include "tensor_core.cuh"

namespace arcs {
namespace {

constexpr float kSpread = 64.0f;  // of the value scales of a tile's pages
constexpr int kInfos = 8;         // ring of tiles' descriptions: the copies are at most seven tiles ahead
constexpr int kLiftLog = 14;

template <int D>
struct Prefix {
    static constexpr int kTokens = D == 256 ? 64 : 128;  // of a tile
    static constexpr int kTiles = D == 256 ? 1 : 2;      // tiles of 128 rows
    static constexpr int kRows = 128 * kTiles;
    static constexpr int kOut = D == 256 ? 128 : D;      // values of the output that a thread adds up
    static constexpr int kGranules = kTokens / 16;
    static constexpr int kThreads = 512;
    static constexpr int kQ = 128 * D * 2;
    static constexpr int kOp = kTokens * D * 2, kOps = D == 64 ? 6 : 3;   // ring of fp16 tiles, K and V in turn
    static constexpr int kRaw = kTokens * D, kRaws = D == 64 ? 8 : 4;     // ring of codes, likewise
    static constexpr int kSmem = kTiles * kQ + kOps * kOp + kRaws * kRaw + 1024;
    static constexpr int kS = 0, kP = D == 256 ? 128 : 0, kO = 256;       // columns of tensor memory
    // registers of a thread once the roles part, of 128 at the launch of 512 threads (4 * 128 = 512)
    static constexpr int kSoftmaxRegs = 200, kConvertRegs = 72, kIssueRegs = 40;
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

struct Info {  // a tile
    int32_t tokens;
    int32_t flags;    // 1: the last of its unit's, 2: the last of all
    float value;      // the tile's largest value scale, times 2^-14
    float key[8];     // of each 16 tokens: key scale,
    float lift[8];    // 14 + the logarithm of the value scale over the largest
};

struct PrefixBars {
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
    uint64_t raw_full[8], raw_empty[8];
    uint64_t op_full[6], op_empty[6];
    uint64_t info_full[kInfos];
    uint64_t drained;
    uint32_t tmem, failed;
    Info info[kInfos];
    float top[2][128];  // heads of 256: the largest of each half of a query row
};

// One thread issues all products: for each tile S of every tile of rows, a tile ahead, and O behind the softmax.
template <int D>
__device__ __forceinline__ bool issue_prefix(PrefixBars& bars, uint32_t q_at, uint32_t ops, uint32_t tmem, int tiles) {
    using X = Prefix<D>;
    constexpr uint32_t s_desc = (1u << 4) | (static_cast<uint32_t>(X::kTokens / 8) << 17) | (8u << 24);
    constexpr uint32_t o_desc = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(D / 8) << 17) | (8u << 24);
    constexpr uint32_t kBlock = X::kTokens * 128;  // 64 values of all tokens
    uint32_t q_phase[2] = {0, 0};
    int flags = 0;
    bool fresh = true;  // the next tile begins a unit
    uint32_t op = 0, op_phase = 0;
    auto next_op = [&]() {
        if (++op == X::kOps) {
            op = 0;
            op_phase ^= 1;
        }
    };
    auto scores = [&](int w, uint32_t stage) {
        const uint64_t a = operand_at(q_at + w * X::kQ), b = operand_at(ops + stage * X::kOp);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
            mma_f16_shared(tmem + X::kS + w * 128, a + (k >> 2) * (128 * 128 / 16) + (k & 3) * 2,
                           b + (k >> 2) * (kBlock / 16) + (k & 3) * 2, s_desc, k != 0);
        commit_to(&bars.s_full[w]);
    };
    for (uint32_t t = 0;; ++t) {  // tile t's scores, then tile t - 1's output; past the last tile its output alone
        const bool more = t == 0 || !(flags & 2);
        uint32_t k_stage = 0;
        const uint32_t v_stage = op, v_phase = op_phase;  // of tile t - 1
        if (t) next_op();
        if (more) {
            k_stage = op;
            if (!bar_wait(&bars.info_full[t % kInfos], (t / kInfos) & 1, &bars.failed)) return false;
            if (!bar_wait(&bars.op_full[k_stage], op_phase, &bars.failed)) return false;
            next_op();
        }
        if (t && !bar_wait(&bars.op_full[v_stage], v_phase, &bars.failed)) return false;
        for (int w = 0; w < tiles; ++w) {
            if (t) {
                if (!bar_wait(&bars.p_full[w], (t - 1) & 1, &bars.failed)) return false;
                fence_after();
                const uint64_t b = operand_across(ops + v_stage * X::kOp, kBlock);
#pragma unroll
                for (int k = 0; k < X::kTokens / 16; ++k)
                    mma_f16(tmem + X::kO + w * D, tmem + X::kP + w * 128 + k * 8, b + k * (2048 / 16), o_desc, k != 0);
                commit_to(&bars.o_full[w]);
            }
            if (more) {
                if (fresh) {
                    if (!bar_wait(&bars.q_full[w], q_phase[w], &bars.failed)) return false;
                    q_phase[w] ^= 1;
                }
                fence_after();
                scores(w, k_stage);
            }
        }
        if (t) commit_to(&bars.op_empty[v_stage]);
        if (!more) return true;
        commit_to(&bars.op_empty[k_stage]);
        flags = bars.info[t % kInfos].flags;
        fresh = flags & 1;
    }
}

template <int D>
__global__ void __launch_bounds__(512, 1) prefix_kernel(const __grid_constant__ PrefixArgs a) {
    using X = Prefix<D>;
    extern __shared__ uint8_t raw_smem[];
    __shared__ PrefixBars bars;
    uint8_t* const dyn = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t{1023});
    uint8_t* const q_tiles = dyn;
    uint8_t* const ops = dyn + X::kTiles * X::kQ;
    uint8_t* const raws = ops + X::kOps * X::kOp;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t from = cut_of(a.total, blockIdx.x, a.pieces), to = cut_of(a.total, blockIdx.x + 1, a.pieces);
    const int tiles = X::kTiles == 2 && a.rows > 128 ? 2 : 1;  // of rows

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            bar_init(&bars.q_full[i], D == 256 ? 8 : 4);
            bar_init(&bars.s_full[i], 1);
            bar_init(&bars.p_full[i], D == 256 ? 8 : 4);
            bar_init(&bars.o_full[i], 1);
        }
        for (int i = 0; i < 8; ++i) {
            bar_init(&bars.raw_full[i], 1);
            bar_init(&bars.raw_empty[i], 4);
        }
        for (int i = 0; i < 6; ++i) {
            bar_init(&bars.op_full[i], 4);
            bar_init(&bars.op_empty[i], 1);
        }
        for (int i = 0; i < kInfos; ++i) bar_init(&bars.info_full[i], 1);
        bar_init(&bars.drained, 1);
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
        if (warp == 12 && elect_one()) {
            // ---- products
            if (!issue_prefix<D>(bars, shared_of(q_tiles), shared_of(ops), tmem, tiles)) {
                commit_to(&bars.drained);
                uint32_t quiet = 0;
                bar_wait(&bars.drained, 0, &quiet);
            }
        }
        if (warp == 13) {
            // ---- copies: a lane for each page of a chunk, whose number and scales are loaded ahead
            const int ps = a.c.page_size, span = ps < X::kTokens ? ps : X::kTokens, per = X::kTokens / span;
            int id[2] = {-1, -1};  // of this chunk and the next
            float key = 0.0f, val = 0.0f;
            auto pages_of = [&](int64_t c, int64_t& head, int& first, int& offset, int& n) {
                const int64_t unit = c / a.chunks;
                const int64_t token = (c - unit * a.chunks) * X::kTokens;
                head = unit / a.row_groups;
                first = static_cast<int>(token / ps);
                offset = static_cast<int>(token - int64_t{first} * ps);
                n = a.prefix_pages - first < per ? a.prefix_pages - first : per;
            };
            auto load_id = [&](int64_t c) {
                int64_t head;
                int first, offset, n;
                if (c >= to) return -1;
                pages_of(c, head, first, offset, n);
                return lane < n ? __ldg(a.pages + first + lane) : -1;
            };
            auto load_scales = [&](int64_t c, int page, float& k, float& v) {
                k = __int_as_float(0x7FC00000);  // a bad page spoils every row, through its scores
                v = 1.0f;
                if (c >= to || static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.c.pages)) return;
                const int64_t at = static_cast<int64_t>(page) * a.c.heads + c / a.chunks / a.row_groups;
                k = __ldg(a.c.k_scale + at);
                v = __ldg(a.c.v_scale + at);
            };
            id[0] = load_id(from);
            id[1] = load_id(from + 1);
            load_scales(from, id[0], key, val);
            uint32_t t = 0;
            bool ok = true;
            for (int64_t c = from; ok && c < to; ++c) {
                float key_next, val_next;
                load_scales(c + 1, id[1], key_next, val_next);
                const int id_next = load_id(c + 2);
                int64_t head;
                int first, offset, n;
                pages_of(c, head, first, offset, n);
                const bool good = lane < n && static_cast<uint32_t>(id[0]) < static_cast<uint32_t>(a.c.pages);
                if (lane < n && !good && a.err) atomicOr(a.err, ARC_KV_ERR_PAGE);
                const int64_t at = (good ? id[0] : 0) * a.c.page_stride + head * a.c.head_stride + int64_t{offset} * D;
                const bool unit_ends = (c + 1) % a.chunks == 0 || c + 1 == to;
                for (int start = 0; ok && start < n; ++t) {
                    // the pages from `start` on whose scales go together
                    float hi = lane >= start && lane < n ? val : 0.0f, lo = hi;
#pragma unroll
                    for (int m = 1; m < 8; m <<= 1) {
                        const float h = __shfl_up_sync(0xFFFFFFFFu, hi, m), l = __shfl_up_sync(0xFFFFFFFFu, lo, m);
                        if (lane - m >= start) {
                            hi = fmaxf(hi, h);
                            lo = fminf(lo, l);
                        }
                    }
                    const uint32_t apart = __ballot_sync(0xFFFFFFFFu, lane > start && lane < n && hi > kSpread * lo);
                    const int end = apart ? __ffs(apart) - 1 : n;
                    const float top = __shfl_sync(0xFFFFFFFFu, hi, end - 1);
                    const uint32_t ks = 2 * t % X::kRaws, vs = (2 * t + 1) % X::kRaws, phase = (2 * t / X::kRaws & 1) ^ 1;
                    ok = warp_wait(&bars.raw_empty[ks], phase, &bars.failed) && warp_wait(&bars.raw_empty[vs], phase, &bars.failed);
                    if (!ok) break;
                    Info& info = bars.info[t % kInfos];
                    const int page = start + lane * 16 / span;  // of the lane's 16 tokens
                    const float k16 = __shfl_sync(0xFFFFFFFFu, key, page & 31), v16 = __shfl_sync(0xFFFFFFFFu, val, page & 31);
                    if (lane < X::kGranules) {
                        const float lift = kLiftLog + (v16 == top ? 0.0f : __log2f(v16 / top));
                        info.key[lane] = k16;
                        info.lift[lane] = lift;
                    }
                    if (lane == 0) {
                        info.tokens = (end - start) * span;
                        info.flags = end == n && unit_ends ? (c + 1 == to ? 3 : 1) : 0;
                        info.value = top * (1.0f / (1 << kLiftLog));
                    }
                    const bool mine = good && lane >= start && lane < end;
                    const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, mine)) * span * D;
                    __syncwarp();
                    if (lane == 0) {
                        bar_arrive(&bars.info_full[t % kInfos]);
                        bar_expect(&bars.raw_full[ks], bytes);
                        bar_expect(&bars.raw_full[vs], bytes);
                    }
                    __syncwarp();
                    if (mine) {
                        const uint32_t dst = shared_of(raws) + (lane - start) * span * D;
                        bulk_copy(dst + ks * X::kRaw, static_cast<const char*>(a.c.k) + at, span * D, &bars.raw_full[ks]);
                        bulk_copy(dst + vs * X::kRaw, static_cast<const char*>(a.c.v) + at, span * D, &bars.raw_full[vs]);
                    }
                    start = end;
                }
                id[0] = id[1];
                id[1] = id_next;
                key = key_next;
                val = val_next;
            }
            // a failed block still waits for its copies in flight before its memory goes away
            if (!ok)
                for (uint32_t i = 0; i < X::kRaws && i < 2 * t; ++i) {
                    const uint32_t u = 2 * t - 1 - i;
                    uint32_t quiet = 0;
                    bar_wait(&bars.raw_full[u % X::kRaws], (u / X::kRaws) & 1, &quiet);
                }
        }
        __syncwarp();
    } else if (warp >= 8) {
        // ---- codes to fp16: 64 values a row of 128 bytes, its 16-byte chunks permuted by the token
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(X::kConvertRegs));
        const int me = tid - 256;
        constexpr int kChunks = D / 16;  // 16 codes each, of a token
        bool ok = true, last = false;
        for (uint32_t t = 0; ok && !last; ++t) {
            ok = warp_wait(&bars.info_full[t % kInfos], (t / kInfos) & 1, &bars.failed);
            if (!ok) break;
            const int tokens = bars.info[t % kInfos].tokens;
            last = bars.info[t % kInfos].flags & 2;
#pragma unroll 1
            for (uint32_t u = 2 * t; u < 2 * t + 2; ++u) {
                const uint32_t rs = u % X::kRaws, os = u % X::kOps;
                ok = warp_wait(&bars.raw_full[rs], (u / X::kRaws) & 1, &bars.failed);
                if (ok) ok = warp_wait(&bars.op_empty[os], ((u / X::kOps) & 1) ^ 1, &bars.failed);
                if (!ok) break;
                const uint8_t* src = raws + rs * X::kRaw;
                uint8_t* dst = ops + os * X::kOp;
#pragma unroll 4
                for (int j = 0; j < X::kTokens * kChunks / 128; ++j) {
                    const int i = j * 128 + me, token = i / kChunks, chunk = i % kChunks;
                    uint4 x = *reinterpret_cast<const uint4*>(src + i * 16);
                    if (token >= tokens) x = make_uint4(0, 0, 0, 0);
                    uint32_t h[8];
                    e4m3x4_to_half2(x.x, h[0], h[1]);
                    e4m3x4_to_half2(x.y, h[2], h[3]);
                    e4m3x4_to_half2(x.z, h[4], h[5]);
                    e4m3x4_to_half2(x.w, h[6], h[7]);
                    uint8_t* row = dst + (chunk >> 2) * (X::kTokens * 128) + token * 128;
                    const int c0 = (chunk & 3) * 2, odd = (chunk >> 2) & 1;  // lanes of two blocks meet in no bank
                    const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
                    *reinterpret_cast<uint4*>(row + (((c0 + odd) ^ (token & 7)) * 16)) = odd ? hi : lo;
                    *reinterpret_cast<uint4*>(row + (((c0 + (odd ^ 1)) ^ (token & 7)) * 16)) = odd ? lo : hi;
                }
                fence_operands();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(&bars.op_full[os]);
                    bar_arrive(&bars.raw_empty[rs]);
                }
            }
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
                    bars.top[who][r] = top;
                    asm volatile("bar.sync 1, 256;" ::: "memory");
                    top = fmaxf(top, bars.top[who ^ 1][r]);
                    asm volatile("bar.sync 1, 256;" ::: "memory");
                }
                // 2^(14 - exponent), kept inside fp32's normal range
                const int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
                const int up = top == 0.0f ? 0 : (14 - ex > 126 ? 126 : (14 - ex < -113 ? -113 : 14 - ex));
                const float f = exp2i(up);
                back = exp2i(-up) * a.scale;
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
            uint64_t o[C / 2];
#pragma unroll
            for (int i = 0; i < C / 2; ++i) o[i] = 0;
            float m = kNothing, l = 0.0f;
            for (bool unit_ends = false; ok && !unit_ends; ++t) {
                ok = warp_wait(&bars.info_full[t % kInfos], (t / kInfos) & 1, &bars.failed);
                if (!ok) break;
                const Info& info = bars.info[t % kInfos];
                const int granules = info.tokens >> 4;
                const float value = info.value;
                unit_ends = info.flags & 1;
                ok = warp_wait(&bars.s_full[w], t & 1, &bars.failed);
                if (!ok) break;
                fence_after();
                float top = kNothing;
#pragma unroll
                for (int b = 0; b < X::kTokens / 32; ++b) {
                    if (2 * b >= granules) break;
                    uint32_t s[32];
                    tmem_load32(s_at + 32 * b, s);
                    tmem_wait_load32(s);
                    // (the key scale is positive, the row's factor has the sign of the call's)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (2 * b + h >= granules) break;
                        const float f = info.key[2 * b + h] * back;
                        float hi = __uint_as_float(s[16 * h]) * f;
#pragma unroll
                        for (int i = 1; i < 16; ++i) hi = fmaxf(hi, __uint_as_float(s[16 * h + i]) * f);
                        top = fmaxf(top, hi);
                    }
                }
                float sum = 0.0f;
#pragma unroll
                for (int b = 0; b < X::kTokens / 32; ++b) {
                    uint32_t p[16];
                    if (2 * b < granules) {
                        uint32_t s[32];
                        tmem_load32(s_at + 32 * b, s);
                        tmem_wait_load32(s);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (2 * b + h < granules) {
                                const float f = info.key[2 * b + h] * back, add = info.lift[2 * b + h] - top;
                                float part = 0.0f;
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const float e0 = ex2(fmaf(__uint_as_float(s[16 * h + 2 * i]), f, add));
                                    const float e1 = ex2(fmaf(__uint_as_float(s[16 * h + 2 * i + 1]), f, add));
                                    part += e0 + e1;
                                    p[8 * h + i] = Half<ARC_F16>::pack(e0, e1);
                                }
                                sum = fmaf(part, ex2(-info.lift[2 * b + h]), sum);
                            } else {
#pragma unroll
                                for (int i = 0; i < 8; ++i) p[8 * h + i] = 0;
                            }
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) p[i] = 0;
                    }
                    if (D != 256 || b == who) tmem_store16(p_at + 16 * b, p);
                }
                tmem_wait_store();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&bars.p_full[w]);
                // what the sums so far and this tile's count from here on
                const float now = fmaxf(m, top), old = ex2(m - now), add = ex2(top - now);
                m = now;
                l = fmaf(l, old, sum * add);
                ok = warp_wait(&bars.o_full[w], t & 1, &bars.failed);
                if (!ok) break;
                fence_after();
                const uint64_t f2 = pack2(add * value, add * value);
                const bool grown = __any_sync(0xFFFFFFFFu, old != 1.0f);
                const uint64_t old2 = pack2(old, old);
#pragma unroll
                for (int b = 0; b < C / 32; ++b) {
                    uint32_t y[32];
                    tmem_load32(o_at + 32 * b, y);
                    tmem_wait_load32(y);
                    if (grown) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[16 * b + i] = mul2(o[16 * b + i], old2);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        o[16 * b + i] = fma2(pack2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1])), f2, o[16 * b + i]);
                }
                fence_before();
            }
            // ---- the unit's partial
            const float inv = 1.0f / l;
            float4* out = reinterpret_cast<float4*>(a.slots) + ((slot * X::kTiles + w) * (D / 4) + o0 / 4) * 128 + r;
#pragma unroll
            for (int i = 0; i < C / 4; ++i)
                out[i * 128] = make_float4(half_of(o[2 * i], 0) * inv, half_of(o[2 * i], 1) * inv, half_of(o[2 * i + 1], 0) * inv,
                                           half_of(o[2 * i + 1], 1) * inv);
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

// 32 rows of a cached head, a lane each; the warps share the output's values.
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
    float top = kNothing, total = 0.0f;
    for (int i = 0; i <= n; ++i) top = fmaxf(top, weight[i][lane]);
    for (int i = 0; i <= n; ++i) total += ex2(weight[i][lane] - top);
    __syncthreads();
    for (int i = warp; i <= n; i += 8) weight[i][lane] = ex2(weight[i][lane] - top) / total;
    __syncthreads();
    constexpr int Q = D / 32;  // four values each
    float4 x[Q];
    const float f0 = weight[n][lane];
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        const float4 v = reinterpret_cast<const float4*>(a.rows)[own * (D / 4) + warp * Q + i];
        x[i] = make_float4(v.x * f0, v.y * f0, v.z * f0, v.w * f0);
    }
    const float4* part = reinterpret_cast<const float4*>(a.slots) + ((slot0 * X::kTiles + in / 128) * (D / 4) + warp * Q) * 128 + in % 128;
#pragma unroll 4
    for (int s = 0; s < n; ++s) {
        const float f = weight[s][lane];
        const float4* p = part + static_cast<int64_t>(s) * X::kTiles * (D / 4) * 128;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            const float4 v = p[i * 128];
            if (f != 0.0f)  // (rows that nothing is joined to)
                x[i] = make_float4(fmaf(v.x, f, x[i].x), fmaf(v.y, f, x[i].y), fmaf(v.z, f, x[i].z), fmaf(v.w, f, x[i].w));
        }
    }
    if (!real) return;
    uint16_t* out = static_cast<uint16_t*>(a.out) + tok * a.out_token_stride +
                    (head * a.group + row - tok * a.group) * a.out_head_stride + warp * Q * 4;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        const uint32_t lo = a.bf16 ? Half<ARC_BF16>::pack(x[i].x, x[i].y) : Half<ARC_F16>::pack(x[i].x, x[i].y);
        const uint32_t hi = a.bf16 ? Half<ARC_BF16>::pack(x[i].z, x[i].w) : Half<ARC_F16>::pack(x[i].z, x[i].w);
        if (a.vec) {
            *reinterpret_cast<uint2*>(out + 4 * i) = make_uint2(lo, hi);
        } else {
            out[4 * i] = static_cast<uint16_t>(lo);
            out[4 * i + 1] = static_cast<uint16_t>(lo >> 16);
            out[4 * i + 2] = static_cast<uint16_t>(hi);
            out[4 * i + 3] = static_cast<uint16_t>(hi >> 16);
        }
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
    const dim3 grid(static_cast<unsigned>((p.rows + 31) / 32), static_cast<unsigned>(cache.heads));
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
