// arc_kv_append: rotate the new queries and keys, quantise keys and values to
// e4m3 with one power-of-two scale for each page and head.
//
// Rotation.  Pair i at position p turns by p * turns[i] modulo 2^64: the low
// 64 bits of the product are the exact fraction of a turn, so a far position
// costs no accuracy.  The fraction is split into a quarter turn and a rest of
// at most an eighth to either side, whose sine and cosine are taken in fp32:
// a rotated value is off by less than 2^-21 (|a| + |b|) times the amplitude.
//
// Rounding.  The stored code is the nearest one to the exact rotated value:
// where the two ends of that error interval round to different codes (about
// one value in 10^5) the value is recomputed in fp64.  The same holds for the
// page's largest magnitude, where the interval's ends give different scales.
#include <atomic>

#include "kv_host.cuh"
#include "serve_util.cuh"

namespace {

using namespace arcs;

constexpr int kThreads = 256;
constexpr float kRotErr = 4.8e-7f;  // 2^-21
constexpr int kKept = 4;            // row passes of a page job whose rows stay in registers

struct AppendArgs {
    arc_kv_cache c;
    arc_kv_step s;
    arc_kv_rows r;
    const uint64_t* turns;
    float amp;
    int32_t rot;
    int32_t layout;
    int32_t vec;      // bit 0: q and q_out, 1: k, 2: v allow 16-byte accesses
    int64_t q_blocks; // blocks that rotate queries; the rest store keys and values
    int32_t head_sets;  // the query heads of a token are shared by this many thread groups
    uint32_t* err;
};

// cos and sin of the pair's angle, fp32, without the amplitude.
__device__ __forceinline__ float2 turn32(uint64_t phase) {
    const uint32_t quarter = static_cast<uint32_t>((phase + (uint64_t{1} << 61)) >> 62);
    const int64_t rest = static_cast<int64_t>(phase - (static_cast<uint64_t>(quarter) << 62));
    // rest / 2^63 half turns, at most a quarter of a half turn to either side
    const float x = static_cast<float>(static_cast<int32_t>(rest >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(x, &s, &c);
    const float a = (quarter & 1) ? s : c, b = (quarter & 1) ? c : s;
    return make_float2(((quarter + 1) & 2) ? -a : a, (quarter & 2) ? -b : b);
}

__device__ __noinline__ double turn64(uint64_t phase, float a, float b, float amp) {
    double s, c;
    sincospi(static_cast<double>(static_cast<int64_t>(phase)) * 0x1p-63, &s, &c);
    return static_cast<double>(amp) * (static_cast<double>(a) * c - static_cast<double>(b) * s);
}

// Round a double to e4m3 once: to odd in fp32 first (fp32 keeps more than two
// bits below an e4m3 step), then to nearest.
__device__ __forceinline__ uint32_t e4m3_of_double(double y) {
    float f = __double2float_rz(y);
    if (static_cast<double>(f) != y) f = __uint_as_float(__float_as_uint(f) | 1u);
    return e4m3x2(f, 0.0f) & 0xFFu;
}

// Which angle and partner the element at `d` of a head has: y[d] = a c - b s
// with a = x[d], b = sgn * x[partner].
struct PairOf {
    int pair, partner;
    float sgn;
};
__device__ __forceinline__ PairOf pair_of(int d, int rot, int layout) {
    if (layout == ARC_ROPE_HALF) {
        const int h = rot >> 1;
        return d < h ? PairOf{d, d + h, 1.0f} : PairOf{d - h, d - h, -1.0f};
    }
    return (d & 1) ? PairOf{d >> 1, d - 1, -1.0f} : PairOf{d >> 1, d + 1, 1.0f};
}

// Eight values d0 .. d0 + 7 of one head: x and, with its sign, the partner of
// each (b); elements past the rotation have b = 0.
template <int DT>
__device__ __forceinline__ void load_pairs(const char* head, int d0, int rot, int layout, bool vec, float (&a)[8],
                                           float (&b)[8]) {
    load8<DT>(head + d0 * 2, vec, a);
    if (d0 >= rot) {
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = 0.0f;
        return;
    }
    if (layout == ARC_ROPE_INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const bool in = d0 + i < rot;
            b[i] = in ? a[i + 1] : 0.0f;
            b[i + 1] = in ? -a[i] : 0.0f;
        }
        return;
    }
    const int h = rot >> 1;
    if ((h & 7) == 0) {  // the whole vector lies on one side
        load8<DT>(head + (d0 < h ? d0 + h : d0 - h) * 2, vec, b);
        if (d0 >= h) {
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] = -b[i];
        }
        return;
    }
    const typename Half<DT>::T* e = reinterpret_cast<const typename Half<DT>::T*>(head);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = d0 + i;
        b[i] = 0.0f;
        if (d < rot) {
            const PairOf p = pair_of(d, rot, layout);
            b[i] = p.sgn * Half<DT>::to_float(e[p.partner]);
        }
    }
}

// cos and sin (times the amplitude) of the eight elements' angles.
__device__ __forceinline__ void load_turns(const AppendArgs& a, int64_t pos, int d0, float (&c)[8], float (&s)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = 1.0f;
        s[i] = 0.0f;
    }
    if (d0 >= a.rot) return;
    if (a.layout == ARC_ROPE_INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            if (d0 + i < a.rot) {
                const float2 t = turn32(static_cast<uint64_t>(pos) * __ldg(a.turns + ((d0 + i) >> 1)));
                c[i] = c[i + 1] = t.x * a.amp;
                s[i] = s[i + 1] = t.y * a.amp;
            }
        }
        return;
    }
    const int h = a.rot >> 1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = d0 + i;
        if (d < a.rot) {
            const float2 t = turn32(static_cast<uint64_t>(pos) * __ldg(a.turns + (d < h ? d : d - h)));
            c[i] = t.x * a.amp;
            s[i] = t.y * a.amp;
        }
    }
}

// The sequence of row t: the last b with row_offsets[b] <= t.
__device__ __forceinline__ int64_t sequence_of(const arc_kv_step& s, int64_t t) {
    if (s.row_offsets == nullptr) return t;
    int64_t lo = 0, hi = s.B - 1;
    while (lo < hi) {
        const int64_t m = (lo + hi + 1) >> 1;
        if (__ldg(s.row_offsets + m) <= t)
            lo = m;
        else
            hi = m - 1;
    }
    return lo;
}

// Rows of sequence b: first and count; a bad pair of offsets counts as none.
__device__ __forceinline__ bool rows_of(const arc_kv_step& s, int64_t b, int64_t& first, int64_t& n) {
    if (s.row_offsets == nullptr) {
        first = b;
        n = 1;
        return true;
    }
    const int64_t lo = __ldg(s.row_offsets + b), hi = __ldg(s.row_offsets + b + 1);
    first = lo;
    n = hi - lo;
    if (lo < 0 || hi < lo || hi > s.T || (b == 0 && lo != 0) || (b == s.B - 1 && hi != s.T)) {
        n = 0;
        return false;
    }
    return true;
}

// A thread owns eight values of a token's heads h0, h0 + sets, ...: the
// angles are computed once for all of them.
template <int DT>
__device__ __forceinline__ void rotate_queries(const AppendArgs& a) {
    const int L = a.c.head_dim >> 3;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int d0 = static_cast<int>(unit % L) * 8;
    const int64_t g = unit / L;
    const int set = static_cast<int>(g % a.head_sets);
    const int64_t t = g / a.head_sets;
    bool on = t < a.s.T;
    int64_t pos = 0;
    if (on) {
        const int64_t b = sequence_of(a.s, t);
        int64_t first, n;
        if (!rows_of(a.s, b, first, n) || t < first || t >= first + n) {
            if (a.err) atomicOr(a.err, ARC_KV_ERR_OFFSETS);
            on = false;
        } else {
            const int p = __ldg(a.s.positions + b);
            pos = p < 0 ? -1 : p + (t - first);
        }
    }
    float c[8], s[8];
    load_turns(a, pos, d0, c, s);
    const bool vec = a.vec & 1;
    for (int h0 = 0; h0 < a.r.q_heads; h0 += a.head_sets) {  // the same trips in every lane
        const int h = h0 + set;
        const bool here = on && h < a.r.q_heads;
        float x[8], y[8];
        if (here)
            load_pairs<DT>(static_cast<const char*>(a.r.q) + (t * a.r.q_token_stride + h * a.r.q_head_stride) * 2, d0,
                           a.rot, a.layout, vec, x, y);
        __syncwarp();  // in place: a head's lanes are in one warp, its loads come before its stores
        if (here) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = pos < 0 ? 0.0f : fmaf(x[i], c[i], -(y[i] * s[i]));
            store8<DT>(static_cast<char*>(a.r.q_out) + (t * a.r.out_token_stride + h * a.r.out_head_stride + d0) * 2,
                       vec, x);
        }
        __syncwarp();
    }
}

// Eight rotated values of a key, or eight values (`turn` false), their error
// bound, and what an exact recomputation needs.
struct Eight {
    float y[8];
    float err;  // 0: exact
};

template <int DT>
__device__ __forceinline__ bool eight(const AppendArgs& a, const char* head, bool turn, int64_t pos, int d0, bool vec,
                                      Eight& e) {
    bool nan = false;
    e.err = 0.0f;
    if (turn && d0 < a.rot) {
        float x[8], b[8], c[8], s[8];
        load_pairs<DT>(head, d0, a.rot, a.layout, vec, x, b);
        load_turns(a, pos, d0, c, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            e.y[i] = fmaf(x[i], c[i], -(b[i] * s[i]));
            e.err = fmaxf(e.err, fabsf(x[i]) + fabsf(b[i]));
        }
        e.err *= kRotErr * a.amp;
    } else {
        load8<DT>(head + d0 * 2, vec, e.y);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (e.y[i] != e.y[i]) {
            e.y[i] = 0.0f;
            nan = true;
        }
    }
    return nan;
}

// The exact value of element d of a rotated head.
template <int DT>
__device__ __noinline__ double exact_value(const AppendArgs& a, const char* head, int64_t pos, int d) {
    const typename Half<DT>::T* e = reinterpret_cast<const typename Half<DT>::T*>(head);
    const float x = Half<DT>::to_float(e[d]);
    if (d >= a.rot) return x;
    const PairOf p = pair_of(d, a.rot, a.layout);
    const double y = turn64(static_cast<uint64_t>(pos) * __ldg(a.turns + p.pair), x,
                            p.sgn * Half<DT>::to_float(e[p.partner]), a.amp);
    return y != y ? 0.0 : y;
}

// The codes of eight values under the scale 2^e.
template <int DT>
__device__ __forceinline__ uint2 codes(const AppendArgs& a, const char* head, int64_t pos, int d0, const Eight& v, int e) {
    const float inv = exp2i(-e);
    uint32_t lo[2], hi[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const float* y = v.y + 4 * w;
        lo[w] = e4m3x2((y[0] - v.err) * inv, (y[1] - v.err) * inv) |
                (e4m3x2((y[2] - v.err) * inv, (y[3] - v.err) * inv) << 16);
        hi[w] = e4m3x2((y[0] + v.err) * inv, (y[1] + v.err) * inv) |
                (e4m3x2((y[2] + v.err) * inv, (y[3] + v.err) * inv) << 16);
    }
    if (lo[0] != hi[0] || lo[1] != hi[1]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int w = i >> 2, sh = (i & 3) * 8;
            if (((lo[w] ^ hi[w]) >> sh) & 0xFFu) {
                const uint32_t code = e4m3_of_double(exact_value<DT>(a, head, pos, d0 + i) * static_cast<double>(inv));
                lo[w] = (lo[w] & ~(0xFFu << sh)) | (code << sh);
            }
        }
    }
    return make_uint2(lo[0], lo[1]);
}

// Four e4m3 codes times `f`, a power of two: shifts exponents, rounds below
// the normal range.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t h = e4m3x2_to_half2(w >> (16 * i));
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
        out |= e4m3x2(x.x * f, x.y * f) << (16 * i);
    }
    return out;
}

// Scale exponent of a page that keeps older tokens (`held`): what is stored is
// a power of two; anything else (never written here) counts as its exponent.
__device__ __forceinline__ int held_exponent(float scale) {
    const int e = static_cast<int>((__float_as_uint(scale) >> 23) & 0xFF) - 127;
    return e < -kScaleExp ? -kScaleExp : (e > kScaleExp ? kScaleExp : e);
}

// One new token of a (sequence, head, key or value): head_dim / 8 lanes.
template <int DT>
__device__ __forceinline__ void store_single(const AppendArgs& a) {
    const int L = a.c.head_dim >> 3;
    const int64_t unit = (static_cast<int64_t>(blockIdx.x) - a.q_blocks) * kThreads + threadIdx.x;
    const int64_t job = unit / L;
    const int d0 = static_cast<int>(unit % L) * 8;
    const bool is_v = job & 1;
    const int64_t bh = job >> 1;
    const int h = static_cast<int>(bh % a.c.heads);
    const int64_t b = bh / a.c.heads;
    bool on = b < a.s.B;
    int pos = on ? __ldg(a.s.positions + b) : -1;
    uint32_t err = 0;
    on = on && pos >= 0;
    const int pi = pos / a.c.page_size, slot = pos - pi * a.c.page_size;
    if (on && pi >= a.s.max_pages) {
        err |= ARC_KV_ERR_POSITION;
        on = false;
    }
    int page = on ? __ldg(a.s.page_table + b * a.s.table_stride + pi) : 0;
    if (on && static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.c.pages)) {
        err |= ARC_KV_ERR_PAGE;
        on = false;
    }
    const char* head = static_cast<const char*>(is_v ? a.r.v : a.r.k) +
                       (b * (is_v ? a.r.v_token_stride : a.r.k_token_stride) +
                        h * (is_v ? a.r.v_head_stride : a.r.k_head_stride)) * 2;
    const bool vec = a.vec & (is_v ? 4 : 2);
    float* scale = (is_v ? a.c.v_scale : a.c.k_scale) + static_cast<int64_t>(page) * a.c.heads + h;
    Eight v;
    v.err = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v.y[i] = 0.0f;
    float was = 0.0f;
    if (on) {
        was = *scale;
        if (eight<DT>(a, head, !is_v, pos, d0, vec, v)) err |= ARC_KV_ERR_NAN;
    }
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fmaxf(lo, fabsf(v.y[i]) - v.err);
        hi = fmaxf(hi, fabsf(v.y[i]) + v.err);
    }
    for (int m = L >> 1 < 16 ? L >> 1 : 16; m; m >>= 1) {
        lo = fmaxf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, m));
        hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, m));
    }
    int e = scale_exponent(lo);
    const bool unsure = on && e != scale_exponent(hi);
    if (__any_sync(0xFFFFFFFFu, unsure)) {
        double y = 0.0;
        if (unsure)
            for (int i = 0; i < 8; ++i) y = fmax(y, fabs(exact_value<DT>(a, head, pos, d0 + i)));
        for (int m = L >> 1 < 16 ? L >> 1 : 16; m; m >>= 1) y = fmax(y, __shfl_xor_sync(0xFFFFFFFFu, y, m));
        // rounding up cannot pass a border from below: 448 * 2^e is an fp32 value
        if (unsure) e = scale_exponent(__double2float_ru(y));
    }
    // the reads of the scale above come before any lane's write below
    __syncwarp();
    if (on) {
        char* base = static_cast<char*>(is_v ? a.c.v : a.c.k) + page * a.c.page_stride + h * a.c.head_stride + d0;
        if (slot > 0) {
            const int old = held_exponent(was);
            if (e > old) {
                const float f = exp2i(old - e);
#pragma unroll 4
                for (int s = 0; s < slot; ++s) {
                    uint2* p = reinterpret_cast<uint2*>(base + static_cast<int64_t>(s) * a.c.head_dim);
                    const uint2 w = *p;
                    *p = make_uint2(rescale4(w.x, f), rescale4(w.y, f));
                }
            } else {
                e = old;
            }
        }
        *reinterpret_cast<uint2*>(base + static_cast<int64_t>(slot) * a.c.head_dim) = codes<DT>(a, head, pos, d0, v, e);
        if (d0 == 0) *scale = exp2i(e);
    }
    if (err && a.err) atomicOr(a.err, err);
}

// All new tokens of a (sequence, page, head, key or value): one block, a row
// of head_dim / 8 lanes for each token, the rows of the first kKept passes in
// registers between the maximum and the rounding.
template <int DT>
__device__ __forceinline__ void store_pages(const AppendArgs& a) {
    __shared__ int64_t wsum[kThreads / 32];
    __shared__ int64_t found[2];  // sequence, page within its new ones
    __shared__ uint32_t red[2][kThreads / 32];
    __shared__ unsigned long long red64[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ps = a.c.page_size;
    const int64_t jobs_per_page = int64_t{2} * a.c.heads;
    const int64_t block = static_cast<int64_t>(blockIdx.x) - a.q_blocks;
    const int64_t want = block / jobs_per_page;
    const int sub = static_cast<int>(block % jobs_per_page);
    const bool is_v = sub & 1;
    const int h = sub >> 1;

    // pages touched by sequence b; the running total finds this block's
    auto touched = [&](int64_t b) -> int64_t {
        int64_t first, n;
        if (!rows_of(a.s, b, first, n)) {
            if (a.err) atomicOr(a.err, ARC_KV_ERR_OFFSETS);
            return 0;
        }
        const int64_t p = __ldg(a.s.positions + b);
        if (p < 0 || n <= 0) return 0;
        return (p + n - 1) / ps - p / ps + 1;
    };
    if (tid == 0) found[0] = -1;
    int64_t before = 0;
    for (int64_t b0 = 0; b0 < a.s.B; b0 += kThreads) {
        const int64_t b = b0 + tid;
        const int64_t mine = b < a.s.B ? touched(b) : 0;
        int64_t incl = mine;
        for (int m = 1; m < 32; m <<= 1) {
            const int64_t o = __shfl_up_sync(0xFFFFFFFFu, incl, m);
            if (lane >= m) incl += o;
        }
        __syncthreads();
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        int64_t off = before, total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) off += wsum[w];
            total += wsum[w];
        }
        const int64_t lo = off + incl - mine;
        if (want >= lo && want < lo + mine) {
            found[0] = b;
            found[1] = want - lo;
        }
        before += total;
        if (before > want) break;
    }
    __syncthreads();
    const int64_t b = found[0];
    if (b < 0) return;
    int64_t first, n;
    rows_of(a.s, b, first, n);
    const int64_t p0 = __ldg(a.s.positions + b);
    const int64_t pi = p0 / ps + found[1];
    if (pi >= a.s.max_pages) {
        if (tid == 0 && a.err) atomicOr(a.err, ARC_KV_ERR_POSITION);
        return;
    }
    const int page = __ldg(a.s.page_table + b * a.s.table_stride + pi);
    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.c.pages)) {
        if (tid == 0 && a.err) atomicOr(a.err, ARC_KV_ERR_PAGE);
        return;
    }
    const int64_t page0 = pi * ps;
    const int slot0 = static_cast<int>(p0 > page0 ? p0 - page0 : 0);
    const int64_t end = p0 + n - page0;
    const int slot1 = static_cast<int>(end < ps ? end : ps);
    const int64_t row0 = first + (page0 + slot0 - p0);  // row of slot0

    const int L = a.c.head_dim >> 3;
    const int per = kThreads / L;  // rows of a pass
    const int my = tid / L, d0 = (tid % L) * 8;
    const int rows = slot1 - slot0, passes = (rows + per - 1) / per;
    const int64_t ts = is_v ? a.r.v_token_stride : a.r.k_token_stride;
    const char* src = static_cast<const char*>(is_v ? a.r.v : a.r.k) +
                      (row0 * ts + h * (is_v ? a.r.v_head_stride : a.r.k_head_stride)) * 2;
    const bool vec = a.vec & (is_v ? 4 : 2);
    float* scale = (is_v ? a.c.v_scale : a.c.k_scale) + static_cast<int64_t>(page) * a.c.heads + h;
    const float was = *scale;
    Eight kept[kKept];
    float lo = 0.0f, hi = 0.0f;
    bool nan = false;
    auto fetch = [&](int r, Eight& v) {
        v.err = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v.y[i] = 0.0f;
        if (r < rows) nan |= eight<DT>(a, src + r * ts * 2, !is_v, page0 + slot0 + r, d0, vec, v);
    };
    auto widen = [&](const Eight& v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo = fmaxf(lo, fabsf(v.y[i]) - v.err);
            hi = fmaxf(hi, fabsf(v.y[i]) + v.err);
        }
    };
#pragma unroll
    for (int p = 0; p < kKept; ++p) {
        if (p < passes) {
            fetch(p * per + my, kept[p]);
            widen(kept[p]);
        }
    }
    for (int p = kKept; p < passes; ++p) {
        Eight v;
        fetch(p * per + my, v);
        widen(v);
    }
    // magnitudes are not negative: their bits order as they do
    const uint32_t wl = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(lo));
    const uint32_t wh = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(hi));
    if (lane == 0) {
        red[0][warp] = wl;
        red[1][warp] = wh;
    }
    if (nan && a.err) atomicOr(a.err, ARC_KV_ERR_NAN);
    __syncthreads();
    uint32_t bl = 0, bh = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        bl = max(bl, red[0][w]);
        bh = max(bh, red[1][w]);
    }
    int e = scale_exponent(__uint_as_float(bl));
    if (e != scale_exponent(__uint_as_float(bh))) {  // the same in every thread
        double y = 0.0;
        for (int p = 0; p < passes; ++p) {
            const int r = p * per + my;
            if (r < rows)
                for (int i = 0; i < 8; ++i)
                    y = fmax(y, fabs(exact_value<DT>(a, src + r * ts * 2, page0 + slot0 + r, d0 + i)));
        }
        for (int m = 16; m; m >>= 1) y = fmax(y, __shfl_xor_sync(0xFFFFFFFFu, y, m));
        if (lane == 0) red64[warp] = static_cast<unsigned long long>(__double_as_longlong(y));
        __syncthreads();
        for (int w = 0; w < kThreads / 32; ++w) y = fmax(y, __longlong_as_double(static_cast<long long>(red64[w])));
        e = scale_exponent(__double2float_ru(y));
    }
    char* base = static_cast<char*>(is_v ? a.c.v : a.c.k) + page * a.c.page_stride + h * a.c.head_stride;
    if (slot0 > 0) {
        const int old = held_exponent(was);
        if (e > old) {
            const float f = exp2i(old - e);
            const int words = slot0 * (a.c.head_dim >> 3);
            for (int w = tid; w < words; w += kThreads) {
                uint2* p = reinterpret_cast<uint2*>(base) + w;
                const uint2 x = *p;
                *p = make_uint2(rescale4(x.x, f), rescale4(x.y, f));
            }
        } else {
            e = old;
        }
    }
    auto put = [&](int r, const Eight& v) {
        if (r < rows)
            *reinterpret_cast<uint2*>(base + static_cast<int64_t>(slot0 + r) * a.c.head_dim + d0) =
                codes<DT>(a, src + r * ts * 2, page0 + slot0 + r, d0, v, e);
    };
#pragma unroll
    for (int p = 0; p < kKept; ++p)
        if (p < passes) put(p * per + my, kept[p]);
    for (int p = kKept; p < passes; ++p) {
        Eight v;
        fetch(p * per + my, v);
        put(p * per + my, v);
    }
    // every thread read the scale before the barrier above
    if (tid == 0) *scale = exp2i(e);
}

template <int DT>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs a) {
    if (static_cast<int64_t>(blockIdx.x) < a.q_blocks)
        rotate_queries<DT>(a);
    else if (a.s.row_offsets == nullptr)
        store_single<DT>(a);
    else
        store_pages<DT>(a);
}

}  // namespace

extern "C" int arc_kv_append(const arc_kv_cache* cache, const arc_kv_step* step, const arc_kv_rows* rows,
                             const arc_rope* rope, uint32_t* err_word, void* stream) {
    int rc = check_cache(cache);
    if (rc == ARC_OK) rc = check_step(cache, step);
    if (rc != ARC_OK) return rc;
    if (rows == nullptr || rows->k == nullptr || rows->v == nullptr) return ARC_E_NULL;
    if (rows->dtype != ARC_BF16 && rows->dtype != ARC_F16) return ARC_E_DTYPE;
    if (rows->q_heads < 0 || rows->q_heads > (1 << 16)) return ARC_E_SHAPE;
    if (rows->q_heads > 0 && (rows->q == nullptr || rows->q_out == nullptr)) return ARC_E_NULL;
    if (!aligned(rows->q, 2) || !aligned(rows->k, 2) || !aligned(rows->v, 2) || !aligned(rows->q_out, 2) ||
        !aligned(err_word, 4))
        return ARC_E_ALIGN;
    if (rows->q_heads > 0 && rows->q == rows->q_out &&
        (rows->q_token_stride != rows->out_token_stride || rows->q_head_stride != rows->out_head_stride))
        return ARC_E_OPTION;
    AppendArgs a;
    a.turns = nullptr;
    a.amp = 1.0f;
    a.rot = 0;
    a.layout = ARC_ROPE_HALF;
    if (rope != nullptr) {
        if (rope->rot_dim < 0 || rope->rot_dim > cache->head_dim || rope->rot_dim % 2 != 0) return ARC_E_SHAPE;
        if (rope->rot_dim > 0 && rope->turns == nullptr) return ARC_E_NULL;
        if ((rope->layout != ARC_ROPE_HALF && rope->layout != ARC_ROPE_INTERLEAVED) || rope->reserved != 0 ||
            !(rope->amplitude > 0.0f) || !(rope->amplitude <= 3.0e38f))
            return ARC_E_OPTION;
        if (!aligned(rope->turns, 8)) return ARC_E_ALIGN;
        a.turns = rope->turns;
        a.amp = rope->amplitude;
        a.rot = rope->rot_dim;
        a.layout = rope->layout;
    }
    a.c = *cache;
    a.s = *step;
    a.r = *rows;
    a.err = err_word;
    a.vec = (rows->q_heads > 0 && vectors(rows->q, rows->q_token_stride, rows->q_head_stride) &&
                     vectors(rows->q_out, rows->out_token_stride, rows->out_head_stride)
                 ? 1
                 : 0) |
            (vectors(rows->k, rows->k_token_stride, rows->k_head_stride) ? 2 : 0) |
            (vectors(rows->v, rows->v_token_stride, rows->v_head_stride) ? 4 : 0);
    const int L = cache->head_dim / 8;
    a.head_sets = 1;
    a.q_blocks = 0;
    if (rows->q_heads > 0) {
        // few tokens: each head its own threads; many: one thread turns all heads of its eight values
        const int64_t units = step->T * L;
        while (a.head_sets < rows->q_heads && units * a.head_sets < 152 * 2048) a.head_sets *= 2;
        if (a.head_sets > rows->q_heads) a.head_sets = rows->q_heads;
        a.q_blocks = (units * a.head_sets + kThreads - 1) / kThreads;
    }
    int64_t kv_blocks;
    if (step->row_offsets == nullptr) {
        kv_blocks = (step->B * cache->heads * 2 * L + kThreads - 1) / kThreads;
    } else {
        // a sequence with n tokens touches at most n / page_size + 2 pages, and at most n
        const int64_t seqs = step->B < step->T ? step->B : step->T;
        const int64_t most = step->T / cache->page_size + 2 * seqs;
        kv_blocks = (most < step->T ? most : step->T) * cache->heads * 2;
    }
    const int64_t grid = a.q_blocks + kv_blocks;
    if (grid > INT_MAX) return ARC_E_SHAPE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (rows->dtype == ARC_BF16)
        append_kernel<ARC_BF16><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(a);
    else
        append_kernel<ARC_F16><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? ARC_OK : ARC_E_CUDA;
}
