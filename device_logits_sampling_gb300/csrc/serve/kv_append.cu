// arc_kv_append: rotate the new queries and keys, quantise keys and values to
// e4m3 with one power-of-two scale for each page and head.
//
// Rotation.  Pair i at position p turns by p * turns[i] modulo 2^64: the low
// 64 bits of the product are the exact fraction of a turn, so a far position
// costs no accuracy.  The fraction is split into quarter turns and a rest of
// at most an eighth to either side, whose sine and cosine are fp32 Taylor sums:
// a rotated value is off by less than 3.4e-7 (|a| + |b|) times the amplitude
// (the angle's two roundings 1.2e-7, the sums' 4e-8, the amplitude's, the
// product's and the difference's 6e-8 each).
//
// Rounding.  The stored code is the nearest one to the exact rotated value:
// where the two ends of that error interval round to different codes (about
// one value in 10^5) the value is recomputed in fp64, with Taylor sums too.  The same holds for the
// page's largest magnitude, where the interval's ends give different scales.
//
// Bounds and figures.  One token of a sequence: latency, a launch and three
// dependent loads (position, page, scale): 4.0 us; 256 tokens of 32 + 8 heads
// of 64: 5.7 us.  Prompts (10,476 tokens of 32 + 8 heads of 128): 72 us against
// 35 us of memory time; the page blocks wait on their own chain (find the page,
// load, maximum, round) at 16 warps an SM, which their registers allow (the half
// layout spills 312 to 384 bytes a thread).  300 sequences of 1 to 5 drafted tokens:
// 50 us, a block a page and four heads.  2 us of these are the look at all offsets
// by every block, 1 us the care for infinities.
// Measured and left: eight values a thread (187 us), one launch for queries and
// pages (135 us: the queries are held to the pages' registers), no load ahead
// of the next head (78 us), eight heads a block (80 us), one pass in registers
// at three blocks an SM (85 us).
#include <cstring>

#include "kv_device.cuh"
#include "kv_host.cuh"
#include "serve_util.cuh"

namespace {

using namespace arcs;

constexpr int kThreads = 256;
constexpr float kRotErr = 3.4e-7f;
// |a| + |b| is at most sqrt(2) of the pair's length, and that at most the sum of the turned pair's magnitudes
constexpr float kTurnedErr = 1.42f * kRotErr;
constexpr int kKept = 2;            // row passes of a page job whose rows stay in registers

struct AppendArgs {
    arc_kv_cache c;
    arc_kv_step s;
    arc_kv_rows r;
    const uint64_t* turns;
    float amp;
    int32_t rot;
    int32_t layout;
    int32_t vec;      // bit 0: q and q_out, 1: k, 2: v allow 16-byte accesses
    int64_t q_blocks; // blocks that rotate queries
    int32_t head_sets;  // the query heads of a token are shared by this many thread groups
    int32_t page_heads; // heads of a page that a block stores
    uint32_t* err;
};

// cos and sin of the pair's angle, fp32, without the amplitude: Taylor sums on
// an eighth of a turn to either side (the first terms left out are below
// 2e-9), then the quarter turns.
__device__ __forceinline__ float2 turn32(uint64_t phase) {
    const uint32_t quarter = static_cast<uint32_t>((phase + (uint64_t{1} << 61)) >> 62);
    const int32_t rest = static_cast<int32_t>(static_cast<uint32_t>(phase >> 32) - (quarter << 30));
    const float x = static_cast<float>(rest) * 1.46291807926715968e-9f;  // 2 pi / 2^32
    const float q = x * x;
    float s = fmaf(q, 2.7557319e-6f, -1.9841270e-4f);  // 1 / 9!, -1 / 7!
    s = fmaf(q, s, 8.3333333e-3f);
    s = fmaf(q, s, -1.6666667e-1f);
    s = fmaf(x * q, s, x);
    float c = fmaf(q, -2.7557319e-7f, 2.4801587e-5f);  // -1 / 10!, 1 / 8!
    c = fmaf(q, c, -1.3888889e-3f);
    c = fmaf(q, c, 4.1666667e-2f);
    c = fmaf(q, c, -0.5f);
    c = fmaf(q, c, 1.0f);
    const float a = (quarter & 1) ? s : c, b = (quarter & 1) ? c : s;
    return make_float2(((quarter + 1) & 2) ? -a : a, (quarter & 2) ? -b : b);
}

// a c - b s in fp64: Taylor sums up to the first term below 2^-53.
__device__ __noinline__ double turn64(uint64_t phase, float a, float b, float amp) {
    const uint32_t quarter = static_cast<uint32_t>((phase + (uint64_t{1} << 61)) >> 62);
    const int64_t rest = static_cast<int64_t>(phase - (static_cast<uint64_t>(quarter) << 62));
    const double x = static_cast<double>(rest) * 3.40612158008655459e-19;  // 2 pi / 2^64
    const double q = x * x;
    double s = -1.0 / 1307674368000.0;  // 15!
    s = fma(q, s, 1.0 / 6227020800.0);
    s = fma(q, s, -1.0 / 39916800.0);
    s = fma(q, s, 1.0 / 362880.0);
    s = fma(q, s, -1.0 / 5040.0);
    s = fma(q, s, 1.0 / 120.0);
    s = fma(q, s, -1.0 / 6.0);
    s = fma(x * q, s, x);
    double c = 1.0 / 20922789888000.0;  // 16!
    c = fma(q, c, -1.0 / 87178291200.0);
    c = fma(q, c, 1.0 / 479001600.0);
    c = fma(q, c, -1.0 / 3628800.0);
    c = fma(q, c, 1.0 / 40320.0);
    c = fma(q, c, -1.0 / 720.0);
    c = fma(q, c, 1.0 / 24.0);
    c = fma(q, c, -0.5);
    c = fma(q, c, 1.0);
    const double u = (quarter & 1) ? s : c, w = (quarter & 1) ? c : s;
    const double cs = ((quarter + 1) & 2) ? -u : u, sn = (quarter & 2) ? -w : w;
    return static_cast<double>(amp) * (static_cast<double>(a) * cs - static_cast<double>(b) * sn);
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

// A thread owns sixteen values of a head: two vectors of eight, at d[0] and
// d[1].  In the half layout (kHalves) they are each other's partners, so that a
// pair is loaded and its angle computed once; vectors past the rotation pair up
// as they lie.  A half rotation whose halves do not start on a vector (kOdd)
// looks its partners up one by one.
enum Turning { kHalves, kNeighbours, kOdd };
struct Place {
    int d[2];
    bool turns;
};
template <int TURN>
__device__ __forceinline__ Place place_of(const AppendArgs& a, int j) {
    if (TURN == kHalves) {
        const int h = a.rot >> 1, n = h >> 3;  // vectors of a half
        if (j < n) return Place{{8 * j, 8 * j + h}, true};
        return Place{{a.rot + 16 * (j - n), a.rot + 16 * (j - n) + 8}, false};
    }
    return Place{{16 * j, 16 * j + 8}, 16 * j < a.rot};
}

// cos and sin (times the amplitude) of the place's eight pairs.
struct Turns {
    float c[8], s[8];
};
template <int TURN>
__device__ __forceinline__ void turns_of(const AppendArgs& a, const Place& p, int64_t pos, Turns& t) {
    if (TURN == kOdd || !p.turns) return;
    const int first = TURN == kHalves ? p.d[0] : p.d[0] >> 1;
    uint64_t f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = TURN == kHalves || first + i < (a.rot >> 1) ? __ldg(a.turns + first + i) : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 cs = turn32(static_cast<uint64_t>(pos) * f[i]);
        t.c[i] = cs.x * a.amp;
        t.s[i] = cs.y * a.amp;
    }
}

// The place's sixteen values of `head`, as they lie, and as fp32.
__device__ __forceinline__ uint4 raw8(const char* p, bool vec) {
    if (vec) return *reinterpret_cast<const uint4*>(p);
    const uint16_t* e = reinterpret_cast<const uint16_t*>(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = e[2 * i] | (static_cast<uint32_t>(e[2 * i + 1]) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}
struct Raw {
    uint4 v[2];
};
__device__ __forceinline__ Raw load16(const Place& p, const char* head, bool vec) {
    return Raw{{raw8(head + p.d[0] * 2, vec), raw8(head + p.d[1] * 2, vec)}};
}
template <int DT>
__device__ __forceinline__ void unpack16(const Raw& r, float (&x)[16]) {
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const uint32_t w[4] = {r.v[v].x, r.v[v].y, r.v[v].z, r.v[v].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = Half<DT>::unpack(w[i]);
            x[8 * v + 2 * i] = f.x;
            x[8 * v + 2 * i + 1] = f.y;
        }
    }
}

// Turn them; for kOdd returns the error bound of the turned values (elsewhere the pair itself gives it later).
template <int DT, int TURN>
__device__ __forceinline__ float turn16(const AppendArgs& a, const Place& p, const Turns& t, const char* head, int64_t pos,
                                        float (&x)[16]) {
    float most = 0.0f;
    if (!p.turns) return 0.0f;
    if (TURN == kOdd) {
        const typename Half<DT>::T* e = reinterpret_cast<const typename Half<DT>::T*>(head);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int d = p.d[0] + i;
            if (d < a.rot) {
                const PairOf q = pair_of(d, a.rot, a.layout);
                const float b = q.sgn * Half<DT>::to_float(e[q.partner]);
                const float2 cs = turn32(static_cast<uint64_t>(pos) * __ldg(a.turns + q.pair));
                most = fmaxf(most, fabsf(x[i]) + fabsf(b));
                x[i] = fmaf(x[i], cs.x * a.amp, -(b * (cs.y * a.amp)));
            }
        }
    } else {
        const int pairs = TURN == kHalves ? 8 : (a.rot - p.d[0]) >> 1;  // neighbours may end inside
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float& u = x[TURN == kHalves ? i : 2 * i];
            float& w = x[TURN == kHalves ? 8 + i : 2 * i + 1];
            if (TURN == kHalves || i < pairs) {
                const float y = fmaf(u, t.c[i], -(w * t.s[i]));
                w = fmaf(w, t.c[i], u * t.s[i]);
                u = y;
            }
        }
    }
    return most * (kRotErr * a.amp);
}

// The sequence of row t: the last b of `sound` with row_offsets[b] <= t.
__device__ __forceinline__ int64_t sequence_of(const arc_kv_step& s, int64_t sound, int64_t t) {
    if (s.row_offsets == nullptr) return t;
    int64_t lo = 0, hi = sound - 1;
    while (lo < hi) {
        const int64_t m = (lo + hi + 1) >> 1;
        if (__ldg(s.row_offsets + m) <= t)
            lo = m;
        else
            hi = m - 1;
    }
    return lo;
}

// The place's values of a row that no sequence has: NaN.
template <int DT>
__device__ __noinline__ void blank_queries(const AppendArgs& a, const Place& p, int64_t t, int set) {
    for (int h = set; h < a.r.q_heads; h += a.head_sets) {
        typename Half<DT>::T* const to =
            static_cast<typename Half<DT>::T*>(a.r.q_out) + t * a.r.out_token_stride + h * a.r.out_head_stride;
#pragma unroll 1
        for (int i = 0; i < 16; ++i) to[p.d[i >> 3] + (i & 7)] = Half<DT>::from_float(__uint_as_float(0x7FC00000u));
    }
}

// A thread owns sixteen values of a token's heads set, set + sets, ...: the
// angles are computed once for all of them; kHeads heads are in flight at once.
constexpr int kHeads = 4;
template <int DT, int TURN>
__device__ __forceinline__ void rotate_queries(const AppendArgs& a) {
    const int L = a.c.head_dim >> 4;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const Place p = place_of<TURN>(a, static_cast<int>(unit % L));
    const int64_t g = unit / L;
    const int set = static_cast<int>(g % a.head_sets);
    const int64_t t = g / a.head_sets;
    bool on = t < a.s.T;
    int64_t pos = 0;
    int64_t sound = a.s.B;
    if (a.s.row_offsets != nullptr) {
        sound = sound_sequences(a.s);
        if (sound < a.s.B) {
            if (threadIdx.x == 0 && a.err) atomicOr(a.err, ARC_KV_ERR_OFFSETS);
            if (on && t >= unclaimed_rows(a.s, sound)) {
                blank_queries<DT>(a, p, t, set);
                on = false;
            }
        }
    }
    if (on) {
        const int64_t b = sequence_of(a.s, sound, t);
        const int64_t first = a.s.row_offsets == nullptr ? b : static_cast<int64_t>(__ldg(a.s.row_offsets + b));
        const int at = __ldg(a.s.positions + b);
        pos = at < 0 ? -1 : at + (t - first);
    }
    Turns turns;
    turns_of<TURN>(a, p, pos, turns);
    const bool vec = a.vec & 1;
    const char* const from = static_cast<const char*>(a.r.q) + t * a.r.q_token_stride * 2;
    char* const to = static_cast<char*>(a.r.q_out) + t * a.r.out_token_stride * 2;
    for (int h0 = 0; h0 < a.r.q_heads; h0 += kHeads * a.head_sets) {  // the same trips in every lane
        Raw r[kHeads];
#pragma unroll
        for (int k = 0; k < kHeads; ++k) {
            const int h = h0 + k * a.head_sets + set;
            if (on && h < a.r.q_heads) r[k] = load16(p, from + h * a.r.q_head_stride * 2, vec);
        }
        if (TURN != kOdd) __syncwarp();  // in place: a head's lanes are in one warp, its loads come before its stores
#pragma unroll
        for (int k = 0; k < kHeads; ++k) {
            const int h = h0 + k * a.head_sets + set;
            const bool here = on && h < a.r.q_heads;
            float x[16];
            if (here) {
                unpack16<DT>(r[k], x);
                turn16<DT, TURN>(a, p, turns, from + h * a.r.q_head_stride * 2, pos, x);
            }
            if (TURN == kOdd) __syncwarp();  // the partners were read just now
            if (here) {
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    float e[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) e[i] = pos < 0 ? 0.0f : x[8 * v + i];
                    store8<DT>(to + (h * a.r.out_head_stride + p.d[v]) * 2, vec, e);
                }
            }
        }
        __syncwarp();
    }
}

// Sixteen turned values of a key, or sixteen values.
struct Sixteen {
    float y[16];
    float err;  // kOdd: their error bound
    float top;  // their largest magnitude
};

// Bounds of the largest magnitude's exact value (EXACT: the value is exact).
template <int TURN, bool EXACT>
__device__ __forceinline__ void bounds(const Place& p, const Sixteen& v, float& lo, float& hi) {
    // two values of a pair are at most the largest one each
    const float err = EXACT || !p.turns ? 0.0f : TURN == kOdd ? v.err : v.top * (2.0f * kTurnedErr);
    lo = fmaxf(lo, v.top - err);
    hi = fmaxf(hi, v.top + err);
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The largest magnitude; NaN values become 0 (true where there was one).
__device__ __forceinline__ bool finish16(Sixteen& v) {
    v.top = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v.top = max_nan(v.top, fabsf(v.y[i]));
    if (v.top == v.top) return false;
    v.top = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (v.y[i] != v.y[i]) v.y[i] = 0.0f;
        v.top = fmaxf(v.top, fabsf(v.y[i]));
    }
    return true;
}

// The exact value of element d of a key's head, turned; NaN counts as 0.
template <int DT>
__device__ __noinline__ double exact_value(const AppendArgs& a, const char* head, int64_t pos, int d) {
    const typename Half<DT>::T* e = reinterpret_cast<const typename Half<DT>::T*>(head);
    const float x = Half<DT>::to_float(e[d]);
    // (beside a pair that turns it is asked for such a value too, whose slack is the pair's)
    if (d >= a.rot) return x != x ? 0.0 : x;
    const PairOf p = pair_of(d, a.rot, a.layout);
    const double y = turn64(static_cast<uint64_t>(pos) * __ldg(a.turns + p.pair), x,
                            p.sgn * Half<DT>::to_float(e[p.partner]), a.amp);
    return y != y ? 0.0 : y;
}

// Store the codes of the place's values under the scale 2^e in the row at `out`.
template <int DT, int TURN, bool EXACT>
__device__ __forceinline__ void put16(const AppendArgs& a, const Place& p, const char* head, int64_t pos, const Sixteen& v,
                                      int e, char* out) {
    const float inv = exp2i(-e);
    // values that do not turn are exact, and often lie on a tie: no slack for them (nor 0 times an infinity)
    const float rel = kTurnedErr * inv;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t lo[2], hi[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const float* y = v.y + 8 * half + 4 * w;
            if (EXACT || !p.turns) {
                lo[w] = e4m3x2(y[0] * inv, y[1] * inv) | (e4m3x2(y[2] * inv, y[3] * inv) << 16);
                hi[w] = lo[w];
            } else {
                float l[4], h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // the other value of the pair
                    const float z = TURN == kHalves ? v.y[8 * (half ^ 1) + 4 * w + i] : y[i ^ 1];
                    const float slack = TURN == kOdd ? v.err * inv : (fabsf(y[i]) + fabsf(z)) * rel;
                    l[i] = fmaf(y[i], inv, -slack);
                    h[i] = fmaf(y[i], inv, slack);
                }
                lo[w] = e4m3x2(l[0], l[1]) | (e4m3x2(l[2], l[3]) << 16);
                hi[w] = e4m3x2(h[0], h[1]) | (e4m3x2(h[2], h[3]) << 16);
            }
        }
        if (!EXACT && (lo[0] != hi[0] || lo[1] != hi[1])) {
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                const int sh = (i & 3) * 8;
                const uint32_t l = i < 4 ? lo[0] : lo[1], g = i < 4 ? hi[0] : hi[1];
                if (((l ^ g) >> sh) & 0xFFu) {
                    const uint32_t code = e4m3_of_double(exact_value<DT>(a, head, pos, p.d[half] + i) * static_cast<double>(inv));
                    const uint32_t n = (l & ~(0xFFu << sh)) | (code << sh);
                    if (i < 4)
                        lo[0] = n;
                    else
                        lo[1] = n;
                }
            }
        }
        *reinterpret_cast<uint2*>(out + p.d[half]) = make_uint2(lo[0], lo[1]);
    }
}

// Four e4m3 codes times `f`, a power of two: shifts exponents, rounds below
// the normal range.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
    uint32_t h[2], out = 0;
    e4m3x4_to_half2(w, h[0], h[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        out |= e4m3x2(x.x * f, x.y * f) << (16 * i);
    }
    return out;
}

// Whether value i can be the largest one, of which `lo` is a lower bound.
__device__ __forceinline__ bool may_be_largest(const Sixteen& v, int i, float lo) {
    float y = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) y = k == i ? fabsf(v.y[k]) : y;
    return !(y + v.err < lo * (1.0f - 4.0f * kTurnedErr));
}

// A page that keeps older tokens under a scale written here: 2^e with e in [-32, 32].
__device__ __forceinline__ bool plain_scale(float was) {
    const uint32_t b = __float_as_uint(was);
    return (b & 0x7FFFFFu) == 0 && (b >> 23) - (127 - kScaleExp) <= 2 * kScaleExp;
}
__device__ __forceinline__ int held_exponent(float was) { return static_cast<int>(__float_as_uint(was) >> 23) - 127; }

// Any other one, which another program wrote: the new tokens' slots of a page's head, all in fp64, by the threads
// `unit` of `units`.  `need` is the least scale for the new tokens; the page's stays where it is as large. Out of
// range: nothing is stored. One call apart from the rest: its registers cost the prompts 5 us where it was inline.
struct Held {
    const char* src;     // the first new token's values
    char* base;          // the page's head
    float* scale;
    int64_t src_stride;  // bytes from token to token
    int64_t pos;         // of the first new token
    float was, need;
    int slot, rows;      // first new slot, new tokens
    int unit, units;
    bool turns;
};
template <int DT>
__device__ __noinline__ void store_held(const AppendArgs& a, const Held& h) {
    if (!(h.was >= exp2i(-kScaleExp) && h.was <= exp2i(kScaleExp))) {
        if (h.unit == 0 && a.err) atomicOr(a.err, ARC_KV_ERR_SCALE);
        return;
    }
    const int dim = a.c.head_dim;
    const float now = h.need > h.was ? h.need : h.was;
    if (now > h.was) {
        const double f = static_cast<double>(h.was) / static_cast<double>(now);  // exact: now is a power of two
        for (int i = h.unit; i < h.slot * dim; i += h.units) {
            uint32_t x, unused;
            e4m3x4_to_half2(static_cast<uint8_t>(h.base[i]), x, unused);
            const double y = static_cast<double>(__half2float(__ushort_as_half(static_cast<unsigned short>(x))));
            h.base[i] = static_cast<char>(e4m3_of_double(y * f));  // a code times a scale: 28 bits
        }
        if (h.unit == 0) *h.scale = now;
    }
    for (int i = h.unit; i < h.rows * dim; i += h.units) {
        const int r = i / dim, d = i - r * dim;
        const char* const head = h.src + r * h.src_stride;
        const float x = Half<DT>::to_float(reinterpret_cast<const typename Half<DT>::T*>(head)[d]);
        const double y = h.turns ? exact_value<DT>(a, head, h.pos + r, d) : (x != x ? 0.0 : static_cast<double>(x));
        h.base[h.slot * dim + i] = static_cast<char>(e4m3_of_double(y / static_cast<double>(now)));
    }
}

// One new token of a (sequence, head, key or value): head_dim / 16 lanes.
template <int DT, int TURN>
__device__ __forceinline__ void store_single(const AppendArgs& a) {
    const int L = a.c.head_dim >> 4;
    const int64_t unit = (static_cast<int64_t>(blockIdx.x) - a.q_blocks) * kThreads + threadIdx.x;
    const int64_t job = unit / L;
    const int j = static_cast<int>(unit % L);
    const bool is_v = job & 1;
    const int64_t bh = job >> 1;
    const int h = static_cast<int>(bh % a.c.heads);
    const int64_t b = bh / a.c.heads;
    bool on = b < a.s.B;
    const char* head = static_cast<const char*>(is_v ? a.r.v : a.r.k) +
                       (b * (is_v ? a.r.v_token_stride : a.r.k_token_stride) +
                        h * (is_v ? a.r.v_head_stride : a.r.k_head_stride)) * 2;
    const Place p = place_of<TURN>(a, j);
    Sixteen v;
    v.err = v.top = 0.0f;
    Raw raw;
    int pos = -1;
    if (on) {
        pos = __ldg(a.s.positions + b);  // these loads do not wait for each other
        raw = load16(p, head, a.vec & (is_v ? 4 : 2));
    }
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
        page = 0;
    }
    float* scale = (is_v ? a.c.v_scale : a.c.k_scale) + static_cast<int64_t>(page) * a.c.heads + h;
    float was = 0.0f;
    if (on) {
        was = *scale;
        unpack16<DT>(raw, v.y);
        if (!is_v) {
            Turns turns;
            turns_of<TURN>(a, p, pos, turns);
            v.err = turn16<DT, TURN>(a, p, turns, head, pos, v.y);
        }
        if (finish16(v)) err |= ARC_KV_ERR_NAN;
    }
    float lo = 0.0f, hi = 0.0f;
    if (is_v)
        bounds<TURN, true>(p, v, lo, hi);
    else
        bounds<TURN, false>(p, v, lo, hi);
    for (int m = L >> 1; m; m >>= 1) {
        lo = fmaxf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, m));
        hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, m));
    }
    int e = scale_exponent(lo);
    const bool unsure = on && e != scale_exponent(hi);
    if (__any_sync(0xFFFFFFFFu, unsure)) {
        double y = 0.0;
        if (unsure)
            // (only values that can be the largest one)
#pragma unroll 1
            for (int i = 0; i < 16; ++i) {
                const int d = p.d[i >> 3] + (i & 7);
                if (may_be_largest(v, i, lo)) y = fmax(y, fabs(exact_value<DT>(a, head, pos, d)));
            }
        for (int m = L >> 1; m; m >>= 1) y = fmax(y, __shfl_xor_sync(0xFFFFFFFFu, y, m));
        // rounding up cannot pass a border from below: 448 * 2^e is an fp32 value
        if (unsure) e = scale_exponent(__double2float_ru(y));
    }
    __syncwarp();  // every lane has read the scale
    if (on && slot > 0 && !plain_scale(was)) {
        char* base = static_cast<char*>(is_v ? a.c.v : a.c.k) + page * a.c.page_stride + h * a.c.head_stride;
        store_held<DT>(a, Held{head, base, scale, 0, pos, was, exp2i(e), slot, 1, j, L, !is_v});
        on = false;
    }
    if (on) {
        char* base = static_cast<char*>(is_v ? a.c.v : a.c.k) + page * a.c.page_stride + h * a.c.head_stride;
        if (slot > 0) {
            const int old = held_exponent(was);
            if (e > old) {
                const float f = exp2i(old - e);
#pragma unroll 4
                for (int s = 0; s < slot; ++s) {
                    uint4* q = reinterpret_cast<uint4*>(base + static_cast<int64_t>(s) * a.c.head_dim + 16 * j);
                    const uint4 w = *q;
                    *q = make_uint4(rescale4(w.x, f), rescale4(w.y, f), rescale4(w.z, f), rescale4(w.w, f));
                }
            } else {
                e = old;
            }
        }
        base += static_cast<int64_t>(slot) * a.c.head_dim;
        if (is_v)
            put16<DT, TURN, true>(a, p, head, pos, v, e, base);
        else
            put16<DT, TURN, false>(a, p, head, pos, v, e, base);
        if (j == 0) *scale = exp2i(e);
    }
    if (err && a.err) atomicOr(a.err, err);
}

// All new tokens of a (sequence, page, keys or values) and a.page_heads of its
// heads, one after another: a block, head_dim / 16 lanes for each token.  The
// angles are the heads' in common; the rows of the first kKept passes stay in
// registers between the maximum and the rounding.
template <int DT, int TURN, bool V>
__device__ __forceinline__ void store_pages(const AppendArgs& a, int64_t want, int set) {
    __shared__ int64_t wsum[kThreads / 32];
    __shared__ int64_t found[2];  // sequence, page within its new ones
    __shared__ uint32_t red[2][2][kThreads / 32];
    __shared__ double red64[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ps = a.c.page_size;
    // pages touched by sequence b; the running total finds this block's
    bool wrong = false;
    auto touched = [&](int64_t b) -> int64_t {
        int64_t first, n;
        if (!rows_of(a.s, b, first, n)) {
            wrong = true;
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
        int64_t mine = b < a.s.B ? touched(b) : 0;
        auto sums = [&]() {
            int64_t incl = mine;
            for (int m = 1; m < 32; m <<= 1) {
                const int64_t o = __shfl_up_sync(0xFFFFFFFFu, incl, m);
                if (lane >= m) incl += o;
            }
            return incl;
        };
        int64_t incl = sums();
        const bool stop = __syncthreads_or(wrong);
        if (stop) {  // the line ends before the first wrong pair of offsets
            if (tid == 0 && a.err) atomicOr(a.err, ARC_KV_ERR_OFFSETS);
            if (b >= sound_sequences(a.s)) mine = 0;
            incl = sums();
        }
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
        if (before > want || stop) break;
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

    const int L = a.c.head_dim >> 4;
    const int per = kThreads / L;  // rows of a pass
    const int my = tid / L;
    const Place p = place_of<TURN>(a, tid % L);
    const int rows = slot1 - slot0, passes = (rows + per - 1) / per;
    const int64_t ts = V ? a.r.v_token_stride : a.r.k_token_stride;
    const int64_t hs = V ? a.r.v_head_stride : a.r.k_head_stride;
    const bool vec = a.vec & (V ? 4 : 2);
    const char* const src0 = static_cast<const char*>(V ? a.r.v : a.r.k) + row0 * ts * 2;
    float* const scales = (V ? a.c.v_scale : a.c.k_scale) + static_cast<int64_t>(page) * a.c.heads;
    Turns turns[kKept];
    if (!V) {
#pragma unroll
        for (int k = 0; k < kKept; ++k)
            if (k * per + my < rows) turns_of<TURN>(a, p, page0 + slot0 + k * per + my, turns[k]);
    }
    Raw ahead[kKept];  // the next head's values
    auto look = [&](int h) {
#pragma unroll
        for (int k = 0; k < kKept; ++k)
            if (k * per + my < rows) ahead[k] = load16(p, src0 + h * hs * 2 + (k * per + my) * ts * 2, vec);
    };
    const int h1 = set * a.page_heads + a.page_heads < a.c.heads ? set * a.page_heads + a.page_heads : a.c.heads;
    look(set * a.page_heads);
    for (int h = set * a.page_heads; h < h1; ++h) {
        const char* src = src0 + h * hs * 2;
        const float was = scales[h];
        bool nan = false;
        auto fetch = [&](int r, const Raw& raw, const Turns& t, Sixteen& v) {
            v.err = v.top = 0.0f;
            if (r < rows) {
                unpack16<DT>(raw, v.y);
                if (!V) v.err = turn16<DT, TURN>(a, p, t, src + r * ts * 2, page0 + slot0 + r, v.y);
                nan |= finish16(v);
            }
        };
        auto again = [&](int k) {
            return k * per + my < rows ? load16(p, src + (k * per + my) * ts * 2, vec) : Raw{};
        };
        Sixteen kept[kKept];
        float lo = 0.0f, hi = 0.0f;
#pragma unroll
        for (int k = 0; k < kKept; ++k) {
            fetch(k * per + my, ahead[k], turns[k], kept[k]);
            bounds<TURN, V>(p, kept[k], lo, hi);
        }
        for (int k = kKept; k < passes; ++k) {
            Sixteen v;
            Turns t;
            if (!V && k * per + my < rows) turns_of<TURN>(a, p, page0 + slot0 + k * per + my, t);
            fetch(k * per + my, again(k), t, v);
            bounds<TURN, V>(p, v, lo, hi);
        }
        if (h + 1 < h1) look(h + 1);
        // magnitudes are not negative: their bits order as they do
        const uint32_t wl = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(lo));
        const uint32_t wh = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(hi));
        if (lane == 0) {
            red[h & 1][0][warp] = wl;
            red[h & 1][1][warp] = wh;
        }
        if (nan && a.err) atomicOr(a.err, ARC_KV_ERR_NAN);
        __syncthreads();  // two sets of sums in turn: the next head's are written before this one's are read by all
        uint32_t bl = 0, bh = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            bl = max(bl, red[h & 1][0][w]);
            bh = max(bh, red[h & 1][1][w]);
        }
        int e = scale_exponent(__uint_as_float(bl));
        if (!V && e != scale_exponent(__uint_as_float(bh))) {  // the same in every thread
            double y = 0.0;
            for (int k = 0; k < passes; ++k) {
                const int r = k * per + my;
                if (r < rows)
                    for (int i = 0; i < 16; ++i)
                        y = fmax(y, fabs(exact_value<DT>(a, src + r * ts * 2, page0 + slot0 + r, p.d[i >> 3] + (i & 7))));
            }
            for (int m = 16; m; m >>= 1) y = fmax(y, __shfl_xor_sync(0xFFFFFFFFu, y, m));
            if (lane == 0) red64[warp] = y;
            __syncthreads();
            for (int w = 0; w < kThreads / 32; ++w) y = fmax(y, red64[w]);
            __syncthreads();
            e = scale_exponent(__double2float_ru(y));
        }
        char* base = static_cast<char*>(V ? a.c.v : a.c.k) + page * a.c.page_stride + h * a.c.head_stride;
        if (slot0 > 0 && !plain_scale(was)) {  // the same in every thread
            store_held<DT>(a, Held{src, base, scales + h, ts * 2, page0 + slot0, was, exp2i(e), slot0, rows, tid, kThreads, !V});
            continue;
        }
        if (slot0 > 0) {
            const int old = held_exponent(was);
            if (e > old) {
                const float f = exp2i(old - e);
                const int words = slot0 * (a.c.head_dim >> 4);
                for (int w = tid; w < words; w += kThreads) {
                    uint4* q = reinterpret_cast<uint4*>(base) + w;
                    const uint4 x = *q;
                    *q = make_uint4(rescale4(x.x, f), rescale4(x.y, f), rescale4(x.z, f), rescale4(x.w, f));
                }
            } else {
                e = old;
            }
        }
        auto put = [&](int r, const Sixteen& v) {
            if (r < rows)
                put16<DT, TURN, V>(a, p, src + r * ts * 2, page0 + slot0 + r, v, e,
                             base + static_cast<int64_t>(slot0 + r) * a.c.head_dim);
        };
#pragma unroll
        for (int k = 0; k < kKept; ++k) put(k * per + my, kept[k]);
        for (int k = kKept; k < passes; ++k) {
            Sixteen v;
            Turns t;
            if (!V && k * per + my < rows) turns_of<TURN>(a, p, page0 + slot0 + k * per + my, t);
            fetch(k * per + my, again(k), t, v);
            put(k * per + my, v);
        }
        if (tid == 0) scales[h] = exp2i(e);  // every thread read it before the barrier
    }
}

// A decode step: queries and new tokens in one launch.
template <int DT, int TURN>
__global__ void __launch_bounds__(kThreads, 3) single_kernel(const __grid_constant__ AppendArgs a) {
    if (static_cast<int64_t>(blockIdx.x) < a.q_blocks)
        rotate_queries<DT, TURN>(a);
    else
        store_single<DT, TURN>(a);
}

// Prompts: two launches side by side, so that the queries' blocks are not held
// to the pages' registers.  The second starts with the first and ends after it.
template <int DT, int TURN>
__global__ void __launch_bounds__(kThreads, 3) rotate_kernel(const __grid_constant__ AppendArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    rotate_queries<DT, TURN>(a);
}

template <int DT, int TURN>
__global__ void __launch_bounds__(kThreads, 2) pages_kernel(const __grid_constant__ AppendArgs a) {
    const int sets = (a.c.heads + a.page_heads - 1) / a.page_heads;
    const int64_t page = blockIdx.x / (2 * sets);
    const int sub = static_cast<int>(blockIdx.x % (2 * sets));
    if (sub & 1)
        store_pages<DT, TURN, true>(a, page, sub >> 1);
    else
        store_pages<DT, TURN, false>(a, page, sub >> 1);
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int DT, int TURN>
int launch(const AppendArgs& a, int64_t kv_blocks, cudaStream_t st) {
    if (a.s.row_offsets == nullptr) {
        single_kernel<DT, TURN><<<static_cast<unsigned>(a.q_blocks + kv_blocks), kThreads, 0, st>>>(a);
        return cudaGetLastError() == cudaSuccess ? ARC_OK : ARC_E_CUDA;
    }
    if (a.q_blocks > 0) {
        rotate_kernel<DT, TURN><<<static_cast<unsigned>(a.q_blocks), kThreads, 0, st>>>(a);
        if (cudaGetLastError() != cudaSuccess) return ARC_E_CUDA;
    }
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>(kv_blocks), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.q_blocks > 0 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, pages_kernel<DT, TURN>, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return ARC_E_CUDA;
    }
    return ARC_OK;
}

template <int DT>
int launch_turning(const AppendArgs& a, int64_t kv_blocks, cudaStream_t st) {
    if (a.layout == ARC_ROPE_INTERLEAVED) return launch<DT, kNeighbours>(a, kv_blocks, st);
    return a.rot % 16 == 0 ? launch<DT, kHalves>(a, kv_blocks, st) : launch<DT, kOdd>(a, kv_blocks, st);
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
    const int L = cache->head_dim / 16;
    a.head_sets = 1;
    a.page_heads = 1;
    a.q_blocks = 0;
    if (rows->q_heads > 0) {
        // few tokens: each head its own threads; many: a thread turns several heads of its sixteen values with one
        // set of angles.  Sets for 155,000 threads against 620,000: 10,476 tokens of 32 heads of 128 73 us against 77,
        // of 64 38 against 46; 5,400 in 16 pieces 47 against 57; 700 16.6 either way
        const int64_t units = step->T * L;
        while (a.head_sets < rows->q_heads && units * a.head_sets < 152 * 1024) a.head_sets *= 2;
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
        // (and a block more, which finds no page and so sees all offsets)
        const int64_t pages = (most < step->T ? most : step->T) + 1;
        // many pages: a block stores several heads with one set of angles.  Four, two and one: 10,476 tokens 73, 76
        // and 90 us; 300 sequences of drafts 50, 71 and 111; 16 pieces 47, 47 and 52
        while (a.page_heads < 4 && a.page_heads < cache->heads && pages * cache->heads / a.page_heads > 512) a.page_heads *= 2;
        kv_blocks = pages * 2 * ((cache->heads + a.page_heads - 1) / a.page_heads);
    }
    const int64_t grid = a.q_blocks + kv_blocks;
    if (grid > INT_MAX) return ARC_E_SHAPE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return rows->dtype == ARC_BF16 ? launch_turning<ARC_BF16>(a, kv_blocks, st) : launch_turning<ARC_F16>(a, kv_blocks, st);
}
