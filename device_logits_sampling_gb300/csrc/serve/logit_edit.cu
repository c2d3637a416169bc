// arc_edit_logits: penalties, biases and a mask of allowed ids on a step's logits, in one pass.
//
// A block has a slice of a row.  It reads the row's lists once, keeps those of its ids in two tables in shared memory
// (how often the history has the id; the last bias entry for it, so that the order in which entries arrive does not
// matter) and marks each group of eight ids that has one; the slice's logits and mask are under way meanwhile.  Eight ids
// are one byte of the mask, one byte of marks and 16 bytes of 16-bit logits.  Eight disallowed ids are written without
// being read; in place, eight that are allowed and unmarked are not touched at all.
//
// Bounds and figures.  A mask alone, in place, 100 x 100,003 fp32: 9.2 us, faster than its 81 MB at the measured copy
// rate (12.1), since what it takes out is not read.  256 rows x 129,280 with histories of up to 4,096 ids, up to 300
// biases and masks: 47 us (20.5 of traffic): instructions, 70% of the issue slots; every block of a row goes through the
// row's lists.  One row 4.4 us: four loads that wait for one another.  Measured and left: all eight ids of a marked group
// looked up with its store (56 us), a second kernel with a hash table a row that edits behind the stream (54, and 12 for
// one row), edits by whoever takes an id's word out of the table (66 to 80), counts and entries in one word (73).
//
// Rows of an odd vocabulary begin anywhere: the groups of eight are laid on the 16-byte boundaries of the output, the
// mask's byte is cut out of two, and logits that are not aligned alike are read one by one.
#include <atomic>
#include <climits>
#include <cstdint>

#include "launch_util.cuh"
#include "serve/arc_edit.h"
#include "serve_util.cuh"

namespace {

using namespace arcs;

constexpr int kThreads = 256;

// G: groups of eight ids a thread has.
template <int G>
struct Slice {
    static constexpr int kSlice = kThreads * G, kIds = kSlice * 8;  // groups and ids of a block
    struct Tables {
        uint32_t count[kIds];  // of the history
        uint32_t entry[kIds];  // 1 + the last bias entry
        uint8_t marks[kSlice];
    };
};

struct EditArgs {
    arc_logit_edits e;
    const void* logits;
    void* out;
    int64_t B, V, ld, out_ld;
    uint32_t* err;
    int32_t in_place;
};

template <int DT>
struct Type {
    using T = typename Half<DT>::T;
};
template <>
struct Type<ARC_F32> {
    using T = float;
};
template <int DT>
__device__ __forceinline__ float widen(typename Type<DT>::T x) {
    if constexpr (DT == ARC_F32)
        return x;
    else
        return Half<DT>::to_float(x);
}
template <int DT>
__device__ __forceinline__ typename Type<DT>::T narrow(float x) {
    if constexpr (DT == ARC_F32)
        return x;
    else
        return Half<DT>::from_float(x);
}

// A row's part of a list; false where its offsets are wrong.
__device__ __forceinline__ bool part_of(const int32_t* offsets, int64_t row, int64_t len, int64_t& lo, int64_t& hi) {
    lo = __ldg(offsets + row);
    hi = __ldg(offsets + row + 1);
    if (lo >= 0 && lo <= hi && hi <= len) return true;
    lo = hi = 0;
    return false;
}

__device__ __forceinline__ bool in_range(float x) { return fabsf(x) <= 3.4028235e38f; }

template <int DT, int OT, bool LISTS, int G>
__global__ void __launch_bounds__(kThreads) edit_kernel(const __grid_constant__ EditArgs a) {
    using T = typename Type<DT>::T;
    using O = typename Type<OT>::T;
    using Tables = typename Slice<G>::Tables;
    constexpr int kIds = Slice<G>::kIds;
    extern __shared__ __align__(16) uint8_t dyn[];
    Tables& tab = *reinterpret_cast<Tables*>(dyn);
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.y + static_cast<int64_t>(gridDim.y) * blockIdx.z;
    if (row >= a.B) return;
    const T* const in = static_cast<const T*>(a.logits) + row * a.ld;
    O* const out = static_cast<O*>(a.out) + row * a.out_ld;
    // ids of the first, short group: those before the output's first 16-byte boundary
    const int head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(out) & 15)) & 15) / static_cast<int>(sizeof(O));
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kIds + (head ? head - 8 : 0);  // first id, maybe below 0
    if (base >= a.V) return;
    const bool first = blockIdx.x == 0;
    uint32_t err = 0;

    int64_t h0 = 0, h1 = 0, b0 = 0, b1 = 0;
    float rep = 1.0f, freq = 0.0f, pres = 0.0f;
    if (a.e.hist_offsets) {
        if (!part_of(a.e.hist_offsets, row, a.e.hist_len, h0, h1)) err |= ARC_EDIT_ERR_HIST;
        const arc_row_params* p = a.e.params + row;
        rep = p->repetition_penalty;
        freq = p->frequency_penalty;
        pres = p->presence_penalty;
        if (!(rep > 0.0f) || !in_range(rep) || !in_range(freq) || !in_range(pres)) {
            err |= ARC_EDIT_ERR_PARAM;
            h1 = h0;
        }
    }
    if (a.e.bias_offsets && !part_of(a.e.bias_offsets, row, a.e.bias_len, b0, b1)) err |= ARC_EDIT_ERR_BIAS;
    const uint32_t* mask = nullptr;
    bool nothing = false;
    if (a.e.allowed) {
        const int64_t m = a.e.allowed_rows ? __ldg(a.e.allowed_rows + row) : row;
        if (m >= a.e.allowed_count) {
            err |= ARC_EDIT_ERR_MASK;
            nothing = true;
        } else if (m >= 0) {
            mask = a.e.allowed + m * a.e.allowed_stride;
        }
    }

    // the mask's eight bits of ids i .. i + 7 (i may lie below 0; no bit from V on is used)
    const int64_t words = (a.V + 31) >> 5;
    auto bits_of = [&](int64_t i) -> uint32_t {
        if (nothing) return 0;
        if (mask == nullptr) return 0xFFu;
        const int64_t w = i >> 5;
        const int s = static_cast<int>(i & 31);
        uint32_t lo = w >= 0 ? __ldg(mask + w) : 0, hi = 0;
        if (s > 24 && w + 1 < words) hi = __ldg(mask + w + 1);
        return __funnelshift_r(lo, hi, s) & 0xFFu;
    };
    const bool lists = LISTS && !nothing && (h1 > h0 || b1 > b0);
    // the history's first ids, the mask and the logits are on their way together
    int32_t early[4] = {0, 0, 0, 0};
    if (lists) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (h0 + tid + k * kThreads < h1) early[k] = __ldg(a.e.hist_ids + h0 + tid + k * kThreads);
    }
    const float none = -__int_as_float(0x7F800000);
    const bool in_vec = ((reinterpret_cast<uintptr_t>(in) + base * static_cast<int64_t>(sizeof(T))) & 15) == 0;
    uint32_t bits[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int64_t i = base + (g * kThreads + tid) * 8;
        bits[g] = i < a.V ? bits_of(i) : 0;
    }
    alignas(16) T x[G][8];  // moved 16 bytes at a time
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int64_t i = base + (g * kThreads + tid) * 8;
        if (i >= a.V || bits[g] == 0 || (a.in_place && bits[g] == 0xFFu)) continue;
        if (in_vec && i >= 0 && i + 8 <= a.V) {
            const uint4* p = reinterpret_cast<const uint4*>(in + i);
            uint4* q = reinterpret_cast<uint4*>(x[g]);
#pragma unroll
            for (int k = 0; k < static_cast<int>(sizeof(T)) / 2; ++k) q[k] = p[k];
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (i + k >= 0 && i + k < a.V) x[g][k] = in[i + k];
        }
    }

    if (lists) {
        uint4* z = reinterpret_cast<uint4*>(dyn);
        for (int i = tid; i < static_cast<int>(sizeof(Tables) / 16); i += kThreads) z[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        // a list's ids, four loads of a thread under way at a time
        auto each = [&](const int32_t* ids, int64_t lo, int64_t hi, uint32_t bit, bool loaded, auto take) {
            for (int64_t i = lo + tid; i < hi; i += 4 * kThreads) {
                int32_t id[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    id[k] = loaded ? early[k] : i + k * kThreads < hi ? __ldg(ids + i + k * kThreads) : 0;
                loaded = false;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (i + k * kThreads >= hi) break;
                    if (id[k] < 0 || id[k] >= a.V) {
                        err |= bit;
                    } else if (static_cast<uint64_t>(id[k] - base) < kIds) {
                        const int at = static_cast<int>(id[k] - base);
                        take(at, static_cast<uint32_t>(i + k * kThreads - lo + 1));
                        tab.marks[at >> 3] = 1;
                    }
                }
            }
        };
        each(a.e.hist_ids, h0, h1, ARC_EDIT_ERR_HIST, true, [&](int at, uint32_t) { atomicAdd(&tab.count[at], 1u); });
        each(a.e.bias_ids, b0, b1, ARC_EDIT_ERR_BIAS, false, [&](int at, uint32_t e) { atomicMax(&tab.entry[at], e); });
        __syncthreads();
    }
    if (err && first && a.err) atomicOr(a.err, err);

#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int64_t i = base + (g * kThreads + tid) * 8;
        if (i >= a.V) continue;
        if (!(a.in_place && bits[g] == 0xFFu)) {
            alignas(16) O y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if constexpr (DT == OT)
                    y[k] = x[g][k];
                else
                    y[k] = narrow<OT>(widen<DT>(x[g][k]));
                if (!(bits[g] >> k & 1)) y[k] = narrow<OT>(none);
            }
            if (i >= 0 && i + 8 <= a.V) {
                const uint4* q = reinterpret_cast<const uint4*>(y);
                uint4* p = reinterpret_cast<uint4*>(out + i);
#pragma unroll
                for (int k = 0; k < static_cast<int>(sizeof(O)) / 2; ++k) p[k] = q[k];
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (i + k >= 0 && i + k < a.V) out[i + k] = y[k];
            }
        }
        if (LISTS && lists && tab.marks[g * kThreads + tid]) {
            // the ids of the eight that the lists have, one by one, over what has just been stored
            const int at = (g * kThreads + tid) * 8;
            uint32_t hit = 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint4 c = reinterpret_cast<const uint4*>(tab.count + at)[k], e = reinterpret_cast<const uint4*>(tab.entry + at)[k];
                hit |= ((c.x | e.x ? 1u : 0u) | (c.y | e.y ? 2u : 0u) | (c.z | e.z ? 4u : 0u) | (c.w | e.w ? 8u : 0u)) << (4 * k);
            }
            for (hit &= bits[g]; hit; hit &= hit - 1) {
                const int k = __ffs(hit) - 1;
                const uint32_t c = tab.count[at + k], e = tab.entry[at + k];
                float z = widen<DT>(in[i + k]);
                if (c) {
                    z = z > 0.0f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
                    z = __fsub_rn(z, __fmul_rn(static_cast<float>(c), freq));
                    z = __fsub_rn(z, pres);
                }
                if (e) z = __fadd_rn(z, __ldg(a.e.bias + b0 + (e - 1)));
                out[i + k] = narrow<OT>(z);
            }
        }
    }
}

template <int DT, int OT, bool LISTS, int G>
int launch(const EditArgs& a, int dev, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    // without tables the whole of an SM's storage holds loads in flight
    if (arc::prepare(edit_kernel<DT, OT, LISTS, G>, dev, done, LISTS ? 100 : 0) != cudaSuccess) return ARC_E_CUDA;
    // the short first group shifts the slices by less than one group
    const int64_t slices = (a.V + 7 + Slice<G>::kIds - 1) / Slice<G>::kIds;
    const int64_t ys = a.B < 65535 ? a.B : 65535, zs = (a.B + ys - 1) / ys;
    const dim3 grid(static_cast<unsigned>(slices), static_cast<unsigned>(ys), static_cast<unsigned>(zs));
    edit_kernel<DT, OT, LISTS, G><<<grid, kThreads, LISTS ? sizeof(typename Slice<G>::Tables) : 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? ARC_OK : ARC_E_CUDA;
}

template <int DT, int OT>
int launch(const EditArgs& a, int dev, cudaStream_t st) {
    // Two groups a thread where there are lists (256 rows x 129,280 46.6 us, 57.2 with one; 512 rows 90 and 111; 32 rows 9.5
    // and 10.5; 64 x 50,003 9.3 and 10.1).  Few rows want more blocks: one row 5.4 us with one, 6.0 with two; 8 rows 6.0 and
    // 7.0; 16 rows 7.0 and 7.6; 20 rows 8.3 and 7.6, 24 rows 7.8 and 8.3.  Without lists the numbers lie within 4%.
    if (a.e.hist_offsets || a.e.bias_offsets)
        return a.B * a.V <= (5 << 19) ? launch<DT, OT, true, 1>(a, dev, st) : launch<DT, OT, true, 2>(a, dev, st);
    return launch<DT, OT, false, 1>(a, dev, st);
}

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

extern "C" int arc_edit_logits(const void* logits, int64_t B, int64_t V, int64_t ld, int32_t dtype, void* out,
                               int64_t out_ld, int32_t out_dtype, const arc_logit_edits* edits, uint32_t* err_word,
                               void* stream) {
    if (logits == nullptr || out == nullptr || edits == nullptr) return ARC_E_NULL;
    const arc_logit_edits& e = *edits;
    if ((e.hist_offsets == nullptr) != (e.hist_ids == nullptr)) return ARC_E_NULL;
    if (e.hist_offsets != nullptr && e.params == nullptr) return ARC_E_NULL;
    if ((e.bias_offsets == nullptr) != (e.bias_ids == nullptr) || (e.bias_offsets == nullptr) != (e.bias == nullptr))
        return ARC_E_NULL;
    if (e.allowed == nullptr && e.allowed_rows != nullptr) return ARC_E_NULL;
    if (dtype != ARC_F32 && dtype != ARC_BF16 && dtype != ARC_F16) return ARC_E_DTYPE;
    if (out_dtype != dtype && out_dtype != ARC_F32) return ARC_E_DTYPE;
    if (B <= 0 || B > INT_MAX || V <= 0 || V > INT_MAX || ld < V || out_ld < V) return ARC_E_SHAPE;
    if (e.hist_offsets && (e.hist_len < 0 || e.hist_len > INT_MAX)) return ARC_E_SHAPE;
    if (e.bias_offsets && (e.bias_len < 0 || e.bias_len > INT_MAX)) return ARC_E_SHAPE;
    if (e.allowed && (e.allowed_stride < (V + 31) / 32 || e.allowed_count <= 0 ||
                      (e.allowed_rows == nullptr && e.allowed_count < B)))
        return ARC_E_SHAPE;
    if (out == logits && (out_dtype != dtype || (B > 1 && out_ld != ld))) return ARC_E_OPTION;
    const uintptr_t in_size = dtype == ARC_F32 ? 4 : 2, out_size = out_dtype == ARC_F32 ? 4 : 2;
    if (!aligned(logits, in_size) || !aligned(out, out_size) || !aligned(err_word, 4) || !aligned(e.hist_offsets, 4) ||
        !aligned(e.hist_ids, 4) || !aligned(e.bias_offsets, 4) || !aligned(e.bias_ids, 4) || !aligned(e.bias, 4) ||
        !aligned(e.allowed, 4) || !aligned(e.allowed_rows, 4) || !aligned(e.params, 8))
        return ARC_E_ALIGN;
    EditArgs a{e, logits, out, B, V, ld, out_ld, err_word, out == logits};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return ARC_E_CUDA;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == ARC_F32) return launch<ARC_F32, ARC_F32>(a, dev, st);
    if (dtype == ARC_BF16) return out_dtype == ARC_F32 ? launch<ARC_BF16, ARC_F32>(a, dev, st) : launch<ARC_BF16, ARC_BF16>(a, dev, st);
    return out_dtype == ARC_F32 ? launch<ARC_F16, ARC_F32>(a, dev, st) : launch<ARC_F16, ARC_F16>(a, dev, st);
}
