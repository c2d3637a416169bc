// arc_kv_attend: attention of a step's new tokens over the paged 8-bit cache.
#include "kv_host.cuh"
#include "serve_util.cuh"

namespace {

using namespace arcs;

constexpr int kThreads = 256;

struct AttendArgs {
    arc_kv_cache c;
    arc_kv_step s;
    arc_kv_query q;
    uint32_t* err;
};

// One warp for each (token, query head): the running maximum, sum and output
// of its softmax over the tokens in turn, head_dim / 32 values a lane.
template <int DT, int D>
__global__ void __launch_bounds__(kThreads) attend_kernel(const __grid_constant__ AttendArgs a) {
    constexpr int V = D / 32;
    using T = typename Half<DT>::T;
    const int lane = threadIdx.x & 31;
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    if (w >= a.s.T * a.q.q_heads) return;
    const int hq = static_cast<int>(w % a.q.q_heads);
    const int64_t t = w / a.q.q_heads;
    const int h = hq / (a.q.q_heads / a.c.heads);
    int64_t b = t, first = t;
    bool bad = false;
    if (a.s.row_offsets != nullptr) {
        int64_t lo = 0, hi = a.s.B - 1;
        while (lo < hi) {
            const int64_t m = (lo + hi + 1) >> 1;
            if (__ldg(a.s.row_offsets + m) <= t)
                lo = m;
            else
                hi = m - 1;
        }
        b = lo;
        first = __ldg(a.s.row_offsets + b);
        const int64_t end = __ldg(a.s.row_offsets + b + 1);
        if (first < 0 || first > t || end <= t || end > a.s.T || (b > 0 && __ldg(a.s.row_offsets + b - 1) > first)) {
            if (a.err && lane == 0) atomicOr(a.err, ARC_KV_ERR_OFFSETS);
            return;
        }
    }
    const int64_t held = __ldg(a.s.positions + b);
    const int64_t pos = held + (t - first);
    T* out = static_cast<T*>(a.q.out) + t * a.q.out_token_stride + hq * a.q.out_head_stride + lane * V;
    float o[V], q[V];
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = 0.0f;
    float m = -INFINITY, l = 0.0f;
    if (held >= 0) {
        const T* qp = static_cast<const T*>(a.q.q) + t * a.q.q_token_stride + hq * a.q.q_head_stride + lane * V;
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] = Half<DT>::to_float(qp[i]) * (a.q.scale * 1.4426950408889634f);
        const int64_t from = a.q.window > 0 && pos + 1 > a.q.window ? pos + 1 - a.q.window : 0;
        if (pos >= int64_t{a.s.max_pages} * a.c.page_size) {
            bad = true;
            if (a.err && lane == 0) atomicOr(a.err, ARC_KV_ERR_POSITION);
        }
        for (int64_t j = from; j <= pos && !bad; ++j) {
            const int64_t pi = j / a.c.page_size;
            const int page = __ldg(a.s.page_table + b * a.s.table_stride + pi);
            if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.c.pages)) {
                bad = true;
                if (a.err && lane == 0) atomicOr(a.err, ARC_KV_ERR_PAGE);
                break;
            }
            const int64_t at = page * a.c.page_stride + h * a.c.head_stride + (j - pi * a.c.page_size) * D + lane * V;
            const uint8_t* kp = static_cast<const uint8_t*>(a.c.k) + at;
            const uint8_t* vp = static_cast<const uint8_t*>(a.c.v) + at;
            const int64_t si = static_cast<int64_t>(page) * a.c.heads + h;
            float s = 0.0f, v[V];
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const uint32_t kw = e4m3x2_to_half2(kp[i] | (kp[i + 1] << 8));
                const uint32_t vw = e4m3x2_to_half2(vp[i] | (vp[i + 1] << 8));
                const float2 kf = __half22float2(*reinterpret_cast<const __half2*>(&kw));
                const float2 vf = __half22float2(*reinterpret_cast<const __half2*>(&vw));
                s = fmaf(q[i], kf.x, fmaf(q[i + 1], kf.y, s));
                v[i] = vf.x;
                v[i + 1] = vf.y;
            }
            for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
            s *= a.c.k_scale[si];
            const float vs = a.c.v_scale[si];
            const float mn = fmaxf(m, s);
            const float keep = m == -INFINITY ? 0.0f : exp2f(m - mn), p = exp2f(s - mn);
            l = l * keep + p;
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = fmaf(o[i], keep, p * vs * v[i]);
            m = mn;
        }
    }
    const float inv = bad ? __int_as_float(0x7FC00000) : (l > 0.0f || l != l ? 1.0f / l : 0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = Half<DT>::from_float(o[i] * inv);
}

template <int DT>
int launch(const AttendArgs& a, cudaStream_t st) {
    const int64_t warps = a.s.T * a.q.q_heads;
    const int64_t grid = (warps * 32 + kThreads - 1) / kThreads;
    if (grid > INT_MAX) return ARC_E_SHAPE;
    const unsigned g = static_cast<unsigned>(grid);
    if (a.c.head_dim == 64)
        attend_kernel<DT, 64><<<g, kThreads, 0, st>>>(a);
    else if (a.c.head_dim == 128)
        attend_kernel<DT, 128><<<g, kThreads, 0, st>>>(a);
    else
        attend_kernel<DT, 256><<<g, kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? ARC_OK : ARC_E_CUDA;
}

}  // namespace

extern "C" {

size_t arc_kv_attend_workspace_bytes(const arc_kv_cache* cache) { return check_cache(cache) == ARC_OK ? 16 : 0; }

int arc_kv_attend(const arc_kv_cache* cache, const arc_kv_step* step, const arc_kv_query* query, uint32_t* err_word,
                  void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_cache(cache);
    if (rc == ARC_OK) rc = check_step(cache, step);
    if (rc != ARC_OK) return rc;
    if (query == nullptr || query->q == nullptr || query->out == nullptr) return ARC_E_NULL;
    if (query->dtype != ARC_BF16 && query->dtype != ARC_F16) return ARC_E_DTYPE;
    if (query->q_heads <= 0 || query->q_heads > (1 << 16) || query->q_heads % cache->heads != 0) return ARC_E_SHAPE;
    if (query->window < 0 || !(query->scale >= -3.0e38f && query->scale <= 3.0e38f)) return ARC_E_OPTION;
    if (!aligned(query->q, 2) || !aligned(query->out, 2) || !aligned(err_word, 4)) return ARC_E_ALIGN;
    if (workspace == nullptr || workspace_bytes < arc_kv_attend_workspace_bytes(cache)) return ARC_E_WORKSPACE;
    if (!aligned(workspace, 16)) return ARC_E_ALIGN;
    AttendArgs a{*cache, *step, *query, err_word};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return query->dtype == ARC_BF16 ? launch<ARC_BF16>(a, st) : launch<ARC_F16>(a, st);
}

}  // extern "C"
