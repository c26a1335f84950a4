// Softmax attention over a sliding window plus the first (sink) tokens:
//   o_t = sum_{s in K(t)} softmax_s(scale q_t . k_s) v_s,
//   K(t) = {s <= t : s > t - window or s < sinks},
// for a whole prompt (queries are the last Tq of Tk tokens), for one token per session
// against a rolling cache, and the copy that fills that cache from a prompt.
//
// The rolling cache of a session holds its visible tokens and no others: token p lies in
// slot p while p < window + sinks and later in the window's turn,
//   slot(p) = p < sinks ? p : sinks + (p - sinks) mod window,
// so the tokens visible at position p are exactly slots 0 .. min(window + sinks, p + 1) - 1,
// in an order that the softmax does not see.
#include "gdn_common.cuh"

namespace gdn {

struct WindowArgs {
    const __nv_bfloat16 *q, *k, *v;
    long long q_batch, q_row, q_head, k_batch, k_row, k_head, v_batch, v_row, v_head;
    const int* lengths;                      // [B] or null: keys at and past lengths[b] are padding
    __nv_bfloat16* out;                      // [B, Tq, Hq, dv]
    int B, Tq, Tk, Hq, Hkv, dk, dv;
    int window, sinks;
    float scale;
};

struct StepArgs {
    const __nv_bfloat16 *q, *k, *v;          // [B, Hq, dk], [B, Hkv, dk], [B, Hkv, dv]
    long long q_batch, k_batch, v_batch;
    __nv_bfloat16 *k_cache, *v_cache;        // [B, window + sinks, Hkv, d]
    const int* pos;                          // [B]: the token's position; negative: nothing is done
    __nv_bfloat16* out;                      // [B, Hq, dv]
    int B, Hq, Hkv, dk, dv, window, sinks;
    float scale;
};

struct AppendArgs {
    const __nv_bfloat16 *k, *v;
    long long k_batch, k_row, v_batch, v_row;
    __nv_bfloat16 *k_cache, *v_cache;
    const int *start, *lengths;              // [B] or null (0 / T)
    int B, T, Hkv, dk, dv, window, sinks;
};

namespace window {

__host__ __device__ __forceinline__ long long cache_slot(long long p, int window, int sinks) {
    return p < sinks ? p : sinks + (p - sinks) % window;
}

// One warp's softmax state for one query: lane i holds the head's elements 2 i, 2 i + 1, 64 + 2 i, 65 + 2 i.
struct Row {
    float q[4], acc[4], m, l;
    __device__ void load(const __nv_bfloat16* p, int d, float scale, int lane) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = 64 * (i >> 1) + 2 * lane + (i & 1);
            q[i] = e < d ? __bfloat162float(p[e]) * scale : 0.0f;
            acc[i] = 0.0f;
        }
        m = -INFINITY;
        l = 0.0f;
    }
    __device__ void key(const __nv_bfloat16* k, const __nv_bfloat16* v, int dk, int dv, int lane) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = 64 * (i >> 1) + 2 * lane + (i & 1);
            if (e < dk) s = fmaf(q[i], __bfloat162float(k[e]), s);
        }
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
        const float mn = fmaxf(m, s), f = __expf(m - mn), p = __expf(s - mn);
        l = l * f + p;
        m = mn;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = 64 * (i >> 1) + 2 * lane + (i & 1);
            acc[i] = acc[i] * f + (e < dv ? p * __bfloat162float(v[e]) : 0.0f);
        }
    }
    __device__ void store(__nv_bfloat16* o, int dv, int lane) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = 64 * (i >> 1) + 2 * lane + (i & 1);
            if (e < dv) o[e] = __float2bfloat16_rn(acc[i] / l);
        }
    }
};

constexpr int kWarps = 8;

__global__ void __launch_bounds__(32 * kWarps)
window_attn_kernel(const WindowArgs a)
{
    const int lane = threadIdx.x & 31, i = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int h = blockIdx.y, b = blockIdx.z, hk = h / (a.Hq / a.Hkv);
    const int n = a.lengths ? min(max(a.lengths[b], 0), a.Tk) : a.Tk;
    const int t = a.Tk - a.Tq + i;
    if (i >= a.Tq || t >= n) return;
    Row r;
    r.load(a.q + b * a.q_batch + i * a.q_row + h * a.q_head, a.dk, a.scale, lane);
    const __nv_bfloat16* k = a.k + b * a.k_batch + hk * a.k_head;
    const __nv_bfloat16* v = a.v + b * a.v_batch + hk * a.v_head;
    const int lo = max(0, t - a.window + 1);
    for (int s = 0; s < min(a.sinks, lo); ++s) r.key(k + s * a.k_row, v + s * a.v_row, a.dk, a.dv, lane);
    for (int s = lo; s <= t; ++s) r.key(k + s * a.k_row, v + s * a.v_row, a.dk, a.dv, lane);
    r.store(a.out + (((long long)b * a.Tq + i) * a.Hq + h) * a.dv, a.dv, lane);
}

// One warp per query head and session.
__global__ void __launch_bounds__(32)
window_step_kernel(const StepArgs a)
{
    const int lane = threadIdx.x, h = blockIdx.x, b = blockIdx.y, G = a.Hq / a.Hkv, hk = h / G;
    const long long p = a.pos[b];
    if (p < 0) return;
    const int cap = a.window + a.sinks;
    const long long slot = cache_slot(p, a.window, a.sinks);
    const __nv_bfloat16* kn = a.k + b * a.k_batch + hk * a.dk;
    const __nv_bfloat16* vn = a.v + b * a.v_batch + hk * a.dv;
    __nv_bfloat16* kc = a.k_cache + ((long long)b * cap * a.Hkv + hk) * a.dk;
    __nv_bfloat16* vc = a.v_cache + ((long long)b * cap * a.Hkv + hk) * a.dv;
    const long long kr = (long long)a.Hkv * a.dk, vr = (long long)a.Hkv * a.dv;
    Row r;
    r.load(a.q + b * a.q_batch + (long long)h * a.dk, a.dk, a.scale, lane);
    const long long seen = p + 1 < cap ? p + 1 : cap;
    for (long long s = 0; s < seen; ++s) {
        const bool own = s == slot;                    // the slot is being written: read the new row itself
        r.key(own ? kn : kc + s * kr, own ? vn : vc + s * vr, a.dk, a.dv, lane);
    }
    if (h == hk * G) {
        for (int e = lane; e < a.dk; e += 32) kc[slot * kr + e] = kn[e];
        for (int e = lane; e < a.dv; e += 32) vc[slot * vr + e] = vn[e];
    }
    r.store(a.out + ((long long)b * a.Hq + h) * a.dv, a.dv, lane);
}

// Copies the tokens that stay visible (the sinks, and the window's last ones) into their
// slots.  Block x takes one token, or, when the call has more tokens than the cache slots,
// one slot and the last token that has its turn; either way a slot has one writer.
__global__ void __launch_bounds__(128)
window_append_kernel(const AppendArgs a)
{
    const int b = blockIdx.y, cap = a.window + a.sinks;
    const int n = a.lengths ? min(max(a.lengths[b], 0), a.T) : a.T;
    const long long start = a.start ? a.start[b] : 0, end = start + n;
    if (start < 0) return;
    long long p;
    if (a.T <= cap) {
        p = start + blockIdx.x;
        if (p >= end || (p >= a.sinks && p < end - a.window)) return;
    } else {
        const long long c = blockIdx.x;
        p = c < a.sinks ? c : end - 1 - ((end - 1 - c) % a.window + a.window) % a.window;
        if (p < c || p < start || p >= end) return;
    }
    const long long slot = (long long)b * cap + cache_slot(p, a.window, a.sinks), t = p - start;
    const int nk = a.Hkv * a.dk / 8, nv = a.Hkv * a.dv / 8;
    const uint4* ks = reinterpret_cast<const uint4*>(a.k + b * a.k_batch + t * a.k_row);
    const uint4* vs = reinterpret_cast<const uint4*>(a.v + b * a.v_batch + t * a.v_row);
    uint4* kd = reinterpret_cast<uint4*>(a.k_cache) + slot * nk;
    uint4* vd = reinterpret_cast<uint4*>(a.v_cache) + slot * nv;
    for (int i = threadIdx.x; i < nk; i += 128) kd[i] = __ldg(ks + i);
    for (int i = threadIdx.x; i < nv; i += 128) vd[i] = __ldg(vs + i);
}

}  // namespace window

cudaError_t launch_window(const WindowArgs& a, cudaStream_t stream)
{
    const dim3 grid((unsigned)((a.Tq + window::kWarps - 1) / window::kWarps), (unsigned)a.Hq, (unsigned)a.B);
    window::window_attn_kernel<<<grid, 32 * window::kWarps, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_window_step(const StepArgs& a, cudaStream_t stream)
{
    window::window_step_kernel<<<dim3((unsigned)a.Hq, (unsigned)a.B), 32, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_window_append(const AppendArgs& a, cudaStream_t stream)
{
    const long long cap = (long long)a.window + a.sinks, items = a.T <= cap ? a.T : cap;
    window::window_append_kernel<<<dim3((unsigned)items, (unsigned)a.B), 128, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn
