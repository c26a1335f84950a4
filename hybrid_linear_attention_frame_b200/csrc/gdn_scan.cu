// Selective state space scan.  Per batch entry and channel d, with N states:
//   delta_t = softplus(dt_t + dt_bias[d]),
//   h_t[n]  = exp(delta_t A[d, n]) h_{t-1}[n] + delta_t x_t B_t[n],
//   y_t     = (sum_n C_t[n] h_t[n] + skip[d] x_t) silu(z_t),
// h in fp32 from state_in to state_out, B_t and C_t shared by all channels.
//
// The work is one exponential per token, channel and state: at N = 16 one clock of an SM's
// special-function unit (16 a clock) per token and channel, against a third of a clock for
// the 8 bytes that the rows need from HBM.  So the layout serves that unit: everything that
// exists once per token and channel (softplus, the gate, conversions) is kept away from the
// threads that own the states.
//
// A CTA owns 16 channels of one batch entry.  Its four scan warps hold the states: 8 threads
// share a channel, N / 8 states each.  Its four helper warps walk the same tokens a tile of 64
// ahead: they read the rows with 16-byte loads (the next tile's into registers while this one
// is worked on), put delta, delta x, B and C into shared memory, and later turn the scan's sums
// into rows of y.  The two sides meet at named barriers, two buffers each way.
#include "gdn_common.cuh"
#include "gdn_sm100.cuh"

namespace gdn {

struct ScanArgs {
    const void *x, *dt, *z, *Bm, *Cm;                 // z may be null
    long long x_batch, x_row, dt_batch, dt_row, z_batch, z_row, b_batch, b_row, c_batch, c_row;
    const float *A, *skip, *dt_bias;                  // [D, N], [D] or null, [D] or null
    const float* state_in;                            // [B, D, N] or null
    float* state_out;                                 // [B, D, N] or null; may be state_in
    const int* lengths;                               // [B] or null
    void* y;                                          // [B, T, D]
    int B, T, D, N;
    bool softplus;
};

namespace scan {

constexpr float kLog2e = 1.4426950408889634f;

// log(1 + e^x) = max(x, 0) + log1p(u), u = e^-|x| in (0, 1], through
// log1p(u) = 2 artanh(s), s = u / (2 + u) <= 1/3, whose series s + s^3/3 + .. + s^13/13 leaves
// out less than 2e-8 of the value: relative accuracy holds where softplus is tiny.
__device__ __forceinline__ float softplus_series(float x) {
    const float u = attn::ex2(-fabsf(x) * kLog2e);
    const float s = __fdividef(u, 2.0f + u), q = s * s;
    float r = fmaf(q, 1.0f / 13.0f, 1.0f / 11.0f);
    r = fmaf(r, q, 1.0f / 9.0f);
    r = fmaf(r, q, 1.0f / 7.0f);
    r = fmaf(r, q, 1.0f / 5.0f);
    r = fmaf(r, q, 1.0f / 3.0f);
    r = fmaf(r, q, 1.0f);
    return fmaf(2.0f * s, r, fmaxf(x, 0.0f));
}

// v silu(g); the quotient of a gate far below 0 is 0
__device__ __forceinline__ float gated(float v, float g) { return v * __fdividef(g, 1.0f + attn::ex2(-g * kLog2e)); }

// Eight consecutive elements of a row.
template <typename IOT> struct Eight;
template <> struct Eight<__nv_bfloat16> {
    uint4 v;
    __device__ void load(const __nv_bfloat16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ float get(int i) const {
        const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
        return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
    }
    __device__ static void store(__nv_bfloat16* p, const float (&f)[8]) {
        *reinterpret_cast<uint4*>(p) = make_uint4(sm100::pack_bf16x2(f[0], f[1]), sm100::pack_bf16x2(f[2], f[3]),
                                                  sm100::pack_bf16x2(f[4], f[5]), sm100::pack_bf16x2(f[6], f[7]));
    }
};
template <> struct Eight<float> {
    float4 a, b;
    __device__ void load(const float* p) {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ void zero() { a = b = make_float4(0, 0, 0, 0); }
    __device__ float get(int i) const {
        const float4& q = i < 4 ? a : b;
        return (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
    }
    __device__ static void store(float* p, const float (&f)[8]) {
        reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
};

constexpr int kC = 16;                     // channels per CTA
constexpr int kL = 8;                      // threads per channel
constexpr int kTile = 64;                  // tokens per tile
constexpr int kScanThreads = kC * kL;      // 128: warps 0-3; the helpers are warps 4-7
constexpr int kThreads = 2 * kScanThreads;
static_assert(kScanThreads == kTile * 2, "a helper thread has one token and 8 channels of a tile");
constexpr int kDRow = kTile + 2;           // (delta, delta x) pairs per channel, padded off the banks
constexpr int kYRow = 20;                  // sums per token: 16 channels, padded so that 8 tokens x 4
                                           // channels, a warp's store, fall on 32 banks
enum { kFull = 1, kEmpty = 3, kYFull = 5, kYEmpty = 7 };   // named barriers, + buffer

template <int N> constexpr int smem_bytes() {
    return 2 * (kC * kDRow * 8 + kTile * 2 * N * 4 + kTile * kYRow * 4);
}

__device__ __forceinline__ void bar_arrive(int id) {
    asm volatile("bar.arrive %0, %1;" :: "r"(id), "n"(kThreads) : "memory");
}
__device__ __forceinline__ void bar_sync(int id) {
    asm volatile("bar.sync %0, %1;" :: "r"(id), "n"(kThreads) : "memory");
}

// S floats per thread from / to shared or global memory
template <int S> __device__ __forceinline__ void ld(float (&r)[S], const float* p) {
    if constexpr (S == 1) r[0] = *p;
    else if constexpr (S == 2) { const float2 v = *reinterpret_cast<const float2*>(p); r[0] = v.x; r[1] = v.y; }
    else {
#pragma unroll
        for (int i = 0; i < S; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + i);
            r[i] = v.x; r[i + 1] = v.y; r[i + 2] = v.z; r[i + 3] = v.w;
        }
    }
}

template <typename IOT, int N>
__global__ void __launch_bounds__(kThreads)
selective_scan_kernel(const ScanArgs a)
{
    constexpr int S = N / kL;
    extern __shared__ __align__(16) uint8_t smem[];
    float2* s_d = reinterpret_cast<float2*>(smem);                       // [2][kC][kDRow]
    float* s_bc = reinterpret_cast<float*>(s_d + 2 * kC * kDRow);        // [2][kTile][kL][B: S | C: S]
    float* s_y = s_bc + 2 * kTile * 2 * N;                               // [2][kTile][kYRow]
    const int b = blockIdx.y, c0 = blockIdx.x * kC;
    const int n = a.lengths ? min(max(a.lengths[b], 0), a.T) : a.T;
    const int tiles = (n + kTile - 1) / kTile;

    if (threadIdx.x < kScanThreads) {
        // ======================= the states =======================
        const int tid = threadIdx.x, l = tid % kL, ch = tid / kL, c = c0 + ch;
        const bool live = c < a.D;
        float h[S], A[S];
        const long long so = ((long long)b * a.D + c) * N + l * S;
#pragma unroll
        for (int i = 0; i < S; ++i) {
            h[i] = (live && a.state_in) ? a.state_in[so + i] : 0.0f;
            A[i] = live ? a.A[(long long)c * N + l * S + i] * kLog2e : 0.0f;
        }
        for (int k = 0; k < tiles; ++k) {
            const int buf = k & 1;
            const float2* d = s_d + (buf * kC + ch) * kDRow;
            const float* bc = s_bc + buf * kTile * 2 * N + l * 2 * S;
            float* y = s_y + buf * kTile * kYRow + ch;
            bar_sync(kFull + buf);
            if (k >= 2) bar_sync(kYEmpty + buf);
            const int groups = (min(kTile, n - k * kTile) + 7) / 8;
#pragma unroll 1
            for (int g = 0; g < groups; ++g) {
                float v[8];
#pragma unroll
                for (int t = 0; t < 8; t += 2) {
                    const float4 dd = *reinterpret_cast<const float4*>(d + g * 8 + t);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float de = u ? dd.z : dd.x, dx = u ? dd.w : dd.y;
                        float B[S], C[S];
                        ld<S>(B, bc + (g * 8 + t + u) * 2 * N);
                        ld<S>(C, bc + (g * 8 + t + u) * 2 * N + S);
                        float s = 0.0f;
#pragma unroll
                        for (int i = 0; i < S; ++i) {
                            h[i] = fmaf(attn::ex2(de * A[i]), h[i], dx * B[i]);
                            s = i == 0 ? h[i] * C[i] : fmaf(h[i], C[i], s);
                        }
                        v[t + u] = s;
                    }
                }
                // the 8 threads of a channel sum 8 tokens, one left with each: thread l ends with token l
#pragma unroll
                for (int w = 4; w > 0; w >>= 1) {
                    const bool up = (l & w) != 0;
#pragma unroll
                    for (int i = 0; i < w; ++i) {
                        const float keep = up ? v[i + w] : v[i], give = up ? v[i] : v[i + w];
                        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
                    }
                }
                y[(g * 8 + l) * kYRow] = v[0];
            }
            bar_arrive(kYFull + buf);
            if (k + 2 < tiles) bar_arrive(kEmpty + buf);
        }
        if (live && a.state_out) {
#pragma unroll
            for (int i = 0; i < S; ++i) a.state_out[so + i] = h[i];
        }
    } else {
        // ======================= rows in, rows out =======================
        const int tid = threadIdx.x - kScanThreads, row = tid >> 1, cv = 8 * (tid & 1), c = c0 + cv;
        const bool live = c < a.D;                                       // D is a multiple of 8
        const IOT* x = static_cast<const IOT*>(a.x) + b * a.x_batch + c;
        const IOT* dt = static_cast<const IOT*>(a.dt) + b * a.dt_batch + c;
        const IOT* z = a.z ? static_cast<const IOT*>(a.z) + b * a.z_batch + c : nullptr;
        const IOT* Bm = static_cast<const IOT*>(a.Bm) + b * a.b_batch;
        const IOT* Cm = static_cast<const IOT*>(a.Cm) + b * a.c_batch;
        IOT* y = static_cast<IOT*>(a.y) + (long long)b * a.T * a.D + c;
        constexpr int kBC = (kTile * N / 8 + kScanThreads - 1) / kScanThreads;   // 8-state pieces of B (and C) a thread
        float bias[8], skip[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            bias[e] = (live && a.dt_bias) ? a.dt_bias[c + e] : 0.0f;
            skip[e] = (live && a.skip) ? a.skip[c + e] : 0.0f;
        }
        Eight<IOT> rx, rd, rz, px, pz, rb[kBC], rc[kBC];
        auto fetch = [&](int k) {
            const int t = k * kTile + row;
            const bool on = live && t < n;
            rx.zero(); rd.zero(); rz.zero();
            if (on) {
                rx.load(x + t * a.x_row);
                rd.load(dt + t * a.dt_row);
                if (z) rz.load(z + t * a.z_row);
            }
#pragma unroll
            for (int i = 0; i < kBC; ++i) {
                const int p = tid + i * kScanThreads, pt = k * kTile + p / (N / 8), ps = 8 * (p % (N / 8));
                rb[i].zero(); rc[i].zero();
                if (p < kTile * N / 8 && pt < n) {
                    rb[i].load(Bm + pt * a.b_row + ps);
                    rc[i].load(Cm + pt * a.c_row + ps);
                }
            }
        };
        auto finish = [&](int k, const Eight<IOT>& fx, const Eight<IOT>& fz) {
            const int buf = k & 1, t = k * kTile + row;
            bar_sync(kYFull + buf);
            float f[8];
            ld<8>(f, s_y + (buf * kTile + row) * kYRow + cv);
            if (k + 2 < tiles) bar_arrive(kYEmpty + buf);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[e] = fmaf(skip[e], fx.get(e), f[e]);
                if (z) f[e] = gated(f[e], fz.get(e));
            }
            if (live && t < n) Eight<IOT>::store(y + (long long)t * a.D, f);
        };
        if (tiles > 0) fetch(0);
        for (int k = 0; k < tiles; ++k) {
            const int buf = k & 1;
            const bool on = live && k * kTile + row < n;
            if (k >= 2) bar_sync(kEmpty + buf);
            // padding leaves the state as it is: delta = 0, and B = C = 0 from fetch
            float2* d = s_d + (buf * kC + cv) * kDRow + row;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float de = rd.get(e) + bias[e];
                if (a.softplus) de = softplus_series(de);
                if (!on) de = 0.0f;
                d[e * kDRow] = make_float2(de, de * rx.get(e));
            }
#pragma unroll
            for (int i = 0; i < kBC; ++i) {
                const int p = tid + i * kScanThreads;
                if (p < kTile * N / 8) {
                    float* w = s_bc + (buf * kTile + p / (N / 8)) * 2 * N + (p % (N / 8)) * 16;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        w[(e / S) * 2 * S + e % S] = rb[i].get(e);
                        w[(e / S) * 2 * S + S + e % S] = rc[i].get(e);
                    }
                }
            }
            bar_arrive(kFull + buf);
            const Eight<IOT> cx = rx, cz = rz;
            if (k + 1 < tiles) fetch(k + 1);
            if (k > 0) finish(k - 1, px, pz);
            px = cx;
            pz = cz;
        }
        if (tiles > 0) finish(tiles - 1, px, pz);
    }
}

// The next token of every session: the states stream through once, so HBM bounds it (8 bytes
// per state).  A thread has 4 states of one channel; N / 4 threads sum a channel's output.
constexpr int kStepThreads = 256;

template <typename IOT, int N>
__global__ void __launch_bounds__(kStepThreads)
selective_scan_step_kernel(const ScanArgs a)
{
    constexpr int L = N / 4;
    const long long id = (long long)blockIdx.x * kStepThreads + threadIdx.x;
    const int l = (int)(id % L);
    const long long ch = id / L;
    const bool live = ch < a.D;
    const int c = live ? (int)ch : 0, b = blockIdx.y;
    const float4 A = *reinterpret_cast<const float4*>(a.A + (long long)c * N + 4 * l);
    const long long so = ((long long)b * a.D + c) * N + 4 * l;
    float4 h = live ? *reinterpret_cast<const float4*>(a.state_in + so) : make_float4(0, 0, 0, 0);
    const float x = to_f32(static_cast<const IOT*>(a.x)[b * a.x_batch + c]);
    float de = to_f32(static_cast<const IOT*>(a.dt)[b * a.dt_batch + c]) + (a.dt_bias ? a.dt_bias[c] : 0.0f);
    if (a.softplus) de = softplus_series(de);
    const IOT* Bm = static_cast<const IOT*>(a.Bm) + b * a.b_batch + 4 * l;
    const IOT* Cm = static_cast<const IOT*>(a.Cm) + b * a.c_batch + 4 * l;
    const float dx = de * x, d2 = de * kLog2e;
    h.x = fmaf(attn::ex2(d2 * A.x), h.x, dx * to_f32(Bm[0]));
    h.y = fmaf(attn::ex2(d2 * A.y), h.y, dx * to_f32(Bm[1]));
    h.z = fmaf(attn::ex2(d2 * A.z), h.z, dx * to_f32(Bm[2]));
    h.w = fmaf(attn::ex2(d2 * A.w), h.w, dx * to_f32(Bm[3]));
    float y = fmaf(h.x, to_f32(Cm[0]), fmaf(h.y, to_f32(Cm[1]), fmaf(h.z, to_f32(Cm[2]), h.w * to_f32(Cm[3]))));
#pragma unroll
    for (int k = L / 2; k > 0; k >>= 1) y += __shfl_xor_sync(0xffffffffu, y, k);
    if (!live) return;
    *reinterpret_cast<float4*>(a.state_out + so) = h;
    if (l == 0) {
        if (a.skip) y = fmaf(a.skip[c], x, y);
        if (a.z) y = gated(y, to_f32(static_cast<const IOT*>(a.z)[b * a.z_batch + c]));
        static_cast<IOT*>(a.y)[(long long)b * a.D + c] = from_f32<IOT>(y);
    }
}

template <typename IOT, int N>
cudaError_t launch(const ScanArgs& a, bool step, cudaStream_t stream)
{
    if (step) {
        const long long threads = (long long)a.D * (N / 4);
        const dim3 grid((unsigned)((threads + kStepThreads - 1) / kStepThreads), (unsigned)a.B);
        selective_scan_step_kernel<IOT, N><<<grid, kStepThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    if (smem_bytes<N>() > 48 * 1024) {     // (a per-device setting of the current context: set on every call)
        const cudaError_t e = cudaFuncSetAttribute(selective_scan_kernel<IOT, N>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<N>());
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)((a.D + kC - 1) / kC), (unsigned)a.B);
    selective_scan_kernel<IOT, N><<<grid, kThreads, smem_bytes<N>(), stream>>>(a);
    return cudaGetLastError();
}

}  // namespace scan

// `step`: T = 1 with the state in place.
template <typename IOT>
cudaError_t launch_scan(const ScanArgs& a, bool step, cudaStream_t stream)
{
    if (a.N == 8) return scan::launch<IOT, 8>(a, step, stream);
    if (a.N == 16) return scan::launch<IOT, 16>(a, step, stream);
    if (a.N == 32) return scan::launch<IOT, 32>(a, step, stream);
    return scan::launch<IOT, 64>(a, step, stream);
}

}  // namespace gdn
