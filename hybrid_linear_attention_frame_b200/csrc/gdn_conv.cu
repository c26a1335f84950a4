// Causal depthwise convolution of width 2 to 4 with an optional SiLU, the short
// convolution that sits in front of a recurrent mixer (q, k, v of a delta rule, x of a
// selective scan):
//   y[b, t, c] = act(bias[c] + sum_{j < W} w[c, j] x[b, t - W + 1 + j, c]),
// rows before the call's first token taken from state_in (its last W - 1 inputs, oldest
// first; zeros without one).  state_out receives the last W - 1 inputs of each sequence.
//
// 2 W + 5 operations and two special functions (the SiLU) per element against two elements of
// traffic: bound by HBM, with the special-function unit busy for 0.7 of that time, so loads and
// arithmetic have to overlap.  A thread owns 4 channels, few enough that blocks of 128 threads share an
// SM, 6 at width 4 to 8 at width 2 in bf16 and 4 to 6 in float32 (8 channels a thread: 206 us against
// 108 us), and walks a stretch of tokens with the
// last W - 1 rows in registers; x is read once but for the W - 1 rows of halo per stretch, and the
// loads of 8 rows are issued before the first is used.  Channels are the fastest thread index, so a
// warp reads and writes whole lines of a row.
// 27,280 tokens of 4480 channels, width 4: bf16 99 us, 4.9 TB/s; float32 167 us, 5.9 TB/s.
#include "gdn_common.cuh"
#include "gdn_sm100.cuh"

namespace gdn {

struct ConvArgs {
    const void* x;
    const float* weight;       // [D, W]
    const float* bias;         // [D] or null
    const void* state_in;      // [B, W - 1, D] or null
    void* state_out;           // [B, W - 1, D] or null; may be state_in
    const int* lengths;        // [B] or null: rows at and past lengths[b] are padding
    void* out;                 // [B, T, D]
    long long x_batch, x_row;  // strides of x in elements
    int B, T, D;
    int stretch;               // set at launch
};

namespace conv {

constexpr int kThreads = 128;
// Tokens per thread: long stretches spare halo rows and weight loads, short ones fill the device (27,280
// tokens of 4480 channels: 103 us in stretches of 64, 132 us of 16; 333 tokens of 1024 channels: 10.3 us
// and 5.0 us; both before the weights came by vector loads).  Even the shortest is longer than the halo, so
// that only stretch 0 reads state_in and state_out may be the same memory.
constexpr int kMaxStretch = 64, kMinStretch = 8;
constexpr int V = 4;           // channels per thread

// Four channels as they lie in memory, and as two pairs of f32 in 64-bit registers, the form of the
// paired FMA.
template <typename IOT> struct Vec;
template <> struct Vec<__nv_bfloat16> {
    using Raw = uint2;
    __device__ static Raw zero() { return make_uint2(0, 0); }
    __device__ static uint64_t pair(const Raw& v, int i) {
        const uint32_t w = i == 0 ? v.x : v.y;
        return attn::f2pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    __device__ static Raw pack(const float (&f)[V]) {
        return make_uint2(sm100::pack_bf16x2(f[0], f[1]), sm100::pack_bf16x2(f[2], f[3]));
    }
};
template <> struct Vec<float> {
    using Raw = uint4;
    __device__ static Raw zero() { return make_uint4(0, 0, 0, 0); }
    __device__ static uint64_t pair(const Raw& v, int i) {
        return i == 0 ? attn::f2pack(__uint_as_float(v.x), __uint_as_float(v.y))
                      : attn::f2pack(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    __device__ static Raw pack(const float (&f)[V]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

// y / (1 + e^-y); the quotient far below 0 is 0
__device__ __forceinline__ float silu_f(float y) {
    return __fdividef(y, 1.0f + attn::ex2(-1.4426950408889634f * y));
}

// Batch: rows loaded at once, 8, or 1 for single tokens.
template <typename IOT, int W, bool SILU, int Batch>
__global__ void __launch_bounds__(kThreads)
causal_conv_kernel(const ConvArgs a)
{
    using Raw = typename Vec<IOT>::Raw;
    const int nvec = a.D / V;
    const int stretches = a.T > 0 ? (a.T - 1) / a.stretch + 1 : 1;   // T = 0 carries the state over
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (id >= (long long)nvec * stretches) return;
    const int b = blockIdx.y;
    const int s = (int)(id / nvec), c = (int)(id - (long long)s * nvec) * V;
    const int n = a.lengths ? min(max(a.lengths[b], 0), a.T) : a.T;
    const int t0 = s * a.stretch, t1 = min(n, t0 + a.stretch);
    const IOT* x = static_cast<const IOT*>(a.x) + b * a.x_batch + c;
    const IOT* st = a.state_in ? static_cast<const IOT*>(a.state_in) + (long long)b * (W - 1) * a.D + c : nullptr;

    // the row of token t; tokens before the call come from the carried state
    auto row = [&](int t) {
        if (t >= 0) return __ldg(reinterpret_cast<const Raw*>(x + t * a.x_row));
        if (st) return *reinterpret_cast<const Raw*>(st + (long long)(t + W - 1) * a.D);
        return Vec<IOT>::zero();
    };

    if (t0 < t1) {
        uint64_t w[W][V / 2], bias[V / 2], win[W - 1][V / 2];
        alignas(16) float wf[V * W];                                  // 4 W consecutive floats
#pragma unroll
        for (int i = 0; i < W; ++i)
            *reinterpret_cast<float4*>(wf + 4 * i) = __ldg(reinterpret_cast<const float4*>(a.weight + (long long)c * W) + i);
        const float4 bf = a.bias ? __ldg(reinterpret_cast<const float4*>(a.bias + c)) : make_float4(0, 0, 0, 0);
        bias[0] = attn::f2pack(bf.x, bf.y);
        bias[1] = attn::f2pack(bf.z, bf.w);
#pragma unroll
        for (int e = 0; e < V / 2; ++e)
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][e] = attn::f2pack(wf[2 * e * W + j], wf[(2 * e + 1) * W + j]);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const Raw v = row(t0 - (W - 1) + j);
#pragma unroll
            for (int e = 0; e < V / 2; ++e) win[j][e] = Vec<IOT>::pair(v, e);
        }
        IOT* o = static_cast<IOT*>(a.out) + ((long long)b * a.T + t0) * a.D + c;
#pragma unroll 1
        for (int t = t0; t < t1; t += Batch) {
            Raw in[Batch];
#pragma unroll
            for (int i = 0; i < Batch; ++i) in[i] = row(min(t + i, t1 - 1));
#pragma unroll
            for (int i = 0; i < Batch; ++i) {
                float r[V];
#pragma unroll
                for (int e = 0; e < V / 2; ++e) {
                    const uint64_t xe = Vec<IOT>::pair(in[i], e);
                    uint64_t y = bias[e];
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) y = attn::fma2(w[j][e], win[j][e], y);
                    y = attn::fma2(w[W - 1][e], xe, y);
#pragma unroll
                    for (int j = 0; j + 1 < W - 1; ++j) win[j][e] = win[j + 1][e];
                    win[W - 2][e] = xe;
                    attn::f2unpack(y, r[2 * e], r[2 * e + 1]);
                    if (SILU) {
                        r[2 * e] = silu_f(r[2 * e]);
                        r[2 * e + 1] = silu_f(r[2 * e + 1]);
                    }
                }
                if (t + i < t1) *reinterpret_cast<Raw*>(o) = Vec<IOT>::pack(r);
                o += a.D;
            }
        }
    }
    if (s == 0 && a.state_out) {
        Raw keep[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) keep[j] = row(n - (W - 1) + j);     // read before the state is written
        IOT* so = static_cast<IOT*>(a.state_out) + (long long)b * (W - 1) * a.D + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) *reinterpret_cast<Raw*>(so + (long long)j * a.D) = keep[j];
    }
}

template <typename IOT, int W, bool SILU>
void launch_w(const ConvArgs& a, dim3 grid, cudaStream_t stream)
{
    if (a.T > 1) causal_conv_kernel<IOT, W, SILU, 8><<<grid, kThreads, 0, stream>>>(a);
    else causal_conv_kernel<IOT, W, SILU, 1><<<grid, kThreads, 0, stream>>>(a);
}

}  // namespace conv

template <typename IOT>
cudaError_t launch_conv(const ConvArgs& a, int width, bool silu, cudaStream_t stream)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    ConvArgs r = a;
    auto items = [&]() { return (long long)(a.D / conv::V) * (a.T > 0 ? (a.T - 1) / r.stretch + 1 : 1); };
    r.stretch = conv::kMaxStretch;
    while (r.stretch > conv::kMinStretch && items() * a.B < 1536ll * sms) r.stretch /= 2;
    const long long blocks = (items() + conv::kThreads - 1) / conv::kThreads;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks, (unsigned)a.B);
    if (silu) {
        if (width == 2) conv::launch_w<IOT, 2, true>(r, grid, stream);
        else if (width == 3) conv::launch_w<IOT, 3, true>(r, grid, stream);
        else conv::launch_w<IOT, 4, true>(r, grid, stream);
    } else {
        if (width == 2) conv::launch_w<IOT, 2, false>(r, grid, stream);
        else if (width == 3) conv::launch_w<IOT, 3, false>(r, grid, stream);
        else conv::launch_w<IOT, 4, false>(r, grid, stream);
    }
    return cudaGetLastError();
}

}  // namespace gdn
