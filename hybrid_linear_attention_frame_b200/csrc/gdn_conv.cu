// Causal depthwise convolution of width 2 to 4 with an optional SiLU, the short
// convolution that sits in front of a recurrent mixer (q, k, v of a delta rule, x of a
// selective scan):
//   y[b, t, c] = act(bias[c] + sum_{j < W} w[c, j] x[b, t - W + 1 + j, c]),
// rows before the call's first token taken from state_in (its last W - 1 inputs, oldest
// first; zeros without one).  state_out receives the last W - 1 inputs of each sequence.
//
// 2 W + 5 operations per element against 2 elements of traffic: bound by HBM.  A thread
// owns one 16-byte vector of channels and walks kStretch tokens with the last W - 1 rows in
// registers, so x is read once but for the W - 1 rows of halo per stretch; the loads of
// kBatch rows are issued before the first is used.  Channels are the fastest thread index,
// so a warp reads and writes 512 contiguous bytes of a row.
#include "gdn_common.cuh"

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
};

namespace conv {

constexpr int kThreads = 128;
constexpr int kStretch = 16;   // tokens per thread; a stretch is longer than the halo, so that only
                               // stretch 0 reads state_in and state_out may be the same memory
constexpr int kBatch = 8;

template <typename IOT> struct Vec {
    static constexpr int n = 16 / sizeof(IOT);
    union { uint4 raw; IOT e[n]; };
    __device__ Vec() {}
};

__device__ __forceinline__ float silu_f(float y) { return y / (1.0f + __expf(-y)); }

template <typename IOT, int W, bool SILU>
__global__ void __launch_bounds__(kThreads)
causal_conv_kernel(const ConvArgs a)
{
    constexpr int V = Vec<IOT>::n;
    const int nvec = a.D / V;
    const int stretches = a.T > 0 ? (a.T - 1) / kStretch + 1 : 1;   // T = 0 carries the state over
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (id >= (long long)nvec * stretches) return;
    const int b = blockIdx.y;
    const int s = (int)(id / nvec), c = (int)(id - (long long)s * nvec) * V;
    const int n = a.lengths ? min(max(a.lengths[b], 0), a.T) : a.T;
    const int t0 = s * kStretch, t1 = min(n, t0 + kStretch);
    const IOT* x = static_cast<const IOT*>(a.x) + b * a.x_batch + c;
    const IOT* st = a.state_in ? static_cast<const IOT*>(a.state_in) + (long long)b * (W - 1) * a.D + c : nullptr;

    // the row of token t; tokens before the call come from the carried state
    auto row = [&](int t) {
        Vec<IOT> v;
        if (t >= 0) v.raw = *reinterpret_cast<const uint4*>(x + t * a.x_row);
        else if (st) v.raw = *reinterpret_cast<const uint4*>(st + (long long)(t + W - 1) * a.D);
        else v.raw = make_uint4(0, 0, 0, 0);
        return v;
    };

    if (t0 < t1) {
        float w[V][W], bias[V], win[W - 1][V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            bias[e] = a.bias ? __ldg(a.bias + c + e) : 0.0f;
#pragma unroll
            for (int j = 0; j < W; ++j) w[e][j] = __ldg(a.weight + (long long)(c + e) * W + j);
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const Vec<IOT> v = row(t0 - (W - 1) + j);
#pragma unroll
            for (int e = 0; e < V; ++e) win[j][e] = to_f32(v.e[e]);
        }
        IOT* o = static_cast<IOT*>(a.out) + ((long long)b * a.T + t0) * a.D + c;
        for (int t = t0; t < t1; t += kBatch) {
            Vec<IOT> in[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (t + i < t1) in[i] = row(t + i);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (t + i >= t1) break;
                Vec<IOT> r;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float xe = to_f32(in[i].e[e]);
                    float y = bias[e];
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) y = fmaf(w[e][j], win[j][e], y);
                    y = fmaf(w[e][W - 1], xe, y);
#pragma unroll
                    for (int j = 0; j + 1 < W - 1; ++j) win[j][e] = win[j + 1][e];
                    win[W - 2][e] = xe;
                    r.e[e] = from_f32<IOT>(SILU ? silu_f(y) : y);
                }
                *reinterpret_cast<uint4*>(o) = r.raw;
                o += a.D;
            }
        }
    }
    if (s == 0 && a.state_out) {
        Vec<IOT> keep[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) keep[j] = row(n - (W - 1) + j);     // read before the state is written
        IOT* so = static_cast<IOT*>(a.state_out) + (long long)b * (W - 1) * a.D + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) *reinterpret_cast<uint4*>(so + (long long)j * a.D) = keep[j].raw;
    }
}

template <typename IOT, int W>
void launch_w(const ConvArgs& a, bool silu, dim3 grid, cudaStream_t stream)
{
    if (silu) causal_conv_kernel<IOT, W, true><<<grid, kThreads, 0, stream>>>(a);
    else causal_conv_kernel<IOT, W, false><<<grid, kThreads, 0, stream>>>(a);
}

}  // namespace conv

template <typename IOT>
cudaError_t launch_conv(const ConvArgs& a, int width, bool silu, cudaStream_t stream)
{
    const int stretches = a.T > 0 ? (a.T - 1) / conv::kStretch + 1 : 1;
    const long long items = (long long)(a.D / conv::Vec<IOT>::n) * stretches;
    const long long blocks = (items + conv::kThreads - 1) / conv::kThreads;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks, (unsigned)a.B);
    if (width == 2) conv::launch_w<IOT, 2>(a, silu, grid, stream);
    else if (width == 3) conv::launch_w<IOT, 3>(a, silu, grid, stream);
    else conv::launch_w<IOT, 4>(a, silu, grid, stream);
    return cudaGetLastError();
}

}  // namespace gdn
