// Selective state space scan.  Per batch entry and channel d, with N states:
//   delta_t = softplus(dt_t + dt_bias[d]),
//   h_t[n]  = exp(delta_t A[d, n]) h_{t-1}[n] + delta_t x_t B_t[n],
//   y_t     = (sum_n C_t[n] h_t[n] + D[d] x_t) silu(z_t),
// h in fp32 from state_in to state_out, B_t and C_t shared by all channels.
//
// One exponential per token, channel and state is the work (one per SM and clock for
// N = 16, three times what HBM needs for the rows), so the special-function unit bounds
// it.  L threads share a channel, each with S = N / L states in registers; a CTA owns
// 128 / L channels of one batch entry and walks the tokens in tiles.
#include "gdn_common.cuh"

namespace gdn {

struct ScanArgs {
    const void *x, *dt, *z, *Bm, *Cm;                 // z may be null
    long long x_batch, x_row, dt_batch, dt_row, z_batch, z_row, b_batch, b_row, c_batch, c_row;
    const float *A, *skip, *dt_bias;                    // [D, N], [D] or null, [D] or null
    const float* state_in;                            // [B, D, N] or null
    float* state_out;                                 // [B, D, N] or null; may be state_in
    const int* lengths;                               // [B] or null
    void* y;                                          // [B, T, D]
    int B, T, D, N;
    bool softplus;
};

namespace scan {

constexpr int kThreads = 128;
constexpr int kTile = 32;

template <typename IOT, int S, int L>
__global__ void __launch_bounds__(kThreads)
selective_scan_kernel(const ScanArgs a)
{
    constexpr int N = S * L, C = kThreads / L;
    __shared__ float2 s_d[kTile][C];                  // delta, delta x
    __shared__ float s_y[kTile][C];
    __shared__ float s_B[kTile][N], s_C[kTile][N];
    const int b = blockIdx.y, c0 = blockIdx.x * C;
    const int tid = threadIdx.x, l = tid % L, ch = tid / L;
    const int c = c0 + ch;
    const bool live = c < a.D;
    const int n = a.lengths ? min(max(a.lengths[b], 0), a.T) : a.T;
    const IOT* x = static_cast<const IOT*>(a.x) + b * a.x_batch;
    const IOT* dt = static_cast<const IOT*>(a.dt) + b * a.dt_batch;
    const IOT* z = a.z ? static_cast<const IOT*>(a.z) + b * a.z_batch : nullptr;
    const IOT* Bm = static_cast<const IOT*>(a.Bm) + b * a.b_batch;
    const IOT* Cm = static_cast<const IOT*>(a.Cm) + b * a.c_batch;

    float h[S], A[S];
    const long long so = ((long long)b * a.D + c) * N + l * S;
#pragma unroll
    for (int i = 0; i < S; ++i) {
        h[i] = (live && a.state_in) ? a.state_in[so + i] : 0.0f;
        A[i] = live ? a.A[(long long)c * N + l * S + i] * 1.4426950408889634f : 0.0f;
    }
    for (int t0 = 0; t0 < n; t0 += kTile) {
        const int m = min(kTile, n - t0);
        for (int i = tid; i < m * C; i += kThreads) {
            const int t = i / C, cc = i % C;
            float2 v = make_float2(0.0f, 0.0f);
            if (c0 + cc < a.D) {
                float d = to_f32(dt[(t0 + t) * a.dt_row + c0 + cc]) + (a.dt_bias ? a.dt_bias[c0 + cc] : 0.0f);
                if (a.softplus) d = softplus_f(d);
                v = make_float2(d, d * to_f32(x[(t0 + t) * a.x_row + c0 + cc]));
            }
            s_d[t][cc] = v;
        }
        for (int i = tid; i < m * N; i += kThreads) {
            s_B[i / N][i % N] = to_f32(Bm[(t0 + i / N) * a.b_row + i % N]);
            s_C[i / N][i % N] = to_f32(Cm[(t0 + i / N) * a.c_row + i % N]);
        }
        __syncthreads();
        for (int t = 0; t < m; ++t) {
            const float2 v = s_d[t][ch];
            float y = 0.0f;
#pragma unroll
            for (int i = 0; i < S; ++i) {
                h[i] = fmaf(exp2f(v.x * A[i]), h[i], v.y * s_B[t][l * S + i]);
                y = fmaf(h[i], s_C[t][l * S + i], y);
            }
#pragma unroll
            for (int k = L / 2; k > 0; k >>= 1) y += __shfl_xor_sync(0xffffffffu, y, k);
            if (l == 0) s_y[t][ch] = y;
        }
        __syncthreads();
        for (int i = tid; i < m * C; i += kThreads) {
            const int t = i / C, cc = i % C;
            if (c0 + cc >= a.D) continue;
            float y = s_y[t][cc];
            if (a.skip) y = fmaf(a.skip[c0 + cc], to_f32(x[(t0 + t) * a.x_row + c0 + cc]), y);
            if (z) {
                const float g = to_f32(z[(t0 + t) * a.z_row + c0 + cc]);
                y *= g / (1.0f + expf(-g));
            }
            static_cast<IOT*>(a.y)[((long long)b * a.T + t0 + t) * a.D + c0 + cc] = from_f32<IOT>(y);
        }
        __syncthreads();
    }
    if (live && a.state_out) {
#pragma unroll
        for (int i = 0; i < S; ++i) a.state_out[so + i] = h[i];
    }
}

template <typename IOT, int S, int L>
void launch(const ScanArgs& a, cudaStream_t stream)
{
    constexpr int C = kThreads / L;
    selective_scan_kernel<IOT, S, L><<<dim3((unsigned)((a.D + C - 1) / C), (unsigned)a.B), kThreads, 0, stream>>>(a);
}

}  // namespace scan

template <typename IOT>
cudaError_t launch_scan(const ScanArgs& a, cudaStream_t stream)
{
    if (a.N == 8) scan::launch<IOT, 2, 4>(a, stream);
    else if (a.N == 16) scan::launch<IOT, 2, 8>(a, stream);
    else if (a.N == 32) scan::launch<IOT, 4, 8>(a, stream);
    else scan::launch<IOT, 4, 16>(a, stream);
    return cudaGetLastError();
}

}  // namespace gdn
