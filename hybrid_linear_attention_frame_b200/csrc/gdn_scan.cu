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
// share a channel, N / 8 states each.  Its eight helper warps walk the same tokens a tile of 128
// ahead: they read the rows with 16-byte loads (the next tile's into registers while this one
// is worked on), put delta, delta x, B and C into shared memory, and later turn the scan's sums
// into rows of y.  The two sides meet at named barriers, two buffers each way.
//
// A step of one CTA's 16 channels (N = 16) takes 20 clocks of the special-function unit and about 27 of
// shared memory (loads and shuffles); one CTA alone on an SM needs 45, two 38 each.  27,280 tokens of
// 2240 channels: 660 us, 1.5 T exponentials a second; N = 64: 2.4 T.
//
// Where channels and batch entries leave SMs idle, the CTAs of a cluster cut the sequence between
// them.  Each first runs its segment from a zero state without outputs, which gives the segment's
// own end state E and the sum of its deltas (the segment decays what enters it by exp(A sum)); they
// read each other's through distributed shared memory, so that each knows the state that enters its
// segment, and the segments then run in full.  Twice the exponentials for up to 8 times the SMs.
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
constexpr float kLog2eLow = (float)(1.4426950408889634 - (double)kLog2e);

// log(1 + e^x) = max(x, 0) + log1p(u), u = e^-|x| in (0, 1], through
// log1p(u) = 2 artanh(s), s = u / (2 + u) <= 1/3, whose series s + s^3/3 + .. + s^13/13 leaves
// out less than 2e-8 of the value: relative accuracy holds where softplus is tiny.  There it is u
// itself, whose exponent's rounding error (|x| 2^-24 of u) is taken along as `low`.  u is 0 in float
// from |x| = 104 on; the bound keeps e finite there, since low would be inf - inf: the lowest value
// of a type and -inf, which mask a token, give 0.  (A select, so that NaN stays NaN.)
__device__ __forceinline__ float softplus_series(float x) {
    const float ax = fabsf(x) > 200.0f ? 200.0f : fabsf(x);
    const float e = -ax * kLog2e;
    const float low = fmaf(-ax, kLog2e, -e) - ax * kLog2eLow;
    float u = attn::ex2(e);
    u = fmaf(u, low * 0.69314718f, u);
    const float s = __fdividef(u, 2.0f + u), q = s * s;
    float r = fmaf(q, 1.0f / 13.0f, 1.0f / 11.0f);
    r = fmaf(r, q, 1.0f / 9.0f);
    r = fmaf(r, q, 1.0f / 7.0f);
    r = fmaf(r, q, 1.0f / 5.0f);
    r = fmaf(r, q, 1.0f / 3.0f);
    r = fmaf(r, q, 1.0f);
    return fmaf(2.0f * s, r, fmaxf(x, 0.0f));
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// a within the finite floats (NaN as it is).  Of A, so that a step of 0 times it is 0 also where the decay
// is unbounded: padding and masked tokens leave the state as it is, any other step forgets all of it.
__device__ __forceinline__ float clamp_finite(float a) {
    constexpr float kTop = 3.4028235e38f;
    return a < -kTop ? -kTop : a > kTop ? kTop : a;
}

// v silu(g); the quotient of a gate far below 0 is 0
__device__ __forceinline__ float gated(float v, float g) { return v * __fdividef(g, 1.0f + attn::ex2(-g * kLog2e)); }

// One state over one token in the float32 mode, e^x h + b.  The hardware's exponential reads low by 1e-8
// to 3e-8 on average below 0, which a memory of a thousand tokens sums up to a hundred roundings; so for
// |x| <= 1/8 the result is h + ((e^x - 1) h + b) with the Taylor polynomial of e^x - 1 (what it leaves out
// is below 5e-8 of itself).  Beyond that a memory is short; and an infinite h, where the difference form
// is inf - inf, takes the plain one too.
__device__ __forceinline__ float exact_step(float x, float h, float b) {
    float p = fmaf(x, 1.0f / 120.0f, 1.0f / 24.0f);
    p = fmaf(p, x, 1.0f / 6.0f);
    p = fmaf(p, x, 0.5f);
    p = fmaf(p, x, 1.0f) * x;
    const float near = h + fmaf(p, h, b), far = fmaf(attn::ex2(x * kLog2e), h, b);
    float r;                               // a select, not a branch: lanes differ (47 us against 20 us, 3 x 517 tokens)
    asm("{\n\t.reg .pred q;\n\tsetp.le.f32 q, %1, 0f3e000000;\n\tsetp.lt.and.f32 q, %4, 0f7f800000, q;\n\t"
        "selp.f32 %0, %2, %3, q;\n\t}"
        : "=f"(r) : "f"(fabsf(x)), "f"(near), "f"(far), "f"(fabsf(h)));
    return r;
}

// Four consecutive elements of a row, 8- or 16-byte aligned.
__device__ __forceinline__ float4 four(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 four(const __nv_bfloat16* p) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xffff0000u));
}

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
constexpr int kTile = 128;                 // tokens per tile
constexpr int kScanThreads = kC * kL;      // warps 0-3
constexpr int kHelpers = 2 * kTile;        // warps 4-11: a helper has one token and 8 channels of a tile
constexpr int kThreads = kScanThreads + kHelpers;
constexpr int kDRow = kTile + 2;           // (delta, delta x) per channel, padded off the banks
constexpr int kYRow = 20;                  // sums per token: 16 channels, padded so that 8 tokens x 4
                                           // channels, a warp's store, fall on 32 banks
enum { kFull = 1, kEmpty = 3, kYFull = 5, kYEmpty = 7 };   // named barriers, + buffer

template <int N> constexpr int smem_bytes() {
    return 2 * (kC * kDRow * 8 + kTile * 2 * N * 4 + kTile * kYRow * 4) + (kC * N + kC) * 4;
}

__device__ __forceinline__ void bar_arrive(int id) {
    asm volatile("bar.arrive %0, %1;" :: "r"(id), "n"(kThreads) : "memory");
}
__device__ __forceinline__ void bar_sync(int id) {
    asm volatile("bar.sync %0, %1;" :: "r"(id), "n"(kThreads) : "memory");
}

// B and C of a tile: a row of 2 N floats per token, in units of 16 bytes.  Thread l of a channel reads
//   S = 1: half a unit (B, C);   S = 2: a unit (B, B, C, C);
//   S = 4, 8: units of B, then of C, the j-th of every thread side by side,
// so that the 8 threads' units are one contiguous line; and the rows are swizzled so that the helpers'
// stores, a few rows at a time, fall on all banks too.
template <int S> __device__ __forceinline__ constexpr int unit_at(int t, int unit) {
    return S == 1 ? unit ^ ((t >> 1) & 3) : S == 2 ? unit ^ (t & 3) : S == 4 ? unit ^ (t & 1) : unit;
}

// What a thread needs of two tokens: (delta, delta x) of each, S values of B and S of C as pairs of f32
// in 64-bit registers.  The loads are written out so that they stay where they are put, some tokens
// ahead of their use.
template <int S> struct Tokens {
    static constexpr int P = S > 1 ? S / 2 : 1;
    float de[2], dx[2];
    uint64_t B[2][P], C[2][P];
    // d: this channel's pairs from the first token on, bc: its row; t: the token within its 8
    __device__ void load(uint32_t d, uint32_t bc, int t, int l) {
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(de[0]), "=f"(dx[0]), "=f"(de[1]), "=f"(dx[1]) : "r"(d));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t row = bc + 8 * (S * kL) * k;
            if constexpr (S == 1) {
                asm volatile("ld.shared.b64 %0, [%1];"
                             : "=l"(B[k][0]) : "r"(row + 16 * unit_at<1>(t + k, l >> 1) + 8 * (l & 1)));
            } else if constexpr (S == 2) {
                lds(row + 16 * unit_at<2>(t + k, l), B[k][0], C[k][0]);
            } else {
#pragma unroll
                for (int j = 0; j < S / 4; ++j) {
                    lds(row + 16 * (8 * j + unit_at<S>(t + k, l)), B[k][2 * j], B[k][2 * j + 1]);
                    lds(row + 16 * (8 * (S / 4 + j) + unit_at<S>(t + k, l)), C[k][2 * j], C[k][2 * j + 1]);
                }
            }
        }
    }
    __device__ static void lds(uint32_t a, uint64_t& x, uint64_t& y) {
        asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "r"(a));
    }
};

// S states of one channel, in pairs for the paired FMA.
template <int S, bool Exact> struct States {
    static constexpr int P = S > 1 ? S / 2 : 1;
    static constexpr float kUnit = Exact ? 1.0f : kLog2e;              // of A
    uint64_t h[P], A[P];
    __device__ void init(const float* a, const float* h0) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int j = S > 1 ? 2 * i + 1 : 0;
            A[i] = a ? attn::f2pack(clamp_finite(a[2 * i] * kUnit), clamp_finite(a[j] * kUnit)) : 0ull;
            h[i] = h0 ? attn::f2pack(h0[2 * i], h0[j]) : 0ull;
        }
    }
    // one token; returns this thread's part of C . h
    __device__ float step(const Tokens<S>& t, int k) {
        float s0, s1;
        if constexpr (S == 1) {
            float B, C, a1, hv, _;
            attn::f2unpack(t.B[k][0], B, C);
            attn::f2unpack(A[0], a1, _);
            attn::f2unpack(h[0], hv, _);
            hv = Exact ? exact_step(t.de[k] * a1, hv, t.dx[k] * B) : fmaf(attn::ex2(t.de[k] * a1), hv, t.dx[k] * B);
            h[0] = attn::f2pack(hv, hv);
            return hv * C;
        }
        const uint64_t de = attn::f2pack(t.de[k], t.de[k]), dx = attn::f2pack(t.dx[k], t.dx[k]);
        uint64_t s = 0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            attn::f2unpack(mul2(de, A[i]), s0, s1);
            if constexpr (Exact) {
                float h0, h1, b0, b1;
                attn::f2unpack(h[i], h0, h1);
                attn::f2unpack(mul2(dx, t.B[k][i]), b0, b1);
                h[i] = attn::f2pack(exact_step(s0, h0, b0), exact_step(s1, h1, b1));
            } else {
                h[i] = attn::fma2(attn::f2pack(attn::ex2(s0), attn::ex2(s1)), h[i], mul2(dx, t.B[k][i]));
            }
            s = i == 0 ? mul2(h[i], t.C[k][i]) : attn::fma2(h[i], t.C[k][i], s);
        }
        attn::f2unpack(s, s0, s1);
        return s0 + s1;
    }
    __device__ void clear() {
#pragma unroll
        for (int i = 0; i < P; ++i) h[i] = 0ull;
    }
    // One state over a whole segment, e^x h + end.  The recurrence keeps a zero (or infinite) state as it is
    // however much the segment grows (or shrinks) it; with the factor of the whole segment that would be 0 inf.
    __device__ static float over(float x, float h, float end) {
        const float r = Exact ? exact_step(x, h, end) : fmaf(attn::ex2(x), h, end);
        return (h == 0.0f || fabsf(h) == INFINITY) ? h + end : r;
    }
    // a whole segment: its sum of deltas and its own end state
    __device__ void pass(float sum, const float (&end)[S]) {
        float a0, a1, h0, h1;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int j = S > 1 ? 2 * i + 1 : 0;
            attn::f2unpack(A[i], a0, a1);
            attn::f2unpack(h[i], h0, h1);
            h[i] = attn::f2pack(over(sum * a0, h0, end[2 * i]), over(sum * a1, h1, end[j]));
        }
    }
    __device__ void store(float* o) const {
        float a, b;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            attn::f2unpack(h[i], a, b);
            o[2 * i] = a;
            if (S > 1) o[2 * i + 1] = b;
        }
    }
};

// One round of the sum over a channel's 8 threads: of 2 w tokens' parts each thread keeps w, those of
// its own bit w, with its partner's added; after rounds 4, 2, 1 thread l has token l's sum.
template <int W> __device__ __forceinline__ void sum_round(float (&v)[8], int l) {
    const bool up = (l & W) != 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const float keep = up ? v[i + W] : v[i], give = up ? v[i] : v[i + W];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, W);
    }
}

// CTAs that an SM holds: two in 80 registers a thread in bf16 at N 8 and 16 (3 sequences of 517 tokens, 1128
// channels, N 8: 14.0 us, one at a time 16.0; 27,280 tokens of 2240 channels, whose 140 CTAs have an SM each
// anyway: 660 and 645 us).  float32 rows take 148 registers; in 80 they spill (517 tokens: 20.5 us against
// 18.7; 2640 tokens of 2240 channels, N 16: 115 against 87).
template <typename IOT, int N> constexpr int resident() { return N <= 16 && sizeof(IOT) == 2 ? 2 : 1; }

// Cut: the clusters' CTAs share a sequence (a kernel of its own, since the uncut one is slower by 9 %
// with that code beside it).
template <typename IOT, int N, bool Cut>
__global__ void __launch_bounds__(kThreads, resident<IOT, N>())
selective_scan_kernel(const ScanArgs a)
{
    constexpr int S = N / kL;
    static_assert(kL == 8 && kC * kL == kScanThreads, "thread l of a channel");
    constexpr int kRing = 2;                                             // pairs of tokens
    extern __shared__ __align__(16) uint8_t smem[];
    float2* s_d = reinterpret_cast<float2*>(smem);                       // [2][kC][kDRow]
    float* s_bc = reinterpret_cast<float*>(s_d + 2 * kC * kDRow);        // [2][kTile][kL][B: S | C: S]
    float* s_y = s_bc + 2 * kTile * 2 * N;                               // [2][kTile][kYRow]
    float* s_end = s_y + 2 * kTile * kYRow;                              // [kC][N] end states, [kC] sums of delta
    const int X = Cut ? (int)sm100::cluster_size() : 1, rank = Cut ? (int)sm100::cluster_rank() : 0;
    const int b = blockIdx.y, c0 = (int)(blockIdx.x / (unsigned)X) * kC;
    const int len = a.lengths ? min(max(a.lengths[b], 0), a.T) : a.T;
    // this CTA's segment: tokens t0 .. n - 1
    const int seg = ((len + X - 1) / X + kTile - 1) / kTile * kTile;
    const int t0 = Cut ? min(rank * seg, len) : 0, n = Cut ? min(t0 + seg, len) : len;
    const int tiles = (n - t0 + kTile - 1) / kTile;

    if (threadIdx.x < kScanThreads) {
        // ======================= the states =======================
        const int tid = threadIdx.x, l = tid % kL, ch = tid / kL, c = c0 + ch;
        const bool live = c < a.D;
        States<S, sizeof(IOT) == 4> s;
        const long long so = ((long long)b * a.D + c) * N + l * S;
        s.init(live ? a.A + (long long)c * N + l * S : nullptr, (live && a.state_in) ? a.state_in + so : nullptr);
        if constexpr (Cut) {
            const States<S, sizeof(IOT) == 4> enter = s;
            s.clear();
            float sum = 0.0f, lost = 0.0f;                               // of delta, compensated
            for (int k = 0; k < tiles; ++k) {
                const int buf = k & 1;
                const uint32_t d = sm100::smem_u32(s_d + (buf * kC + ch) * kDRow);
                const uint32_t bc = sm100::smem_u32(s_bc + buf * kTile * 2 * N);
                bar_sync(kFull + buf);
                Tokens<S> ring[kRing];
#pragma unroll
                for (int u = 0; u < kRing - 1; ++u) ring[u].load(d + 16 * u, bc + 16 * N * u, 2 * u, l);
                const int groups = (min(kTile, n - t0 - k * kTile) + 7) / 8;
#pragma unroll 1
                for (int g = 0; g < groups; ++g) {
                    float part = 0.0f;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int ahead = u + kRing - 1;
                        ring[ahead % kRing].load(d + 16 * (4 * g + ahead), bc + 16 * N * (4 * g + ahead), 2 * ahead & 7, l);
                        const Tokens<S>& now = ring[u % kRing];
                        part += now.de[0] + now.de[1];
                        (void)s.step(now, 0);
                        (void)s.step(now, 1);
                    }
                    const float add = part - lost, next = sum + add;
                    lost = fabsf(next) < INFINITY ? (next - sum) - add : 0.0f;  // (of a sum past the range: nothing)
                    sum = next;
                }
                if (k + 2 < tiles) bar_arrive(kEmpty + buf);
            }
            sum = clamp_finite(sum);                                             // (A = 0 keeps the state all the same)
            s.store(s_end + ch * N + l * S);
            if (l == 0) s_end[kC * N + ch] = sum;
            sm100::cluster_sync();
            s = enter;
            const uint32_t end = sm100::smem_u32(s_end);
            for (int r = 0; r < rank; ++r) {
                float e[S];
#pragma unroll
                for (int i = 0; i < S; ++i) e[i] = sm100::ld_remote(end + 4 * (ch * N + l * S + i), r);
                s.pass(sm100::ld_remote(end + 4 * (kC * N + ch), r), e);
            }
            sm100::cluster_sync();                                              // no one reads s_end any more
        }
        for (int k = 0; k < tiles; ++k) {
            const int buf = k & 1;
            const uint32_t d = sm100::smem_u32(s_d + (buf * kC + ch) * kDRow);
            const uint32_t bc = sm100::smem_u32(s_bc + buf * kTile * 2 * N);
            float* y = s_y + buf * kTile * kYRow + ch + l * kYRow;
            bar_sync(kFull + buf);
            if (k >= 2) bar_sync(kYEmpty + buf);
            // A ring of tokens, loaded kRing - 1 ahead (past the tile's end: other data of this block's
            // shared memory, not used); the sum of one group of 8 goes on beside the next group's tokens.
            Tokens<S> ring[kRing];
#pragma unroll
            for (int u = 0; u < kRing - 1; ++u) ring[u].load(d + 16 * u, bc + 16 * N * u, 2 * u, l);
            const int groups = (min(kTile, n - t0 - k * kTile) + 7) / 8;
            float last[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 1
            for (int g = 0; g < groups; ++g) {
                float v[8];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int ahead = u + kRing - 1;
                    ring[ahead % kRing].load(d + 16 * (4 * g + ahead), bc + 16 * N * (4 * g + ahead), 2 * ahead & 7, l);
                    v[2 * u] = s.step(ring[u % kRing], 0);
                    v[2 * u + 1] = s.step(ring[u % kRing], 1);
                    if (u == 0) sum_round<4>(last, l);
                    if (u == 1) sum_round<2>(last, l);
                    if (u == 2) sum_round<1>(last, l);
                    if (u == 3 && g > 0) y[8 * (g - 1) * kYRow] = last[0];
                }
#pragma unroll
                for (int t = 0; t < 8; ++t) last[t] = v[t];
            }
            sum_round<4>(last, l);
            sum_round<2>(last, l);
            sum_round<1>(last, l);
            y[8 * (groups - 1) * kYRow] = last[0];
            bar_arrive(kYFull + buf);
            if (k + 2 < tiles) bar_arrive(kEmpty + buf);
        }
        if (live && a.state_out && rank == X - 1) s.store(a.state_out + so);
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
        constexpr int kBC = (kTile * N / 8 + kHelpers - 1) / kHelpers;   // 8-state pieces of B (and C) a thread
        float bias[8], skip[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            bias[e] = (live && a.dt_bias) ? a.dt_bias[c + e] : 0.0f;
            skip[e] = (live && a.skip) ? a.skip[c + e] : 0.0f;
        }
        Eight<IOT> rx, rd, rz, px, pz, rb[kBC], rc[kBC];
        auto fetch = [&](int k) {
            const int t = t0 + k * kTile + row;
            const bool on = live && t < n;
            rx.zero(); rd.zero(); rz.zero();
            if (on) {
                rx.load(x + t * a.x_row);
                rd.load(dt + t * a.dt_row);
                if (z) rz.load(z + t * a.z_row);
            }
#pragma unroll
            for (int i = 0; i < kBC; ++i) {
                const int p = tid + i * kHelpers, pt = t0 + k * kTile + p / (N / 8), ps = 8 * (p % (N / 8));
                rb[i].zero(); rc[i].zero();
                if (p < kTile * N / 8 && pt < n) {
                    rb[i].load(Bm + pt * a.b_row + ps);
                    rc[i].load(Cm + pt * a.c_row + ps);
                }
            }
        };
        auto finish = [&](int k, const Eight<IOT>& fx, const Eight<IOT>& fz) {
            const int buf = k & 1, t = t0 + k * kTile + row;
            bar_sync(kYFull + buf);
            float f[8];
            const float4* v = reinterpret_cast<const float4*>(s_y + (buf * kTile + row) * kYRow + cv);
            const float4 v0 = v[0], v1 = v[1];
            f[0] = v0.x; f[1] = v0.y; f[2] = v0.z; f[3] = v0.w;
            f[4] = v1.x; f[5] = v1.y; f[6] = v1.z; f[7] = v1.w;
            if (k + 2 < tiles) bar_arrive(kYEmpty + buf);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[e] = fmaf(skip[e], fx.get(e), f[e]);
                if (z) f[e] = gated(f[e], fz.get(e));
            }
            if (live && t < n) Eight<IOT>::store(y + (long long)t * a.D, f);
        };
        auto produce = [&](int k) {
            const int buf = k & 1;
            const bool on = live && t0 + k * kTile + row < n;
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
                const int p = tid + i * kHelpers;
                if (p < kTile * N / 8) {
                    const int pt = p / (N / 8), pu = p % (N / 8);
                    float4* w = reinterpret_cast<float4*>(s_bc + (buf * kTile + pt) * 2 * N);
                    const auto& B = rb[i];
                    const auto& C = rc[i];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        if constexpr (S == 1)
                            w[unit_at<1>(pt, u)] = make_float4(B.get(2 * u), C.get(2 * u), B.get(2 * u + 1), C.get(2 * u + 1));
                        else if constexpr (S == 2)
                            w[unit_at<2>(pt, 4 * pu + u)] =
                                make_float4(B.get(2 * u), B.get(2 * u + 1), C.get(2 * u), C.get(2 * u + 1));
                        else {
                            // states 4 (u & 1) .. of the 8: unit j of thread l
                            const auto& V = u < 2 ? B : C;
                            const int s4 = 2 * pu + (u & 1), l = s4 * 4 / S, j = s4 % (S / 4) + (u < 2 ? 0 : S / 4), e = 4 * (u & 1);
                            w[8 * j + unit_at<S>(pt, l)] = make_float4(V.get(e), V.get(e + 1), V.get(e + 2), V.get(e + 3));
                        }
                    }
                }
            }
            bar_arrive(kFull + buf);
        };
        if constexpr (Cut) {
            if (tiles > 0) fetch(0);
            for (int k = 0; k < tiles; ++k) {
                produce(k);
                if (k + 1 < tiles) fetch(k + 1);
            }
            sm100::cluster_sync();
            sm100::cluster_sync();
        }
        if (tiles > 0) fetch(0);
        for (int k = 0; k < tiles; ++k) {
            produce(k);
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
// per state).  A thread has 4 states of one channel, in kMany sessions at once where there are enough
// of them: their loads are in flight together, and A is read once for all.  N / 4 threads sum a
// channel's output.
constexpr int kStepThreads = 256, kMany = 4;

template <typename IOT, int N, int Sessions>
__global__ void __launch_bounds__(kStepThreads)
selective_scan_step_kernel(const ScanArgs a)
{
    constexpr int L = N / 4;
    const long long id = (long long)blockIdx.x * kStepThreads + threadIdx.x;
    const int l = (int)(id % L);
    const long long ch = id / L;
    const bool live = ch < a.D;
    const int c = live ? (int)ch : 0, b0 = blockIdx.y * Sessions;
    const long long so = ((long long)b0 * a.D + c) * N + 4 * l, sb = (long long)a.D * N;
    float4 h[Sessions];
    float x[Sessions], de[Sessions], z[Sessions];
#pragma unroll
    for (int k = 0; k < Sessions; ++k) {
        const int b = min(b0 + k, a.B - 1);                // (a session past the last: read, not written)
        h[k] = *reinterpret_cast<const float4*>(a.state_in + so + (b - b0) * sb);
        x[k] = to_f32(static_cast<const IOT*>(a.x)[b * a.x_batch + c]);
        de[k] = to_f32(static_cast<const IOT*>(a.dt)[b * a.dt_batch + c]);
        z[k] = a.z ? to_f32(static_cast<const IOT*>(a.z)[b * a.z_batch + c]) : 0.0f;
    }
    float4 A = *reinterpret_cast<const float4*>(a.A + (long long)c * N + 4 * l);
    A = make_float4(clamp_finite(A.x), clamp_finite(A.y), clamp_finite(A.z), clamp_finite(A.w));
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.0f, skip = a.skip ? a.skip[c] : 0.0f;
#pragma unroll
    for (int k = 0; k < Sessions; ++k) {
        const int b = min(b0 + k, a.B - 1);
        const float4 B = four(static_cast<const IOT*>(a.Bm) + b * a.b_batch + 4 * l);
        const float4 C = four(static_cast<const IOT*>(a.Cm) + b * a.c_batch + 4 * l);
        float d = de[k] + bias;
        if (a.softplus) d = softplus_series(d);
        const float dx = d * x[k];
        if constexpr (sizeof(IOT) == 4) {
            h[k].x = exact_step(d * A.x, h[k].x, dx * B.x);
            h[k].y = exact_step(d * A.y, h[k].y, dx * B.y);
            h[k].z = exact_step(d * A.z, h[k].z, dx * B.z);
            h[k].w = exact_step(d * A.w, h[k].w, dx * B.w);
        } else {
            const float d2 = d * kLog2e;
            h[k].x = fmaf(attn::ex2(d2 * A.x), h[k].x, dx * B.x);
            h[k].y = fmaf(attn::ex2(d2 * A.y), h[k].y, dx * B.y);
            h[k].z = fmaf(attn::ex2(d2 * A.z), h[k].z, dx * B.z);
            h[k].w = fmaf(attn::ex2(d2 * A.w), h[k].w, dx * B.w);
        }
        float y = fmaf(h[k].x, C.x, fmaf(h[k].y, C.y, fmaf(h[k].z, C.z, h[k].w * C.w)));
#pragma unroll
        for (int w = L / 2; w > 0; w >>= 1) y += __shfl_xor_sync(0xffffffffu, y, w);
        if (!live || b0 + k >= a.B) continue;
        *reinterpret_cast<float4*>(a.state_out + so + k * sb) = h[k];
        if (l == 0) {
            y = fmaf(skip, x[k], y);
            if (a.z) y = gated(y, z[k]);
            static_cast<IOT*>(a.y)[(long long)b * a.D + c] = from_f32<IOT>(y);
        }
    }
}

template <typename IOT, int N>
cudaError_t launch(const ScanArgs& a, bool step, cudaStream_t stream)
{
    if (step) {
        int dev = 0, sms = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        const long long threads = (long long)a.D * (N / 4);
        const unsigned blocks = (unsigned)((threads + kStepThreads - 1) / kStepThreads);
        // several sessions a thread as long as the threads still fill the device twice
        if (threads * a.B >= 2 * 2048ll * kMany * sms)
            selective_scan_step_kernel<IOT, N, kMany>
                <<<dim3(blocks, (unsigned)((a.B + kMany - 1) / kMany)), kStepThreads, 0, stream>>>(a);
        else
            selective_scan_step_kernel<IOT, N, 1><<<dim3(blocks, (unsigned)a.B), kStepThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    // Sequences are cut in 4 or 8 while all CTAs are resident at once and a segment has a tile; in 2 it
    // does not pay.  8192 tokens of N = 16: 64 CTAs 211 us whole, 147 us in 4; 32 CTAs 210 us whole, 90 us
    // in 4, 75 us in 8; 94 CTAs, beyond the rule, 213 us whole and 218 us in 4.
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const long long blocks = (a.D + kC - 1) / kC, ctas = blocks * a.B;
    int X = 8;
    while (X > 2 && (ctas * X > (long long)resident<IOT, N>() * sms || a.T < kTile * X)) X /= 2;
    if (X == 2) X = 1;
    auto kernel = X > 1 ? selective_scan_kernel<IOT, N, true> : selective_scan_kernel<IOT, N, false>;
    if (smem_bytes<N>() > 48 * 1024) {     // (a per-device setting of the current context: set on every call)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<N>());
        if (e != cudaSuccess) return e;
    }
    if (X == 1) {
        kernel<<<dim3((unsigned)blocks, (unsigned)a.B), kThreads, smem_bytes<N>(), stream>>>(a);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks * X), (unsigned)a.B);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes<N>();
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)X;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
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
