// C ABI of the other sequence mixers: argument checks and dispatch of the causal
// convolution, the selective scan, and window attention with its rolling cache.
// As everywhere, every argument is checked before any CUDA call and nothing is enqueued
// on an error.  (Part of the translation unit: uses the helpers of gdn_api.cu.)
#include "gdn.h"

namespace {

// A [B, T, inner] tensor read through batch and row strides (in elements): vector loads
// need 16-byte aligned rows; a stride over a single batch entry or row is not looked at.
struct Rows {
    const void* p;
    long long batch, row;
};

int check_rows(Rows* r, int B, int T, long long inner, size_t elem, size_t* bytes)
{
    *bytes = 0;
    if (!aligned(r->p, 16)) return GDN_ERR_INVALID_ARG;
    if (B == 1) r->batch = 0;
    if (T <= 1) r->row = inner;
    const long long v = 16 / (long long)elem;
    if (r->row < inner || r->batch < 0 || r->row % v || r->batch % v) return GDN_ERR_INVALID_ARG;
    if (T < 1) return GDN_OK;
    if (r->row > INT64_MAX / 32 / T || r->batch > INT64_MAX / 32 / B) return GDN_ERR_INVALID_ARG;
    *bytes = (size_t)((B - 1) * r->batch + (T - 1) * r->row + inner) * elem;
    return GDN_OK;
}

struct Span {
    const void* p;
    size_t bytes;
};

template <int N>
bool overlaps_any(const void* p, size_t bytes, const Span (&s)[N])
{
    for (const Span& e : s)
        if (overlaps(p, bytes, e.p, e.bytes)) return true;
    return false;
}

int run_conv(gdn::ConvArgs a, int width, int silu, size_t elem, cudaStream_t stream)
{
    if (a.B < 1 || a.T < 0 || a.D < 1 || (silu != 0 && silu != 1)) return GDN_ERR_INVALID_ARG;
    if (width < 2 || width > 4 || a.D % 8 || a.B > 65535 || a.T > INT32_MAX - 1024) return GDN_ERR_UNSUPPORTED;
    if (!a.weight || (a.T > 0 && (!a.x || !a.out))) return GDN_ERR_INVALID_ARG;
    if (!aligned(a.out, 16) || !aligned(a.state_in, 16) || !aligned(a.state_out, 16) || !aligned(a.weight, 16) ||
        !aligned(a.bias, 16) || !aligned(a.lengths, 4))
        return GDN_ERR_INVALID_ARG;
    Rows x{a.x, a.x_batch, a.x_row};
    size_t nx = 0;
    const int st = check_rows(&x, a.B, a.T, a.D, elem, &nx);
    if (st != GDN_OK) return st;
    a.x_batch = x.batch;
    a.x_row = x.row;
    const size_t no = (size_t)a.B * a.T * a.D * elem, ns = (size_t)a.B * (width - 1) * a.D * elem;
    const Span in[] = {{a.x, nx}, {a.weight, (size_t)a.D * width * 4}, {a.bias, (size_t)a.D * 4},
                       {a.lengths, (size_t)a.B * 4}};
    if (overlaps_any(a.out, no, in) || overlaps(a.out, no, a.state_in, ns) || overlaps(a.out, no, a.state_out, ns))
        return GDN_ERR_INVALID_ARG;
    if (a.state_out && (overlaps_any(a.state_out, ns, in) ||
                        (a.state_out != a.state_in && overlaps(a.state_out, ns, a.state_in, ns))))
        return GDN_ERR_INVALID_ARG;
    return to_status(elem == 2 ? gdn::launch_conv<__nv_bfloat16>(a, width, silu != 0, stream)
                               : gdn::launch_conv<float>(a, width, silu != 0, stream));
}

int run_scan(gdn::ScanArgs a, int softplus, size_t elem, bool step, cudaStream_t stream)
{
    if (a.B < 1 || a.T < 0 || a.D < 1 || a.N < 1 || (softplus != 0 && softplus != 1)) return GDN_ERR_INVALID_ARG;
    if ((a.N != 8 && a.N != 16 && a.N != 32 && a.N != 64) || a.D % 8 || a.B > 65535 || a.T > INT32_MAX - 1024 ||
        a.D > INT32_MAX - 1024)
        return GDN_ERR_UNSUPPORTED;
    if (!a.A || (a.T > 0 && (!a.x || !a.dt || !a.Bm || !a.Cm || !a.y))) return GDN_ERR_INVALID_ARG;
    if (!aligned(a.y, 16) || !aligned(a.A, 16) || !aligned(a.state_in, 16) || !aligned(a.state_out, 16) ||
        !aligned(a.skip, 4) || !aligned(a.dt_bias, 4) || !aligned(a.lengths, 4))
        return GDN_ERR_INVALID_ARG;
    Rows x{a.x, a.x_batch, a.x_row}, dt{a.dt, a.dt_batch, a.dt_row}, z{a.z, a.z_batch, a.z_row};
    Rows bm{a.Bm, a.b_batch, a.b_row}, cm{a.Cm, a.c_batch, a.c_row};
    size_t nx, ndt, nz = 0, nb, nc;
    int st = check_rows(&x, a.B, a.T, a.D, elem, &nx);
    if (st == GDN_OK) st = check_rows(&dt, a.B, a.T, a.D, elem, &ndt);
    if (st == GDN_OK && a.z) st = check_rows(&z, a.B, a.T, a.D, elem, &nz);
    if (st == GDN_OK) st = check_rows(&bm, a.B, a.T, a.N, elem, &nb);
    if (st == GDN_OK) st = check_rows(&cm, a.B, a.T, a.N, elem, &nc);
    if (st != GDN_OK) return st;
    a.x_batch = x.batch; a.x_row = x.row; a.dt_batch = dt.batch; a.dt_row = dt.row;
    a.z_batch = z.batch; a.z_row = z.row; a.b_batch = bm.batch; a.b_row = bm.row;
    a.c_batch = cm.batch; a.c_row = cm.row;
    a.softplus = softplus != 0;
    const size_t ny = (size_t)a.B * a.T * a.D * elem, ns = (size_t)a.B * a.D * a.N * 4, nd = (size_t)a.D * 4;
    const Span in[] = {{a.x, nx}, {a.dt, ndt}, {a.z, nz}, {a.Bm, nb}, {a.Cm, nc}, {a.A, nd * a.N},
                       {a.skip, nd}, {a.dt_bias, nd}, {a.lengths, (size_t)a.B * 4}};
    if (overlaps_any(a.y, ny, in) || overlaps(a.y, ny, a.state_in, ns) || overlaps(a.y, ny, a.state_out, ns))
        return GDN_ERR_INVALID_ARG;
    if (a.state_out && (overlaps_any(a.state_out, ns, in) ||
                        (a.state_out != a.state_in && overlaps(a.state_out, ns, a.state_in, ns))))
        return GDN_ERR_INVALID_ARG;
    return to_status(elem == 2 ? gdn::launch_scan<__nv_bfloat16>(a, step, stream)
                               : gdn::launch_scan<float>(a, step, stream));
}

bool head_dim_ok(int d) { return d >= 16 && d <= 128 && d % 16 == 0; }

int check_window(int B, int Hq, int Hkv, int dk, int dv, int window, int sinks, float scale)
{
    if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || dk < 1 || dv < 1 || window < 1 || sinks < 0)
        return GDN_ERR_INVALID_ARG;
    if (!(scale > 0.0f && scale <= 3.4028235e38f)) return GDN_ERR_INVALID_ARG;      // NaN fails too
    if (!head_dim_ok(dk) || !head_dim_ok(dv) || B > 65535 || Hq > 65535) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

// A [B, T, H, d] tensor read through batch, row and head strides; d contiguous.
int check_heads(const void* p, long long* batch, long long* row, long long* head, int B, int T, int H, int d,
                size_t* bytes)
{
    *bytes = 0;
    if (!p || !aligned(p, 16)) return GDN_ERR_INVALID_ARG;
    if (B == 1) *batch = (long long)H * d;           // (a valid stride, multiplied by 0)
    if (T <= 1) *row = (long long)H * d;
    if (H == 1) *head = d;
    if (*head < d || *row < d || *batch < d || *head % 8 || *row % 8 || *batch % 8) return GDN_ERR_INVALID_ARG;
    // the strides of a tensor map stay below 2^40 bytes
    if (*head >= (1ll << 38) || *row >= (1ll << 38) || *batch >= (1ll << 38)) return GDN_ERR_UNSUPPORTED;
    if (T > 0)
        *bytes = 2 * ((size_t)(B - 1) * (size_t)*batch + (size_t)(T - 1) * (size_t)*row +
                      (size_t)(H - 1) * (size_t)*head + (size_t)d);
    return GDN_OK;
}

int run_window_step(const void* q, long long q_batch_stride, const void* k, long long k_batch_stride,
                    const void* v, long long v_batch_stride, void* k_cache, void* v_cache,
                    const int* pos, void* out, int B, int Hq, int Hkv, int d_k, int d_v,
                    int window, int sinks, float scale, bool zero_idle, cudaStream_t stream)
{
    int st = check_window(B, Hq, Hkv, d_k, d_v, window, sinks, scale);
    if (st != GDN_OK) return st;
    if ((int64_t)window + sinks > INT32_MAX - 64) return GDN_ERR_UNSUPPORTED;
    if (!q || !k || !v || !k_cache || !v_cache || !pos || !out) return GDN_ERR_INVALID_ARG;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) || !aligned(pos, 4))
        return GDN_ERR_INVALID_ARG;
    Rows rq{q, q_batch_stride, 0}, rk{k, k_batch_stride, 0}, rv{v, v_batch_stride, 0};
    size_t nq, nk, nv;
    st = check_rows(&rq, B, 1, (long long)Hq * d_k, 2, &nq);
    if (st == GDN_OK) st = check_rows(&rk, B, 1, (long long)Hkv * d_k, 2, &nk);
    if (st == GDN_OK) st = check_rows(&rv, B, 1, (long long)Hkv * d_v, 2, &nv);
    if (st != GDN_OK) return st;
    const size_t slots = (size_t)B * ((size_t)window + sinks) * Hkv, nkc = slots * d_k * 2, nvc = slots * d_v * 2;
    const size_t no = (size_t)B * Hq * d_v * 2;
    const Span in[] = {{q, nq}, {k, nk}, {v, nv}, {pos, (size_t)B * 4}};
    if (overlaps_any(k_cache, nkc, in) || overlaps_any(v_cache, nvc, in) || overlaps(k_cache, nkc, v_cache, nvc) ||
        overlaps_any(out, no, in) || overlaps(out, no, k_cache, nkc) || overlaps(out, no, v_cache, nvc))
        return GDN_ERR_INVALID_ARG;
    gdn::StepArgs a;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.q_batch = rq.batch; a.k_batch = rk.batch; a.v_batch = rv.batch;
    a.k_cache = static_cast<__nv_bfloat16*>(k_cache);
    a.v_cache = static_cast<__nv_bfloat16*>(v_cache);
    a.pos = pos;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.dk = d_k; a.dv = d_v; a.window = window; a.sinks = sinks;
    a.scale = scale;
    a.zero_idle = zero_idle;
    return to_status(gdn::launch_window_step(a, stream));
}

}  // namespace

extern "C" {

int gdn_causal_conv(const void* x, long long x_batch_stride, long long x_row_stride,
                    const float* weight, const float* bias, const void* state_in, void* state_out,
                    const int* lengths, void* out, int B, int T, int D, int width, int silu, cudaStream_t stream)
{
    return run_conv({x, weight, bias, state_in, state_out, lengths, out, x_batch_stride, x_row_stride, B, T, D},
                    width, silu, 2, stream);
}

int gdn_causal_conv_f32(const float* x, long long x_batch_stride, long long x_row_stride,
                        const float* weight, const float* bias, const float* state_in, float* state_out,
                        const int* lengths, float* out, int B, int T, int D, int width, int silu, cudaStream_t stream)
{
    return run_conv({x, weight, bias, state_in, state_out, lengths, out, x_batch_stride, x_row_stride, B, T, D},
                    width, silu, 4, stream);
}

int gdn_causal_conv_step(const void* x, long long x_batch_stride, const float* weight, const float* bias,
                         void* state, void* out, int B, int D, int width, int silu, cudaStream_t stream)
{
    if (!state) return GDN_ERR_INVALID_ARG;
    return run_conv({x, weight, bias, state, state, nullptr, out, x_batch_stride, D, B, 1, D}, width, silu, 2, stream);
}

int gdn_causal_conv_step_f32(const float* x, long long x_batch_stride, const float* weight, const float* bias,
                             float* state, float* out, int B, int D, int width, int silu, cudaStream_t stream)
{
    if (!state) return GDN_ERR_INVALID_ARG;
    return run_conv({x, weight, bias, state, state, nullptr, out, x_batch_stride, D, B, 1, D}, width, silu, 4, stream);
}

int gdn_selective_scan(const void* x, long long x_batch_stride, long long x_row_stride,
                       const void* dt, long long dt_batch_stride, long long dt_row_stride,
                       const float* A,
                       const void* Bm, long long b_batch_stride, long long b_row_stride,
                       const void* Cm, long long c_batch_stride, long long c_row_stride,
                       const float* skip, const void* z, long long z_batch_stride, long long z_row_stride,
                       const float* dt_bias, const float* state_in, float* state_out, const int* lengths, void* y,
                       int B, int T, int D, int N, int dt_softplus, cudaStream_t stream)
{
    return run_scan({x, dt, z, Bm, Cm, x_batch_stride, x_row_stride, dt_batch_stride, dt_row_stride, z_batch_stride,
                     z_row_stride, b_batch_stride, b_row_stride, c_batch_stride, c_row_stride, A, skip, dt_bias,
                     state_in, state_out, lengths, y, B, T, D, N, false}, dt_softplus, 2, false, stream);
}

int gdn_selective_scan_f32(const float* x, long long x_batch_stride, long long x_row_stride,
                           const float* dt, long long dt_batch_stride, long long dt_row_stride,
                           const float* A,
                           const float* Bm, long long b_batch_stride, long long b_row_stride,
                           const float* Cm, long long c_batch_stride, long long c_row_stride,
                           const float* skip, const float* z, long long z_batch_stride, long long z_row_stride,
                           const float* dt_bias, const float* state_in, float* state_out, const int* lengths, float* y,
                           int B, int T, int D, int N, int dt_softplus, cudaStream_t stream)
{
    return run_scan({x, dt, z, Bm, Cm, x_batch_stride, x_row_stride, dt_batch_stride, dt_row_stride, z_batch_stride,
                     z_row_stride, b_batch_stride, b_row_stride, c_batch_stride, c_row_stride, A, skip, dt_bias,
                     state_in, state_out, lengths, y, B, T, D, N, false}, dt_softplus, 4, false, stream);
}

int gdn_selective_scan_step(const void* x, long long x_batch_stride, const void* dt, long long dt_batch_stride,
                            const float* A, const void* Bm, long long b_batch_stride,
                            const void* Cm, long long c_batch_stride, const float* skip,
                            const void* z, long long z_batch_stride, const float* dt_bias, float* state, void* y,
                            int B, int D, int N, int dt_softplus, cudaStream_t stream)
{
    if (!state) return GDN_ERR_INVALID_ARG;
    return run_scan({x, dt, z, Bm, Cm, x_batch_stride, D, dt_batch_stride, D, z_batch_stride, D, b_batch_stride, N,
                     c_batch_stride, N, A, skip, dt_bias, state, state, nullptr, y, B, 1, D, N, false},
                    dt_softplus, 2, true, stream);
}

int gdn_selective_scan_step_f32(const float* x, long long x_batch_stride, const float* dt, long long dt_batch_stride,
                                const float* A, const float* Bm, long long b_batch_stride,
                                const float* Cm, long long c_batch_stride, const float* skip,
                                const float* z, long long z_batch_stride, const float* dt_bias, float* state, float* y,
                                int B, int D, int N, int dt_softplus, cudaStream_t stream)
{
    if (!state) return GDN_ERR_INVALID_ARG;
    return run_scan({x, dt, z, Bm, Cm, x_batch_stride, D, dt_batch_stride, D, z_batch_stride, D, b_batch_stride, N,
                     c_batch_stride, N, A, skip, dt_bias, state, state, nullptr, y, B, 1, D, N, false},
                    dt_softplus, 4, true, stream);
}

int gdn_window_attention(const void* q, long long q_batch_stride, long long q_row_stride, long long q_head_stride,
                         const void* k, long long k_batch_stride, long long k_row_stride, long long k_head_stride,
                         const void* v, long long v_batch_stride, long long v_row_stride, long long v_head_stride,
                         const int* lengths, void* out, int B, int Tq, int Tk, int Hq, int Hkv, int d_k, int d_v,
                         int window, int sinks, float scale, cudaStream_t stream)
{
    int st = check_window(B, Hq, Hkv, d_k, d_v, window, sinks, scale);
    if (st != GDN_OK) return st;
    if (Tq < 0 || Tk < Tq) return GDN_ERR_INVALID_ARG;
    if (Tk > INT32_MAX - 1024) return GDN_ERR_UNSUPPORTED;
    if (Tq == 0) return GDN_OK;                      // no query: nothing to write, no pointer is looked at
    if (!out || !aligned(out, 16) || !aligned(lengths, 4)) return GDN_ERR_INVALID_ARG;
    size_t nq, nk, nv;
    st = check_heads(q, &q_batch_stride, &q_row_stride, &q_head_stride, B, Tq, Hq, d_k, &nq);
    if (st == GDN_OK) st = check_heads(k, &k_batch_stride, &k_row_stride, &k_head_stride, B, Tk, Hkv, d_k, &nk);
    if (st == GDN_OK) st = check_heads(v, &v_batch_stride, &v_row_stride, &v_head_stride, B, Tk, Hkv, d_v, &nv);
    if (st != GDN_OK) return st;
    const Span in[] = {{q, nq}, {k, nk}, {v, nv}, {lengths, (size_t)B * 4}};
    if (overlaps_any(out, (size_t)B * Tq * Hq * d_v * 2, in)) return GDN_ERR_INVALID_ARG;
    gdn::WindowArgs a;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.q_batch = q_batch_stride; a.q_row = q_row_stride; a.q_head = q_head_stride;
    a.k_batch = k_batch_stride; a.k_row = k_row_stride; a.k_head = k_head_stride;
    a.v_batch = v_batch_stride; a.v_row = v_row_stride; a.v_head = v_head_stride;
    a.lengths = lengths;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.B = B; a.Tq = Tq; a.Tk = Tk; a.Hq = Hq; a.Hkv = Hkv; a.dk = d_k; a.dv = d_v;
    a.window = window < Tk ? window : Tk;            // a longer window sees no more
    a.sinks = sinks < Tk ? sinks : Tk;
    a.scale = scale;
    return to_status(gdn::launch_window(a, stream));
}

int gdn_window_cache_append(const void* k, long long k_batch_stride, long long k_row_stride,
                            const void* v, long long v_batch_stride, long long v_row_stride,
                            void* k_cache, void* v_cache, const int* start, const int* lengths,
                            int B, int T, int Hkv, int d_k, int d_v, int window, int sinks, cudaStream_t stream)
{
    int st = check_window(B, Hkv, Hkv, d_k, d_v, window, sinks, 1.0f);
    if (st != GDN_OK) return st;
    if (T < 0) return GDN_ERR_INVALID_ARG;
    if ((int64_t)window + sinks > INT32_MAX - 64) return GDN_ERR_UNSUPPORTED;
    if (T == 0) return GDN_OK;
    if (!k || !v || !k_cache || !v_cache || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(start, 4) ||
        !aligned(lengths, 4))
        return GDN_ERR_INVALID_ARG;
    Rows rk{k, k_batch_stride, k_row_stride}, rv{v, v_batch_stride, v_row_stride};
    size_t nk, nv;
    st = check_rows(&rk, B, T, (long long)Hkv * d_k, 2, &nk);
    if (st == GDN_OK) st = check_rows(&rv, B, T, (long long)Hkv * d_v, 2, &nv);
    if (st != GDN_OK) return st;
    const size_t slots = (size_t)B * ((size_t)window + sinks) * Hkv, nkc = slots * d_k * 2, nvc = slots * d_v * 2;
    const Span in[] = {{k, nk}, {v, nv}, {start, (size_t)B * 4}, {lengths, (size_t)B * 4}};
    if (overlaps_any(k_cache, nkc, in) || overlaps_any(v_cache, nvc, in) || overlaps(k_cache, nkc, v_cache, nvc))
        return GDN_ERR_INVALID_ARG;
    gdn::AppendArgs a;
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.k_batch = rk.batch; a.k_row = rk.row; a.v_batch = rv.batch; a.v_row = rv.row;
    a.k_cache = static_cast<__nv_bfloat16*>(k_cache);
    a.v_cache = static_cast<__nv_bfloat16*>(v_cache);
    a.start = start;
    a.lengths = lengths;
    a.B = B; a.T = T; a.Hkv = Hkv; a.dk = d_k; a.dv = d_v; a.window = window; a.sinks = sinks;
    return to_status(gdn::launch_window_append(a, stream));
}

int gdn_window_attention_step(const void* q, long long q_batch_stride, const void* k, long long k_batch_stride,
                              const void* v, long long v_batch_stride, void* k_cache, void* v_cache,
                              const int* pos, void* out, int B, int Hq, int Hkv, int d_k, int d_v,
                              int window, int sinks, float scale, cudaStream_t stream)
{
    return run_window_step(q, q_batch_stride, k, k_batch_stride, v, v_batch_stride, k_cache, v_cache, pos, out, B, Hq,
                           Hkv, d_k, d_v, window, sinks, scale, false, stream);
}

int gdn_window_attention_step_zero_idle(const void* q, long long q_batch_stride, const void* k, long long k_batch_stride,
                                        const void* v, long long v_batch_stride, void* k_cache, void* v_cache,
                                        const int* pos, void* out, int B, int Hq, int Hkv, int d_k, int d_v,
                                        int window, int sinks, float scale, cudaStream_t stream)
{
    return run_window_step(q, q_batch_stride, k, k_batch_stride, v, v_batch_stride, k_cache, v_cache, pos, out, B, Hq,
                           Hkv, d_k, d_v, window, sinks, scale, true, stream);
}

}  // extern "C"
