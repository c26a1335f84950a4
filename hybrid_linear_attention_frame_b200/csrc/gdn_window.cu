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
#include "gdn_sm100.cuh"

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
    const int* pos;                          // [B]: the token's position; negative: an idle session
    __nv_bfloat16* out;                      // [B, Hq, dv]
    int B, Hq, Hkv, dk, dv, window, sinks;
    float scale;
    bool zero_idle;                          // an idle session's row of out: zeros, else as it was
    uint64_t wait_limit_ns;
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

// 4-D bf16 map over a strided [B, T, H, d] tensor, box {64, 1, rows, 1}, 128-byte swizzle.
bool make_map(CUtensorMap* map, const void* ptr, int d, int H, long long T, int B, int rows, long long head,
              long long row, long long batch)
{
    PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)T, (cuuint64_t)B};
    cuuint64_t strides[3] = {(cuuint64_t)head * 2, (cuuint64_t)row * 2, (cuuint64_t)batch * 2};
    cuuint32_t box[4] = {64, 1, (cuuint32_t)rows, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---- whole prompts: tcgen05 ----
//
// One CTA per pair of 128-query tiles (two query heads that share a key head where there are
// such, else two tiles of consecutive queries), which read the same K and V tiles:
//   S_q = Q_q K^T on the tensor cores into TMEM, q = 0, 1;
//   softmax of tile q by its own eight warps, two threads per query row, against a reference m, 16 (in
//     powers of 2) above the row's largest score in its first tile: it moves only when a thread's 64
//     weights of a tile sum to more than 64, so later tiles need no maximum and O is hardly ever
//     rescaled (the division by the running sum at the end is right for any m).  So no sum is larger
//     than if every weight were at most 1, and the 2^-16 that O may be small by is within what float
//     has below bf16's smallest values;
//   P in bf16 over the score columns it came from, O_q += P_q V with P as the A operand.
// P enters its product in bf16, each weight off by up to 2^-8 of itself, while the row's sum keeps them in
// f32: outputs are 0.0019 to 0.0023 from the formula (relative, root mean square) where their own rounding to
// bf16 makes 0.0016.  The remainders in a second bf16 word, as the form for one token has them, would take 32
// more registers a thread, held until the row's other thread was looked at (18 warps leave 96), and half
// again the P V products.
// S and P of a query tile have two buffers of 64 keys, the halves of a 128-key tile and one thread of
// each row.  Warp 16 issues, half by half, PV_0(j-1) S_0(j) PV_1(j-1) S_1(j); the tensor cores execute
// in order, so S(j) may overwrite P(j-1) of its half, and while a softmax weighs one half, the other
// half's products run.  Warp 17 keeps K (3 stages) and V (2 stages) coming by TMA.  Key tiles are
// counted from the window's first key, sink tiles before them when the two do not touch, so no key is
// visited twice; a tile that a query tile sees nothing of is skipped for it.  Every wait is bounded.
//
// A step (two query tiles, 128 keys, d 128) needs 2.0 K cycles of the tensor cores and as many of the
// special-function unit; it takes about 3.6 K, the two taking turns at each buffer.  27,280 tokens,
// 20 heads on 4, d 128, window 2640 + 880 sinks: 840 to 930 us as the power cap allows, about 1,020
// TFLOP/s; causal over 8192 tokens, 32 heads on 8: 528 us, 1,040 TFLOP/s.  What the form rests on: one
// thread per row weighing 128 keys held the chain from scores to weights to scores at 4.2 K cycles; with
// S and P in one buffer per tile the softmax waited for both products; an issuing thread that sleeps at
// its barriers adds 300 cycles to every hand-off (1,008 against 972 us).
namespace tc {

using namespace sm100;

constexpr int kBM = 128, kBN = 128;            // queries per tile, keys per tile
constexpr int kTileWarps = 8;                  // softmax warps per query tile: two threads per row
constexpr int kMmaWarp = 2 * kTileWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kLoadWarp + 1);
constexpr uint32_t kBox = 128u * 128u;         // one 64-column SW128 box of 128 rows
constexpr uint32_t kOp = 2u * kBox;            // a 128 x (d <= 128) operand
constexpr int kKStages = 3, kVStages = 2;
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = kOffQ + 2 * kOp;
constexpr uint32_t kOffV = kOffK + kKStages * kOp;
constexpr uint32_t kOffBar = kOffV + kVStages * kOp;
enum : uint32_t { kBarQ = 0, kBarKFull = 1, kBarKFree = kBarKFull + kKStages, kBarVFull = kBarKFree + kKStages,
                  kBarVFree = kBarVFull + kVStages, // [query tile][half of the key tile]:
                  kBarS = kBarVFree + kVStages,          // scores ready
                  kBarP = kBarS + 4,           // P written, O rescaled (one arrival per softmax warp)
                  kBarH = kBarP + 4,           // P V done
                  kBarO = kBarH + 4,           // [2] last P V of the tile done
                  kBarL = kBarO + 2,           // a row's word written (its maximum, at the end its sum)
                  kBarDrain = kBarL + 4,       // every MMA done
                  kNumBars = kBarDrain + 1 };
__host__ __device__ constexpr uint32_t bar_count(uint32_t i) {
    return ((i >= kBarP && i < kBarP + 4) || (i >= kBarL && i < kBarL + 4)) ? 4u : 1u;
}
constexpr uint32_t kOffAbort = kOffBar + 8u * kNumBars;
constexpr uint32_t kOffTmemSlot = kOffAbort + 8u;
constexpr uint32_t kOffM = kOffTmemSlot + 8u;  // [2][128] the rows' references, at the end their sums
constexpr uint32_t kSmemBytes = kOffM + 2u * kBM * 4u + 1024u;   // + slack for 1024-byte alignment
static_assert(kSmemBytes <= 232448, "shared memory budget");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;     // + 128 q each; S: two buffers of 64 columns
// The reference lies kAbove over the largest score that it was taken from, and moves when a thread's 64
// weights sum to more than kMaxSum: scores may rise by 2^16 at least (one alone by 2^22) before it does.
constexpr float kAbove = 16.0f, kMaxSum = 64.0f;
constexpr uint32_t kIdS = idesc_bf16(128, 64, false, false);

struct Args {
    const __nv_bfloat16 *q, *k, *v;            // (as the tensor maps have them; for the rows that are done again)
    long long q_batch, q_row, q_head, k_batch, k_row, k_head, v_batch, v_row, v_head;
    const int* lengths;
    __nv_bfloat16* out;
    int Tq, Tk, Hq, group, dk, dv, window, sinks;
    int pair_heads;                            // the CTA's two tiles: two heads, or two tiles of one head
    int row_blocks, head_blocks;
    float scale_log2;
    uint64_t wait_limit_ns;
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32"
                 " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                   "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                   "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Waits for this thread's TMEM loads; x is what they bring (nothing that uses it moves before the wait).
__device__ __forceinline__ void tmem_wait32(float (&x)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7]),
                   "+f"(x[8]), "+f"(x[9]), "+f"(x[10]), "+f"(x[11]), "+f"(x[12]), "+f"(x[13]), "+f"(x[14]),
                   "+f"(x[15]), "+f"(x[16]), "+f"(x[17]), "+f"(x[18]), "+f"(x[19]), "+f"(x[20]), "+f"(x[21]),
                   "+f"(x[22]), "+f"(x[23]), "+f"(x[24]), "+f"(x[25]), "+f"(x[26]), "+f"(x[27]), "+f"(x[28]),
                   "+f"(x[29]), "+f"(x[30]), "+f"(x[31])
                 :: "memory");
}

// the n lowest bits, none below 0, all above 31
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

// What a CTA visits: its two query tiles' rows and the key tiles of their union.
struct Plan {
    int head[2], row0[2];                      // query head and first query of tile q
    int p_lo[2], p_hi[2];                      // positions of its first and last live query; none if p_hi < p_lo
    int sink, startB, nA, n;                   // sink tiles 0 .. nA-1, then tiles from startB on
    // tile q sees keys of tiles 0 .. first_end - 1 (sinks) and near .. end - 1 (its window)
    int first_end[2], near[2], end[2];
    __device__ int start(int j) const { return j < nA ? kBN * j : startB + kBN * (j - nA); }
    __device__ bool active(int q, int j) const { return j < first_end[q] || (j >= near[q] && j < end[q]); }
};

__device__ __forceinline__ Plan make_plan(const Args& a, int n_keys, uint32_t block) {
    Plan p;
    const int off = a.Tk - a.Tq;
    // later queries see more: their blocks come first
    const int rb = a.row_blocks - 1 - (int)(block / (uint32_t)a.head_blocks);
    const int hb = (int)(block % (uint32_t)a.head_blocks);
    int lo = INT32_MAX, hi = -1;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        p.head[q] = a.pair_heads ? 2 * hb + q : hb;
        p.row0[q] = a.pair_heads ? rb * kBM : (2 * rb + q) * kBM;
        p.p_lo[q] = off + p.row0[q];
        p.p_hi[q] = min(off + min(p.row0[q] + kBM, a.Tq), n_keys) - 1;
        if (p.p_hi[q] >= p.p_lo[q]) {
            lo = min(lo, p.p_lo[q]);
            hi = max(hi, p.p_hi[q]);
        }
    }
    const int w_lo = max(0, lo - a.window + 1);
    p.sink = min(a.sinks, n_keys);
    const bool split = w_lo > p.sink;
    p.nA = split ? (p.sink + kBN - 1) / kBN : 0;
    p.startB = split ? w_lo : 0;
    p.n = hi < 0 ? 0 : p.nA + (hi + 1 - p.startB + kBN - 1) / kBN;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const bool live = p.p_hi[q] >= p.p_lo[q];
        const int w = max(0, p.p_lo[q] - a.window + 1);
        p.end[q] = live ? p.nA + (p.p_hi[q] - p.startB) / kBN + 1 : 0;
        p.near[q] = live ? p.nA + (w - p.startB) / kBN : 0;
        p.first_end[q] = live ? min(split ? p.nA : (p.sink + kBN - 1) / kBN, p.end[q]) : 0;
    }
    return p;
}

__device__ __forceinline__ uint64_t kmaj(uint32_t addr) { return smem_desc(addr, 16, 1024, kSwizzle128); }

// The issuing thread's wait: polls without suspending (a suspended thread takes ~300 cycles to resume,
// which here would stand between a softmax and its next scores), bounded like every wait.
__device__ __forceinline__ bool mbar_poll(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit_ns,
                                          int code) {
    uint64_t t0 = 0;
    for (uint32_t it = 1; !mbar_test_wait(bar, parity); ++it) {
        if ((it & 255u) == 0) {
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (*abort) return false;
            if (now - t0 > limit_ns) {
                *abort = 1;
                atomicCAS(&g_device_status, 0, code);
                return false;
            }
        }
    }
    return true;
}

// One MMA of the calling thread whose A operand is in TMEM (row m in lane m, a bf16 pair per column).
__device__ __forceinline__ void mma_bf16_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// The weights of tokens that a row does not see are 0, and 0 times an infinity or NaN in their values is NaN:
// on the tensor cores such a token of a visited tile reaches rows that it must not.  So a warp that wrote a NaN
// does again, key by key in f32, those of its 32 rows (64 columns) that have such a token beside what they see.
// The tokens that row t's query tile visits and that t does not see lie in [min(sink, t + 1), ws) from the
// window's first tile on, and in (t, end of the last tile).
__device__ __forceinline__ void redo_rows(const Args& a) {
    // (Everything anew, the plan too: kept in the kernel's registers for this, or in a function of its own, it
    // costs calls that never come here 5 %: 43.9 us instead of 41.2 for 2640 tokens, window 880.)
    uint32_t block, tid;
    int b;
    asm volatile("mov.u32 %0, %%ctaid.x;\n\tmov.u32 %1, %%ctaid.y;\n\tmov.u32 %2, %%tid.x;" : "=r"(block), "=r"(b), "=r"(tid));
    const int warp = (int)tid >> 5, lane = tid & 31, q_tile = warp / kTileWarps, half = (warp >> 2) & 1;
    const int n_keys = a.lengths ? min(max(a.lengths[b], 0), a.Tk) : a.Tk, cols = min(64, a.dv - 64 * half);
    const Plan p = make_plan(a, n_keys, block);
    const int head = p.head[q_tile], t0 = p.p_lo[q_tile] + 32 * (warp & 3), live = min(32, p.p_hi[q_tile] + 1 - t0);
    if (live <= 0 || cols <= 0) return;
    const int near_key = p.startB > 0 || p.nA > 0 ? p.start(p.near[q_tile]) : 0;
    const int end = min(n_keys, p.start(p.end[q_tile] - 1) + kBN), off = a.Tk - a.Tq;
    if (lane == 0) bulk_wait_group0();         // the warp's rows are out before any is written again
    __syncwarp();
    const __nv_bfloat16* k = a.k + b * a.k_batch + head / a.group * a.k_head;
    const __nv_bfloat16* v = a.v + b * a.v_batch + head / a.group * a.v_head + 64 * half;
    for (int t = t0; t < t0 + live; ++t) {
        const int i = t - off, ws = max(0, t - a.window + 1);
        // four tokens at a time: is there one?
        bool hit = false;
        for (int part = 0; part < 2 && !hit; ++part) {
            const int lo = part ? t + 1 : max(min(p.sink, t + 1), near_key), hi = part ? end : ws;
            for (int s0 = lo; s0 < hi && !hit; s0 += 4) {
                const int s = s0 + (lane >> 3), c = 8 * (lane & 7);
                bool bad = false;
                if (s < hi && c < cols) {
                    const uint4 w = __ldg(reinterpret_cast<const uint4*>(v + s * a.v_row + c));
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        bad |= (u[e] & 0x7f80u) == 0x7f80u || (u[e] & 0x7f800000u) == 0x7f800000u;
                }
                hit = __any_sync(0xffffffffu, bad);
            }
        }
        if (!hit) continue;
        const uint4* q = reinterpret_cast<const uint4*>(a.q + b * a.q_batch + i * a.q_row + head * a.q_head);
        float m = -INFINITY, l = 0.0f, o0 = 0.0f, o1 = 0.0f;      // l: this lane's keys; o: columns 2 lane, 2 lane + 1
        bool whole = true;                     // (until every column is NaN)
        for (int part = 0; part < 2; ++part) {
            const int lo = part ? ws : 0, hi = part ? t + 1 : min(p.sink, ws);
            for (int s0 = lo; s0 < hi && whole; s0 += 32) {
                float x = -INFINITY;
                if (s0 + lane < hi) {          // a lane's key
                    const uint4* kq = reinterpret_cast<const uint4*>(k + (s0 + lane) * a.k_row);
                    x = 0.0f;
                    for (int c = 0; c < a.dk / 8; ++c) {
                        const uint4 w = __ldg(kq + c), g = __ldg(q + c);
                        const uint32_t u[4] = {w.x, w.y, w.z, w.w}, h[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x = fmaf(__uint_as_float(u[e] << 16), __uint_as_float(h[e] << 16), x);
                            x = fmaf(__uint_as_float(u[e] & 0xffff0000u), __uint_as_float(h[e] & 0xffff0000u), x);
                        }
                    }
                    x *= a.scale_log2;
                }
                float mn = x;
                for (int w = 16; w > 0; w >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, w));
                mn = fmaxf(m, mn);
                const float f = mn > m ? attn::ex2(m - mn) : 1.0f, pr = attn::ex2(x - (mn == -INFINITY ? 0.0f : mn));
                m = mn;
                l = fmaf(l, f, pr);
                o0 *= f;
                o1 *= f;
                const int n = min(32, hi - s0);
                for (int j = 0; j < n; ++j) {
                    const float w = __shfl_sync(0xffffffffu, pr, j);
                    if (2 * lane < cols) {
                        const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(v + (s0 + j) * a.v_row) + lane);
                        o0 = fmaf(w, __uint_as_float(u << 16), o0);
                        o1 = fmaf(w, __uint_as_float(u & 0xffff0000u), o1);
                    }
                }
                whole = !__all_sync(0xffffffffu, 2 * lane >= cols || (isnan(o0) && isnan(o1)));
            }
        }
        for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
        if (2 * lane < cols)
            reinterpret_cast<uint32_t*>(a.out + (((long long)b * a.Tq + i) * a.Hq + head) * a.dv + 64 * half)[lane] =
                pack_bf16x2(o0 / l, o1 / l);
    }
}

__global__ void __launch_bounds__(kThreads, 1)
window_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                   const __grid_constant__ Args a)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gb = smem_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.y;
    const int n_keys = a.lengths ? min(max(a.lengths[b], 0), a.Tk) : a.Tk;
    const Plan p = make_plan(a, n_keys, blockIdx.x);
    if (p.n == 0) return;                      // all padding
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gb + kOffAbort);
    auto bar = [&](uint32_t i) { return base + kOffBar + 8u * i; };
    const uint64_t lim = a.wait_limit_ns;
    const int nbk = (a.dk + 63) / 64, nbv = (a.dv + 63) / 64;       // 64-column boxes per operand

    if (warp == 0) {
        tmem_alloc(base + kOffTmemSlot, kTmemCols);
        tmem_relinquish();
    }
    auto load_k = [&](int j) {
        const uint32_t s = (uint32_t)(j % kKStages), full = bar(kBarKFull + s);
        mbar_arrive_expect_tx(full, (uint32_t)nbk * kBox);
        for (int c = 0; c < nbk; ++c)
            tma_load_4d(base + kOffK + s * kOp + c * kBox, &tm_k, full, 64 * c, p.head[0] / a.group, p.start(j), b);
    };
    auto load_v = [&](int j) {
        const uint32_t s = (uint32_t)(j % kVStages), full = bar(kBarVFull + s);
        mbar_arrive_expect_tx(full, (uint32_t)nbv * kBox);
        for (int c = 0; c < nbv; ++c)
            tma_load_4d(base + kOffV + s * kOp + c * kBox, &tm_v, full, 64 * c, p.head[0] / a.group, p.start(j), b);
    };
    if (warp == kLoadWarp && lane == 0) {
        // the first copies start beside the allocation
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        for (uint32_t i = 0; i < kNumBars; ++i) mbar_init(bar(i), bar_count(i));
        fence_mbar_init();
        *abort_flag = 0;
        const uint32_t live = (p.p_hi[0] >= p.p_lo[0] ? 1u : 0u) + (p.p_hi[1] >= p.p_lo[1] ? 1u : 0u);
        mbar_arrive_expect_tx(bar(kBarQ), live * (uint32_t)nbk * kBox);
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (p.p_hi[q] >= p.p_lo[q])
                for (int c = 0; c < nbk; ++c)
                    tma_load_4d(base + kOffQ + q * kOp + c * kBox, &tm_q, bar(kBarQ), 64 * c, p.head[q], p.row0[q], b);
        load_k(0);
        load_v(0);
        tma_prefetch_desc(&tm_o);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gb + kOffTmemSlot);

    if (warp == kLoadWarp) {
        // ======================= copies =======================
        if (lane == 0) {
            bool ok = true;
            int k_issued = 1, v_issued = 1;
            for (int j = 1; ok && j < p.n; ++j) {
                if (j >= kKStages)
                    ok = mbar_wait(bar(kBarKFree + j % kKStages), (uint32_t)((j / kKStages - 1) & 1), abort_flag, lim, 41);
                if (!ok) break;
                load_k(j);
                k_issued = j + 1;
                if (j >= kVStages)
                    ok = mbar_wait(bar(kBarVFree + j % kVStages), (uint32_t)((j / kVStages - 1) & 1), abort_flag, lim, 42);
                if (!ok) break;
                load_v(j);
                v_issued = j + 1;
            }
            // copies land before shared memory goes away, whoever gave up: the last one of each stage is
            // enough (a stage is refilled only after its tile was read)
            drain_wait(bar(kBarQ), 0);
            for (int j = max(0, k_issued - kKStages); j < k_issued; ++j)
                drain_wait(bar(kBarKFull + j % kKStages), (uint32_t)((j / kKStages) & 1));
            for (int j = max(0, v_issued - kVStages); j < v_issued; ++j)
                drain_wait(bar(kBarVFull + j % kVStages), (uint32_t)((j / kVStages) & 1));
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ======================= MMAs (one thread issues them all) =======================
        if (elect_one()) {
            const int nks = a.dk / 16;
            const uint32_t idpv = idesc_bf16(128, a.dv, false, true);
            const uint64_t q0desc = kmaj(base + kOffQ), k0desc = kmaj(base + kOffK);
            const uint64_t v0desc = smem_desc(base + kOffV, kBox, 1024, kSwizzle128);
            uint32_t sk = 0, pk = 0, sv = 0, pv = 0;       // stage and phase of K(j) and of V(j - 1)
            uint32_t steps[2] = {0, 0};                    // key tiles whose P V was issued
            bool ok = mbar_poll(bar(kBarQ), 0, abort_flag, lim, 43);
#pragma unroll 1
            for (int j = 0; ok && j <= p.n; ++j) {
                const bool dopv[2] = {j >= 1 && p.active(0, j - 1), j >= 1 && p.active(1, j - 1)};
                const bool doqk[2] = {j < p.n && p.active(0, j), j < p.n && p.active(1, j)};
                if (j >= 1) ok = mbar_poll(bar(kBarVFull + sv), pv, abort_flag, lim, 44);
                if (j < p.n) ok = ok && mbar_poll(bar(kBarKFull + sk), pk, abort_flag, lim, 46);
                if (!ok) break;
                const uint64_t vdesc = v0desc + sv * (kOp >> 4), kdesc = k0desc + sk * (kOp >> 4);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint32_t s = tmem + kColS + 128u * q + 64u * h;
                        if (dopv[q]) {
                            ok = ok && mbar_poll(bar(kBarP + 2 * q + h), steps[q] & 1u, abort_flag, lim, 45);
                            if (!ok) break;
                            tc_fence_after();
                            // a K step of 16 keys: 8 columns of P, 2048 bytes (128 descriptor units) of V
#pragma unroll
                            for (int ks = 0; ks < kBN / 32; ++ks)
                                mma_bf16_tmem_a(tmem + kColO + 128u * q, s + 8u * ks, vdesc + 128u * (4 * h + ks), idpv,
                                                (steps[q] > 0 || h + ks > 0) ? 1u : 0u);
                            mma_commit(bar(kBarH + 2 * q + h));
                            if (h == 1) {
                                ++steps[q];
                                if (q == 1 || !dopv[1]) mma_commit(bar(kBarVFree + sv));
                                if (j == p.end[q]) mma_commit(bar(kBarO + q));
                            }
                        }
                        if (doqk[q]) {
                            // keys 64 h .. of the tile (8192 bytes on); a K step of 16 head elements: 32 bytes inside a
                            // box, four of them per box
                            const uint64_t qdesc = q0desc + q * (kOp >> 4), kd = kdesc + 512u * h;
#pragma unroll
                            for (int ks = 0; ks < 8; ++ks)
                                if (ks < nks)
                                    mma_bf16(s, qdesc + (ks >> 2) * (kBox >> 4) + 2u * (ks & 3),
                                             kd + (ks >> 2) * (kBox >> 4) + 2u * (ks & 3), kIdS, ks > 0);
                            mma_commit(bar(kBarS + 2 * q + h));
                            if (h == 1 && (q == 1 || !doqk[1])) mma_commit(bar(kBarKFree + sk));
                        }
                    }
                    if (!ok) break;
                }
                if (j >= 1 && ++sv == kVStages) { sv = 0; pv ^= 1u; }
                if (++sk == kKStages) { sk = 0; pk ^= 1u; }
            }
            // every MMA is done before shared memory and TMEM go away, whoever gave up
            mma_commit(bar(kBarDrain));
            drain_wait(bar(kBarDrain), 0);
        }
        __syncwarp();
    } else {
        // ======================= softmax of tile q, two threads per row =======================
        // Thread 0 of a row has keys 0-63 of each tile, thread 1 keys 64-127.  The row's reference m is both
        // threads': each weighs with the last it knows, and before it stores its weights (thread 0's of tile
        // i after thread 1's of tile i - 1, thread 1's after thread 0's of the same tile) it looks whether the
        // other has moved m meanwhile; whoever moves it rescales O.
        const int q = warp / kTileWarps, half = (warp >> 2) & 1;
        const int p_lo = q ? p.p_lo[1] : p.p_lo[0], p_hi = q ? p.p_hi[1] : p.p_hi[0];
        const int row0 = q ? p.row0[1] : p.row0[0], head = q ? p.head[1] : p.head[0];
        const int first_end = q ? p.first_end[1] : p.first_end[0], near = q ? p.near[1] : p.near[0];
        const int end = q ? p.end[1] : p.end[0];
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ts = lane_base + kColS + 128u * q, th = ts + 64u * half, to = lane_base + kColO + 128u * q;
        const uint32_t bar_s = bar(kBarS + 2 * q + half), bar_p = bar(kBarP + 2 * q + half);
        const uint32_t bar_other = bar(kBarP + 2 * q + (half ^ 1));
        const int row = (warp & 3) * 32 + lane;
        const int t = p_lo + row;                             // this row's position
        const int ws = max(0, t - a.window + 1);
        const bool split = p.startB > 0 || p.nA > 0;
        volatile float* m_row = reinterpret_cast<volatile float*>(gb + kOffM) + q * kBM + row;
        float m_ref = -INFINITY, l = 0.0f;
        bool ok = true, settled = false;                      // settled: every row of the warp has a reference
        int i = 0;                                            // key tiles taken
        auto wait = [&](uint32_t b_, uint32_t parity, int code) {
            ok = __all_sync(0xffffffffu, mbar_wait(b_, parity & 1u, abort_flag, lim, code));
            return ok;
        };
        // Both threads of a row end up with join(thread 0's word), computed by thread 1.
        auto swap = [&](auto&& join, float& word, uint32_t parity) {
            if (half == 1) {
                if (!wait(bar(kBarL + 2 * q), parity, 54)) return false;
                word = join(*m_row);
            }
            *m_row = word;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarL + 2 * q + half));
            if (half == 0) {
                if (!wait(bar(kBarL + 2 * q + 1), parity, 54)) return false;
                word = *m_row;
            }
            return true;
        };
        // the first tile from j on that this query tile sees
        auto seen = [&](int j) { return j < first_end ? j : j < near ? near : j; };
#pragma unroll 1
        for (int j = seen(0); j < end; j = seen(j + 1)) {
            const int s0 = p.start(j);
            const bool sink_tile = j < p.nA;
            // columns [lo, hi] are in the row's window, columns below sk among the sinks
            const int hi = sink_tile ? -1 : min(t, n_keys - 1) - s0;
            const int lo = ws - s0, sk = (split && !sink_tile) ? 0 : min(p.sink, t + 1) - s0;
            const bool masked = __any_sync(0xffffffffu, !((lo <= 0 && hi >= kBN - 1) || sk >= kBN));
            auto mask = [&](float (&x)[32], int c) {          // x: columns 32 c ..
                if (masked) {
                    const uint32_t keep = (low_bits(hi + 1 - 32 * c) & ~low_bits(lo - 32 * c)) | low_bits(sk - 32 * c);
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = (keep & (1u << e)) ? x[e] : -INFINITY;
                }
            };
            // rows of V past what any query of this tile sees (padding; beside the sinks of a tile that is no
            // window's) hold anything: zero times that must be zero
            const int v_end = sink_tile ? p.sink : n_keys;
            if (half == 0 && v_end - s0 < kBN && (sink_tile || n_keys < a.Tk)) {
                const uint32_t v = base + kOffV + (uint32_t)(j % kVStages) * kOp;
                if (!wait(bar(kBarVFull + j % kVStages), (uint32_t)(j / kVStages), 49)) break;
                for (int r = (v_end - s0) * 8 + row; r < kBN * 8; r += kBM)
                    for (int c = 0; c < nbv; ++c) st_shared_v4(v + c * kBox + 16u * r, 0, 0, 0, 0);
                fence_proxy_async_smem();
            }
            // what the other thread made of the reference, once its weights before these are stored
            auto follow = [&]() {
                if (half == 0 && i == 0) return true;
                if (!wait(bar_other, (uint32_t)(half ? i : i - 1), 51)) return false;
                const float mn = *m_row;
                if (mn != m_ref) {
                    l *= attn::ex2(m_ref - mn);
                    m_ref = mn;
                }
                return true;
            };
            // a reference for the row: above the largest score among this thread's columns
            auto above = [&]() {
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float x[32];
                    tmem_ld32(th + 32u * c, x);
                    tmem_wait32(x);
                    mask(x, 2 * half + c);
#pragma unroll
                    for (int e = 0; e < 16; ++e) mx[e & 3] = attn::max3f(mx[e & 3], x[2 * e], x[2 * e + 1]);
                }
                return fmaf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), a.scale_log2, kAbove);
            };
            // Moves the references up to it, and O along, once it is complete up to here.
            auto look_up = [&]() {
                const bool none = half == 0 && i == 0;        // no P V yet
                if (!none && !wait(bar(kBarH + 2 * q + (half ^ 1)), (uint32_t)(half ? i : i - 1), 50)) return false;
                tc_fence_after();
                const float mn = fmaxf(m_ref, above());
                const float alpha = mn > m_ref ? attn::ex2(m_ref - mn) : 1.0f;
                l *= alpha;
                m_ref = mn;
                *m_row = mn;
                // (TMEM accesses are warp-collective: the other rows' alpha is 1)
                if (!none) {
#pragma unroll 1
                    for (int c = 0; c < a.dv / 16; ++c) {
                        float o[16];
                        tmem_ld16(to + 16u * c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] *= alpha;
                        attn::tmem_st16(to + 16u * c, o);
                    }
                }
                return true;
            };
            if (!wait(bar_s, (uint32_t)i, 47)) break;
            tc_fence_after();
            if (i == 0) {
                m_ref = above();
                if (!swap([&](float other) { m_ref = fmaxf(m_ref, other); return m_ref; }, m_ref, 0)) break;
                settled = !__any_sync(0xffffffffu, m_ref == -INFINITY);
            } else if (!settled) {
                if (!follow()) break;
                if (__any_sync(0xffffffffu, m_ref == -INFINITY) && !look_up()) break;
                settled = !__any_sync(0xffffffffu, m_ref == -INFINITY);
            }
            // 2^(x scale - m) without looking for the maximum first: m is above a score of an earlier tile.
            uint32_t pk[32];
            float sum;
            bool looked = !settled;
            while (true) {
                const float neg_mr = (m_ref == -INFINITY) ? 0.0f : -m_ref;
                const uint64_t sc2 = attn::f2pack(a.scale_log2, a.scale_log2), nm2 = attn::f2pack(neg_mr, neg_mr);
                uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float x[32];
                    tmem_ld32(th + 32u * c, x);
                    tmem_wait32(x);
                    mask(x, 2 * half + c);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float p0, p1;
                        attn::f2unpack(attn::fma2(attn::f2pack(x[2 * e], x[2 * e + 1]), sc2, nm2), p0, p1);
                        p0 = attn::ex2(p0);
                        p1 = attn::ex2(p1);
                        acc[e & 3] = attn::add2(acc[e & 3], attn::f2pack(p0, p1));
                        pk[16 * c + e] = pack_bf16x2(p0, p1);
                    }
                }
                float sm[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) attn::f2unpack(acc[e], sm[2 * e], sm[2 * e + 1]);
                sum = ((sm[0] + sm[1]) + (sm[2] + sm[3])) + ((sm[4] + sm[5]) + (sm[6] + sm[7]));
                // a reference that the other thread has moved, or a score far above it
                const float m_old = m_ref;
                if (half == 1 || i > 0) {
                    if (!wait(bar_other, (uint32_t)(half ? i : i - 1), 51)) break;
                    m_ref = *m_row;
                }
                const bool stale = m_ref != m_old, far = !(sum <= kMaxSum) && !looked;
                if (!__any_sync(0xffffffffu, stale || far)) break;
                l *= stale ? attn::ex2(m_old - m_ref) : 1.0f;
                if (!__any_sync(0xffffffffu, stale)) {
                    if (!look_up()) break;
                    looked = true;
                }
            }
            if (!ok) break;
            l += sum;
            attn::tmem_st16u(th, pk);
            attn::tmem_st16u(th + 16u, pk + 16);
            attn::tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_p);
            ++i;
        }
        // (thread 0 may have to follow thread 1 once more)
        if (ok && i > 0 && wait(bar(kBarO + q), 0, 48) && (half == 1 || wait(bar_other, (uint32_t)(i - 1), 51))) {
            tc_fence_after();
            if (half == 0 && *m_row != m_ref) l *= attn::ex2(m_ref - *m_row);
            float total = l;
            if (swap([&](float other) { return l + other; }, total, 1)) {
                // thread `half` of a row takes 64 columns, one box; O / l in bf16 goes out through the tile's
                // place in Q (its last S is done), 32 rows a warp by one copy, which leaves rows past the
                // last query alone.  A tile that `lengths` cuts short writes its rows one by one.
                const float inv = 1.0f / total;
                const int groups = min(4, a.dv / 16 - 4 * half);
                const bool cut = p_hi + 1 < a.Tk - a.Tq + min(row0 + kBM, a.Tq);
                const uint32_t stage = base + kOffQ + q * kOp + half * kBox + (uint32_t)row * 128u;
                __nv_bfloat16* orow = a.out + (((long long)b * a.Tq + row0 + row) * a.Hq + head) * a.dv + 64 * half;
                uint64_t zero = 0ull;                         // O times 0: NaN where O is not finite
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c >= groups) break;
                    float o[16];
                    tmem_ld16(to + 64u * half + 16u * c, o);
                    tmem_wait_ld();
                    uint32_t w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        zero = attn::fma2(attn::f2pack(o[2 * e], o[2 * e + 1]), 0ull, zero);
                        w[e] = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
                    }
                    if (!cut) {
                        st_shared_v4(stage + (uint32_t)(((2 * c) ^ (row & 7)) << 4), w[0], w[1], w[2], w[3]);
                        st_shared_v4(stage + (uint32_t)(((2 * c + 1) ^ (row & 7)) << 4), w[4], w[5], w[6], w[7]);
                    } else if (t <= p_hi) {
                        reinterpret_cast<uint4*>(orow + 16 * c)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                        reinterpret_cast<uint4*>(orow + 16 * c)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                    }
                }
                const int first = row0 + 32 * (warp & 3);
                float z0, z1;
                attn::f2unpack(zero, z0, z1);
                const bool redo = __any_sync(0xffffffffu, t <= p_hi && !(z0 + z1 == 0.0f));
                if (!cut && groups > 0 && first < a.Tq) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_4d(&tm_o, stage, 64 * half, head, first, b);
                        bulk_commit_group();
                        bulk_wait_group_read0();
                    }
                    __syncwarp();
                }
                if (redo) redo_rows(a);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

}  // namespace tc

// ---- one token per session ----
//
// The cache is read once for all query heads of a key head, so HBM bounds it.  Sixteen query
// heads are the rows of mma.sync m16n8k16 tiles (tcgen05 takes 64 rows at least, of which a
// group fills a few): with 16 slots a tile, a warp's scores, softmax and P V stay in its
// registers, and a warp needs no other one until the end.  Each warp streams its tiles
// (every warp of the cluster takes its turn) through a private ring of TMA boxes, so
// kStages - 1 tiles per warp are in flight, a tile costs one thread a few instructions to fetch,
// and no barrier of the CTA stands in the loop.  The cluster's CTAs
// split one session and key head; the warps' partial sums (maximum, sum, O) meet in shared
// memory, the CTAs' through distributed shared memory in a fixed order: one launch, no
// workspace, the same bits every time.  P enters as a bf16 pair (value and remainder), since
// the tensor cores have time to spare here: the result is rounded once, like a plain form's.
namespace step {

using namespace sm100;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kRows = 16, kSlots = 16;         // query heads, cache slots per tile
constexpr int kMaxCluster = 8;
// Three stages and two CTAs per SM (96 KB of copies in flight at d 128); two stages and three CTAs
// measured 139 against 138 us on 64 sessions of up to 4160 slots, 184 against 162 us on full ones.
constexpr int kStages = 3, kCtas = 2;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// One stage: 16 rows of K and of V as 64-column boxes of 16 x 128 bytes in the 128-byte swizzle,
// under which the 8 rows of an ldmatrix fall on different banks.
constexpr uint32_t kBox = kSlots * 128u;
__host__ __device__ constexpr uint32_t boxes(int d) { return (uint32_t)(d + 63) / 64u; }
__host__ __device__ constexpr uint32_t stage_bytes(int dk, int dv) { return kBox * (boxes(dk) + boxes(dv)); }
__device__ __forceinline__ uint32_t chunk_offset(int row, int chunk) {      // of 16 bytes of a row
    return (uint32_t)(chunk >> 3) * kBox + (uint32_t)row * 128u + (uint32_t)(((chunk & 7) ^ (row & 7)) << 4);
}
__host__ __device__ constexpr uint32_t part_floats(int dv) { return kRows * (dv + 2); }   // m, l and O of 16 rows
__host__ __device__ constexpr uint32_t smem_bytes(int dk, int dv) {
    const uint32_t ring = kWarps * kStages * stage_bytes(dk, dv), parts = (kWarps + 1) * part_floats(dv) * 4;
    return (ring > parts ? ring : parts) + 8u * kWarps * kStages + 16u + 1024u;   // + barriers, the abort flag, alignment
}

// DK16, DV16: the head sizes in units of 16, rounded up to whole boxes; the columns past a head's
// size are zeros (the copies fill them, Q has zeros there) and are not stored.
template <int DK16, int DV16>
__global__ void __launch_bounds__(kThreads, kCtas)
window_step_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const StepArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int X = (int)cluster_size(), rank = (int)cluster_rank();
    const int G = a.Hq / a.Hkv, parts = (G + kRows - 1) / kRows;
    const int unit = blockIdx.x / X, hk = unit / parts, g0 = (unit % parts) * kRows, b = blockIdx.y;
    const long long pos = a.pos[b];
    const uint32_t nbk = boxes(a.dk), nbv = boxes(a.dv), sb = stage_bytes(a.dk, a.dv);
    const uint32_t ring = smem_u32(smem) + warp * kStages * sb;
    const uint32_t tail = smem_bytes(a.dk, a.dv) - 8u * kWarps * kStages - 16u - 1024u;
    const uint32_t bars = smem_u32(smem) + tail + 8u * kStages * warp;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + tail + 8u * kStages * kWarps);
    if (lane < kStages) mbar_init(bars + 8u * lane, 1);
    if (tid == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        *abort_flag = 0;
    }
    fence_mbar_init();
    __syncthreads();
    if (pos < 0) {                             // idle: the whole cluster leaves
        uint4* row = reinterpret_cast<uint4*>(a.out + ((long long)b * a.Hq + hk * G + g0) * a.dv);
        if (a.zero_idle && rank == 0)
            for (int i = tid; i < min(kRows, G - g0) * a.dv / 8; i += kThreads) row[i] = make_uint4(0, 0, 0, 0);
        return;
    }
    const int cap = a.window + a.sinks;
    const int slot = (int)cache_slot(pos, a.window, a.sinks);
    const int seen = pos + 1 < cap ? (int)(pos + 1) : cap;
    const int rows = min(kRows, G - g0);
    const int nk = a.dk / 16, nv = a.dv / 16;
    const __nv_bfloat16* kn = a.k + b * a.k_batch + hk * a.dk;
    const __nv_bfloat16* vn = a.v + b * a.v_batch + hk * a.dv;
    __nv_bfloat16* kc = a.k_cache + ((long long)b * cap * a.Hkv + hk) * a.dk;
    __nv_bfloat16* vc = a.v_cache + ((long long)b * cap * a.Hkv + hk) * a.dv;
    const long long kr = (long long)a.Hkv * a.dk, vr = (long long)a.Hkv * a.dv;

    const int tiles = (seen + kSlots - 1) / kSlots, stride = X * kWarps, first = rank * kWarps + warp;
    auto fetch = [&](int tile, int stage) {
        if (lane == 0) {
            const uint32_t dst = ring + stage * sb, bar = bars + 8u * stage;
            mbar_arrive_expect_tx(bar, sb);
            for (uint32_t c = 0; c < nbk; ++c) tma_load_4d(dst + c * kBox, &tm_k, bar, 64 * c, hk, tile * kSlots, b);
            for (uint32_t c = 0; c < nbv; ++c)
                tma_load_4d(dst + (nbk + c) * kBox, &tm_v, bar, 64 * c, hk, tile * kSlots, b);
        }
        __syncwarp();
    };

    int issued = 0, taken = 0;                 // tiles of this warp
    for (; issued < kStages - 1 && first + issued * stride < tiles; ++issued) fetch(first + issued * stride, issued);

    // Q as A fragments: row r = lane / 4 (and + 8), columns 2 (lane % 4) (and + 8) of each 16
    uint32_t qa[DK16][4];
    {
        const __nv_bfloat16* q = a.q + b * a.q_batch + (long long)(hk * G + g0) * a.dk;
        const int r = lane >> 2, c = 2 * (lane & 3);
#pragma unroll
        for (int i = 0; i < DK16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int rr = r + 8 * (e & 1), cc = 16 * i + c + 8 * (e >> 1);
                qa[i][e] = (rr < rows && i < nk) ? *reinterpret_cast<const uint32_t*>(q + (long long)rr * a.dk + cc) : 0u;
            }
    }

    float o[2 * DV16][4];
#pragma unroll
    for (int i = 0; i < 2 * DV16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};     // rows lane / 4 and + 8; l: this thread's columns
    const float sc = a.scale * 1.4426950408889634f;

    // this lane's rows of an ldmatrix: the 16-byte chunk of step i is this one with bits 5 and 6 flipped by i
    const uint32_t ka0 = chunk_offset((lane & 7) + 8 * (lane >> 4), (lane >> 3) & 1);
    const uint32_t va0 = chunk_offset(lane & 15, lane >> 4);
    for (int tile = first; tile < tiles; tile += stride) {
        const int st = taken % kStages;
        if (!__all_sync(0xffffffffu, mbar_wait(bars + 8u * st, (uint32_t)(taken / kStages) & 1u, abort_flag, a.wait_limit_ns, 51)))
            break;
        ++taken;
        // the stage read last (its reads are over for the whole warp) takes the next tile
        if (first + issued * stride < tiles) {
            fetch(first + issued * stride, issued % kStages);
            ++issued;
        }
        const uint32_t kd = ring + st * sb, vd = kd + nbk * kBox;
        // The copy may have brought what must not count: the new token's rows stand in k and v, not in
        // their slot, and V rows past the last slot seen (zero times which must be zero) hold anything.
        const int mine = slot - tile * kSlots, past = seen - tile * kSlots;
        if ((mine >= 0 && mine < kSlots) || past < kSlots) {
            if (mine >= 0 && mine < kSlots) {
                for (int c = lane; c < a.dk / 8; c += 32) {
                    const uint4 w = __ldg(reinterpret_cast<const uint4*>(kn) + c);
                    st_shared_v4(kd + chunk_offset(mine, c), w.x, w.y, w.z, w.w);
                }
                for (int c = lane; c < a.dv / 8; c += 32) {
                    const uint4 w = __ldg(reinterpret_cast<const uint4*>(vn) + c);
                    st_shared_v4(vd + chunk_offset(mine, c), w.x, w.y, w.z, w.w);
                }
            }
            for (int i = max(past, 0) * 8 + lane; i < kSlots * 8; i += 32)
                for (uint32_t c = 0; c < nbv; ++c) st_shared_v4(vd + c * kBox + 16u * i, 0, 0, 0, 0);
            fence_proxy_async_smem();          // before a later copy into this stage
            __syncwarp();
        }
        // S [16 x 16] = Q K^T: K rows are the columns of B; a x4 load brings slots 0-7 and 8-15, both halves of 16 d
        // (two sums of every other 16 d: half as long a chain of dependent products)
        float s[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}}, s2[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        const uint32_t ka = kd + ka0;
#pragma unroll
        for (int i = 0; i < DK16; ++i) {
            uint32_t f[4];
            ldsm4(f, (ka ^ (uint32_t)((i & 3) << 5)) + (i >> 2) * kBox);
            mma16816((i & 1) ? s2[0] : s[0], qa[i], f[0], f[1]);
            mma16816((i & 1) ? s2[1] : s[1], qa[i], f[2], f[3]);
        }
        // online softmax of this warp's slots; columns 2 (lane % 4) + {0, 1} of each 8
        const int left = seen - tile * kSlots;
        float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int col = 8 * h + 2 * (lane & 3) + (e & 1);
                s[h][e] = col < left ? (s[h][e] + s2[h][e]) * sc : -INFINITY;
                mt[e >> 1] = fmaxf(mt[e >> 1], s[h][e]);
            }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            mt[r] = fmaxf(mt[r], __shfl_xor_sync(0xffffffffu, mt[r], 1));
            mt[r] = fmaxf(mt[r], __shfl_xor_sync(0xffffffffu, mt[r], 2));
        }
        // -inf as long as every score was; then the weights are 0, against a reference of 0
        const float mn[2] = {fmaxf(m[0], mt[0]), fmaxf(m[1], mt[1])};
        if (__any_sync(0xffffffffu, mn[0] > m[0] || mn[1] > m[1])) {
            const float f[2] = {mn[0] == -INFINITY ? 1.0f : attn::ex2(m[0] - mn[0]),
                                mn[1] == -INFINITY ? 1.0f : attn::ex2(m[1] - mn[1])};
            l[0] *= f[0];
            l[1] *= f[1];
#pragma unroll
            for (int i = 0; i < 2 * DV16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] *= f[e >> 1];
            m[0] = mn[0];
            m[1] = mn[1];
        }
        // P as A fragments (the layout of S as it is), split into a bf16 value and its remainder
        uint32_t ph[4], pl[4];
        const float ref[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float p0 = attn::ex2(s[h][2 * r] - ref[r]), p1 = attn::ex2(s[h][2 * r + 1] - ref[r]);
                l[r] += p0 + p1;
                const uint32_t hi = pack_bf16x2(p0, p1);
                ph[2 * h + r] = hi;
                pl[2 * h + r] = pack_bf16x2(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u));
            }
        // O += P V: V rows are the K axis of B, read transposed; a x4 load brings 16 slots of 16 columns
        const uint32_t va = vd + va0;
#pragma unroll
        for (int i = 0; i < DV16; ++i) {
            uint32_t f[4];
            ldsm4t(f, (va ^ (uint32_t)((i & 3) << 5)) + (i >> 2) * kBox);
            mma16816(o[2 * i], ph, f[0], f[1]);
            mma16816(o[2 * i + 1], ph, f[2], f[3]);
            mma16816(o[2 * i], pl, f[0], f[1]);
            mma16816(o[2 * i + 1], pl, f[2], f[3]);
        }
    }
    // after a wait that gave up: the copies in flight land before the ring is used for anything else
    if (lane == 0)
        for (int i = taken; i < issued; ++i) drain_wait(bars + 8u * (i % kStages), (uint32_t)(i / kStages) & 1u);
    __syncwarp();
    // the new token goes into the cache (one writer; no one reads that slot from it in this call)
    if (g0 == 0 && slot / kSlots % stride == first) {
        for (int i = lane; i < a.dk / 8; i += 32)
            reinterpret_cast<uint4*>(kc + slot * kr)[i] = __ldg(reinterpret_cast<const uint4*>(kn) + i);
        for (int i = lane; i < a.dv / 8; i += 32)
            reinterpret_cast<uint4*>(vc + slot * vr)[i] = __ldg(reinterpret_cast<const uint4*>(vn) + i);
    }

    // ---- partial results: [warp][16 rows][m, l, O], then the CTA's over warp 0 .. kWarps - 1 ----
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    __syncthreads();                           // every warp is done with its ring
    float* part = reinterpret_cast<float*>(smem);
    const int pr = a.dv + 2, pw = kRows * pr;
    {
        float* w = part + (warp + 1) * pw;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if ((lane >> 2) + 8 * r >= rows) continue;
            float* row = w + ((lane >> 2) + 8 * r) * pr;
            if ((lane & 3) == 0) {
                row[0] = m[r];
                row[1] = l[r];
            }
#pragma unroll
            for (int i = 0; i < 2 * DV16; ++i)
                if (i < 2 * nv) {
                    row[2 + 8 * i + 2 * (lane & 3)] = o[i][2 * r];
                    row[3 + 8 * i + 2 * (lane & 3)] = o[i][2 * r + 1];
                }
        }
    }
    __syncthreads();
    // merge the warps of this CTA into part 0; rows past the group's heads are not looked at
    for (int i = tid; i < rows * a.dv; i += kThreads) {
        const int r = i / a.dv, c = i - r * a.dv;
        float M = -INFINITY, L = 0.0f, O = 0.0f;
#pragma unroll
        for (int w = 1; w <= kWarps; ++w) M = fmaxf(M, part[w * pw + r * pr]);
#pragma unroll
        for (int w = 1; w <= kWarps; ++w) {
            const float* row = part + w * pw + r * pr;
            const float f = row[0] == -INFINITY ? 0.0f : attn::ex2(row[0] - M);
            L = fmaf(f, row[1], L);
            O = fmaf(f, row[2 + c], O);
        }
        part[r * pr + 2 + c] = O;
        if (c == 0) {
            part[r * pr] = M;
            part[r * pr + 1] = L;
        }
    }
    if (X > 1) cluster_sync();
    else __syncthreads();
    // each CTA of the cluster finishes its share of the outputs
    const uint32_t p0 = smem_u32(part);
    __nv_bfloat16* out = a.out + ((long long)b * a.Hq + hk * G + g0) * a.dv;
    for (int i = rank * kThreads + tid; i < rows * a.dv; i += X * kThreads) {
        const int r = i / a.dv, c = i - r * a.dv;
        float M = -INFINITY, L = 0.0f, O = 0.0f;
        float mk[kMaxCluster], lk[kMaxCluster], ok[kMaxCluster];
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {          // all loads on their way before the first is used
            mk[k] = k < X ? ld_remote(p0 + 4 * (r * pr), k) : -INFINITY;
            lk[k] = k < X ? ld_remote(p0 + 4 * (r * pr + 1), k) : 0.0f;
            ok[k] = k < X ? ld_remote(p0 + 4 * (r * pr + 2 + c), k) : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) M = fmaxf(M, mk[k]);
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
            const float f = mk[k] == -INFINITY ? 0.0f : attn::ex2(mk[k] - M);
            L = fmaf(f, lk[k], L);
            O = fmaf(f, ok[k], O);
        }
        out[(long long)r * a.dv + c] = __float2bfloat16_rn(O / L);
    }
    if (X > 1) cluster_sync();                 // no CTA leaves while another reads its part
}

template <int DK16, int DV16>
cudaError_t launch(const StepArgs& a, int X, cudaStream_t stream)
{
    const uint32_t smem = smem_bytes(a.dk, a.dv);
    CUtensorMap mk, mv;
    const long long slots = (long long)a.window + a.sinks, H = a.Hkv;
    if (!make_map(&mk, a.k_cache, a.dk, a.Hkv, slots, a.B, kSlots, a.dk, H * a.dk, slots * H * a.dk) ||
        !make_map(&mv, a.v_cache, a.dv, a.Hkv, slots, a.B, kSlots, a.dv, H * a.dv, slots * H * a.dv))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(window_step_kernel<DK16, DV16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    const int parts = (a.Hq / a.Hkv + kRows - 1) / kRows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.Hkv * parts * X), (unsigned)a.B);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)X;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, window_step_kernel<DK16, DV16>, mk, mv, a);
}

}  // namespace step

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
    using namespace window::tc;
    CUtensorMap mq, mk, mv, mo;
    const long long orow = (long long)a.Hq * a.dv;
    if (!window::make_map(&mo, a.out, a.dv, a.Hq, a.Tq, a.B, 32, a.dv, orow, orow * a.Tq) ||
        !window::make_map(&mq, a.q, a.dk, a.Hq, a.Tq, a.B, kBM, a.q_head, a.q_row, a.q_batch) ||
        !window::make_map(&mk, a.k, a.dk, a.Hkv, a.Tk, a.B, kBM, a.k_head, a.k_row, a.k_batch) ||
        !window::make_map(&mv, a.v, a.dv, a.Hkv, a.Tk, a.B, kBM, a.v_head, a.v_row, a.v_batch))
        return cudaErrorInvalidValue;
    // (a per-device setting of the current context: set on every call)
    cudaError_t e = cudaFuncSetAttribute(window_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    Args r;
    r.q = a.q; r.k = a.k; r.v = a.v;
    r.q_batch = a.q_batch; r.q_row = a.q_row; r.q_head = a.q_head;
    r.k_batch = a.k_batch; r.k_row = a.k_row; r.k_head = a.k_head;
    r.v_batch = a.v_batch; r.v_row = a.v_row; r.v_head = a.v_head;
    r.lengths = a.lengths;
    r.out = a.out;
    r.Tq = a.Tq; r.Tk = a.Tk; r.Hq = a.Hq; r.group = a.Hq / a.Hkv; r.dk = a.dk; r.dv = a.dv;
    r.window = a.window; r.sinks = a.sinks;
    r.pair_heads = r.group % 2 == 0;
    const int tiles = (a.Tq + kBM - 1) / kBM;
    r.row_blocks = r.pair_heads ? tiles : (tiles + 1) / 2;
    r.head_blocks = r.pair_heads ? a.Hq / 2 : a.Hq;
    r.scale_log2 = 1.4426950408889634f * a.scale;
    r.wait_limit_ns = g_wait_limit_ns;
    const long long blocks = (long long)r.row_blocks * r.head_blocks;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    window_attn_kernel<<<dim3((unsigned)blocks, (unsigned)a.B), kThreads, kSmemBytes, stream>>>(mq, mk, mv, mo, r);
    return cudaGetLastError();
}

cudaError_t launch_window_step(const StepArgs& a, cudaStream_t stream)
{
    // CTAs per session and key head: doubled while they all fit on the device at once (two per SM) and
    // each warp keeps a tile of its own.  Beyond one wave splitting loses: 64 sessions of 4160 slots on
    // 8 key heads (512 units) take 162 us unsplit and 177 us in halves; 16 sessions of 32,832 slots
    // (128 units) 425 us unsplit and 306 us in halves.
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    StepArgs r = a;
    r.wait_limit_ns = g_wait_limit_ns;
    const long long units = (long long)a.B * a.Hkv * ((a.Hq / a.Hkv + window::step::kRows - 1) / window::step::kRows);
    const long long cap = (long long)a.window + a.sinks;
    int X = 1;
    while (X < window::step::kMaxCluster && units * X <= sms && 2ll * X * window::step::kWarps * window::step::kSlots <= cap) X *= 2;
    if (units * X / a.B > INT32_MAX) return cudaErrorInvalidValue;
    if (a.dk <= 64) return a.dv <= 64 ? window::step::launch<4, 4>(r, X, stream) : window::step::launch<4, 8>(r, X, stream);
    return a.dv <= 64 ? window::step::launch<8, 4>(r, X, stream) : window::step::launch<8, 8>(r, X, stream);
}

cudaError_t launch_window_append(const AppendArgs& a, cudaStream_t stream)
{
    const long long cap = (long long)a.window + a.sinks, items = a.T <= cap ? a.T : cap;
    window::window_append_kernel<<<dim3((unsigned)items, (unsigned)a.B), 128, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn
