// Dense matrix product with its epilogue, FP16 or e4m3 operands:
//
//   y[t][n] = RN16( act( s * sum_k x[t][k] W[n][k] + bias[n] ) + residual[t][n] )
//   s = x_scale[t] * w_scale[n] (e4m3), 1 (FP16);  FP32 sums and epilogue
//
// Both operands are read as rows of 16-byte chunks along k, so FP16 (8 values
// a chunk) and e4m3 (16) share all addressing and differ in the matrix
// instruction only.  In every kernel the weights are the row operand of the
// instruction and the tokens its columns: a lane's four results are four
// consecutive outputs n of one token.
//   linear_stream_kernel: few tokens, bound by reading W once from HBM;
//   linear_tile_kernel: many tokens, bound by the matrix cores and LDS; where
//   its tiles are too few for the GPU, k is divided among blocks and
//   linear_join_kernel adds the splits in their order.
#include "moe_internal.h"

#include <algorithm>

namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;

struct LinearArgs {
    const uint8_t *x, *w;
    long long ldx, ldw;                  // bytes
    const float *x_scale, *w_scale;      // e4m3 only
    const float *bias;                   // [N] or null
    const uint16_t *res;                 // [T][ldr] or null
    long long ldr;
    uint16_t *y;
    long long ldy;
    int T, N, chunks;                    // chunks: 16-byte chunks of a row
    int act;
    float *planes;                       // [splits][T][plane_ld] partial sums, or null: k is not divided
    int plane_ld;                        // N rounded up to 8
    int split_steps;                     // 128-byte steps of k per split
};

// Rows of y and of the residual may start at any element: 16-byte accesses
// that assume element alignment only.
struct __attribute__((packed, aligned(2))) Out8 { half8 v; };

// v / (1 + exp(-u)) with the hardware's reciprocal and exponential (each within
// about a step of FP32, far below the output's FP16 rounding); exp overflows to
// infinity for far negative u and the result is then 0.
__device__ inline float gate(float v, float u)
{
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u * -1.44269504f));
}

// v Phi(v) = max(v, 0) - |v|/2 erfc(|v| / sqrt 2).  erfc(z) = exp(-z^2) P(t),
// t = 1 / (1 + 0.37 z), P of degree 7 without a constant term: a weighted
// least-squares fit of exp(z^2) erfc(z), made equal-rippled by reweighting;
// relative error 1.7e-6 in FP32 over z <= 12 (past it the product is 0 in FP16).
__device__ inline float gelu(float v)
{
    const float u = fminf(fabsf(v), 64.0f);
    const float t = __builtin_amdgcn_rcpf(fmaf(u, 0.26162952f, 1.0f));
    float p = -0.138180092f;
    p = fmaf(p, t, 0.419946969f);
    p = fmaf(p, t, -0.163837433f);
    p = fmaf(p, t, 0.300842702f);
    p = fmaf(p, t, 0.159155518f);
    p = fmaf(p, t, 0.21359317f);
    p = fmaf(p, t, 0.208480641f);
    const float tail = 0.5f * u * t * p * __builtin_amdgcn_exp2f(u * u * -0.72134752f);
    return (v < 0.0f ? 0.0f : v) - tail;         // a NaN stays one
}

// What the epilogue needs of outputs n .. n+7, read once per lane.
template <bool E4M3>
struct Columns {
    float scale[8], bias[8];
    int n, m;                            // first output, and how many of the 8 are inside the matrix

    __device__ inline void load(const LinearArgs &a, int first)
    {
        n = first;
        m = min(8, a.N - n);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            scale[r] = E4M3 ? a.w_scale[min(n + r, a.N - 1)] : 1.0f;
            bias[r] = 0.0f;
        }
        if (!a.bias) return;
#pragma unroll
        for (int r = 0; r < 8; ++r) bias[r] = a.bias[min(n + r, a.N - 1)];
    }

    __device__ inline half8 residual(const LinearArgs &a, int t) const
    {
        half8 h = {};
        if (!a.res || t >= a.T || m <= 0) return h;
        const uint16_t *res = a.res + (long long)t * a.ldr + n;
        if (m == 8) return reinterpret_cast<const Out8 *>(res)->v;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const _Float16 f = __builtin_bit_cast(_Float16, res[min(r, m - 1)]);
            h[r] = f;
        }
        return h;
    }

    // The 8 sums of token t as they are, to split `split`'s plane.
    __device__ inline void store_plane(const LinearArgs &a, int split, int t, f32x4 lo, f32x4 hi) const
    {
        if (t >= a.T || m <= 0) return;
        f32x4 *o = reinterpret_cast<f32x4 *>(a.planes + ((long long)split * a.T + t) * a.plane_ld + n);
        o[0] = lo;
        o[1] = hi;
    }

    // The 8 outputs of tokens t[0 .. U) from their sums (lo, hi), the tokens' scales and residuals.
    template <int U>
    __device__ inline void finish(const LinearArgs &a, const int (&t)[U], const f32x4 (&lo)[U], const f32x4 (&hi)[U],
                                  const float (&sx)[U], const half8 (&res)[U]) const
    {
        float v[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const float s = r < 4 ? lo[u][r] : hi[u][r - 4];
                v[u][r] = E4M3 ? fmaf(s, sx[u] * scale[r], bias[r]) : s + bias[r];
            }
        if (a.act == MOE_ACT_SILU) {
#pragma unroll
            for (int i = 0; i < 8 * U; ++i) v[i / 8][i % 8] = gate(v[i / 8][i % 8], v[i / 8][i % 8]);
        } else if (a.act == MOE_ACT_GELU) {
#pragma unroll
            for (int i = 0; i < 8 * U; ++i) v[i / 8][i % 8] = gelu(v[i / 8][i % 8]);
        } else if (a.act == MOE_ACT_GELU_TANH) {
            // 0.5 v (1 + tanh u) = v / (1 + exp(-2u)), u = sqrt(2/pi) (v + 0.044715 v^3)
#pragma unroll
            for (int i = 0; i < 8 * U; ++i) {
                const float w = v[i / 8][i % 8];
                v[i / 8][i % 8] = gate(w, w * fmaf(0.07135481627f * w, w, 1.5957691216f));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            half8 o;
#pragma unroll
            for (int r = 0; r < 8; ++r) o[r] = (_Float16)(v[u][r] + (float)res[u][r]);
            if (t[u] >= a.T || m <= 0) continue;
            uint16_t *y = a.y + (long long)t[u] * a.ldy + n;
            if (m == 8) {
                reinterpret_cast<Out8 *>(y)->v = o;
            } else {
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const _Float16 h = o[r];
                    if (r < m) y[r] = __builtin_bit_cast(uint16_t, h);
                }
            }
        }
    }
    __device__ inline void finish(const LinearArgs &a, int t, f32x4 lo, f32x4 hi, float sx, half8 res) const
    {
        const int ts[1] = {t};
        const f32x4 los[1] = {lo}, his[1] = {hi};
        const float sxs[1] = {sx};
        const half8 ress[1] = {res};
        finish<1>(a, ts, los, his, sxs, ress);
    }
};

__device__ inline i32x8 join(i32x4 a, i32x4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

// One 128-byte step along k of an MT x MT output: lane (g, r) = (lane / MT,
// lane % MT) reads its row r's chunks, kParts matrix instructions long (which
// k a chunk stands for is the same for both operands, and the order of the sum
// is free).  Its results 4b .. 4b + 3 are outputs n = 8b (32) + 4g .. + 3 of
// token r.
template <bool E4M3, int MT>
struct Step;
template <>
struct Step<true, 16> {
    static constexpr int kParts = 1;
    typedef i32x8 Operand;
    typedef f32x4 Acc;
    static __device__ inline Operand pick(const i32x4 (&c)[2], int) { return join(c[0], c[1]); }
    static __device__ inline Operand read(const i32x4 *row, int g, int swz, int)
    {
        return join(row[g ^ swz], row[(g + 4) ^ swz]);
    }
    static __device__ inline Acc mma(Operand w, Operand x, Acc c)
    {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 0, 0, 0, 0, 0, 0);
    }
};
template <>
struct Step<false, 16> {
    static constexpr int kParts = 2;
    typedef i32x4 Operand;
    typedef f32x4 Acc;
    static __device__ inline Operand pick(const i32x4 (&c)[2], int part) { return c[part]; }
    static __device__ inline Operand read(const i32x4 *row, int g, int swz, int part) { return row[(g + 4 * part) ^ swz]; }
    static __device__ inline Acc mma(Operand w, Operand x, Acc c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, w), __builtin_bit_cast(half8, x), c, 0, 0, 0);
    }
};
template <>
struct Step<false, 32> {
    static constexpr int kParts = 4;
    typedef i32x4 Operand;
    typedef f32x16 Acc;
    static __device__ inline Operand read(const i32x4 *row, int g, int swz, int part) { return row[(g + 2 * part) ^ swz]; }
    static __device__ inline Acc mma(Operand w, Operand x, Acc c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, w), __builtin_bit_cast(half8, x), c, 0, 0, 0);
    }
};

__device__ inline __amdgpu_buffer_rsrc_t rows_rsrc(const uint8_t *base, long long ld, int rows, int chunks)
{
    // reads past the last row's chunks return zeros
    const long long bytes = (long long)(rows - 1) * ld + (long long)chunks * 16;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), (short)0, (int)(uint32_t)bytes, 0x00020000);
}

// An offset past every buffer, also with a step's offset along k added: the
// load returns zeros.
constexpr uint32_t kOutside = 0xC0000000u;

// ------------------------------------------------------------ at most 16 tokens
// Block: 16 R rows of W, all of k; wavefront w takes the 128-byte steps w, w + NW,
// ... and the NW partial sums meet in LDS.  Every lane asks for U steps of both
// operands before it uses the first.  Bound by one round of loads for small W
// (1 x 2048 x 2048 4.6 us FP16, 3.6 e4m3), by HBM for large ones (1 x 65536 x 2048
// FP16 51 us, 5.2 TB/s; e4m3 26 us, 5.1 TB/s).
constexpr int kStreamT = 16;

template <bool E4M3, int NW, int R>
__global__ __launch_bounds__(NW * 64) void linear_stream_kernel(LinearArgs a)
{
    typedef Step<E4M3, 16> S;
    constexpr int U = 4;
    static_assert(2 * kStreamT * R <= NW * 64, "two lanes a token and 16 rows");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int g = lane >> 4, r = lane & 15;
    const int n0 = blockIdx.x * (16 * R);
    __shared__ f32x4 s_acc[NW][R][64];
    const __amdgpu_buffer_rsrc_t rw = rows_rsrc(a.w + n0 * a.ldw, a.ldw, min(16 * R, a.N - n0), a.chunks);
    const __amdgpu_buffer_rsrc_t rx = rows_rsrc(a.x, a.ldx, a.T, a.chunks);
    uint32_t row_w[R];
#pragma unroll
    for (int i = 0; i < R; ++i) row_w[i] = n0 + 16 * i + r < a.N ? (uint32_t)((16 * i + r) * a.ldw) : kOutside;
    const uint32_t row_x = r < a.T ? (uint32_t)(r * a.ldx) : kOutside;
    f32x4 acc[R];
#pragma unroll
    for (int i = 0; i < R; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    // the epilogue's operands first: they arrive while the products are made.
    // Two lanes a token: outputs 8h .. 8h + 7 of 16 rows are the results of lanes (2h, r) and (2h + 1, r)
    const int et = tid >> 1 & 15, eh = tid & 1, ei = tid >> 5;
    Columns<E4M3> cols;
    half8 res = {};
    float sx = 1.0f;
    if (tid < 2 * kStreamT * R) {
        cols.load(a, n0 + 16 * ei + 8 * eh);
        res = cols.residual(a, et);
        if constexpr (E4M3) sx = a.x_scale[min(et, a.T - 1)];
    }
    for (int s = wave; 8 * s < a.chunks; s += NW * U) {
        i32x4 w[R][U][2], x[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = 8 * (s + u * NW) + 4 * h + g;
#pragma unroll
                for (int i = 0; i < R; ++i)
                    w[i][u][h] =
                        __builtin_amdgcn_raw_buffer_load_b128(rw, c < a.chunks ? row_w[i] + 16u * c : kOutside, 0, 0);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = 8 * (s + u * NW) + 4 * h + g;
                x[u][h] = __builtin_amdgcn_raw_buffer_load_b128(rx, c < a.chunks ? row_x + 16u * c : kOutside, 0, 0);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < S::kParts; ++h)
#pragma unroll
                for (int i = 0; i < R; ++i) acc[i] = S::mma(S::pick(w[i][u], h), S::pick(x[u], h), acc[i]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) s_acc[wave][i][lane] = acc[i];
    __syncthreads();
    if (tid < 2 * kStreamT * R) {
        const int at = 32 * eh + et;
        f32x4 lo = s_acc[0][ei][at], hi = s_acc[0][ei][at + 16];
#pragma unroll
        for (int w = 1; w < NW; ++w) {
            lo += s_acc[w][ei][at];
            hi += s_acc[w][ei][at + 16];
        }
        cols.finish(a, et, lo, hi, sx, res);
    }
}

// ------------------------------------------------------------ many tokens
// Block tile BN outputs x BT tokens by 4 wavefronts, 2 x 2, each BN/2 x BT/2 in
// registers (or KG such groups of 4, each taking every KG-th step of k, whose
// sums meet in LDS: for tiles too few to fill the GPU, and to have two
// wavefronts a SIMD where one block fills a CU's LDS); 128 bytes of k a step.
// A step's operands lie in LDS in three parts: the tokens X, and the first and
// second half (WA, WB) of every wavefront's output rows, for B steps at once.
// Per step:
//     barrier; ask for WB of step k + B - 1; read WB(k); multiply WA(k) . X(k)
//     barrier; ask for X, WA of step k + B; read X, WA of step k + 1; multiply WB(k) . X(k)
// A part is overwritten after the barrier that follows the products it was
// read for: every wavefront's reads of it have then returned, so the barriers
// wait for loads from memory only.  Each load has B - 1 steps to arrive, and the
// reads of LDS run under the matrix instructions: those of the next step's token
// tile j replace tile j once it has met every row of WB.
//   A row of a step is 8 chunks of 16 bytes; chunk c of row r sits in slot
// c ^ (r / 2 & 7) (two groups: 16 chunks, those of both groups' steps, in slot
// c ^ (r & 15)), so the lanes that read one chunk of many rows spread over all
// banks (a load's 64 lanes fill 1024 consecutive bytes of LDS: the swizzle is
// in the addresses they read from).
//   Bound by the matrix cores for large products, whose clock then falls (8192^3
// FP16 821 us = 1.34 PFLOP/s, e4m3 386 us = 2.85; 8192 x 5632 x 4096 e4m3 163 us =
// 2.32, 172 with bias and SiLU, whose two transcendental instructions a value
// nothing overlaps; FP16 312 us = 1.21), by LDS with 128 x 128 tiles (64 KB read and
// 32 KB written a step against 512 cycles of matrix instructions: 1333 x 2817 x
// 2048 FP16 22 us).  Of a 256 x 256 tile's 111 k cycles (e4m3, K 4096) the loop takes
// 85 k (65 k of matrix instructions), the epilogue 19 k (28 k with SiLU); finishing
// one token at a time, each wait for a residual one for the stores before it, it
// took 42 k.  Rows that do not start at multiples of 128 bytes cost a second cache
// line a step (K 2064 26 to 28 us); two groups load both their steps of a row
// together so that they share lines (5 % off that), while one group that loads two
// steps ahead together has a step less for them to arrive (aligned rows 10 % slower).
template <int OUTSTANDING>
__device__ inline void arrive()
{
    // all but the newest of this wavefront's loads have landed in LDS, then everyone's
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"i"(OUTSTANDING) : "memory");
}

// The parts of stage `STAGE` (0 X, 1 WA, 2 WB), each an LDS array of its own:
// the compiler then knows which loads a read of LDS depends on.
template <bool E4M3, int BN, int BT, int MT, int KG, int STAGE, int WHICH>
__device__ inline i32x4 *part()
{
    static __shared__ i32x4 s[KG * (WHICH == 0 ? BT * 8 : BN * 4)];
    return s;
}

constexpr int kNoLoads = 0x0F70;                                 // s_waitcnt operand: vmcnt(0)

template <int V>
struct Const {
    static constexpr int value = V;
};

template <bool E4M3, int BN, int BT, int MT, int B, int KG>
__device__ inline void linear_tile(const LinearArgs &a, int tiles_n, int tiles_t)
{
    typedef Step<E4M3, MT> S;
    constexpr int P = S::kParts;
    constexpr int FT = BT / 2 / MT, HN = BN / 4 / MT;            // MT x MT tiles of a wavefront: along t; along half its n
    constexpr int LX = BT / 32, LW = BN / 64;                    // loads (1 KB) of X and of a half of W a wavefront
    __shared__ float s_scale[E4M3 ? BT : 1];
    const int lane = threadIdx.x & 63, all_waves = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wave = all_waves & 3, grp = KG > 1 ? all_waves >> 2 : 0;
    const int g = lane / MT, r = lane % MT;

    // blocks are dealt to the 8 XCDs in turn: give each a contiguous run of
    // tiles, so its L2 serves the rows its blocks share
    const int total = tiles_n * tiles_t;
    int tile;
    {
        const int xcd = blockIdx.x & 7, i = blockIdx.x >> 3, base = total / 8, extra = total % 8;
        tile = xcd * base + min(xcd, extra) + i;
    }
    // runs of 8 token tiles, outputs outermost within a run
    const int run = 8 * tiles_n, first = tile / run * 8, height = min(8, tiles_t - first);
    const int in_run = tile % run;
    const int t0 = (first + in_run % height) * BT, n0 = in_run / height * BN;

    if constexpr (E4M3) {
        if ((int)threadIdx.x < BT) s_scale[threadIdx.x] = a.x_scale[min(t0 + (int)threadIdx.x, a.T - 1)];
    }
    // this split's steps of k (all of them unless k is divided)
    const int step0 = blockIdx.y * a.split_steps;
    const int chunks = min(a.chunks - 8 * step0, 8 * a.split_steps), steps = (chunks + 8 * KG - 1) / (8 * KG);
    const __amdgpu_buffer_rsrc_t rw = rows_rsrc(a.w + n0 * a.ldw + 128 * step0, a.ldw, min(BN, a.N - n0), chunks);
    const __amdgpu_buffer_rsrc_t rx = rows_rsrc(a.x + t0 * a.ldx + 128 * step0, a.ldx, min(BT, a.T - t0), chunks);
    // Two groups: a row of LDS holds both groups' steps, 16 chunks that all wavefronts load together (256
    // consecutive bytes of a row touch fewer cache lines than twice 128 where they straddle them).
    constexpr bool WIDE = KG == 2;
    static_assert(!WIDE || MT == 16, "the swizzle of 16 chunks is of 16 rows");
    constexpr int RC = WIDE ? 16 : 8, LR = 64 / RC;                             // chunks of a row; rows of a load
    constexpr int NW = WIDE ? 8 : 4;                                            // wavefronts that load a part
    const int lw = WIDE ? all_waves : wave, lr = lane / RC;                     // row within a load
    const int lc = (lane % RC) ^ (WIDE ? 4 * (all_waves & 3) + lr : (lr >> 1) + 4 * (wave & 1));   // chunk of it
    uint32_t off_x[LX], off_a[LW], off_b[LW];
#pragma unroll
    for (int i = 0; i < LX; ++i) {
        const int row = LR * (i * NW + lw) + lr;
        off_x[i] = t0 + row < a.T ? (uint32_t)(row * a.ldx) + 16u * lc : kOutside;
    }
#pragma unroll
    for (int i = 0; i < LW; ++i) {
        const int h = LR * (i * NW + lw) + lr, row = h / (BN / 4) * (BN / 2) + h % (BN / 4);
        off_a[i] = n0 + row < a.N ? (uint32_t)(row * a.ldw) + 16u * lc : kOutside;
        off_b[i] = n0 + row + BN / 4 < a.N ? (uint32_t)((row + BN / 4) * a.ldw) + 16u * lc : kOutside;
    }
    // load i of a part of step `step` (zeros past the last chunk)
    auto fetch = [&](uint32_t off, const __amdgpu_buffer_rsrc_t &rsrc, i32x4 *s, int i, int step) {
        // uniform, but not always seen to be: a divergent scalar offset would become a loop over lanes
        const int at = __builtin_amdgcn_readfirstlane(WIDE ? step : step * KG + grp);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)(s + (i * NW + lw) * 64), 16,
                                                 RC * at + lc < chunks ? off : kOutside, 16 * RC * at, 0, 0);
    };
    // a stage's X; its WA (1) or WB (2)
    auto stage_x = [&](auto st) {
        return part<E4M3, BN, BT, MT, KG, decltype(st)::value, 0>() + (WIDE ? 0 : grp) * (BT * 8);
    };
    auto stage_w = [&](auto st, auto ab) {
        return part<E4M3, BN, BT, MT, KG, decltype(st)::value, decltype(ab)::value>() + (WIDE ? 0 : grp) * (BN * 4);
    };
    // loads [i0, i1) of X, then WA; of WB
    auto fetch_xa = [&](auto st, int i0, int i1, int step) {
#pragma unroll
        for (int i = i0; i < i1; ++i) {
            if (i < LX) fetch(off_x[i], rx, stage_x(st), i, step);
            else fetch(off_a[i - LX], rw, stage_w(st, Const<1>{}), i - LX, step);
        }
    };
    auto fetch_b = [&](auto st, int i0, int i1, int step) {
#pragma unroll
        for (int i = i0; i < i1; ++i) fetch(off_b[i], rw, stage_w(st, Const<2>{}), i, step);
    };
    const int swz = WIDE ? r : (r >> 1) & 7, rg = WIDE ? 8 * grp + g : g;
    const int at_x = ((wave & 1) * (BT / 2) + r) * RC, at_w = ((wave >> 1) * (BN / 4) + r) * RC;
    auto read = [&](const i32x4 *s, int at, int part) { return S::read(s + at, rg, swz, part); };
    typename S::Acc acc[2][FT][HN];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < FT; ++j)
#pragma unroll
            for (int i = 0; i < HN; ++i) acc[h][j][i] = (typename S::Acc)(0.0f);

    // four groups: a lane finishes 8 outputs of one token at the end, whose operands arrive meanwhile
    constexpr int ITEMS = BT * BN / 8;
    static_assert(KG != 4 || ITEMS <= 256 * KG, "one item a thread");
    const int it = threadIdx.x / (BN / 8), ic = threadIdx.x % (BN / 8) * 2;    // its token; its 4-output chunk
    Columns<E4M3> cols;
    half8 own = {};
    if constexpr (KG == 4) {
        if ((int)threadIdx.x < ITEMS) {
            cols.load(a, n0 + 4 * ic);
            if (!a.planes) own = cols.residual(a, t0 + it);
        }
    }

    typename S::Operand x[P][FT], wa[P][HN], wb[P][HN];
    constexpr int XA = LX + LW;
    fetch_xa(Const<0>{}, 0, XA, 0);
    fetch_b(Const<0>{}, 0, LW, 0);
    fetch_xa(Const<1>{}, 0, XA, 1);
    if constexpr (B > 2) {
        fetch_b(Const<1>{}, 0, LW, 1);
        fetch_xa(Const<2>{}, 0, XA, 2);
    }
    if constexpr (B > 3) {
        fetch_b(Const<2>{}, 0, LW, 2);
        fetch_xa(Const<3>{}, 0, XA, 3);
    }
    arrive<(B - 1) * (XA + LW)>();
#pragma unroll
    for (int h = 0; h < P; ++h) {
#pragma unroll
        for (int j = 0; j < FT; ++j) x[h][j] = read(stage_x(Const<0>{}), at_x + j * (MT * RC), h);
#pragma unroll
        for (int i = 0; i < HN; ++i) wa[h][i] = read(stage_w(Const<0>{}, Const<1>{}), at_w + i * (MT * RC), h);
    }
    // Step k, its parts in stage st.  The scheduling barriers keep each token
    // tile's few loads and reads among its matrix instructions.
    auto do_step = [&](auto st, int k) {
        constexpr int ST = decltype(st)::value, NEXT = (ST + 1) % B, LAST = (ST + B - 1) % B;
        arrive<(B - 1) * XA + (B - 2) * LW>();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < P * FT; ++q) {
            const int h = q / FT, j = q % FT;
            if (q < P * HN) wb[q / HN][q % HN] = read(stage_w(Const<ST>{}, Const<2>{}), at_w + q % HN * (MT * RC), q / HN);
            fetch_b(Const<LAST>{}, q * LW / (P * FT), (q + 1) * LW / (P * FT), k + B - 1);
#pragma unroll
            for (int i = 0; i < HN; ++i) acc[0][j][i] = S::mma(wa[h][i], x[h][j], acc[0][j][i]);
            __builtin_amdgcn_sched_barrier(0);
        }
        arrive<(B - 2) * XA + (B - 1) * LW>();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < P * FT; ++q) {
            const int h = q / FT, j = q % FT;
            if (q < P * HN) wa[q / HN][q % HN] = read(stage_w(Const<NEXT>{}, Const<1>{}), at_w + q % HN * (MT * RC), q / HN);
            fetch_xa(st, q * XA / (P * FT), (q + 1) * XA / (P * FT), k + B);
#pragma unroll
            for (int i = 0; i < HN; ++i) acc[1][j][i] = S::mma(wb[h][i], x[h][j], acc[1][j][i]);
            x[h][j] = read(stage_x(Const<NEXT>{}), at_x + j * (MT * RC), h);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    if constexpr (B == 2) {
        for (int k = 0; k < steps; k += 2) {                     // an odd last step is followed by one of zeros
            do_step(Const<0>{}, k);
            do_step(Const<1>{}, k + 1);
        }
    } else {
        for (int k = 0;; k += B) {
            do_step(Const<0>{}, k);
            if (k + 1 >= steps) break;
            do_step(Const<1>{}, k + 1);
            if (k + 2 >= steps) break;
            do_step(Const<2>{}, k + 2);
            if (k + 3 >= steps) break;
            if constexpr (B > 3) {
                do_step(Const<3>{}, k + 3);
                if (k + 4 >= steps) break;
            }
        }
    }
    constexpr int NH = KG == 2 ? 1 : 2;                          // halves of its output rows a wavefront finishes
    constexpr int CW = BN / 16 * NH, LPT = CW / 2;               // 4-output chunks of its row; lanes that finish a token
    if constexpr (KG != 4) cols.load(a, n0 + (wave >> 1) * (BN / 2) + (KG == 2 ? grp * (BN / 4) : 0) + lane % LPT * 8);
    // tokens finished at once, and the first ones' residuals; the next ones' follow, a round ahead
    constexpr int TPI = 64 / LPT, U = 32 / TPI < 4 ? 32 / TPI : 4;   // tokens a wavefront holds; rounds of them at once
    const int t_wave = (wave & 1) * (BT / 2);
    half8 next[U];
    if constexpr (KG != 4)
#pragma unroll
        for (int u = 0; u < U; ++u) next[u] = cols.residual(a, t0 + t_wave + lane / LPT + u * TPI);
    // No load is on its way to LDS any more.  The builtin tells the compiler, which would else wait for
    // memory (and so for the stores before) at every use of LDS below.
    __builtin_amdgcn_s_waitcnt(kNoLoads);
    arrive<0>();

    if constexpr (KG == 4) {
        // the groups' sums meet in LDS, [group][token][output], two groups a
        // stage of X; then a lane finishes 8 outputs of a token
        constexpr int ROW = BN / 4;                              // 4-output chunks of a token
        static_assert(MT == 16 && 2 * BT * ROW <= KG * BT * 8, "two groups' sums fit a stage");
        i32x4 *const x0 = part<E4M3, BN, BT, MT, KG, 0, 0>(), *const x1 = part<E4M3, BN, BT, MT, KG, 1, 0>();
        i32x4 *mine = (grp & 2 ? x1 : x0) + (grp & 1) * (BT * ROW);
#pragma unroll
        for (int j = 0; j < FT; ++j)
#pragma unroll
            for (int i = 0; i < 2 * HN; ++i) {
                const int t = (wave & 1) * (BT / 2) + 16 * j + r, c = (wave >> 1) * (ROW / 2) + 4 * i + g;
                mine[t * ROW + (c ^ (t & 7))] = __builtin_bit_cast(i32x4, acc[i / HN][j][i % HN]);
            }
        __syncthreads();
        if ((int)threadIdx.x < ITEMS) {
            f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
#pragma unroll
            for (int q = 0; q < KG; ++q) {
                const i32x4 *p = (q & 2 ? x1 : x0) + (q & 1) * (BT * ROW) + it * ROW;
                lo += __builtin_bit_cast(f32x4, p[ic ^ (it & 7)]);
                hi += __builtin_bit_cast(f32x4, p[(ic + 1) ^ (it & 7)]);
            }
            if (a.planes) cols.store_plane(a, blockIdx.y, t0 + it, lo, hi);
            else cols.finish(a, t0 + it, lo, hi, E4M3 ? s_scale[it] : 1.0f, own);
        }
        return;
    } else {
    if constexpr (KG == 2) {
        // group g finishes half g of its wavefronts' output rows (in acc[0] from here): it hands the
        // other's sums over and adds what it gets
        constexpr int CH = MT * MT / 256;                        // 16-byte chunks of a tile's sums in a lane
        static_assert(4 * 64 * FT * HN * CH <= KG * BT * 8, "a group's half of the sums fits a stage of X");
        i32x4 *const x0 = part<E4M3, BN, BT, MT, KG, 0, 0>(), *const x1 = part<E4M3, BN, BT, MT, KG, 1, 0>();
        i32x4 *const give = (grp ? x1 : x0) + wave * (64 * FT * HN * CH) + lane;
        const i32x4 *const get = (grp ? x0 : x1) + wave * (64 * FT * HN * CH) + lane;
#pragma unroll
        for (int j = 0; j < FT; ++j)
#pragma unroll
            for (int i = 0; i < HN; ++i) {
                const typename S::Acc v = grp ? acc[0][j][i] : acc[1][j][i];
                acc[0][j][i] = grp ? acc[1][j][i] : acc[0][j][i];
#pragma unroll
                for (int c = 0; c < CH; ++c)
                    give[((j * HN + i) * CH + c) * 64] =
                        __builtin_bit_cast(i32x4, f32x4{v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]});
            }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < FT; ++j)
#pragma unroll
            for (int i = 0; i < HN; ++i)
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const f32x4 v = __builtin_bit_cast(f32x4, get[((j * HN + i) * CH + c) * 64]);
#pragma unroll
                    for (int b = 0; b < 4; ++b) acc[0][j][i][4 * c + b] += v[b];
                }
        __syncthreads();                                         // the same LDS serves the epilogue
    }
    // Epilogue: the sums pass through LDS, 2 x 16 tokens of a wavefront at a
    // time, so that a lane finishes 8 neighbouring outputs of a token.
    constexpr int PT = 32 / MT;                                  // token tiles at a time
    static_assert(32 * CW * 2 <= BT * 8, "two wavefronts' sums fit one token part");
    i32x4 *const sums = (wave & 2) ? part<E4M3, BN, BT, MT, KG, 1, 0>() : part<E4M3, BN, BT, MT, KG, 0, 0>();
    i32x4 *const mine = sums + grp * (BT * 8) + (wave & 1) * (32 * CW);
    const int lane_n = lane % LPT;
#pragma unroll 1
    for (int p = 0; p < FT / PT; ++p) {
#pragma unroll
        for (int q = 0; q < FT / PT; ++q) {
            if (q != p) continue;
#pragma unroll
            for (int u = 0; u < PT; ++u)
#pragma unroll
                for (int i = 0; i < NH * HN; ++i)
#pragma unroll
                    for (int c = 0; c < MT / 16 * MT / 16; ++c) {
                        const typename S::Acc v = acc[i / HN][q * PT + u][i % HN];
                        mine[(MT * u + r) * CW + ((MT / 4 * i + 2 * c + g) ^ (r & 7))] =
                            __builtin_bit_cast(i32x4, f32x4{v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]});
                    }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        // U tokens a lane at a time: one wavefront a SIMD hides no latency of another's.  Without residuals
        // nothing in the loop waits for memory (a wait for a load is one for the stores before it).
        const int t_first = t_wave + p * 32;
        auto tokens = [&](auto residuals) {
            constexpr bool RES = decltype(residuals)::value != 0;
#pragma unroll 1
            for (int tb = lane / LPT; tb < 32; tb += U * TPI) {
                int t[U];
                f32x4 lo[U], hi[U];
                float sx[U];
                half8 res[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int tt = tb + u * TPI;
                    t[u] = t0 + t_first + tt;
                    lo[u] = __builtin_bit_cast(f32x4, mine[tt * CW + ((2 * lane_n) ^ (tt & 7))]);
                    hi[u] = __builtin_bit_cast(f32x4, mine[tt * CW + ((2 * lane_n + 1) ^ (tt & 7))]);
                    sx[u] = E4M3 ? s_scale[t_first + tt] : 1.0f;
                    res[u] = RES ? next[u] : half8{};
                }
                if constexpr (RES)
#pragma unroll
                    for (int u = 0; u < U; ++u) next[u] = cols.residual(a, t[u] + U * TPI);
                cols.finish(a, t, lo, hi, sx, res);
            }
        };
        if (a.res) tokens(Const<1>{});
        else tokens(Const<0>{});
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    }
}

template <bool E4M3, int BN, int BT, int MT, int B, int KG>
__global__ __launch_bounds__(256 * KG, BN + BT > 256 ? 1 : 2) void linear_tile_kernel(LinearArgs a, int tiles_n, int tiles_t)
{
    linear_tile<E4M3, BN, BT, MT, B, KG>(a, tiles_n, tiles_t);
}

// ------------------------------------------------------------ k divided
// Sums the splits' planes in their order and finishes: one lane 8 outputs of a
// token.
template <bool E4M3>
__global__ __launch_bounds__(256) void linear_join_kernel(LinearArgs a, int splits)
{
    const int per_token = a.plane_ld / 8;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    const int t = (int)(i / per_token), c = (int)(i % per_token);
    if (t >= a.T) return;
    const f32x4 *p = reinterpret_cast<const f32x4 *>(a.planes + (long long)t * a.plane_ld + 8 * c);
    const long long stride = (long long)a.T * a.plane_ld / 4;
    Columns<E4M3> cols;
    cols.load(a, 8 * c);
    const half8 res = cols.residual(a, t);
    const float sx = E4M3 ? a.x_scale[t] : 1.0f;
    f32x4 lo = p[0], hi = p[1];
#pragma unroll 4
    for (int s = 1; s < splits; ++s) {
        lo += p[s * stride];
        hi += p[s * stride + 1];
    }
    cols.finish(a, t, lo, hi, sx, res);
}

// Splits of k: only for long sums (kSplitFrom 128-byte steps or more: 8192 FP16 or
// 16384 e4m3 values), into parts of kSplitSteps steps or more, until the blocks
// fill the 256 CUs, with planes of at most kPlaneBytes in all.  The second launch
// costs what about 100 steps of one block take: 64 x 512 x 8192 FP16 15.2 us in
// one part, 9.9 in 4; 64 x 512 x 8192 e4m3 (64 steps) 9.7 in one, 10.1 in 2.
constexpr int kSplitFrom = 128, kSplitSteps = 32, kMaxSplits = 16;
constexpr long long kPlaneBytes = 32 << 20;

int plane_ld(int N) { return (N + 7) / 8 * 8; }

int splits_of(const LinearArgs &a, long long tiles)
{
    const int steps = (a.chunks + 7) / 8;
    if (steps < kSplitFrom) return 1;
    const long long plane = (long long)a.T * plane_ld(a.N) * 4;
    const long long want = min(min(256 / tiles, kPlaneBytes / plane), (long long)min(kMaxSplits, steps / kSplitSteps));
    if (want <= 1) return 1;
    const int per = (int)((steps + want - 1) / want);
    return (steps + per - 1) / per;              // no split is empty
}

template <bool E4M3, int BN, int BT, int MT, int B, int KG = 1>
void launch_tile(LinearArgs a, int splits, void *ws, hipStream_t s)
{
    const int tn = (a.N + BN - 1) / BN, tt = (a.T + BT - 1) / BT, steps = (a.chunks + 7) / 8;
    a.split_steps = (steps + splits - 1) / splits;
    a.planes = splits > 1 ? (float *)ws : nullptr;
    a.plane_ld = plane_ld(a.N);
    hipLaunchKernelGGL((linear_tile_kernel<E4M3, BN, BT, MT, B, KG>), dim3((unsigned int)(tn * tt), (unsigned int)splits),
                       dim3(256 * KG), 0, s, a, tn, tt);
    if (splits > 1) {
        const long long lanes = (long long)a.T * (a.plane_ld / 8);
        hipLaunchKernelGGL(linear_join_kernel<E4M3>, dim3((unsigned int)((lanes + 255) / 256)), dim3(256), 0, s, a, splits);
    }
}

// Time of `tiles` blocks where `slots` run at once and a full round takes `cost`: whole rounds, and
// a last one that takes at least `least` of a full round, as a block alone is not that much faster.
double rounds(long long tiles, int slots, double cost, double least)
{
    const double part = (double)(tiles % slots) / slots;
    return cost * ((double)(tiles / slots) + (part > 0.0 ? least + (1.0 - least) * part : 0.0));
}

// Which kernel.  At most kStreamT tokens: the streaming kernel, unless its blocks' reads of x, as many
// bytes as of W at 16 tokens, are in the way (FP16, many outputs); with as many wavefronts as take the
// steps of k in one round of loads, and 32 rows a block where that leaves a block a CU and k still is
// one round (FP16 W of more than that streams at HBM's rate with 16 rows).  Then the 64 x 32 tiles (k
// in four groups of wavefronts; two stages of LDS for up to four steps a group, else three) while they
// fill no more than one round of the 256 CUs.  Then by the time of the rounds, whose costs relative to
// 128 x 128 tiles with two blocks a CU are measured ones (FP16 64 us and e4m3 34 us a round at K 4096; a
// 256 x 256 tile's start and end weigh more when k is short).
// Measured (us, FP16 / e4m3; 128 x 128 with two groups of wavefronts (g) and two blocks a CU (b)):
//   1 x 2048 x 1024: stream with 4 wavefronts 3.2 / 3.3, 8 3.8 / 3.7; K 2048: 5.6 / 3.6, 4.8 / 4.0
//   16 x 5632 x 2048: 8 wavefronts, 16 rows 10.5 / 7.9, 32 rows 8.3 / 6.0; e4m3 4 wavefronts, 32 rows 5.4
//   1 x 65536 x 2048: 8 wavefronts, 16 rows 51 / 44, 32 rows 61 / 35; e4m3 4 wavefronts, 32 rows 26
//   16 x 2048 x 2048: stream 6.1 / 4.3, 64 x 32 tiles 8.1 / 5.5
//   4, 8, 16 x 16384 x 4096 FP16: stream 28.6, 31.7, 38.2, 64 x 32 tiles 29.2, 29.3, 29.6
//   4, 8, 16 x 65536 x 2048 FP16: stream 53.6, 60.1, 72.4, 64 x 32 tiles 61.4, 62.3, 63.5
//   32 x 5632 x 2048: stream 13.2 / 9.3, 64 x 32 tiles with two stages 8.9 / 6.3, three 8.2 / 6.4
//   17 x 2048 x 1024 e4m3: 64 x 32 tiles with two stages 4.4, three 4.5
//   256 x 2048 x 2048: 64 x 32 tiles 8.1 / 6.0, 64 x 64 9.1 / 6.5
//   256 x 5632 x 2048: 64 x 32 tiles 21 / 15, 64 x 64 14 / 9.9, 128 x 128 (g) 18 / 12
//   512 x 5632 x 4096: 64 x 64 43 / 23, 128 x 128 (g) 32 / 19, (b) 39 / 23, 256 x 256 69 / 45
//   1333 x 2817 x 2064: 64 x 64 39 / 23, 128 x 128 (g) 27 / 17, (b) 31 / 18, 256 x 256 46 / 33
//   2048 x 4096 x 4096: 128 x 128 (g) 74 / 41, (b) 64 / 34, 256 x 256 82 / 51
//   2048 x 5632 x 4096: 128 x 128 (g) 113 / 59, (b) 114 / 53, 256 x 256 92 / 52
//   3000 x 5632 x 2048: 128 x 128 (g) 97 / 58, (b) 83 / 47, 256 x 256 100 / 62
//   4096 x 4096 x 512: 128 x 128 (b) 26 / 20, 256 x 256 27 / 21
//   4096 x 4096 x 4096: 128 x 128 (g) 160 / 82, (b) 136 / 66, 256 x 256 116 / 58
//   500 x 65536 x 2048: 64 x 64 274 / 162, 128 x 128 (b) 167 / 100, 256 x 256 140 / 82
//   70 x 65536 x 2048: 64 x 64 82 / 47, 128 x 128 (b) 74 / 34, 256 x 256 84 / 46
// 128 x 128 tiles in FP16 with 32 x 32 instructions: (g) 5 %, (b) 2 to 8 % slower; 256 x 256 ones with
// 16 x 16 instructions 10 % and more, as their accumulators do not stay in place.  With four stages
// instead of two groups a 128 x 128 tile took 33 / 19 at 1333 x 2817 x 2064 (two groups then 29 / 18).
template <bool E4M3>
void launch(const LinearArgs &a, void *ws, hipStream_t s)
{
    auto tiles = [&](int bn, int bt) { return (long long)((a.N + bn - 1) / bn) * ((a.T + bt - 1) / bt); };
    const int steps = (a.chunks + 7) / 8;
    if (a.T <= kStreamT && (E4M3 || a.T <= 8 || a.N <= 8192 || steps <= 16)) {
        auto stream = [&](auto nw, auto r) {
            constexpr int NW = decltype(nw)::value, R = decltype(r)::value;
            hipLaunchKernelGGL((linear_stream_kernel<E4M3, NW, R>), dim3((unsigned int)((a.N + 16 * R - 1) / (16 * R))),
                               dim3(64 * NW), 0, s, a);
        };
        if (steps <= 16 && a.N <= 4096) stream(Const<4>{}, Const<1>{});
        else if (steps <= 16) stream(Const<4>{}, Const<2>{});
        else if (steps <= 32 && a.N > 4096 && (E4M3 || a.N <= 8192)) stream(Const<8>{}, Const<2>{});
        else stream(Const<8>{}, Const<1>{});
        return;
    }
    if (tiles(64, 32) <= 256) {
        const int splits = splits_of(a, tiles(64, 32));
        if (steps <= 16) return launch_tile<E4M3, 64, 32, 16, 2, 4>(a, splits, ws, s);
        return launch_tile<E4M3, 64, 32, 16, 3, 4>(a, splits, ws, s);
    }
    const double small = rounds(tiles(64, 64), 512, 0.45, 0.5), deep = rounds(tiles(128, 128), 256, 0.6, 0.5);
    const double two = rounds(tiles(128, 128), 512, 1.0, 0.5);
    const double large = rounds(tiles(256, 256), 256, 1.55 + 12.0 / (steps + 16), 0.65);
    const double best = std::min(std::min(small, deep), std::min(two, large));
    if (small == best) return launch_tile<E4M3, 64, 64, 16, 4>(a, 1, ws, s);
    if (deep == best) return launch_tile<E4M3, 128, 128, 16, 2, 2>(a, 1, ws, s);
    if (two == best) return launch_tile<E4M3, 128, 128, 16, 2>(a, 1, ws, s);
    launch_tile<E4M3, 256, 256, E4M3 ? 16 : 32, 2>(a, 1, ws, s);
}

constexpr int kMaxLd = 1 << 22;                  // elements: 256 rows stay within 32-bit offsets
constexpr int kMaxK = 1 << 20, kMaxN = 1 << 24;

}  // namespace

extern "C" {

size_t moe_linear_workspace_size(int T, int N, int K, int type)
{
    if (T < 0 || T > 65536 || N < 1 || N > kMaxN || K < 16 || K > kMaxK || K % 16) return 0;
    if (type != MOE_LINEAR_FP16 && type != MOE_LINEAR_E4M3) return 0;
    // the planes of every T' <= T
    const long long most = (long long)kMaxSplits * T * plane_ld(N) * 4;
    return 256 + (size_t)(most < kPlaneBytes ? most : kPlaneBytes);
}

int moe_linear(const void *x_dev, long long ldx, const float *x_scale_dev, const void *w_dev, long long ldw,
               const float *w_scale_dev, const float *bias_dev, const void *residual_dev, long long ldr, int T, int N,
               int K, int type, int act, void *y_dev, long long ldy, void *ws_dev, size_t ws_bytes, void *stream)
{
    moe::clear_error();
    const char *who = "moe_linear";
    if (type != MOE_LINEAR_FP16 && type != MOE_LINEAR_E4M3)
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: unknown type %d", who, type);
    if (act < MOE_ACT_NONE || act > MOE_ACT_GELU_TANH)
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: unknown activation %d", who, act);
    if (T < 0 || T > 65536) return moe::fail(MOE_ERR_UNSUPPORTED, "%s: T=%d outside [0, 65536]", who, T);
    if (N < 1 || N > kMaxN) return moe::fail(MOE_ERR_UNSUPPORTED, "%s: N=%d outside [1, %d]", who, N, kMaxN);
    if (K < 16 || K > kMaxK || K % 16)
        return moe::fail(MOE_ERR_UNSUPPORTED, "%s: K=%d must be a multiple of 16 in [16, %d]", who, K, kMaxK);
    if (T == 0) return MOE_OK;
    const bool e4m3 = type == MOE_LINEAR_E4M3;
    if (!x_dev || !w_dev || !y_dev) return moe::fail(MOE_ERR_INVALID_ARG, "%s: null pointer argument", who);
    if (e4m3 != (x_scale_dev != nullptr) || e4m3 != (w_scale_dev != nullptr))
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: x_scale and w_scale go with e4m3 operands, and only with them", who);
    const int size = e4m3 ? 1 : 2;
    if (ldx < K || ldw < K || ldy < N || (residual_dev && ldr < N))
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: a row stride is below its row (K=%d, N=%d)", who, K, N);
    if (ldx > kMaxLd || ldw > kMaxLd)
        return moe::fail(MOE_ERR_UNSUPPORTED, "%s: row strides of x and w are at most %d", who, kMaxLd);
    if (!moe::aligned(x_dev, 16) || !moe::aligned(w_dev, 16) || ldx * size % 16 || ldw * size % 16)
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: rows of x and w must start at multiples of 16 bytes", who);
    if (!moe::aligned(y_dev, 2) || !moe::aligned(residual_dev, 2) || !moe::aligned(bias_dev, 4) ||
        !moe::aligned(x_scale_dev, 4) || !moe::aligned(w_scale_dev, 4))
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: y and residual must be 2-byte, bias and scales 4-byte aligned", who);
    const size_t need = moe_linear_workspace_size(T, N, K, type);
    if (!ws_dev || ws_bytes < need || !moe::aligned(ws_dev, 256))
        return moe::fail(MOE_ERR_WORKSPACE, "%s: the workspace needs %zu bytes, 256-byte aligned", who, need);
    LinearArgs a;
    a.x = (const uint8_t *)x_dev;
    a.w = (const uint8_t *)w_dev;
    a.ldx = ldx * size;
    a.ldw = ldw * size;
    a.x_scale = x_scale_dev;
    a.w_scale = w_scale_dev;
    a.bias = bias_dev;
    a.res = (const uint16_t *)residual_dev;
    a.ldr = ldr;
    a.y = (uint16_t *)y_dev;
    a.ldy = ldy;
    a.T = T;
    a.N = N;
    a.chunks = K * size / 16;
    a.act = act;
    a.planes = nullptr;
    a.plane_ld = a.split_steps = 0;
    if (e4m3) launch<true>(a, ws_dev, (hipStream_t)stream);
    else launch<false>(a, ws_dev, (hipStream_t)stream);
    return moe::check_launch(who);
}

}  // extern "C"
