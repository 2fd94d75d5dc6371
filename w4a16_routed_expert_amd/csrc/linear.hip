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
//   linear_tile_kernel: many tokens, bound by the matrix cores and LDS.
#include "moe_internal.h"

namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
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
    int quads;                           // y and residual rows are 8-byte aligned: four outputs at once
};

__device__ inline float activate(float v, int act)
{
    if (act == MOE_ACT_SILU) return v / (1.0f + __expf(-v));
    if (act == MOE_ACT_GELU) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    if (act == MOE_ACT_GELU_TANH) {
        // 0.5 v (1 + tanh u) = v / (1 + exp(-2u))
        const float u = 0.79788456080286536f * (v + 0.044715f * v * v * v);
        return v / (1.0f + __expf(-2.0f * u));
    }
    return v;
}

// Epilogue of outputs n .. n+3 of token t (those inside the matrix).
template <bool E4M3>
__device__ inline void finish4(const LinearArgs &a, int t, int n, f32x4 v)
{
    if (t >= a.T || n >= a.N) return;
    const int m = min(4, a.N - n);
    if constexpr (E4M3) {
        const float sx = a.x_scale[t];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] *= sx * a.w_scale[n + min(r, m - 1)];
    }
    if (a.bias) {
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] += a.bias[n + min(r, m - 1)];
    }
    if (a.act != MOE_ACT_NONE) {
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = activate(v[r], a.act);
    }
    uint16_t *y = a.y + (long long)t * a.ldy + n;
    const uint16_t *res = a.res ? a.res + (long long)t * a.ldr + n : nullptr;
    if (m == 4 && a.quads) {
        if (res) {
            const half4 h = *reinterpret_cast<const half4 *>(res);
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] += (float)h[r];
        }
        half4 o;
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] = (_Float16)v[r];
        *reinterpret_cast<half4 *>(y) = o;
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (r >= m) break;
            float f = v[r];
            if (res) f += (float)__builtin_bit_cast(_Float16, res[r]);
            const _Float16 o = (_Float16)f;
            y[r] = __builtin_bit_cast(uint16_t, o);
        }
    }
}

__device__ inline i32x8 join(i32x4 a, i32x4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

// One 128-byte step along k of a 16 x 16 output: lane (g, r) = (lane / 16,
// lane % 16) holds chunks g and g + 4 of its row of each operand (which k
// they stand for is the same on both sides, and the order of the sum is free).
template <bool E4M3>
__device__ inline f32x4 mma(i32x4 w0, i32x4 w1, i32x4 x0, i32x4 x1, f32x4 c)
{
    if constexpr (E4M3)
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(w0, w1), join(x0, x1), c, 0, 0, 0, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, w0), __builtin_bit_cast(half8, x0), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, w1), __builtin_bit_cast(half8, x1), c, 0, 0, 0);
}

__device__ inline __amdgpu_buffer_rsrc_t rows_rsrc(const uint8_t *base, long long ld, int rows, int chunks)
{
    // reads past the last row's chunks return zeros
    const long long bytes = (long long)(rows - 1) * ld + (long long)chunks * 16;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), (short)0, (int)(uint32_t)bytes, 0x00020000);
}

constexpr uint32_t kOutside = 0xFFFFFF00u;       // an offset past every buffer: the load returns zeros

// ------------------------------------------------------------ few tokens
// Block: 16 rows of W, FT x 16 tokens, all of k; wavefront w takes the 128-byte
// steps w, w + NW, ... and the NW partial sums meet in LDS.  Every lane asks
// for U steps of W before it uses the first.
template <bool E4M3, int FT, int NW>
__global__ __launch_bounds__(NW * 64) void linear_stream_kernel(LinearArgs a)
{
    constexpr int U = FT >= 4 ? 2 : 4;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int g = lane >> 4, r = lane & 15;
    const int n0 = blockIdx.x * 16, t0 = blockIdx.y * (16 * FT);
    __shared__ f32x4 s_acc[NW][FT][64];
    const __amdgpu_buffer_rsrc_t rw = rows_rsrc(a.w + n0 * a.ldw, a.ldw, min(16, a.N - n0), a.chunks);
    const __amdgpu_buffer_rsrc_t rx = rows_rsrc(a.x + t0 * a.ldx, a.ldx, min(16 * FT, a.T - t0), a.chunks);
    const uint32_t row_w = (uint32_t)(r * a.ldw);
    uint32_t row_x[FT];
#pragma unroll
    for (int f = 0; f < FT; ++f) row_x[f] = t0 + 16 * f + r < a.T ? (uint32_t)((16 * f + r) * a.ldx) : kOutside;
    f32x4 acc[FT];
#pragma unroll
    for (int f = 0; f < FT; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
    const bool real_w = n0 + r < a.N;
    for (int s = wave; 8 * s < a.chunks; s += NW * U) {
        i32x4 w[U][2], x[U][FT][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = 8 * (s + u * NW) + 4 * h + g;
                const bool in = c < a.chunks;
                w[u][h] = __builtin_amdgcn_raw_buffer_load_b128(rw, in && real_w ? row_w + 16u * c : kOutside, 0, 0);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int f = 0; f < FT; ++f)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = 8 * (s + u * NW) + 4 * h + g;
                    const bool in = c < a.chunks && row_x[f] != kOutside;
                    x[u][f][h] = __builtin_amdgcn_raw_buffer_load_b128(rx, in ? row_x[f] + 16u * c : kOutside, 0, 0);
                }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int f = 0; f < FT; ++f) acc[f] = mma<E4M3>(w[u][0], w[u][1], x[u][f][0], x[u][f][1], acc[f]);
    }
#pragma unroll
    for (int f = 0; f < FT; ++f) s_acc[wave][f][lane] = acc[f];
    __syncthreads();
    for (int f = wave; f < FT; f += NW) {
        f32x4 v = s_acc[0][f][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) v += s_acc[w][f][lane];
        finish4<E4M3>(a, t0 + 16 * f + r, n0 + 4 * g, v);
    }
}

// ------------------------------------------------------------ many tokens
// Block tile BN outputs x BT tokens, WN x WT wavefronts, 128 bytes of k a
// step, two steps in LDS: the loads of step k + 1 go straight to LDS while
// step k is multiplied, one barrier a step.  A row of a step is 8 chunks;
// chunk c of row r sits in slot c ^ (r & 7), so the 16 lanes that read one
// chunk of 16 rows spread over all banks (the swizzle is in the addresses the
// loads read from: a load's 64 lanes fill 1024 consecutive bytes of LDS).
template <bool E4M3, int BN, int BT, int WN, int WT>
__device__ inline void linear_tile(const LinearArgs &a, int tiles_n, int tiles_t)
{
    constexpr int NW = WN * WT;
    constexpr int FN = BN / WN / 16, FT = BT / WT / 16;
    constexpr int GW = BN / 8 / NW, GX = BT / 8 / NW;      // loads of 8 rows per wavefront
    static_assert(GW * 8 * NW == BN && GX * 8 * NW == BT, "whole loads");
    // one array per step in LDS: the compiler then knows that the loads into
    // one do not feed the reads of the other
    __shared__ i32x4 s0[(BN + BT) * 8], s1[(BN + BT) * 8];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int g = lane >> 4, r = lane & 15;

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

    const __amdgpu_buffer_rsrc_t rw = rows_rsrc(a.w + n0 * a.ldw, a.ldw, min(BN, a.N - n0), a.chunks);
    const __amdgpu_buffer_rsrc_t rx = rows_rsrc(a.x + t0 * a.ldx, a.ldx, min(BT, a.T - t0), a.chunks);
    const int lr = lane >> 3, lc = (lane & 7) ^ lr;        // row within a load, chunk of it
    uint32_t off_w[GW], off_x[GX];
#pragma unroll
    for (int i = 0; i < GW; ++i) {
        const int row = 8 * (i * NW + wave) + lr;
        off_w[i] = n0 + row < a.N ? (uint32_t)(row * a.ldw) + 16u * lc : kOutside;
    }
#pragma unroll
    for (int i = 0; i < GX; ++i) {
        const int row = 8 * (i * NW + wave) + lr;
        off_x[i] = t0 + row < a.T ? (uint32_t)(row * a.ldx) + 16u * lc : kOutside;
    }
    auto fetch = [&](i32x4 *s, int step) {
        const bool in = 8 * step + lc < a.chunks;
#pragma unroll
        for (int i = 0; i < GW; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void *)(s + (i * NW + wave) * 64), 16,
                                                     in && off_w[i] != kOutside ? off_w[i] + 128u * step : kOutside, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < GX; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void *)(s + BN * 8 + (i * NW + wave) * 64), 16,
                                                     in && off_x[i] != kOutside ? off_x[i] + 128u * step : kOutside, 0, 0, 0);
    };
    const int wn = wave / WT * (BN / WN), wt = wave % WT * (BT / WT);
    f32x4 acc[FN][FT];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int c0 = g ^ (r & 7), c1 = (g + 4) ^ (r & 7);
    auto multiply = [&](const i32x4 *s) {
        const i32x4 *pw = s + (wn + r) * 8, *px = s + (BN + wt + r) * 8;
        i32x4 x[FT][2];
#pragma unroll
        for (int j = 0; j < FT; ++j) {
            x[j][0] = px[j * 128 + c0];
            x[j][1] = px[j * 128 + c1];
        }
#pragma unroll
        for (int i = 0; i < FN; ++i) {
            const i32x4 w0 = pw[i * 128 + c0], w1 = pw[i * 128 + c1];
#pragma unroll
            for (int j = 0; j < FT; ++j) acc[i][j] = mma<E4M3>(w0, w1, x[j][0], x[j][1], acc[i][j]);
        }
    };
    const int steps = (a.chunks + 7) / 8;
    auto arrive = [&]() {
        __builtin_amdgcn_s_waitcnt(0x0F70);                // vmcnt(0): this wavefront's loads are in LDS
        __syncthreads();
    };
    fetch(s0, 0);
    for (int k = 0; k + 2 <= steps; k += 2) {
        arrive();
        fetch(s1, k + 1);
        multiply(s0);
        arrive();
        fetch(s0, k + 2);                                  // past the end: zeros, never read
        multiply(s1);
    }
    if (steps & 1) {
        arrive();
        multiply(s0);
    }
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FT; ++j) finish4<E4M3>(a, t0 + wt + 16 * j + r, n0 + wn + 16 * i + 4 * g, acc[i][j]);
}

template <bool E4M3, int BN, int BT, int WN, int WT>
__global__ __launch_bounds__(WN * WT * 64) void linear_tile_kernel(LinearArgs a, int tiles_n, int tiles_t)
{
    linear_tile<E4M3, BN, BT, WN, WT>(a, tiles_n, tiles_t);
}

template <bool E4M3, int FT>
void launch_stream(const LinearArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned int)((a.N + 15) / 16), (unsigned int)((a.T + 16 * FT - 1) / (16 * FT)));
    hipLaunchKernelGGL((linear_stream_kernel<E4M3, FT, 8>), grid, dim3(512), 0, s, a);
}

template <bool E4M3, int BN, int BT, int WN, int WT>
void launch_tile(const LinearArgs &a, hipStream_t s)
{
    const int tn = (a.N + BN - 1) / BN, tt = (a.T + BT - 1) / BT;
    hipLaunchKernelGGL((linear_tile_kernel<E4M3, BN, BT, WN, WT>), dim3((unsigned int)(tn * tt)), dim3(WN * WT * 64), 0,
                       s, a, tn, tt);
}

template <bool E4M3>
void launch(const LinearArgs &a, hipStream_t s)
{
    if (a.T <= 16) return launch_stream<E4M3, 1>(a, s);
    if (a.T <= 32) return launch_stream<E4M3, 2>(a, s);
    if (a.T <= 64) return launch_stream<E4M3, 4>(a, s);
    const long long big = (long long)((a.N + 255) / 256) * ((a.T + 255) / 256);
    const long long mid = (long long)((a.N + 127) / 128) * ((a.T + 127) / 128);
    if (big >= 200) return launch_tile<E4M3, 256, 256, 2, 4>(a, s);
    if (mid >= 200) return launch_tile<E4M3, 128, 128, 2, 2>(a, s);
    launch_tile<E4M3, 64, 64, 2, 2>(a, s);
}

constexpr int kMaxLd = 1 << 22;                  // elements: 256 rows stay within 32-bit offsets
constexpr int kMaxK = 1 << 20, kMaxN = 1 << 24;

}  // namespace

extern "C" {

size_t moe_linear_workspace_size(int T, int N, int K, int type)
{
    if (T < 0 || T > 65536 || N < 1 || N > kMaxN || K < 16 || K > kMaxK || K % 16) return 0;
    if (type != MOE_LINEAR_FP16 && type != MOE_LINEAR_E4M3) return 0;
    return 256;
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
    a.quads = moe::aligned(y_dev, 8) && ldy % 4 == 0 && (!residual_dev || (moe::aligned(residual_dev, 8) && ldr % 4 == 0));
    if (e4m3) launch<true>(a, (hipStream_t)stream);
    else launch<false>(a, (hipStream_t)stream);
    return moe::check_launch(who);
}

}  // extern "C"
