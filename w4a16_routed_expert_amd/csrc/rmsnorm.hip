// Residual addition and root-mean-square norm of the rows that pass from one
// layer to the next, with FP16 and/or e4m3 outputs.
//
//   v = RN16(x + y)                    the residual stream (moe_residual_add's sum)
//   r = RN32(1 / sqrt(sum v^2 / H + eps))
//   n = RN32(RN32(v * r) * w)
//   norm = RN16(n)
//   a = max(max_i |n_i|, 2^-100), scale = RN32(a / 448),
//   q = RN_e4m3(RN32(n * RN32(448 / a)))
//
// The squares of FP16 values are exact in FP32 and are summed in fp64, whose
// error (2^-53 per addition) reaches r's FP32 rounding about once in 2^20
// rows; every later step is one IEEE FP32 operation on a value, and a maximum
// does not depend on order.  So the results do not depend on how a row is
// divided among lanes, and 8-bit codes next to a rounding border are the same
// on every run and for every kernel shape.
//
// The row stays in registers between its one read and its writes: bound by
// HBM for long batches (8192 x 4096 with y and all outputs, 302 MB: 61.4 us =
// 4.9 TB/s; a 1 GiB device copy moves 5.0 TB/s), by one load round trip and the
// two reductions for single rows (1 x 2048 2.2 us, 32 x 2048 with 8-bit codes
// 3.4 us).
#include "moe_internal.h"

namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
// Rows may start at any element (odd H, strides): 16-byte accesses that
// assume element alignment only.
struct __attribute__((packed, aligned(2))) Chunk16 { half8 v; };
struct __attribute__((packed, aligned(1))) Chunk8 { uint32_t lo, hi; };

constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 0x1p-100f;      // smallest amax a scale is made for (an all-zero row: codes 0)

struct NormArgs {
    const uint16_t *x, *y, *w;               // y may be null
    long long ldx, ldy;
    uint16_t *sum, *norm;                    // each may be null
    long long lds, ldn;
    uint8_t *q;                              // may be null
    long long ldq;
    float *q_scale;
    double eps;
    int T, H;
};

// The C chunks of 8 values of lane `sub`: chunk i * NT + sub of a row of H
// values (what lies past the row is 0).  Whole chunks are one 16-byte load
// each, all in flight together; the values behind the last whole chunk are
// single loads by the one lane that holds them.
template <int NT, int C>
__device__ inline void load_row(half8 (&v)[C], const uint16_t *row, int sub, int H)
{
    const int whole = H / 8;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = i * NT + sub;
        v[i] = half8{};
        if (c < whole) v[i] = reinterpret_cast<const Chunk16 *>(row + 8 * c)->v;
    }
    if (H % 8 && sub == whole % NT) {
        half8 t;
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = __builtin_bit_cast(_Float16, row[min(8 * whole + j, H - 1)]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (8 * whole + j >= H) t[j] = (_Float16)0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (i == whole / NT) v[i] = t;
    }
}

template <int NT, int C>
__device__ inline void store_row(uint16_t *row, const half8 (&v)[C], int sub, int H)
{
    const int whole = H / 8;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = i * NT + sub;
        if (c < whole) reinterpret_cast<Chunk16 *>(row + 8 * c)->v = v[i];
    }
    if (H % 8 && sub == whole % NT) {
        half8 t = {};
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (i == whole / NT) t = v[i];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const _Float16 h = t[j];
            if (8 * whole + j < H) row[8 * whole + j] = __builtin_bit_cast(uint16_t, h);
        }
    }
}

// Maximum over the wavefront, in every lane, of the bits of non-negative
// floats (their order as integers; a NaN is above infinity).
__device__ inline uint32_t wave_max_u32(uint32_t v)
{
    v = max(v, moe::ror_u32<1>(v));
    v = max(v, moe::ror_u32<2>(v));
    v = max(v, moe::ror_u32<4>(v));
    v = max(v, moe::ror_u32<8>(v));
    v = max(v, moe::partner_u32<true>(v));
    v = max(v, moe::partner_u32<false>(v));
    return v;
}

// NT threads per row (a wavefront, or a block of several), each holding C
// chunks of 8 values: chunk number c * NT + lane.
template <int NT, int C>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void residual_rmsnorm_kernel(NormArgs a)
{
    constexpr int ROWS = NT < 256 ? 256 / NT : 1;          // rows per block
    constexpr int WAVES = NT / 64;
    static_assert(NT == 64 || ROWS == 1, "a row is one wavefront or one block");
    const int sub = threadIdx.x % NT;
    const long long t = (long long)blockIdx.x * ROWS + threadIdx.x / NT;
    if (t >= a.T) return;                                  // whole wavefronts; no barrier follows for NT = 64
    const int H = a.H;
    __shared__ double s_sum[WAVES];
    __shared__ uint32_t s_max[WAVES];

    half8 v[C], w[C];
    load_row<NT, C>(v, a.x + t * a.ldx, sub, H);
    if (a.y) {
        load_row<NT, C>(w, a.y + t * a.ldy, sub, H);
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] += w[i];          // one FP16 rounding of the exact sum
    }
    load_row<NT, C>(w, a.w, sub, H);
    if (a.sum) store_row<NT, C>(a.sum + t * a.lds, v, sub, H);
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float f = (float)v[i][j];
            ss += (double)(f * f);                         // the square is exact in FP32
        }
    ss = moe::sum_phases<1>(ss);
    if constexpr (WAVES == 1) {                            // lanes add in different orders: one lane's sum for all
        const uint64_t b = __builtin_bit_cast(uint64_t, ss);
        const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
        ss = __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
    } else {
        if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = ss;
        __syncthreads();
        ss = 0.0;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) ss += s_sum[i];
    }
    const float r = (float)(1.0 / sqrt(ss / (double)H + a.eps));
    float n[C][8];
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) n[i][j] = (float)v[i][j] * r * (float)w[i][j];
    if (a.norm) {
        half8 h[C];
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = (_Float16)n[i][j];
        store_row<NT, C>(a.norm + t * a.ldn, h, sub, H);
    }
    if (!a.q) return;
    uint32_t m = 0;                                        // values past the row are +-0
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __builtin_bit_cast(uint32_t, n[i][j]) & 0x7fffffffu);
    m = wave_max_u32(m);
    if constexpr (WAVES > 1) {
        if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = m;
        __syncthreads();
        m = 0;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) m = max(m, s_max[i]);
    }
    m = max(m, __builtin_bit_cast(uint32_t, kAmaxFloor));
    const float amax = __builtin_bit_cast(float, m);       // NaN if the row holds one
    const float inv = kE4m3Max / amax;
    if (sub == 0) a.q_scale[t] = amax / kE4m3Max;
    uint8_t *q = a.q + t * a.ldq;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = i * NT + sub;
        if (8 * c >= H) continue;
        int p[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            p[j] = __builtin_amdgcn_cvt_pk_fp8_f32(n[i][4 * j] * inv, n[i][4 * j + 1] * inv, p[j], false);
            p[j] = __builtin_amdgcn_cvt_pk_fp8_f32(n[i][4 * j + 2] * inv, n[i][4 * j + 3] * inv, p[j], true);
        }
        if (8 * c + 8 <= H) {
            *reinterpret_cast<Chunk8 *>(q + 8 * c) = Chunk8{(uint32_t)p[0], (uint32_t)p[1]};
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (8 * c + j < H) q[8 * c + j] = (uint8_t)((uint32_t)p[j >> 2] >> (8 * (j & 3)));
        }
    }
}

template <int NT, int C>
void launch(const NormArgs &a, hipStream_t s)
{
    constexpr int ROWS = NT < 256 ? 256 / NT : 1;
    hipLaunchKernelGGL((residual_rmsnorm_kernel<NT, C>), dim3((unsigned int)(((long long)a.T + ROWS - 1) / ROWS)),
                       dim3(NT * ROWS), 0, s, a);
}

constexpr int kMaxNormH = 65536;

}  // namespace

extern "C" int moe_residual_rmsnorm(const void *x_dev, long long ldx, const void *y_dev, long long ldy,
                                    const void *w_dev, float eps, int T, int H, void *sum_dev, long long lds,
                                    void *norm_dev, long long ldn, void *q_dev, long long ldq, float *q_scale_dev,
                                    void *stream)
{
    moe::clear_error();
    const char *who = "moe_residual_rmsnorm";
    if (T < 0 || H < 1 || H > kMaxNormH)
        return moe::fail(MOE_ERR_UNSUPPORTED, "%s: T=%d must be >= 0 and H=%d in [1, %d]", who, T, H, kMaxNormH);
    if (!(eps > 0.0f) || eps > 1.0f)
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: eps=%g must be in (0, 1]", who, (double)eps);
    if (T == 0) return MOE_OK;
    if (!x_dev || !w_dev) return moe::fail(MOE_ERR_INVALID_ARG, "%s: null pointer argument", who);
    if (!sum_dev && !norm_dev && !q_dev)
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: no output (sum, norm and q are all NULL)", who);
    if ((q_dev == nullptr) != (q_scale_dev == nullptr))
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: q and q_scale must both be given or both NULL", who);
    if (ldx < H || (y_dev && ldy < H) || (sum_dev && lds < H) || (norm_dev && ldn < H) || (q_dev && ldq < H))
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: a row stride is below H=%d", who, H);
    if (!moe::aligned(x_dev, 2) || !moe::aligned(y_dev, 2) || !moe::aligned(w_dev, 2) || !moe::aligned(sum_dev, 2) ||
        !moe::aligned(norm_dev, 2) || !moe::aligned(q_scale_dev, 4))
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: FP16 pointers must be 2-byte and q_scale 4-byte aligned", who);
    if (sum_dev && sum_dev == norm_dev)
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: sum and norm are the same buffer", who);
    NormArgs a;
    a.x = (const uint16_t *)x_dev; a.y = (const uint16_t *)y_dev; a.w = (const uint16_t *)w_dev;
    a.ldx = ldx; a.ldy = ldy;
    a.sum = (uint16_t *)sum_dev; a.norm = (uint16_t *)norm_dev;
    a.lds = lds; a.ldn = ldn;
    a.q = (uint8_t *)q_dev; a.ldq = ldq; a.q_scale = q_scale_dev;
    a.eps = (double)eps;
    a.T = T; a.H = H;
    hipStream_t s = (hipStream_t)stream;
    // Threads a row.  Few rows want more of them, for shorter chains of loads and sums; many want fewer
    // reductions.  Measured (us, T = 1 / 64 / 1024 / 8192, FP16 outputs):
    //   H 512: a wavefront 2.1 / 2.4 / 2.7 / 9.0, 256 threads 2.2 / 2.5 / 3.3 / 13.6
    //   H 1024: a wavefront 2.5 / 2.9 / 4.4 / 13.8, 256 threads 2.3 / 2.5 / 4.6 / 18.1
    //   H 2048: a wavefront 3.0 / 3.5 / 5.7 / 26.6, 256 threads 2.3 / 2.6 / 5.7 / 27.6
    //   H 4096: 256 threads 2.8 / 3.1 / 8.8 / 52.3, 512 threads 2.6 / 2.8 / 9.3 / 49.6
    //   H 8192: 256 threads 3.4 / 3.8 / 13.8 / 97.1, 1024 threads 3.2 / 3.7 / 17.5 / 94.2
    //   H 16384: 256 threads 4.7 / 6.0 / 27.0 / 198, 1024 threads 3.9 / 5.5 / 28.2 / 196
    if (H <= 512) launch<64, 1>(a, s);
    else if (H <= 1024 && T > 256) launch<64, 2>(a, s);
    else if (H <= 2048) launch<256, 1>(a, s);
    else if (H <= 4096) launch<256, 2>(a, s);
    else if (H <= 8192) launch<256, 4>(a, s);
    else if (H <= 16384) launch<1024, 2>(a, s);
    else launch<1024, 8>(a, s);
    return moe::check_launch(who);
}
