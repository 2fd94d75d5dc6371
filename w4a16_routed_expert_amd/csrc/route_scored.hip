// Routing by scores: router logits, softmax or sigmoid scores over all
// experts, an optional balance bias and expert groups for the choice,
// optionally renormalised weights, then moe_route's grouping.
//
//   l[e] = RN32(exact x . W[:, e])
//   s[e] = exp(l[e] - max l) / sum exp(l - max l), or 1 / (1 + exp(-l[e]))
//   c[e] = s[e] + bias[e]                         (a NaN counts as -inf)
//   groups: expert e is in group e / (E / n_group); a group's value is its
//     largest c or the sum of its two largest; the topk_group groups of
//     largest value stay (ties to the lower group)
//   ids = the k largest c of the groups that stay, descending, ties to the
//     lower expert; w[j] = scale * s[ids[j]] (/ sum_j s[ids[j]])
//
// The logits are the correctly rounded FP32 values of route.hip, and scores,
// choice values and group values are in fp64, so a selection does not depend
// on summation order or batch size.
//
// Small batches: one launch, a block per token and 8 experts; the block that
// completes a token's logits selects its experts, the one that completes the
// batch groups the pairs.  Larger ones: route_tile_kernel computes the logits of
// 16 tokens with the fp64 matrix instruction (the experts divided among blocks
// while there are too few tiles for the GPU) and the block that completes a
// tile selects; then one launch places the pairs.  No block waits for another.
#include "moe_internal.h"

#include <climits>

#include "route_dev.h"

namespace {

struct ScoreRule {
    const float *bias;       // [E] or null: added to the score for the choice only
    int softmax, n_group, topk_group, top2, renorm;
    double scale;
};

// LDS of one wavefront's selection.  A wavefront's LDS operations complete in
// order, so its lanes exchange values through it without a barrier.
typedef int Int4 __attribute__((ext_vector_type(4), may_alias));
struct __attribute__((aligned(16))) SelectLds {
    double s[64], c[64];     // scores, choice values
    double top[2][64];       // a group's two largest choice values
    double value[64];        // group values
    int key[64];             // choice values rounded to FP32, as ordered integers
    int slot[MOE_MAX_TOPK];  // expert + 1 of each slot
};

// The value of lane 0 for all (lanes add in different orders: one lane's sum
// keeps equal logits at equal scores).
__device__ inline double first_lane(double v)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
    return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}

// How many of v[0 .. n) are above x, or equal to it and before place `at`.
__device__ inline int rank_among(const double *v, int n, double x, int at)
{
    int rank = 0;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const double o = v[i];
        rank += (o > x || (o == x && i < at)) ? 1 : 0;
    }
    return rank;
}

// Scores, choice and weights of one token by one wavefront (lane = expert, lv
// its logit).  Lane j < k ends with slot j's expert and weight.  Bound by the
// latency of its chain of steps, so ranks are counted against values read from
// LDS (all reads in flight) rather than found by rounds of wavefront maxima.
//
// The ranks compare the FP32 roundings of the choice values, which keep their
// order except that different values may become equal: only then (a slot
// without an expert, or more than k experts ranked below k) are the fp64
// values ranked.
__device__ inline void select_wave(const ScoreRule &rule, int E, int k, int lane, float lv, SelectLds &S, int &id,
                                   float &weight)
{
    const double l = (double)lv;
    double s;
    if (rule.softmax) {
        const int top = wave_max(lane < E ? order_key(lv) : INT_MIN);
        const float mx = __builtin_bit_cast(float, top ^ ((top >> 31) & 0x7FFFFFFF));
        const double e = lane < E ? exp(l - (double)mx) : 0.0;
        s = e / first_lane(sum_phases<1>(e));
    } else {
        s = 1.0 / (1.0 + exp(-l));
    }
    double c = s;
    if (rule.bias) c += (double)rule.bias[min(lane, E - 1)];
    if (isnan(c)) c = -INFINITY;
    S.s[lane] = s;
    S.c[lane] = c;
    bool in = lane < E;
    if (rule.n_group > 1) {
        const int gs = E / rule.n_group, g = min(lane / gs, rule.n_group - 1), m = lane - g * gs;
        const int r = rank_among(&S.c[g * gs], gs, c, m);
        if (in && r < 2) S.top[r][g] = c;
        if (in && r == 0) {
            double v = S.top[0][g];
            if (rule.top2) v += S.top[1][g];
            S.value[g] = isnan(v) ? -INFINITY : v;
        }
        in = in && rank_among(S.value, rule.n_group, S.value[g], g) < rule.topk_group;
    }
    const int key = in ? order_key((float)c) : INT_MIN;
    S.key[lane] = key;
    if (lane < MOE_MAX_TOPK) S.slot[lane] = 0;
    int rank = 0;
    const Int4 *keys = reinterpret_cast<const Int4 *>(S.key);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const Int4 o = keys[i];
        rank += (o[0] > key ? 1 : 0) + (o[1] > key ? 1 : 0) + (o[2] > key ? 1 : 0) + (o[3] > key ? 1 : 0);
    }
    const bool chosen = in && rank < k;
    if (chosen) S.slot[rank] = lane + 1;
    id = S.slot[min(lane, MOE_MAX_TOPK - 1)] - 1;
    if (__popcll(__ballot(chosen)) != k || __ballot(lane < k && id < 0)) {
        S.c[lane] = in ? c : -INFINITY;
        rank = 0;
        for (int i = 0; i < E; ++i) {
            const double o = S.c[i];
            // an expert left out ranks after one whose value is -infinity
            if (S.key[i] != INT_MIN) rank += (o > c || (o == c && i < lane)) ? 1 : 0;
        }
        if (in && rank < k) S.slot[rank] = lane + 1;
        id = S.slot[min(lane, MOE_MAX_TOPK - 1)] - 1;
    }
    double w = S.s[max(id, 0)];
    if (rule.renorm) {
        double den = lane < k ? w : 0.0;                   // k <= 8: the slots lie in the first row of 16 lanes
        den = add_row_ror<1>(den);
        den = add_row_ror<2>(den);
        den = add_row_ror<4>(den);
        den = first_lane(add_row_ror<8>(den));
        w = den != 0.0 ? w / den : 0.0;                    // every chosen score underflowed: weights 0
    }
    weight = (float)(w * rule.scale);
}

// ------------------------------------------------------------ small batches: one launch
// Bound by a chain of latencies: a load round trip, the sums, the logits handed
// over at device scope, the selection, for more than one token the hand-over
// to the block that groups.  H 2048, E 64, k 8: T = 1 7.8 us, T = 32 11.4 us.
// Largest batch routed so (one thread a pair in the grouping): T = 64 12.5 us,
// 15.9 by tiles; T = 17 9.7 and 15.8.
constexpr int kScoredSmallT = 64;
constexpr int kSmallE = 8;                   // experts per block of its logits (16: T = 1 9.3 us)

union SmallLds {
    LogitsLds lg;
    SelectLds sel;
    int cnt[kSelWaves][MOE_MAX_EXPERTS];
};

// moe_route's grouping of a small batch whose pair p has expert e in lane p % 64
// of wavefront p / 64 (e < 0: no pair); `waves` wavefronts hold pairs.  A pair's
// rank among the equal experts of its wavefront comes from ballots; the
// wavefronts' counts, exchanged through LDS once, give each its start per expert.
__device__ inline void group_small(const RouteArgs &a, int e, int waves, int (*cnt)[MOE_MAX_EXPERTS])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const unsigned long long below = (1ull << lane) - 1ull, peers = same_expert_lanes(e);
    const int rank = __popcll(peers & below);
    cnt[wave][lane] = 0;
    if (e >= 0 && rank == 0) cnt[wave][e] = __popcll(peers);
    if (waves > 1) __syncthreads();
    int total = 0, before = 0;                   // of expert `lane`: all pairs, those of earlier wavefronts
    for (int w = 0; w < waves; ++w) {
        const int c = cnt[w][lane];
        total += c;
        before += w < wave ? c : 0;
    }
    const int incl = moe::wave_inclusive_sum(total), start = incl - total + before;
    if (wave == 0) {
        const unsigned long long act = __ballot(total > 0);
        const int na = __popcll(act);
        if (lane < a.E) {
            a.offsets[lane] = incl - total;
            if (total > 0) a.active[__popcll(act & below)] = lane;
            if (lane >= na) a.active[lane] = -1;
            if (lane == a.E - 1) a.offsets[a.E] = incl;
        }
        if (lane == 0) a.n_active[0] = na;
    }
    const int pos = __builtin_amdgcn_ds_bpermute(4 * max(e, 0), start) + rank;
    if (e >= 0) {
        a.sorted_pairs[pos] = (int)threadIdx.x;
        a.pair_pos[threadIdx.x] = pos;
    }
}

// done[t]: blocks that have stored their logits of token t; done[kScoredSmallT]:
// tokens selected.  All zero before and after the call.
template <int VEC>
__global__ __launch_bounds__(kSelThreads) void route_scored_small_kernel(RouteArgs a, ScoreRule rule,
                                                                         unsigned int *done)
{
    static_assert(kScoredSmallT * MOE_MAX_TOPK <= kSelThreads, "one thread a pair");
    __shared__ SmallLds S;
    __shared__ int s_last, s_all;
    const int G = (a.E + kSmallE - 1) / kSmallE;
    const int t = blockIdx.x / G, lane = threadIdx.x & 63;
    logits_block<VEC, true, true, kSmallE>(a, S.lg, t, blockIdx.x % G);
    moe::wait_stores();                                     // this wave's logits are complete
    __syncthreads();
    if (threadIdx.x == 0) {
        const unsigned int before = __hip_atomic_fetch_add(&done[t], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_last = before == (unsigned int)G - 1;
    }
    __syncthreads();
    if (!s_last) return;
    if (threadIdx.x < 64) {
        const float lv = moe::load_dev(a.lbuf + (size_t)t * a.E + min(lane, a.E - 1));
        int id;
        float w;
        select_wave(rule, a.E, a.k, lane, lv, S.sel, id, w);
        if (a.logits && lane < a.E) a.logits[(size_t)t * a.E + lane] = lv;
        if (lane < a.k) {
            moe::store_dev(&a.ids[(size_t)t * a.k + lane], (int32_t)id);
            a.w[(size_t)t * a.k + lane] = w;
        }
        if (lane == 0) done[t] = 0u;
        if (a.T == 1) {                                     // the whole batch is in this wavefront
            group_small(a, lane < a.k ? id : -1, 1, S.cnt);
        } else {
            moe::wait_stores();                             // the ids are complete
            if (lane == 0) {
                unsigned int *all = done + kScoredSmallT;
                const unsigned int before = __hip_atomic_fetch_add(all, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                s_all = before == (unsigned int)a.T - 1;
                if (s_all) *all = 0u;
            }
        }
    }
    if (a.T == 1) return;
    __syncthreads();
    if (!s_all) return;
    const int p = threadIdx.x;
    group_small(a, p < a.T * a.k ? moe::load_dev(&a.ids[p]) : -1, (a.T * a.k + 63) / 64, S.cnt);
}

// ------------------------------------------------------------ larger batches
// Block: 16 tokens x 16 NT experts.  Its 16 wavefronts split H; a wavefront's step
// takes 32 values of H: lane 16q + j holds 8 of token j (values 8q .. 8q + 7 of
// the step) and, per value, the NT experts NT*j .. NT*j + NT - 1 of that router
// row, so one load of NT experts feeds NT matrix instructions (tile n's column
// j is expert NT*j + n; the columns are a permutation of the experts).  The
// loads of a step are in flight while the one before it is multiplied.
//   fp64 matrix instruction, 16x16x4: the products of FP16 values are exact in
//   fp64; a wavefront's chain has H/16 additions per output and the 16 partial
//   sums are added in order: at most H/16 + 16 additions on a path.
// 16 wavefronts: the instruction's unit is shared with the conversions to fp64,
// which four wavefronts a SIMD overlap better than two, and each then selects
// for one token.
//   T = 4096, H 2048, E 64: 30.8 us.  The products alone would take 14.7 us at the
// 72 TFLOP/s of a large fp64 matrix product; of a block's 65 k cycles the loop
// takes 54 k (33 k of matrix instructions; without the loop's loads 47 k, without
// its conversions too 36 k) and the selection 8 k.  Weights moved to fp64 by
// integer operations instead of conversions, packed sums of squares and other
// orders of the steps between blocks left the loop at 55 k.
constexpr int kTileT = 16;
constexpr int kTileThreads = 1024;
constexpr int kTileWaves = kTileThreads / 64;

typedef double f64x4 __attribute__((ext_vector_type(4)));

template <int NT>
struct TileLds {
    union {
        double red[kTileWaves][NT][kTileT][16];
        SelectLds sel[kTileWaves];               // once the sums are taken
    };
    float wsq[kTileWaves][NT * 16];
    float xsq[kTileWaves][kTileT];
    uint32_t xmin[kTileWaves][kTileT];
    float logit[kTileT][64];
    unsigned long long redo[kTileT];
    int any;                                         // some logit needs the integer path
    double ered[kTileWaves][2];
    int cnt[MOE_MAX_EXPERTS];
    int last;
};

// One step's operands of a lane.
template <int NT, bool WIDE>
struct TileStep {
    typename WLoad<8>::T x;
    typename WLoad<NT>::T w[8];
    uint16_t w1[8][WIDE ? 1 : NT];

    // wide: the lane's NT experts lie in one aligned word; else `m` of them, singly
    __device__ inline void load(const uint16_t *xrow, const uint16_t *wcol, int h, int E, int m)
    {
        x = WLoad<8>::ld(xrow + h);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint16_t *row = wcol + (size_t)(h + i) * E;
            if constexpr (WIDE) {
                w[i] = WLoad<NT>::ld(row);
            } else {
#pragma unroll
                for (int n = 0; n < NT; ++n) w1[i][n] = row[min(n, m - 1)];
            }
        }
    }
    __device__ inline uint16_t weight(int i, int n) const { return WIDE ? WLoad<NT>::get(w[i], n) : w1[i][WIDE ? 0 : n]; }
};

// s + c of a running sum after adding p: s the rounded sum, c the sum of the
// additions' errors (each exact, by the error-free transformation of a sum).
__device__ inline void add_exact(double &s, double &c, double p)
{
    const double t = s + p, z = t - s;
    c += (s - (t - z)) + (p - z);
    s = t;
}

// The correctly rounded logit of token t and expert e by the whole block, for
// the rare sum near a rounding border.  Products and partial sums of FP16 x FP16
// are multiples of 2^-48 below 2^44, so s holds their leading 53 bits and c (a
// sum of multiples of 2^-48 below 2^5) the rest: s + c is the exact sum.  Rounding
// hi + lo to odd before the rounding to FP32 makes that one correct rounding.
// Few instructions: this code is seldom in the instruction cache, and a launch
// waits for its slowest tile.  Valid in every thread.
__device__ inline float exact_logit_block(const RouteArgs &a, int t, int e, double (*red)[2])
{
    const int tid = threadIdx.x;
    double s = 0.0, c = 0.0;
    const uint16_t *x = a.x + (size_t)t * a.H, *w = a.wr + e;
#pragma unroll 1
    for (int h0 = tid; h0 < a.H; h0 += 4 * kTileThreads) {              // four pairs of loads in flight
        uint16_t xv[4], wv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int h = h0 + i * kTileThreads, hc = min(h, a.H - 1);
            xv[i] = h < a.H ? x[hc] : (uint16_t)0;
            wv[i] = w[(size_t)hc * a.E];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) add_exact(s, c, h2d(xv[i]) * h2d(wv[i]));
    }
#pragma unroll 1
    for (int off = 32; off >= 1; off >>= 1) {
        const double os = __shfl_xor(s, off);
        c += __shfl_xor(c, off);
        add_exact(s, c, os);
    }
    if ((tid & 63) == 0) {
        red[tid >> 6][0] = s;
        red[tid >> 6][1] = c;
    }
    __syncthreads();
    s = red[0][0];
    c = red[0][1];
#pragma unroll 1
    for (int i = 1; i < kTileWaves; ++i) {
        c += red[i][1];
        add_exact(s, c, red[i][0]);
    }
    __syncthreads();                                                   // red is reused by the next call
    const double hi = s + c, lo = c - (hi - s);
    uint64_t b = __builtin_bit_cast(uint64_t, hi);
    if (lo != 0.0 && !(b & 1)) b += (lo > 0.0) == (hi > 0.0) ? 1 : -1;
    return (float)__builtin_bit_cast(double, b);
}

// Grid: tiles x parts (part p: experts 16 NT p and on).  With more than one
// part the logits meet in a.lbuf ([T][E], device scope) and done[tile] counts
// the parts stored (zero before and after).  counts[tile][E]: the tile's pairs per expert.
template <int NT, bool WIDE>
__global__ __launch_bounds__(kTileThreads) void route_tile_kernel(RouteArgs a, ScoreRule rule, int *counts,
                                                                 unsigned int *done)
{
    __shared__ TileLds<NT> S;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int E = a.E, H = a.H, T = a.T, k = a.k;
    const int tile = blockIdx.x, t0 = tile * kTileT;
    const int first = blockIdx.y * (16 * NT), mine = min(E - first, 16 * NT);   // this block's experts
    const int j = lane & 15, q = lane >> 4;

    f64x4 acc[NT];
    float wsq[NT], xsq = 0.0f;
    uint32_t xmin = ~0u;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        acc[n] = f64x4{0.0, 0.0, 0.0, 0.0};
        wsq[n] = 0.0f;
    }
    const uint16_t *xrow = a.x + (size_t)min(t0 + j, T - 1) * H + 8 * q;
    const int e0 = NT * j < mine ? NT * j : 0;       // lanes past the experts repeat the first (their columns are not read)
    const uint16_t *wcol = a.wr + (size_t)(8 * q) * E + first + e0;
    // single router loads (an odd number of experts, or an unaligned router) leave no registers for a second step
    TileStep<NT, WIDE> cur, nxt;
    if (WIDE && 32 * wave < H) cur.load(xrow, wcol, 32 * wave, E, mine - e0);
    for (int h0 = 32 * wave; h0 < H; h0 += 32 * kTileWaves) {
        if (!WIDE) cur.load(xrow, wcol, h0, E, mine - e0);
        else if (h0 + 32 * kTileWaves < H) nxt.load(xrow, wcol, h0 + 32 * kTileWaves, E, mine - e0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float xf = (float)__builtin_bit_cast(_Float16, WLoad<8>::get(cur.x, i));
            xsq = fmaf(xf, xf, xsq);
            xmin = min(xmin, magnitude_less_one(WLoad<8>::get(cur.x, i)));
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float wf = (float)__builtin_bit_cast(_Float16, cur.weight(i, n));
                wsq[n] = fmaf(wf, wf, wsq[n]);
                acc[n] = __builtin_amdgcn_mfma_f64_16x16x4f64((double)xf, (double)wf, acc[n], 0, 0, 0);
            }
        }
        if (WIDE) cur = nxt;
    }
    // partial sums of this wavefront: lane (q, j) holds tokens q + 4r of column j
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) S.red[wave][n][q + 4 * r][j] = acc[n][r];
    xsq = sum_phases<16>(xsq);
    xmin = min(xmin, moe::partner_u32<true>(xmin));
    xmin = min(xmin, moe::partner_u32<false>(xmin));
#pragma unroll
    for (int n = 0; n < NT; ++n) wsq[n] = sum_phases<16>(wsq[n]);
    if (q == 0) {
        S.xsq[wave][j] = xsq;
        S.xmin[wave][j] = xmin;
#pragma unroll
        for (int n = 0; n < NT; ++n) S.wsq[wave][NT * j + n] = wsq[n];
    }
    if (tid < kTileT) S.redo[tid] = 0ull;
    if (tid == 0) S.any = 0;
    if (tid < MOE_MAX_EXPERTS) S.cnt[tid] = 0;
    __syncthreads();
    constexpr int OUT = kTileT * NT * 16;
#pragma unroll
    for (int o0 = 0; o0 < OUT; o0 += kTileThreads) {
        const int o = o0 + tid;
        const int n = o / (kTileT * 16), tt = o / 16 % kTileT, e = NT * (o % 16) + n;
        if (o >= OUT || e >= mine || t0 + tt >= T) continue;
        double v = 0.0;
        float X = 0.0f, W = 0.0f, most = 0.0f, high = 0.0f;
        uint32_t least = ~0u;
#pragma unroll
        for (int w = 0; w < kTileWaves; ++w) {
            v += S.red[w][n][tt][o % 16];
            least = min(least, S.xmin[w][tt]);
            X += S.xsq[w][tt];
            W += S.wsq[w][e];
            most = fmaxf(most, S.xsq[w][tt] * S.wsq[w][e]);
            high = fmaxf(high, fabsf((float)v));
        }
        // |v - exact| <= n 2^-53 (1 + n 2^-53) sum|x w| for paths of at most n additions, and
        // sum|x w| <= sqrt(X W).  The FP32 sums of exact squares (at most H <= 4096 roundings) are
        // within a factor 1 + 2^-11 of their true values, the root and the products below within
        // 1 + 2^-20.
        const float bound = __builtin_amdgcn_sqrtf(X * W) * (1.0f + 0x1p-9f);
        const float err = (float)(H / kTileWaves + 32 + kTileWaves) * 0x1p-53f * bound;
        // No addition has rounded where the bound of each wavefront's own sum and the sums over the
        // wavefronts as they came out are small (sums_exact): then v is the exact logit.  The bound of
        // the whole sum is some ten times a wavefront's, and with it alone about one logit in 3e4 was
        // redone (normal activations, H 2048), which cost the slowest tile 15 k cycles (T = 4096: 36.7 us
        // against 31.0).
        const bool exact = sums_exact(least, fmaxf(__builtin_amdgcn_sqrtf(most), high) * (1.0f + 0x1p-9f));
        S.logit[tt][e] = (float)v;
        if (isfinite(v) && !exact && !rn32_certain(v, (double)err)) {
            atomicOr(&S.redo[tt], 1ull << e);
            S.any = 1;
        }
    }
    __syncthreads();
    for (int tt = 0; S.any && tt < kTileT; ++tt) {
        unsigned long long redo = S.redo[tt];
        while (redo) {                               // rare: exact recomputation by the whole block
            const int e = __builtin_ctzll(redo);
            redo &= redo - 1ull;
            const float l = exact_logit_block(a, t0 + tt, first + e, S.ered);
            if (tid == 0) S.logit[tt][e] = l;
        }
    }
    __syncthreads();
    if (gridDim.y > 1) {
        for (int o = tid; o < OUT; o += kTileThreads) {
            const int tt = o / (NT * 16), e = o % (NT * 16);
            if (e < mine && t0 + tt < T) moe::store_dev(&a.lbuf[(size_t)(t0 + tt) * E + first + e], S.logit[tt][e]);
        }
        moe::wait_stores();
        __syncthreads();
        if (tid == 0) {
            const unsigned int before =
                __hip_atomic_fetch_add(&done[tile], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            S.last = before == gridDim.y - 1;
            if (S.last) done[tile] = 0u;
        }
        __syncthreads();
        if (!S.last) return;
    }
    const int tt = wave, t = t0 + tt;
    if (t < T) {
        const int e = min(lane, E - 1);
        const float lv = gridDim.y > 1 ? moe::load_dev(&a.lbuf[(size_t)t * E + e]) : S.logit[tt][e];
        if (a.logits && lane < E) a.logits[(size_t)t * E + lane] = lv;
        int id;
        float w;
        select_wave(rule, E, k, lane, lv, S.sel[wave], id, w);
        if (lane < k) {
            const size_t p = (size_t)t * k + lane;
            a.ids[p] = id;
            a.w[p] = w;
            atomicAdd(&S.cnt[id], 1);
        }
    }
    __syncthreads();
    if (tid < E) counts[(size_t)tile * E + tid] = S.cnt[tid];
}

// Bound by its launch and two dependent loads: T = 611, k 4 4.0 us, T = 4096, k 8 4.7.
// Places the pairs of `tiles` 16-token tiles per block: expert e's pairs of
// tile g start at the expert's offset (all tiles' counts of the experts before
// it) plus the counts of e in the tiles before g.
constexpr int kPlaceWaves = 16;

__global__ __launch_bounds__(kPlaceWaves * 64) void route_place_kernel(RouteArgs a, const int *counts, int G, int tiles)
{
    __shared__ int s_tot[kPlaceWaves][64], s_pre[kPlaceWaves][64], s_cnt[kPlaceWaves][64], s_base[kPlaceWaves][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int E = a.E, n = a.T * a.k, ec = min(lane, E - 1);
    const int g0 = blockIdx.x * tiles;
    int tot = 0, pre = 0;
    constexpr int U = 8;
    for (int g = wave; g < G; g += kPlaceWaves * U) {
        int c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int gg = g + u * kPlaceWaves;
            c[u] = gg < G ? counts[(size_t)gg * E + ec] : 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            tot += c[u];
            pre += g + u * kPlaceWaves < g0 ? c[u] : 0;
        }
    }
    // this block's pairs, each wavefront a contiguous range
    const int b0 = g0 * kTileT * a.k, b1 = min(n, b0 + tiles * kTileT * a.k);
    const int len = b1 - b0;
    const int p0 = b0 + (int)((long long)len * wave / kPlaceWaves);
    const int p1 = b0 + (int)((long long)len * (wave + 1) / kPlaceWaves);
    s_tot[wave][lane] = tot;
    s_pre[wave][lane] = pre;
    s_cnt[wave][lane] = 0;
    for (int p = p0 + lane; p < p1; p += 64) atomicAdd(&s_cnt[wave][a.ids[p] & 63], 1);
    __syncthreads();
    if (wave == 0) {
        int c = 0, before = 0;
#pragma unroll
        for (int w = 0; w < kPlaceWaves; ++w) {
            c += s_tot[w][lane];
            before += s_pre[w][lane];
        }
        if (lane >= E) c = 0;
        const int incl = moe::wave_inclusive_sum(c), excl = incl - c;
        int run = excl + before;
        for (int w = 0; w < kPlaceWaves; ++w) {
            s_base[w][lane] = run;
            run += s_cnt[w][lane];
        }
        if (blockIdx.x == 0) {
            const unsigned long long act = __ballot(lane < E && c > 0);
            const int na = __popcll(act);
            if (lane < E) {
                a.offsets[lane] = excl;
                if (c > 0) a.active[__popcll(act & ((1ull << lane) - 1ull))] = lane;
                if (lane >= na) a.active[lane] = -1;
                if (lane == E - 1) a.offsets[E] = incl;
            }
            if (lane == 0) a.n_active[0] = na;
        }
    }
    __syncthreads();
    const unsigned long long below = (1ull << lane) - 1ull;
    for (int c0 = p0; c0 < p1; c0 += 64) {
        const int p = c0 + lane;
        const int e = p < p1 ? a.ids[p] & 63 : -1;
        const unsigned long long peers = same_expert_lanes(e);
        if (e >= 0) {
            const int rank = __popcll(peers & below);
            const int pos = s_base[wave][e] + rank;
            a.sorted_pairs[pos] = p;
            a.pair_pos[p] = pos;
            if (rank == 0) s_base[wave][e] = pos + __popcll(peers);   // one leader per expert and chunk
        }
    }
}

// Tiles whose experts are divided among blocks: enough blocks for the GPU's
// 256 CUs.  Measured with 16, 32, 64 experts a block (H 2048, E 64, whole call,
// us): T = 512 16.9, 21.7, 30.9; T = 1024 18.2, 22.2, 31.2; T = 2048 28.4, 23.5,
// 31.7; T = 4096 with 64 34.1.
constexpr int kSplitTiles = 128;

// Workspace: the counters (zero between calls), then the logits handed between
// blocks, then the tiles' counts.
constexpr size_t kScoredCtrl = 1024;
static_assert(kTileWaves == kTileT, "one wavefront selects for one token");
static_assert(kScoredCtrl >= (kScoredSmallT + 1) * sizeof(int) && kScoredCtrl >= kSplitTiles * sizeof(int), "counters");

size_t scored_lbuf_bytes(int T, int E)
{
    const int rows = T < kSplitTiles * kTileT ? T : kSplitTiles * kTileT;
    return ((size_t)rows * E * sizeof(float) + 255) / 256 * 256;
}

size_t scored_ws_bytes(int T, int E)
{
    const size_t counts = (size_t)((T + kTileT - 1) / kTileT) * E * sizeof(int);
    return kScoredCtrl + scored_lbuf_bytes(T, E) + (counts + 255) / 256 * 256;
}

template <int NT>
void launch_tiles(const RouteArgs &a, const ScoreRule &rule, int *counts, unsigned int *done, hipStream_t s)
{
    const dim3 grid((unsigned int)((a.T + kTileT - 1) / kTileT), (unsigned int)((a.E + 16 * NT - 1) / (16 * NT)));
    if (a.E % NT == 0 && moe::aligned(a.wr, 2 * NT))
        hipLaunchKernelGGL((route_tile_kernel<NT, true>), grid, dim3(kTileThreads), 0, s, a, rule, counts, done);
    else hipLaunchKernelGGL((route_tile_kernel<NT, false>), grid, dim3(kTileThreads), 0, s, a, rule, counts, done);
}

}  // namespace

extern "C" {

size_t moe_route_scored_workspace_size(int T, int H, int E)
{
    (void)H;
    if (T < 0 || T > 65536 || E < 1 || E > MOE_MAX_EXPERTS) return 0;
    return scored_ws_bytes(T, E);
}

int moe_route_scored(const void *x_dev, const void *w_router_dev, const float *select_bias_dev, int T, int H, int E,
                     int k, const moe_route_rule *rule, float *logits_dev, int32_t *topk_ids_dev, float *topk_w_dev,
                     int32_t *expert_offsets_dev, int32_t *sorted_pairs_dev, int32_t *pair_pos_dev,
                     int32_t *active_list_dev, int32_t *n_active_dev, void *ws_dev, size_t ws_bytes, void *stream)
{
    moe::clear_error();
    const char *who = "moe_route_scored";
    int rc = moe::check_shape(T, H, 0, E, k, false);
    if (rc) return rc;
    if (H > kMaxH) return moe::fail(MOE_ERR_UNSUPPORTED, "%s: H=%d > %d", who, H, kMaxH);
    if (!rule) return moe::fail(MOE_ERR_INVALID_ARG, "%s: null rule", who);
    if (rule->score != MOE_SCORE_SOFTMAX && rule->score != MOE_SCORE_SIGMOID)
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: unknown score %d", who, rule->score);
    if (rule->group_score != MOE_GROUP_MAX && rule->group_score != MOE_GROUP_TOP2)
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: unknown group score %d", who, rule->group_score);
    const int G = rule->n_group;
    if (G < 1 || G > E || E % G)
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: n_group=%d must divide E=%d", who, G, E);
    if (rule->topk_group < 1 || rule->topk_group > G)
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: topk_group=%d outside [1, n_group=%d]", who, rule->topk_group, G);
    if (k > rule->topk_group * (E / G))
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: k=%d exceeds the %d experts of topk_group=%d groups", who, k,
                         rule->topk_group * (E / G), rule->topk_group);
    if (G > 1 && rule->group_score == MOE_GROUP_TOP2 && E / G < 2)
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: groups of one expert have no two largest", who);
    if (!(rule->scale > 0.0f) || rule->scale > 3.0e38f)
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: scale=%g must be positive and finite", who, (double)rule->scale);
    if (T == 0) return MOE_OK;
    if (!x_dev || !w_router_dev || !topk_ids_dev || !topk_w_dev || !expert_offsets_dev || !sorted_pairs_dev ||
        !pair_pos_dev || !active_list_dev || !n_active_dev)
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: null pointer argument", who);
    if (!moe::aligned(x_dev, 16) || !moe::aligned(w_router_dev, 2) || !moe::aligned(select_bias_dev, 4))
        return moe::fail(MOE_ERR_INVALID_ARG, "%s: x must be 16-byte, w_router 2-byte and select_bias 4-byte aligned", who);
    if (!ws_dev || ws_bytes < scored_ws_bytes(T, E) || !moe::aligned(ws_dev, 256))
        return moe::fail(MOE_ERR_WORKSPACE, "%s: the workspace needs %zu bytes, 256-byte aligned", who,
                         scored_ws_bytes(T, E));

    RouteArgs a;
    a.x = (const uint16_t *)x_dev;
    a.wr = (const uint16_t *)w_router_dev;
    a.bias = nullptr;
    a.T = T; a.H = H; a.E = E; a.k = k;
    a.logits = logits_dev;
    a.ids = topk_ids_dev;
    a.w = topk_w_dev;
    a.offsets = expert_offsets_dev;
    a.sorted_pairs = sorted_pairs_dev;
    a.pair_pos = pair_pos_dev;
    a.active = active_list_dev;
    a.n_active = n_active_dev;
    a.force_exact = 0;
    a.lbuf = (float *)((uint8_t *)ws_dev + kScoredCtrl);
    ScoreRule r;
    r.bias = select_bias_dev;
    r.softmax = rule->score == MOE_SCORE_SOFTMAX;
    r.n_group = G;
    r.topk_group = rule->topk_group;
    r.top2 = rule->group_score == MOE_GROUP_TOP2;
    r.renorm = rule->renormalize != 0;
    r.scale = (double)rule->scale;
    hipStream_t s = (hipStream_t)stream;
    if (T <= kScoredSmallT) {
        unsigned int *done = (unsigned int *)ws_dev;
        const unsigned int blocks = (unsigned int)T * (unsigned int)((E + kSmallE - 1) / kSmallE);
        if (E % 2 == 0 && moe::aligned(w_router_dev, 4))
            hipLaunchKernelGGL(route_scored_small_kernel<2>, dim3(blocks), dim3(kSelThreads), 0, s, a, r, done);
        else hipLaunchKernelGGL(route_scored_small_kernel<1>, dim3(blocks), dim3(kSelThreads), 0, s, a, r, done);
        return moe::check_launch(who);
    }
    int *counts = (int *)((uint8_t *)a.lbuf + scored_lbuf_bytes(T, E));
    unsigned int *done = (unsigned int *)ws_dev;
    const int tiles_total = (T + kTileT - 1) / kTileT;
    // one block has the tile's experts where that fills the GPU, else 2 or 4 divide them
    const int column_tiles = (E + 15) / 16;
    if (column_tiles > 2 && tiles_total > kSplitTiles) launch_tiles<4>(a, r, counts, done, s);
    else if (column_tiles > 1 && tiles_total > kSplitTiles / 2) launch_tiles<2>(a, r, counts, done, s);
    else launch_tiles<1>(a, r, counts, done, s);
    rc = moe::check_launch("moe_route_scored (select)");
    if (rc) return rc;
    // at least 4 tiles per block, and at most 256 blocks: every block reads all tiles' counts.  Whole call
    // with 1, 2, 4, 8, 16 tiles a block (H 128, us): T = 512 10.2, 10.3, 10.3, 10.3, 11.1; T = 16384 48.7,
    // 40.1, 36.4, 35.8, 37.2; T = 65536 336, 227, 171, 142, 131
    const int tiles = tiles_total > 1024 ? (tiles_total + 255) / 256 : 4;
    hipLaunchKernelGGL(route_place_kernel, dim3((unsigned int)((tiles_total + tiles - 1) / tiles)),
                       dim3(kPlaceWaves * 64), 0, s, a, (const int *)counts, tiles_total, tiles);
    return moe::check_launch("moe_route_scored (grouping)");
}

}  // extern "C"
