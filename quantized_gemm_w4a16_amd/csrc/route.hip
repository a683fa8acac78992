// route.hip -- which experts a token takes (spear_route): logits, softmax or
// sigmoid scores, a bias for the choice, groups, top-k and renormalised
// weights (gfx950).
//
//   z_me = sum_k x[m][k] w[e][k], s = softmax(z) or sigmoid(z), c = s + bias;
//   the topk largest c of the kept groups, weights from s.
//
// The choice is that of logits summed in fp64.  Three forms reach it:
//  * few tokens, two launches: the logits in fp64 by the whole chip (each bf16 x
//    bf16 product is exact there), then one wave a token chooses;
//  * some tokens and a small router, one launch: a workgroup a token does both;
//  * many tokens, two launches: the logits by bf16 MFMA in fp32, each with a
//    bound of its error, then 16 lanes a token choose in fp32.  Where the bounds
//    leave the order of two candidates open, the logits in question are summed
//    again in fp64, so the choice is the same.  How many tokens that takes, and so
//    the time, depends on the logits (the choice's comment).
#include <math.h>

#include <type_traits>

#include "spear_internal.hpp"

namespace spear {

namespace {

constexpr int64_t MAX_TOKENS = 1 << 27;                   // a launch stays below 2^32 threads

struct RouteArgs {
    const uint16_t *x, *w;
    const float *bias;
    float *weights;
    int32_t *ids;
    float *z;                                             // [ks][M][E] partial logits (two launches)
    float *xn;                                            // [ks][M]: partial squares of x's rows
    float *wn;                                            // [ks][32]: the largest of 16 rows of w each
    int64_t M, K;
    int32_t E, topk, score, n_group, topk_group, group_best, renorm;
    float scale;
    float zerr;                                           // error of a logit over the rows' 2-norms
    int32_t ks, net;                                      // K slices, expert tiles
};

// ---------------------------------------------------------- wave reductions
// By DPP on the vector ALU: within rows of 16 lanes by shifts of 1, 2, 4 and 8,
// then the row totals handed on; lane 63 holds the total, read as a scalar.
// (Through the LDS crossbar, as shuffles go, the 8192-token choice was bound by
// it: 82 us of which two thirds were shuffles.)
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t v, uint32_t ident)
{
    return (uint32_t)__builtin_amdgcn_update_dpp((int)ident, (int)v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double v, double ident)
{
    const uint64_t a = __builtin_bit_cast(uint64_t, v), i = __builtin_bit_cast(uint64_t, ident);
    const uint64_t r = (uint64_t)dpp<CTRL, ROWS>((uint32_t)a, (uint32_t)i) |
                       ((uint64_t)dpp<CTRL, ROWS>((uint32_t)(a >> 32), (uint32_t)(i >> 32)) << 32);
    return __builtin_bit_cast(double, r);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float v, float ident)
{
    return __uint_as_float(dpp<CTRL, ROWS>(__float_as_uint(v), __float_as_uint(ident)));
}
__device__ __forceinline__ uint32_t lane_of(uint32_t v, int l)
{
    return (uint32_t)__builtin_amdgcn_readlane((int)v, l);
}
__device__ __forceinline__ float lane_of(float v, int l) { return __uint_as_float(lane_of(__float_as_uint(v), l)); }
__device__ __forceinline__ double lane_of(double v, int l)
{
    const uint64_t a = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)lane_of((uint32_t)a, l) |
                                          ((uint64_t)lane_of((uint32_t)(a >> 32), l) << 32));
}
template <typename T, typename F>
__device__ __forceinline__ T wave_reduce(T v, T ident, F op)
{
    v = op(v, dpp<0x111, 0xF>(v, ident));                 // row_shr 1, 2, 4, 8
    v = op(v, dpp<0x112, 0xF>(v, ident));
    v = op(v, dpp<0x114, 0xF>(v, ident));
    v = op(v, dpp<0x118, 0xF>(v, ident));
    v = op(v, dpp<0x142, 0xA>(v, ident));                 // row_bcast 15 into rows 1 and 3
    v = op(v, dpp<0x143, 0xC>(v, ident));                 // row_bcast 31 into rows 2 and 3
    return lane_of(v, 63);
}
__device__ __forceinline__ double wave_sum(double v)
{
    return wave_reduce(v, 0.0, [](double p, double q) { return p + q; });
}
__device__ __forceinline__ double wave_max(double v)
{
    return wave_reduce(v, -(double)INFINITY, [](double p, double q) { return q > p ? q : p; });
}
__device__ __forceinline__ float wave_max(float v)
{
    return wave_reduce(v, -INFINITY, [](float p, float q) { return q > p ? q : p; });
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    return wave_reduce(v, 0u, [](uint32_t p, uint32_t q) { return q > p ? q : p; });
}

// Four sums over the wave at once, z[l % 4] in lane l: the first two steps halve
// what is left to add.
__device__ __forceinline__ double wave_sum4(const double (&z)[4], int lane)
{
    const bool b0 = lane & 1, b1 = lane & 2;
    double p = b0 ? z[1] : z[0], q = b0 ? z[3] : z[2], o = b0 ? z[0] : z[1];
    p += dpp<0xB1, 0xF>(o, o);                            // quad_perm 1 0 3 2
    o = b0 ? z[2] : z[3];
    q += dpp<0xB1, 0xF>(o, o);
    o = b1 ? p : q;
    p = b1 ? q : p;
    p += dpp<0x4E, 0xF>(o, o);                            // quad_perm 2 3 0 1
    p += dpp<0x124, 0xF>(p, p);                           // row_ror 4, 8
    p += dpp<0x128, 0xF>(p, p);
    p += __shfl_xor(p, 16);
    p += __shfl_xor(p, 32);
    return p;
}

// acc + the products of 8 bf16 of x and w: every product exact, the sum in fp64.
__device__ __forceinline__ double dot8(u32x4 x, u32x4 w, double acc)
{
#pragma unroll
    for (int q = 0; q < 4; q++) {
        acc = fma((double)__uint_as_float(x[q] << 16), (double)__uint_as_float(w[q] << 16), acc);
        acc = fma((double)__uint_as_float(x[q] & 0xFFFF0000u), (double)__uint_as_float(w[q] & 0xFFFF0000u),
                  acc);
    }
    return acc;
}

// ---------------------------------------------------------------------- choice
// Logits of token m and n listed experts in fp64, by one wave: two experts at a
// time, 2048 depths of loads in flight.
__device__ __forceinline__ void exact_logits(const RouteArgs &a, int64_t m, int lane, const uint16_t *list, int n,
                                             double *z)
{
    const uint16_t *xr = a.x + m * a.K;
#pragma unroll 1
    for (int p = 0; p < n; p += 2) {
        const int p1 = p + 1 < n ? p + 1 : p;
        const uint16_t *w0 = a.w + (int64_t)list[p] * a.K, *w1 = a.w + (int64_t)list[p1] * a.K;
        double s0 = 0.0, s1 = 0.0;
#pragma unroll 1
        for (int64_t k0 = 0; k0 < a.K; k0 += 2048) {
            u32x4 xv[4], v0[4], v1[4];
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int64_t k = k0 + 512 * q + 8 * lane;
                const bool in = k < a.K;
                xv[q] = in ? ld16(xr + k) : zero4();
                v0[q] = in ? ld16(w0 + k) : zero4();
                v1[q] = in ? ld16(w1 + k) : zero4();
            }
#pragma unroll
            for (int q = 0; q < 4; q++) {
                s0 = dot8(xv[q], v0[q], s0);
                s1 = dot8(xv[q], v1[q], s1);
            }
        }
        s0 = wave_sum(s0);
        s1 = wave_sum(s1);
        if (lane == 0) {
            z[p] = s0;
            z[p1] = s1;
        }
    }
    wait_lgkmcnt0();
}

// Appends v of the lanes where `in` holds to a list in LDS; returns its length.
__device__ __forceinline__ int append(uint16_t *list, int n, bool in, int v, int lane)
{
    const uint64_t mask = __ballot(in);
    if (in)
        list[n + __popcll(mask & ((1ull << lane) - 1ull))] = (uint16_t)v;
    return n + __popcll(mask);
}

__device__ __forceinline__ double score_of(const RouteArgs &a, double z, double mx, double sum)
{
    return a.score == SPEAR_SCORE_SOFTMAX ? exp(z - mx) / sum : 1.0 / (1.0 + exp(-z));
}

// The choice: score and bias, -inf where there is none to be made.
__device__ __forceinline__ double choice_of(const RouteArgs &a, double s, int e)
{
    const double v = a.bias ? s + (double)a.bias[e] : s;
    return v == v ? v : -(double)INFINITY;
}

// Winner t's weight and id, by lane t.
__device__ __forceinline__ void write_choice(const RouteArgs &a, int64_t m, int lane, int id, double s)
{
    s = id < 0 ? 0.0 : s;
    if (a.renorm) {
        const double total = wave_sum(s);
        s = total == 0.0 ? 0.0 : s / total;
    }
    if (lane < a.topk) {
        a.ids[m * a.topk + lane] = id;
        a.weights[m * a.topk + lane] = id < 0 ? 0.f : (float)(s * (double)a.scale);
    }
}

// The whole choice of token m by one wave, from all its logits z[0..E) in fp64
// (LDS, as is c[0..E)).  Loops are kept rolled: straight-line code that each
// wave runs once costs more in instruction fetches than in instructions.
__device__ __forceinline__ void choose_all(const RouteArgs &a, int64_t m, int lane, const double *z, double *c)
{
    const double ninf = -INFINITY;
    const int E = a.E, G = a.n_group, gs = E / G;
    double mx = 0.0, sum = 1.0;
    if (a.score == SPEAR_SCORE_SOFTMAX) {
        double t = ninf, u = 0.0;
        bool nan = false;
#pragma unroll 1
        for (int e = lane; e < E; e += 64) {
            t = z[e] > t ? z[e] : t;
            nan |= z[e] != z[e];
        }
        mx = __any(nan) ? __builtin_nan("") : wave_max(t);
#pragma unroll 1
        for (int e = lane; e < E; e += 64)
            u += exp(z[e] - mx);
        sum = wave_sum(u);
    }
#pragma unroll 1
    for (int e = lane; e < E; e += 64)
        c[e] = choice_of(a, score_of(a, z[e], mx, sum), e);
    wait_lgkmcnt0();
    if (a.topk_group < G) {
        // lane g: the sum of group g's best one or two choices
        double b0 = ninf, b1 = ninf;
        if (lane < G)
#pragma unroll 4
            for (int i = 0; i < gs; i++) {
                const double v = c[lane * gs + i];
                b1 = v > b0 ? b0 : (v > b1 ? v : b1);
                b0 = v > b0 ? v : b0;
            }
        double gv = lane < G ? ((a.group_best == 2 && gs > 1) ? b0 + b1 : b0) : ninf;
        gv = gv == gv ? gv : ninf;                        // +inf and -inf biases in one group
        int rank = 0;
#pragma unroll 1
        for (int g = 0; g < G; g++) {
            const double o = lane_of(gv, g);
            rank += o > gv || (o == gv && g < lane);
        }
        const uint64_t kept = __ballot(lane < G && rank < a.topk_group);
#pragma unroll 1
        for (int e = lane; e < E; e += 64)
            if (!((kept >> (e / gs)) & 1))
                c[e] = ninf;
    }
    // rounds: the best candidate left, the lowest expert of equal ones
    int id = -1;
#pragma unroll 1
    for (int t = 0; t < a.topk; t++) {
        double bv = ninf;
        uint32_t be = 0;
#pragma unroll 1
        for (int e = lane; e < E; e += 64)
            if (c[e] > bv) {
                bv = c[e];
                be = (uint32_t)e;
            }
        const double best = wave_max(bv);
        if (best == ninf)
            break;                                        // no candidate is left
        const uint64_t who = __ballot(bv == best);
        uint32_t e = lane_of(be, __builtin_ctzll(who));
        if (who & (who - 1))
            e = ~wave_max(bv == best ? ~be : 0u);
        if ((int)(e & 63u) == lane)
            c[e] = ninf;
        id = lane == t ? (int)e : id;
    }
    write_choice(a, m, lane, id, id < 0 ? 0.0 : score_of(a, z[id], mx, sum));
}

// ------------------------------------------------------------------ one launch
// One workgroup (16 waves) a token.  Wave w sums the logits of experts w,
// w + 16, ... in fp64, four at a time with their loads in flight together; the
// first wave then chooses.  Bound by one CU's fp64 conversions and the choice's
// dependent steps (256 tokens, 64 experts x 2048: 11.7 us in a graph).
constexpr int RF_WAVES = 16;

__global__ __launch_bounds__(64 * RF_WAVES) void route_fused_kernel(const RouteArgs a)
{
    __shared__ double s_z[SPEAR_MAX_EXPERTS], s_c[SPEAR_MAX_EXPERTS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t m = blockIdx.x, K = a.K;
    const int E = a.E;
    const uint16_t *xr = a.x + m * K;
    for (int e0 = wave; e0 < E; e0 += 4 * RF_WAVES) {
        const uint16_t *wr[4];
        double acc[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
        for (int i = 0; i < 4; i++)
            wr[i] = a.w + (int64_t)(e0 + RF_WAVES * i < E ? e0 + RF_WAVES * i : e0) * K;
        for (int64_t k0 = 0; k0 < K; k0 += 2048) {
            u32x4 xv[4], wv[4][4];
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int64_t k = k0 + 512 * q + 8 * lane;
                xv[q] = k < K ? ld16(xr + k) : zero4();
#pragma unroll
                for (int i = 0; i < 4; i++)
                    wv[q][i] = k < K ? ld16(wr[i] + k) : zero4();
            }
#pragma unroll
            for (int q = 0; q < 4; q++)
#pragma unroll
                for (int i = 0; i < 4; i++)
                    acc[i] = dot8(xv[q], wv[q][i], acc[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            acc[i] = wave_sum(acc[i]);
            if (lane == 0 && e0 + RF_WAVES * i < E)
                s_z[e0 + RF_WAVES * i] = acc[i];
        }
    }
    __syncthreads();
    if (wave != 0)
        return;
    choose_all(a, m, lane, s_z, s_c);
}

// ------------------------------------------------------- two launches, few tokens
// A wave sums the logits of one token and two experts in fp64 (to the
// workspace); in the second launch one wave a token chooses.  One token is bound
// by the two round trips to memory and the launches (8.7 us in a graph), more of
// them by fp64 conversions (64 tokens, 256 experts x 4096: 21.7 us).
constexpr int RX_WAVES = 4;

__global__ __launch_bounds__(64 * RX_WAVES) void route_exact_kernel(const RouteArgs a)
{
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t m = blockIdx.y, K = a.K;
    const int E = a.E, e0 = 2 * ((int)blockIdx.x * RX_WAVES + wave);
    if (e0 >= E)
        return;
    const uint16_t *xr = a.x + m * K, *w0 = a.w + (int64_t)e0 * K, *w1 = e0 + 1 < E ? w0 + K : w0;
    double s0 = 0.0, s1 = 0.0;
#pragma unroll 1
    for (int64_t k0 = 0; k0 < K; k0 += 4096) {
        u32x4 xv[8], v0[8], v1[8];
#pragma unroll
        for (int q = 0; q < 8; q++) {
            const int64_t k = k0 + 512 * q + 8 * lane;
            const int64_t kk = k < K ? k : 8 * lane % K;  // (past K: the rows' first ones, made zeros)
            xv[q] = ld16(xr + kk);
            v0[q] = ld16(w0 + kk);
            v1[q] = ld16(w1 + kk);
        }
        // both operands: zero times an infinite weight is no zero
#pragma unroll
        for (int q = 0; q < 8; q++)
            if (k0 + 512 * q + 8 * lane >= K)
                xv[q] = v0[q] = v1[q] = zero4();
#pragma unroll
        for (int q = 0; q < 8; q++) {
            s0 = dot8(xv[q], v0[q], s0);
            s1 = dot8(xv[q], v1[q], s1);
        }
    }
    s0 = wave_sum(s0);
    s1 = wave_sum(s1);
    double *z = reinterpret_cast<double *>(a.z) + m * E + e0;
    if (lane == 0) {
        z[0] = s0;
        if (e0 + 1 < E)
            z[1] = s1;
    }
}

__global__ __launch_bounds__(64) void route_pick_kernel(const RouteArgs a)
{
    __shared__ double s_z[SPEAR_MAX_EXPERTS], s_c[SPEAR_MAX_EXPERTS];
    const int lane = threadIdx.x;
    const int64_t m = blockIdx.x;
    const double *z = reinterpret_cast<const double *>(a.z) + m * a.E;
    for (int e = lane; e < a.E; e += 64)
        s_z[e] = z[e];
    wait_lgkmcnt0();
    choose_all(a, m, lane, s_z, s_c);
}

// ------------------------------------------------------ two launches, many tokens
// Logits by MFMA: a workgroup of 8 waves takes 64 WN experts and 128 tokens
// over one of ks K slices, in stages of 64 depths that go from global memory
// to a ring of LDS buffers by DMA (128 bytes a row, 16-byte chunks swizzled by
// row % 8), one barrier a stage.  Wave (wn, wm) takes 64 experts x 16 FM
// tokens.  The slices' partial sums are added by the choice.  Bound by what goes
// from L2 to LDS: 8192 tokens x 256 experts x 4096 29 us, 201 MB by DMA (6.9 TB/s)
// and 33 MB of partial sums; operands straight from memory took 100 us.
//
// Error: a product passes through at most 32 roundings inside a matrix
// instruction (whatever its order), 8 along a chain of them (the chain's sum
// then moves to a second accumulator), one for each of a slice's chains and
// one for each slice, of a step (2^-23) at most (the hardware rounds to nearest
// and fewer times: with sums of one sign, with a first product 3000 times the
// others, and with exponents spread over 12 bits, K of 256 to 8192, the largest
// error of a logit was 5.8 such units where this allows 52).  So a logit is off by at most
// (32 + 8 + chains + ks) 2^-23 sum |x w|, and sum |x w| is at most the product
// of the rows' 2-norms, whose squares are formed on the way.
constexpr int RL_TM = 128;
constexpr int RL_FRAGS = SPEAR_MAX_EXPERTS / 16;
constexpr int RL_CHAIN = 4;                               // stages (of two instructions) a chain

__device__ __forceinline__ float sq8(u32x4 v, float acc)
{
#pragma unroll
    for (int q = 0; q < 4; q++)
        acc = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(v[q]), as_bf16x2(v[q]), acc, false);
    return acc;
}

// Columns of 64 experts in a tile.
__host__ __device__ __forceinline__ int tile_waves(int32_t E) { return E <= 64 ? 1 : E <= 128 ? 2 : 4; }

template <int WN>
__global__ __launch_bounds__(512) void route_logits_kernel(const RouteArgs a)
{
    constexpr int WM = 8 / WN, FM = RL_TM / (16 * WM), TE = 64 * WN;
    constexpr int SB = (TE + RL_TM) * 128;                // bytes of a stage
    constexpr int NI = SB / 8192;                         // DMAs a wave issues per stage
    constexpr int RING = WN == 4 ? 3 : WN == 2 ? 4 : 6;
    constexpr int WAIT = (RING - 2) * NI;
    static_assert(NI * 8192 == SB && WAIT < 64, "stage split");
    __shared__ __attribute__((aligned(16))) uint8_t s_r0[SB], s_r1[SB], s_r2[SB];
    __shared__ __attribute__((aligned(16))) uint8_t s_r3[RING > 3 ? SB : 16], s_r4[RING > 4 ? SB : 16],
        s_r5[RING > 5 ? SB : 16];
    uint8_t *const ring[6] = {s_r0, s_r1, s_r2, s_r3, s_r4, s_r5};
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4;
    const int wn = wave % WN, wm = wave / WN;
    const int64_t M = a.M, K = a.K;
    const int E = a.E;
    // An XCD takes a contiguous run of units, the token tiles fastest, so that
    // its L2 keeps one slice of w for all of them.
    const int64_t ntt = (M + RL_TM - 1) / RL_TM, units = ntt * a.net * a.ks;
    const int64_t q8 = units / 8, r8 = units % 8, xcd = blockIdx.x % 8;
    const int64_t unit = xcd * q8 + (xcd < r8 ? xcd : r8) + blockIdx.x / 8;
    const int64_t m0 = unit % ntt * RL_TM;
    const int e0 = (int)(unit / ntt % a.net) * TE, ks = (int)(unit / (ntt * a.net));
    const int64_t S = (K + 63) / 64, sb = ks * S / a.ks, se = (ks + 1) * S / a.ks, slast = se - 1;

    // DMA i of a wave fills 1 KB: rows 8 (NI wave + i) .. + 7, lane l position
    // l % 8 of row l / 8.  A chunk past K re-reads the row's last one inside it
    // (its step is not taken).
    const uint16_t *src[NI];
    int coff[NI];
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int r = 8 * (NI * wave + i) + (lane >> 3);
        coff[i] = 8 * ((lane & 7) ^ (r & 7));
        if (r < TE)
            src[i] = a.w + (int64_t)(e0 + r < E ? e0 + r : E - 1) * K;
        else
            src[i] = a.x + (m0 + r - TE < M ? m0 + r - TE : M - 1) * K;
    }
    auto issue = [&](int64_t st, uint8_t *buf) {
        const int64_t k0 = 64 * (st < slast ? st : slast);
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const int64_t k = k0 + coff[i] < K ? k0 + coff[i] : K - 8;
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)(src[i] + k),
                                             (__attribute__((address_space(3))) void *)(buf + (NI * wave + i) * 1024),
                                             16, 0, 0);
        }
    };
    f32x4 acc[4][FM], tot[4][FM];
    float xs[FM], ws[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        ws[i] = 0.f;
#pragma unroll
        for (int f = 0; f < FM; f++)
            acc[i][f] = tot[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int f = 0; f < FM; f++)
        xs[f] = 0.f;
    auto flush = [&]() {
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int f = 0; f < FM; f++) {
                tot[i][f] += acc[i][f];
                acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
    };
    const bool sqw = wm == 0 && m0 == 0, sqx = wn == 0 && e0 == 0;   // who forms the squares
#pragma unroll
    for (int j = 0; j < RING - 1; j++)
        issue(sb + j, ring[j]);
    for (int64_t s0 = sb; s0 < se; s0 += RING) {
#pragma unroll
        for (int j = 0; j < RING; j++) {
            const int64_t st = s0 + j;
            wait_vmcnt<WAIT>();                           // this wave's part of stage st
            read_barrier();                               // every wave's part; stage st - 1 free
            issue(st + RING - 1, ring[(j + RING - 1) % RING]);
            if (st < se) {
                const uint8_t *buf = ring[j];
#pragma unroll
                for (int dd = 0; dd < 2; dd++) {
                    if (dd == 1 && 64 * st + 32 >= K)
                        break;
                    const int off = ((4 * dd + lg) ^ (lr & 7)) << 4;
                    u32x4 wf[4], xf[FM];
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        wf[i] = *reinterpret_cast<const u32x4 *>(buf + (64 * wn + 16 * i + lr) * 128 + off);
#pragma unroll
                    for (int f = 0; f < FM; f++)
                        xf[f] = *reinterpret_cast<const u32x4 *>(buf + (TE + 16 * (FM * wm + f) + lr) * 128 + off);
#pragma unroll
                    for (int i = 0; i < 4; i++)
#pragma unroll
                        for (int f = 0; f < FM; f++)
                            acc[i][f] = mfma16(wf[i], xf[f], acc[i][f]);
                    if (sqw) {
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            ws[i] = sq8(wf[i], ws[i]);
                    }
                    if (sqx) {
#pragma unroll
                        for (int f = 0; f < FM; f++)
                            xs[f] = sq8(xf[f], xs[f]);
                    }
                }
                if ((st - sb) % RL_CHAIN == RL_CHAIN - 1)
                    flush();
            }
        }
    }
    wait_vmcnt<0>();                                      // the clamped tail DMAs
    flush();
    // lane (lr, lg): experts + 16 i + 4 lg + q of token + 16 f + lr
#pragma unroll
    for (int f = 0; f < FM; f++) {
        const int64_t m = m0 + 16 * (FM * wm + f) + lr;
        if (m >= M)
            continue;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int e = e0 + 64 * wn + 16 * i + 4 * lg;
            float *z = a.z + ((int64_t)ks * M + m) * E + e;
            if (e + 3 < E && E % 4 == 0)
                *reinterpret_cast<f32x4 *>(z) = tot[i][f];
            else
                for (int q = 0; q < 4; q++)
                    if (e + q < E)
                        z[q] = tot[i][f][q];
        }
    }
    if (sqx) {
#pragma unroll
        for (int f = 0; f < FM; f++) {
            float v = xs[f];
            v += __shfl_xor(v, 16);
            v += __shfl_xor(v, 32);
            const int64_t m = m0 + 16 * (FM * wm + f) + lr;
            if (lg == 0 && m < M)
                a.xn[(int64_t)ks * M + m] = v;
        }
    }
    if (sqw) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float v = ws[i];
            v += __shfl_xor(v, 16);
            v += __shfl_xor(v, 32);
            // rows past E repeat the last one: the largest of the 16
            for (int o = 1; o < 16; o <<= 1) {
                const float u = __shfl_xor(v, o);
                v = u > v || u != u ? u : v;              // (NaN stays)
            }
            if (lane == 0)
                a.wn[ks * RL_FRAGS + (e0 + 64 * wn + 16 * i) / 16] = v;
        }
    }
}

// Reductions over 16 lanes (a DPP row), the result in all of them: swaps within
// quads, then of the quads and halves by mirrors, each step the same two
// operands on both sides.
template <typename T, typename F>
__device__ __forceinline__ T row_reduce(T v, F op)
{
    v = op(v, dpp<0xB1, 0xF>(v, v));                      // quad_perm 1 0 3 2
    v = op(v, dpp<0x4E, 0xF>(v, v));                      // quad_perm 2 3 0 1
    v = op(v, dpp<0x141, 0xF>(v, v));                     // row_half_mirror
    v = op(v, dpp<0x140, 0xF>(v, v));                     // row_mirror
    return v;
}
__device__ __forceinline__ uint32_t row_max(uint32_t v)
{
    return row_reduce(v, [](uint32_t p, uint32_t q) { return q > p ? q : p; });
}
__device__ __forceinline__ float row_max(float v)
{
    return row_reduce(v, [](float p, float q) { return q > p ? q : p; });
}
__device__ __forceinline__ float row_sum(float v)
{
    return row_reduce(v, [](float p, float q) { return p + q; });
}
__device__ __forceinline__ double row_sum(double v)
{
    return row_reduce(v, [](double p, double q) { return p + q; });
}

// A wave's LDS in the choice (an array for each type: nothing is reused as
// another).
template <int Q>
struct ChooseShared {
    uint32_t key[4][64 * Q];                              // by token and expert
    float logit[4][64 * Q];
    uint32_t gval[4][SPEAR_MAX_GROUPS], gthr[4][SPEAR_MAX_GROUPS];
    uint64_t kept[4];
    double z[64 * Q], c[64 * Q], slot_z[SPEAR_MAX_TOPK];
    int32_t slot_id[SPEAR_MAX_TOPK];
    uint16_t list[64 * Q];
};

// Waves of a workgroup of the choice, four tokens each.  Tokens in doubt are the
// whole workgroup's: it sums their logits together, then each wave settles the
// next one (settled by its own wave alone, a token took 10 to 20 thousand
// cycles and the last wave of 8192 tokens had four of them).  Two waves for more
// than 256 experts, so that LDS holds the same tokens a CU.
template <int Q>
constexpr int RC_WAVES = Q == 8 ? 2 : 4;
constexpr int RC_JOINT = 16;                              // logits a token that are summed together

// A token that has to be settled.
struct Doubt {
    int64_t m;
    float mx, sum, zd;
    uint32_t clear;                                       // choices further apart are in order
    uint32_t slots, last;                                 // winners whose order is open; the last one's key
    int32_t n, hard, rest;                                // experts in the list (up to RC_JOINT of them)
    int32_t id[SPEAR_MAX_TOPK];                           // winners
    alignas(8) uint16_t list[RC_JOINT];
};

template <int Q>
struct Joint {
    static constexpr int NW = RC_WAVES<Q>;
    Doubt t[4 * NW];
    double part[4 * NW][RC_JOINT][NW];                    // logits by K range
    uint32_t open[2][NW];                                 // a wave's tokens in doubt, a bit each: groups, order
};

// Logits of the listed experts of all tokens in `todo` over this wave's share of
// K, in units of four experts and 1024 depths, two with their loads in flight.
// Lists and rows are read as scalars: every load then is a base and a lane's
// offset (addresses by lane made a unit 3200 cycles; 2500 so).
template <int Q>
__device__ __forceinline__ void joint_logits(const RouteArgs &a, Joint<Q> &jt, uint32_t todo, int wave, int lane)
{
    constexpr int NW = RC_WAVES<Q>, UNITS = 2;
    const int64_t kb = a.K / 8 * wave / NW * 8, ke = a.K / 8 * (wave + 1) / NW * 8;
    int u = 0, n = 0, p = 0;
    int64_t k = ke;
    const uint16_t *xr = a.x, *wr[4] = {a.w, a.w, a.w, a.w};
    bool more = true;
    auto next = [&]() __attribute__((always_inline)) {    // (an empty share of K has one unit, of zeros)
        k += 1024;
        if (k < ke)
            return;
        k = kb;
        p += 4;
        while (more && p >= n) {
            p = n = 0;
            more = todo != 0;
            if (more) {
                u = __builtin_ctz(todo);
                todo &= todo - 1;
                const Doubt &t = jt.t[u];
                n = __builtin_amdgcn_readfirstlane(t.n);
                n = n > RC_JOINT ? 0 : n;
                const uint64_t m = (uint64_t)t.m;
                xr = a.x + (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(m >> 32)) << 32) |
                                     (uint32_t)__builtin_amdgcn_readfirstlane((int)m)) * a.K;
            }
        }
        if (more) {
            const uint32_t *list = reinterpret_cast<const uint32_t *>(&jt.t[u].list[p]);
            const uint32_t l0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)list[0]),
                           l1 = (uint32_t)__builtin_amdgcn_readfirstlane((int)list[1]);
            wr[0] = a.w + (int64_t)(l0 & 0xFFFF) * a.K;
            wr[1] = p + 1 < n ? a.w + (int64_t)(l0 >> 16) * a.K : wr[0];
            wr[2] = p + 2 < n ? a.w + (int64_t)(l1 & 0xFFFF) * a.K : wr[0];
            wr[3] = p + 3 < n ? a.w + (int64_t)(l1 >> 16) * a.K : wr[0];
        }
    };
    next();
#pragma unroll 1
    while (more) {
        u32x4 xv[UNITS][2], wv[UNITS][4][2];
        int uu[UNITS], pp[UNITS], nn[UNITS];
        bool begin[UNITS], inside[UNITS][2];
#pragma unroll
        for (int i = 0; i < UNITS; i++) {
            uu[i] = u;
            pp[i] = p;
            nn[i] = more ? n : 0;
            begin[i] = k == kb;
            if (more) {
                const int64_t kc = k < a.K - 8 ? k : a.K - 8;
#pragma unroll
                for (int q = 0; q < 2; q++) {
                    // (a chunk past the share reads its first one, times zero)
                    const uint32_t l = 512 * q + 8 * lane;
                    const bool in = (int64_t)l < ke - k;
                    const uint32_t off = in ? l : 0;
                    xv[i][q] = ld16(xr + kc + off);
                    inside[i][q] = in;
#pragma unroll
                    for (int r = 0; r < 4; r++)
                        wv[i][r][q] = ld16(wr[r] + kc + off);
                }
                next();
            }
        }
#pragma unroll
        for (int i = 0; i < UNITS; i++)
            if (nn[i] != 0) {
                double z[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
                for (int q = 0; q < 2; q++)
                    xv[i][q] = inside[i][q] ? xv[i][q] : zero4();
#pragma unroll
                for (int r = 0; r < 4; r++)
                    if (pp[i] + r < nn[i])
                        z[r] = dot8(xv[i][1], wv[i][r][1], dot8(xv[i][0], wv[i][r][0], 0.0));
                const double t = wave_sum4(z, lane);
                if (lane < 4 && pp[i] + lane < nn[i]) {
                    double &d = jt.part[uu[i]][pp[i] + lane][wave];
                    d = begin[i] ? t : d + t;
                }
            }
    }
}

// The list of token u and its logits to the wave's own LDS, after joint_logits.
template <int Q>
__device__ __forceinline__ void take_joint(ChooseShared<Q> &sh, const Joint<Q> &jt, int u, int n, int lane)
{
    if (lane < n) {
        double z = 0.0;
#pragma unroll
        for (int w = 0; w < RC_WAVES<Q>; w++)
            z += jt.part[u][lane][w];
        sh.z[lane] = z;
        sh.list[lane] = jt.t[u].list[lane];
    }
    wait_lgkmcnt0();
}

// Groups of the token in row `row` whose order the bounds leave open (lane g for
// group g): og those, sure the ones kept whatever their order.
template <int Q>
__device__ __forceinline__ void open_groups(const RouteArgs &a, const ChooseShared<Q> &sh, int row, uint32_t clear,
                                            int lane, uint64_t &og, uint64_t &sure)
{
    const int G = a.n_group;
    const uint32_t tol = (a.group_best == 2 && a.E / G > 1 ? 2u : 1u) * clear;
    const uint32_t gv = lane < G ? sh.gval[row][lane] : 0u;
    uint32_t rank = 0;
#pragma unroll 1
    for (int g = 0; g < G; g++) {
        const uint32_t o = sh.gval[row][g];
        rank += o > gv || (o == gv && g < lane) ? 1u : 0u;
    }
    const bool in = lane < G && rank < (uint32_t)a.topk_group;
    const uint32_t least = ~wave_max(in ? ~gv : 0u), most = wave_max(lane < G && !in ? gv : 0u);
    const bool open = lane < G && (in ? gv <= most + tol : gv + tol >= least);
    og = __ballot(open);
    sure = __ballot(in && !open);
}

// The experts that may be among the best of those groups in fp64, to sh.list of
// the wave `to`; returns their number.
template <int Q>
__device__ __forceinline__ int list_groups(const RouteArgs &a, const ChooseShared<Q> &sh, ChooseShared<Q> &to, int row,
                                           uint32_t clear, int lane)
{
    const int E = a.E, gs = E / a.n_group;
    uint64_t og, sure;
    open_groups(a, sh, row, clear, lane, og, sure);
    int n = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < E; e0 += 64) {
        const int e = e0 + lane, g = e < E ? e / gs : 0;
        const uint32_t k = e < E ? sh.key[row][e] : 0u;
        n = append(to.list, n, e < E && ((og >> g) & 1) && k != 0u && (k >> 9) + clear >= sh.gthr[row][g], e, lane);
    }
    wait_lgkmcnt0();
    return n;
}

// The groups to keep, by the n listed logits in my.z; own: the LDS of the token's
// own wave.
template <int Q>
__device__ __forceinline__ void settle_groups(const RouteArgs &a, ChooseShared<Q> &my, ChooseShared<Q> &own, int row,
                                              const Doubt &t, int n, int lane)
{
    const int G = a.n_group, gs = a.E / G;
    const bool two = a.group_best == 2 && gs > 1;
    uint64_t og, sure;
    open_groups(a, own, row, t.clear, lane, og, sure);
#pragma unroll 1
    for (int p = lane; p < n; p += 64)
        my.c[p] = choice_of(a, score_of(a, my.z[p], t.mx, t.sum), my.list[p]);
    wait_lgkmcnt0();
    double b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll 1
    for (int p = 0; p < n; p++)
        if (my.list[p] / gs == lane) {
            const double v = my.c[p];
            b1 = v > b0 ? b0 : (v > b1 ? v : b1);
            b0 = v > b0 ? v : b0;
        }
    const double v = two ? b0 + b1 : b0;
    int place = 0;
#pragma unroll 1
    for (int g = 0; g < G; g++) {
        const double o = lane_of(v, g);
        place += ((og >> g) & 1) && (o > v || (o == v && g < lane));
    }
    const uint64_t kept = sure | __ballot(((og >> lane) & 1) && place < a.topk_group - __popcll(sure));
    if (lane == 0)
        own.kept[row] = kept;
}

// The winners whose order is open, and (rest) the candidates behind the last one
// that may come before it, to to.list; returns their number.
template <int Q>
__device__ __forceinline__ int list_order(const RouteArgs &a, const ChooseShared<Q> &own, ChooseShared<Q> &to, int row,
                                          int id, uint32_t slots, bool rest, uint32_t last, uint32_t clear, int lane)
{
    int n = append(to.list, 0, lane < SPEAR_MAX_TOPK && ((slots >> (lane & 31)) & 1), id, lane);
    if (rest)
#pragma unroll 1
        for (int e0 = 0; e0 < a.E; e0 += 64) {
            const uint32_t k = e0 + lane < a.E ? own.key[row][e0 + lane] : 0u;
            n = append(to.list, n, k != 0u && last - (k >> 9) <= clear, e0 + lane, lane);
        }
    wait_lgkmcnt0();
    return n;
}

// The n listed experts take the token's open slots in the order of their logits
// in my.z (to my.slot_id, my.slot_z); the other winners are clear of them all.
// False: all logits are needed.
template <int Q>
__device__ __forceinline__ bool settle_order(const RouteArgs &a, ChooseShared<Q> &my, const Doubt &t, int n, int lane)
{
    const int open = __popc(t.slots);
    bool decided = true;
    const bool shift = a.score == SPEAR_SCORE_SOFTMAX && a.bias;   // s + bias: the sum's own error matters
#pragma unroll 1
    for (int p = lane; p < n; p += 64)
        my.c[p] = choice_of(a, score_of(a, my.z[p], t.mx, t.sum), my.list[p]);
    wait_lgkmcnt0();
#pragma unroll 1
    for (int p = lane; p < n; p += 64) {
        const double c = my.c[p], z = my.z[p], s = shift ? score_of(a, z, t.mx, t.sum) : 0.0;
        const int e = my.list[p];
        int place = 0;
#pragma unroll 1
        for (int q = 0; q < n; q++) {
            const double o = my.c[q];
            const int oe = my.list[q];
            place += o > c || (o == c && oe < e);
            if (shift && q != p && !(fabs(o - c) > 1.25 * (double)t.zd * fabs(score_of(a, my.z[q], t.mx, t.sum) - s)))
                decided = false;
        }
        if (place < open) {
            uint32_t m = t.slots;                         // the place-th open slot
#pragma unroll 1
            for (int i = 0; i < place; i++)
                m &= m - 1;
            const int slot = __builtin_ctz(m);
            my.slot_id[slot] = e;
            my.slot_z[slot] = z;
        }
    }
    wait_lgkmcnt0();
    return __all(decided);
}

// All logits of token t in fp64 to my.z.  A row of x that is all zero has zeros
// (zd == 0: then w has no infinity or NaN either), without reading w.
template <int Q>
__device__ __forceinline__ void all_logits(const RouteArgs &a, ChooseShared<Q> &my, const Doubt &t, int lane)
{
    bool zero = t.zd == 0.f;
    if (zero) {
        uint32_t any = 0;
        const uint16_t *xr = a.x + t.m * a.K;
#pragma unroll 1
        for (int64_t k = 8 * lane; k < a.K; k += 512) {
            const u32x4 v = ld16(xr + k);
            any |= (v[0] | v[1] | v[2] | v[3]) & 0x7FFF7FFFu;
        }
        zero = !__any(any != 0);
    }
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64) {
        my.list[e] = (uint16_t)e;
        my.z[e] = 0.0;
    }
    wait_lgkmcnt0();
    if (!zero)
        exact_logits(a, t.m, lane, my.list, a.E, my.z);
}

// The choice, four tokens a wave: 16 lanes a token, 4 Q experts a lane
// (64 i + 4 l + q).  A choice becomes a key of 23 bits of fixed point and 9 bits
// of 511 - expert, so that a round is a maximum of unsigned words and its winner
// is in the word (one wave a token, its candidates searched for each winner,
// took 70 us of vector instructions for 8192 tokens x 256 experts).  Where
// neighbours in the order are nearer than the bounds and the fixed point allow,
// the workgroup settles the token with a few logits in fp64.  Bound by dependent
// steps: 8192 tokens x 256 experts 36 us, of which the partial logits 7, keys,
// groups and rounds 7, the slowest workgroup's tokens in doubt the rest.  A choice's
// error is taken at the steepest slope of its score, so the tokens in doubt grow
// with the logits where the scores do not, and where a bias ranks small scores.
// Whole calls, 8192 tokens x 256 experts x 4096, us by the logits' deviation
// 0.5 / 1 / 2 / 4 / 8 / 16: biased sigmoid, 4 of 8 groups 63 / 65 / 71 / 84 / 109 /
// 136; softmax 53 throughout (its order is the logits'); softmax with a bias 391 /
// 635 / 763 / 926 / 791 / 977.
template <int Q>
__global__ __launch_bounds__(64 * RC_WAVES<Q>, 2) void route_choose_kernel(const RouteArgs a)
{
    constexpr int NW = RC_WAVES<Q>;
    __shared__ __attribute__((aligned(16))) ChooseShared<Q> s_sh[NW];
    __shared__ Joint<Q> jt;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    ChooseShared<Q> &sh = s_sh[wave];
    const int lr = lane & 15, row = lane >> 4;
    const int64_t M = a.M, first = (int64_t)blockIdx.x * (4 * NW), m0 = first + 4 * wave;
    const int64_t m = m0 + row < M ? m0 + row : M - 1;
    const int E = a.E, G = a.n_group, gs = E / G;
    // logits: the slices' sums; |x|^2, and the largest |w_e|^2 of 16 experts a lane
    const int frag = lane & (RL_FRAGS - 1), frags = 4 * tile_waves(E) * a.net;
    float wn2 = 0.f;
    float c[4 * Q], xn = 0.f;
#pragma unroll
    for (int i = 0; i < 4 * Q; i++)
        c[i] = 0.f;
    float bias[4 * Q];
#pragma unroll
    for (int i = 0; i < 4 * Q; i++) {
        const int e = 64 * (i / 4) + 4 * lr + i % 4;
        bias[i] = a.bias && e < E ? a.bias[e] : 0.f;
    }
    constexpr int U = Q <= 4 ? 4 : 2;        // slices in flight, by the registers they take
#pragma unroll U
    for (int k = 0; k < a.ks; k++) {
        const float *zp = a.z + (k * M + m) * E;
        xn += a.xn[k * M + m];
        wn2 += a.wn[k * RL_FRAGS + (frag < frags ? frag : 0)];
#pragma unroll
        for (int i = 0; i < Q; i++) {
            const int e = 64 * i + 4 * lr;
            if (E % 4 == 0) {
                const f32x4 v = *reinterpret_cast<const f32x4 *>(zp + (e < E ? e : E - 4));
#pragma unroll
                for (int q = 0; q < 4; q++)
                    c[4 * i + q] += v[q];
            } else {
#pragma unroll
                for (int q = 0; q < 4; q++)
                    c[4 * i + q] += zp[e + q < E ? e + q : E - 1];
            }
        }
    }
    wn2 = __any(wn2 != wn2) ? __builtin_nanf("") : wave_max(wn2);
    const float zd = 1.02f * a.zerr * sqrtf(xn) * sqrtf(wn2);   // 2 %: the norms' own roundings
#pragma unroll
    for (int i = 0; i < Q; i++)                           // kept for the winners' weights
        *reinterpret_cast<f32x4 *>(&sh.logit[row][64 * i + 4 * lr]) =
            f32x4{c[4 * i], c[4 * i + 1], c[4 * i + 2], c[4 * i + 3]};
    auto expert = [&](int i) { return 64 * (i / 4) + 4 * lr + i % 4; };
    auto real = [&](int i) { return expert(i) < E; };
    const bool soft = a.score == SPEAR_SCORE_SOFTMAX;
    const bool by_z = soft && !a.bias && (a.topk_group == G || a.group_best == 1 || gs == 1);
    bool hard = !(zd < 0.05f);                            // all logits in fp64
#pragma unroll
    for (int i = 0; i < 4 * Q; i++)
        hard |= real(i) && !(fabsf(c[i]) < INFINITY);

    // softmax: largest logit and sum
    float mx = 0.f, sum = 1.f;
    if (soft) {
        float t = -INFINITY, u = 0.f;
#pragma unroll
        for (int i = 0; i < 4 * Q; i++)
            t = real(i) && c[i] > t ? c[i] : t;
        mx = row_max(t);
#pragma unroll
        for (int i = 0; i < 4 * Q; i++)
            u += real(i) ? __expf(c[i] - mx) : 0.f;
        sum = row_sum(u);
    }
    // Choices to [0, 1): by the logits themselves where only their order counts
    // (softmax, no bias, no sums of groups), else by score and bias.  d bounds
    // the error: of the logit, or its slope times that and 1e-5 for the fp32
    // exponential (2 steps and as many as the argument's magnitude, which is
    // below 90 where the score is not 0 or 1).
    float lo, unit, d;                                    // choice = lo + unit * key
    if (by_z) {
        lo = -64.f;                                       // further down all keys are alike: in doubt
        unit = 64.f;
        d = zd + 2e-5f;
#pragma unroll
        for (int i = 0; i < 4 * Q; i++)
            c[i] -= mx;
    } else {
        float mb = 0.f;
        const float inv = 1.f / sum;
#pragma unroll
        for (int i = 0; i < 4 * Q; i++) {
            const float s = soft ? __expf(c[i] - mx) * inv : __builtin_amdgcn_rcpf(1.f + __expf(-c[i]));
            const float b = bias[i];
            mb = fabsf(b) < INFINITY && fabsf(b) > mb ? fabsf(b) : mb;
            hard |= b == INFINITY;
            c[i] = s + b;
        }
        mb = a.bias ? row_max(mb) : 0.f;
        lo = -mb;
        unit = 1.f + 2.f * mb;
        d = (soft ? 2.5f : 0.25f) * zd + 1e-5f + 5e-7f * unit;
    }
    // keys: 1 + 23 bits of the place in the range; 0 for what cannot be chosen
    constexpr float TOP = 8388000.f;
    const float up = TOP / unit;
    uint32_t key[4 * Q];
#pragma unroll
    for (int i = 0; i < 4 * Q; i++) {
        const float t = fminf(fmaxf((c[i] - lo) * up, 0.f), TOP);
        const bool can = real(i) && c[i] > -INFINITY;     // (false for NaN)
        key[i] = can ? (((uint32_t)t + 1u) << 9) | (uint32_t)(SPEAR_MAX_EXPERTS - 1 - expert(i)) : 0u;
    }
    // two choices further apart than this (in key steps) are in order
    const float gap = 2.f * d * up + 3.f;
    const uint32_t clear = gap < 8e6f ? (uint32_t)gap : 0x7FFFFFu;

    if (a.topk_group < G) {
        // 16 lanes a token: groups lr, lr + 16, ...
#pragma unroll
        for (int i = 0; i < Q; i++)
            *reinterpret_cast<u32x4 *>(&sh.key[row][64 * i + 4 * lr]) =
                u32x4{key[4 * i], key[4 * i + 1], key[4 * i + 2], key[4 * i + 3]};
        wait_lgkmcnt0();
        const bool two = a.group_best == 2 && gs > 1;
#pragma unroll 1
        for (int g = lr; g < G; g += 16) {
            // (each lane from another place: all lanes in step through one
            // bank took 7700 cycles for 8 groups of 32, 3600 so)
            uint32_t b0 = 0, b1 = 0;
            int j = lane % gs;
#pragma unroll 8
            for (int i = 0; i < gs; i++) {
                const uint32_t v = sh.key[row][g * gs + j] >> 9, w = v < b0 ? v : b0;
                j = j + 1 == gs ? 0 : j + 1;
                b0 = v > b0 ? v : b0;
                b1 = w > b1 ? w : b1;
            }
            sh.gval[row][g] = !two ? b0 : b1 ? b0 + b1 : 0u;   // (0: not enough candidates)
            sh.gthr[row][g] = two ? b1 : b0;
        }
        wait_lgkmcnt0();
        uint32_t least = 0xFFFFFFFFu, most = 0;
        uint64_t kept = 0;
#pragma unroll 1
        for (int g0 = 0; g0 < G; g0 += 16) {
            const int g = g0 + lr;
            const uint32_t gv = g < G ? sh.gval[row][g] : 0u;
            uint32_t rank = 0;
#pragma unroll 4
            for (int q = 0; q < G; q++) {
                const uint32_t o = sh.gval[row][q];
                rank += o > gv || (o == gv && q < g) ? 1u : 0u;
            }
            const bool in = g < G && rank < (uint32_t)a.topk_group;
            least = in && gv < least ? gv : least;
            most = g < G && !in && gv > most ? gv : most;
            kept |= ((__ballot(in) >> (16 * row)) & 0xFFFFull) << g0;
        }
        least = ~row_max(~least);
        most = row_max(most);
        const bool open = !(least > most && least - most > (two ? 2u : 1u) * clear);
        if (lr == 0)
            sh.kept[row] = kept;
        const bool all = soft && a.bias;                  // its sum's error: all logits are needed
        const uint64_t todo = __ballot(open && !hard && !all && m0 + row < M);
        hard |= open && all;
        wait_lgkmcnt0();
        uint32_t fail = 0;
        if (todo != 0) {
#pragma unroll 1
            for (int r = 0; r < 4; r++) {
                if (((todo >> (16 * r)) & 1) == 0)
                    continue;
                Doubt &t = jt.t[4 * wave + r];
                const uint32_t cl = lane_of(clear, 16 * r);
                const int n = list_groups(a, sh, sh, r, cl, lane);
                if (n > RC_JOINT) {
                    fail |= 1u << r;
                } else if (lane < n) {
                    t.list[lane] = sh.list[lane];
                }
                if (lane == 16 * r) {
                    t.m = m;
                    t.mx = mx;
                    t.sum = sum;
                    t.zd = zd;
                    t.clear = cl;
                    t.n = n;
                }
            }
        }
        hard |= (fail >> row) & 1;
        if (lane == 0)
            jt.open[0][wave] = ((todo & 1) | ((todo >> 15) & 2) | ((todo >> 30) & 4) | ((todo >> 45) & 8)) & ~fail;
        __syncthreads();
        uint32_t open_all = 0;
#pragma unroll
        for (int w = 0; w < NW; w++)
            open_all |= __builtin_amdgcn_readfirstlane(jt.open[0][w]) << (4 * w);
        if (open_all != 0) {                              // (the same for all waves)
            joint_logits(a, jt, open_all, wave, lane);
            __syncthreads();
            int turn = 0;
#pragma unroll 1
            for (uint32_t o = open_all; o; o &= o - 1) {
                if (turn++ % NW != wave)
                    continue;
                const int u = __builtin_ctz(o);
                const int n = __builtin_amdgcn_readfirstlane(jt.t[u].n);
                take_joint(sh, jt, u, n, lane);
                settle_groups(a, sh, s_sh[u / 4], u % 4, jt.t[u], n, lane);
            }
            __syncthreads();
        }
        kept = sh.kept[row];
        const uint32_t magic = ((1u << 20) + gs - 1) / gs;    // e / gs for e < 512, gs <= 512
#pragma unroll
        for (int i = 0; i < 4 * Q; i++)
            key[i] = (kept >> ((expert(i) * magic) >> 20)) & 1u ? key[i] : 0u;
    }

    // rounds: winner t to lane t % 16, slot t / 16
    int id[2] = {-1, -1};
    uint32_t val[2] = {0u, 0u}, prev = 0xFFFFFFFFu, behind = 0;
    bool so[2] = {false, false};                          // slots whose order is open
#pragma unroll 1
    for (int t = 0; t <= a.topk; t++) {                   // one more: the best of the rest
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < 4 * Q; i++)
            best = key[i] > best ? key[i] : best;
        best = row_max(best);
        const uint32_t v = best >> 9;
        if (t == a.topk) {
            behind = v;
            break;
        }
        const bool won = best != 0u, open = won && t > 0 && prev - v <= clear;
        const int e = SPEAR_MAX_EXPERTS - 1 - (int)(best & 511u);
        if ((t & 15) == lr) {
            id[0] = won && t < 16 ? e : id[0];
            id[1] = won && t >= 16 ? e : id[1];
            val[0] = won && t < 16 ? v : val[0];
            val[1] = won && t >= 16 ? v : val[1];
            so[0] |= open && t < 16;
            so[1] |= open && t >= 16;
        }
        if (((t - 1) & 15) == lr) {
            so[0] |= open && t <= 16;
            so[1] |= open && t > 16;
        }
        prev = won ? v : prev;
#pragma unroll
        for (int i = 0; i < 4 * Q; i++)
            key[i] = key[i] == best ? 0u : key[i];
    }
    // candidates behind the last winner that may come before it, and the
    // winners that they may come before
    const bool rest = behind != 0u && prev - behind <= clear;
#pragma unroll
    for (int h = 0; h < 2; h++)
        so[h] |= rest && id[h] >= 0 && val[h] - behind <= clear;
    const uint64_t so0 = __ballot(so[0]), so1 = __ballot(so[1]), hd = __ballot(hard), rs = __ballot(rest);
    auto of_row = [](uint64_t b, int r) { return (b >> (16 * r)) & 0xFFFFull; };
    const uint64_t doubt = so0 | so1 | hd;

    // the weights, in fp64 from the winners' logits
    const bool quick = of_row(doubt, row) == 0 && m0 + row < M;
    double s[2] = {0.0, 0.0};
#pragma unroll
    for (int h = 0; h < 2; h++)
        if (quick && id[h] >= 0)
            s[h] = score_of(a, (double)sh.logit[row][id[h]], (double)mx, (double)sum);
    double f = (double)a.scale;
    if (a.renorm) {
        const double total = row_sum(s[0] + s[1]);
        f = total == 0.0 ? 0.0 : f / total;
    }
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int t = 16 * h + lr;
        if (quick && t < a.topk) {
            a.ids[m * a.topk + t] = id[h];
            a.weights[m * a.topk + t] = id[h] < 0 ? 0.f : (float)(s[h] * f);
        }
    }
    // tokens in doubt: their lists
    if (rs != 0) {
#pragma unroll
        for (int i = 0; i < Q; i++)
            *reinterpret_cast<u32x4 *>(&sh.key[row][64 * i + 4 * lr]) =
                u32x4{key[4 * i], key[4 * i + 1], key[4 * i + 2], key[4 * i + 3]};
    }
    const bool mine = of_row(doubt, row) != 0 && m0 + row < M;
    if (mine) {
        Doubt &t = jt.t[4 * wave + row];
        t.id[lr] = id[0];
        t.id[16 + lr] = id[1];
        if (lr == 0) {
            t.m = m;
            t.mx = mx;
            t.sum = sum;
            t.zd = zd;
            t.clear = clear;
            t.slots = (uint32_t)(of_row(so0, row) | (of_row(so1, row) << 16));
            t.last = prev;
            t.n = 0;
            t.hard = of_row(hd, row) != 0;
            t.rest = rest;
        }
    }
    const uint64_t todo = __ballot(mine);
    wait_lgkmcnt0();
    if (todo != 0) {
#pragma unroll 1
        for (int r = 0; r < 4; r++) {
            Doubt &t = jt.t[4 * wave + r];
            if (((todo >> (16 * r)) & 1) == 0 || t.hard)
                continue;
            const int n = list_order(a, sh, sh, r, lane < SPEAR_MAX_TOPK ? t.id[lane] : -1, t.slots,
                                     t.rest != 0, t.last, t.clear, lane);
            if (lane < n && n <= RC_JOINT)
                t.list[lane] = sh.list[lane];
            if (lane == 0) {
                t.n = n;
                t.hard = n > 64;                          // so many: rounds over all of them are quicker
            }
        }
    }
    if (lane == 0)
        jt.open[1][wave] = (todo & 1) | ((todo >> 15) & 2) | ((todo >> 30) & 4) | ((todo >> 45) & 8);
    __syncthreads();
    uint32_t open_all = 0;
#pragma unroll
    for (int w = 0; w < NW; w++)
        open_all |= __builtin_amdgcn_readfirstlane(jt.open[1][w]) << (4 * w);
    if (open_all == 0)                                    // (the same for all waves)
        return;
    joint_logits(a, jt, open_all, wave, lane);
    __syncthreads();
    int turn = 0;
#pragma unroll 1
    for (uint32_t o = open_all; o; o &= o - 1) {
        if (turn++ % NW != wave)
            continue;
        const int u = __builtin_ctz(o), r = u % 4;
        const Doubt &t = jt.t[u];
        const ChooseShared<Q> &own = s_sh[u / 4];
        bool done = false;
        if (!t.hard) {
            const int my = lane < SPEAR_MAX_TOPK ? t.id[lane] : -1;
            const int n = __builtin_amdgcn_readfirstlane(t.n);
            if (n <= RC_JOINT) {
                take_joint(sh, jt, u, n, lane);
            } else {
                list_order(a, own, sh, r, my, t.slots, t.rest != 0, t.last, t.clear, lane);
                exact_logits(a, t.m, lane, sh.list, n, sh.z);
            }
            done = settle_order(a, sh, t, n, lane);
            if (done) {
                int e = my;
                double z = 0.0;
                if (lane < a.topk && ((t.slots >> lane) & 1)) {
                    e = sh.slot_id[lane];
                    z = sh.slot_z[lane];
                } else if (lane < a.topk && e >= 0) {
                    z = (double)own.logit[r][e];
                }
                write_choice(a, t.m, lane, lane < a.topk ? e : -1, score_of(a, z, (double)t.mx, (double)t.sum));
            }
        }
        if (!done) {
            all_logits(a, sh, t, lane);
            choose_all(a, t.m, lane, sh.z, sh.c);
        }
    }
}

// The three forms, us in graphs (two launches in fp64 / one launch / MFMA logits):
//   64 experts x 2048 (256 KiB)   1 token 8.7 / 10.6 / 14.3, 64: 10.4 / 10.9 / 18.8, 128: 13.1 / 11.1 / 19.2,
//                                 256: - / 11.7 / 20.1, 384: - / 21.0 / 20.2
//   128 x 2048 (512 KiB)          1: 9.6 / 15.9 / 17.4, 64: 14.2 / 16.5 / 22.1, 128: 19.7 / 16.9 / 22.7
//   128 x 4096 (1 MiB)            1: 9.6 / 24.3 / 19.3, 64: 14.4 / 25.6 / 23.9, 128: 20.0 / 26.2 / 25.6
//   256 x 4096 (2 MiB)            1: 11.4 / 43.3 / 29.7, 64: 21.7 / 44.3 / 36.6, 128: 31.8 / 45.7 / 37.6
//   512 x 4096 (4 MiB)            1: 15.2 / 80.1 / 42.2, 64: 36.4 / 81.8 / 52.4, 128: 54.6 / 83.3 / 54.6
// So: fp64 by the whole chip for few tokens, one launch while every token has a CU
// of its own and the router's weights are small enough for a CU to read, else MFMA.
constexpr int64_t RX_TOKENS = 64, RX_MOST = 128;
constexpr int64_t RF_TOKENS = 256;
constexpr int64_t RF_BYTES = 512 << 10;

bool fused(int64_t M, int32_t E, int64_t K) { return M > RX_TOKENS && M <= RF_TOKENS && 2 * K * E <= RF_BYTES; }
bool spread(int64_t M, int32_t E, int64_t K) { return M <= RX_TOKENS || (M <= RX_MOST && 2 * K * E > RF_BYTES); }

// K slices: about 256 workgroups, at most 8 slices (their sums go through
// memory; 777 tokens, 60 experts, logits + choice: 7.4 + 15.2 us with 16 slices,
// 7.9 + 9.5 with 8, 9.7 + 8.6 with 4); K's own limit is applied by the launch.
int64_t most_slices(int64_t tiles)
{
    const int64_t ks = 256 / tiles;
    return ks < 1 ? 1 : ks > 8 ? 8 : ks;
}

hipError_t launch_route(const RouteArgs &a, hipStream_t s)
{
    if (fused(a.M, a.E, a.K)) {
        hipLaunchKernelGGL(route_fused_kernel, dim3((unsigned)a.M), dim3(64 * RF_WAVES), 0, s, a);
        return hipGetLastError();
    }
    if (spread(a.M, a.E, a.K)) {
        const int per = 2 * RX_WAVES;
        hipLaunchKernelGGL(route_exact_kernel, dim3((unsigned)((a.E + per - 1) / per), (unsigned)a.M),
                           dim3(64 * RX_WAVES), 0, s, a);
        hipLaunchKernelGGL(route_pick_kernel, dim3((unsigned)a.M), dim3(64), 0, s, a);
        return hipGetLastError();
    }
    const unsigned grid = (unsigned)((a.M + RL_TM - 1) / RL_TM * a.net * a.ks);
    switch (tile_waves(a.E)) {
    case 1: hipLaunchKernelGGL(route_logits_kernel<1>, dim3(grid), dim3(512), 0, s, a); break;
    case 2: hipLaunchKernelGGL(route_logits_kernel<2>, dim3(grid), dim3(512), 0, s, a); break;
    default: hipLaunchKernelGGL(route_logits_kernel<4>, dim3(grid), dim3(512), 0, s, a); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    auto choose = [&](auto q) {
        constexpr int NW = RC_WAVES<decltype(q)::value>;
        hipLaunchKernelGGL(route_choose_kernel<decltype(q)::value>, dim3((unsigned)((a.M + 4 * NW - 1) / (4 * NW))),
                           dim3(64 * NW), 0, s, a);
    };
    if (a.E <= 64)
        choose(std::integral_constant<int, 1>{});
    else if (a.E <= 128)
        choose(std::integral_constant<int, 2>{});
    else if (a.E <= 256)
        choose(std::integral_constant<int, 4>{});
    else
        choose(std::integral_constant<int, 8>{});
    return hipGetLastError();
}

struct RouteLayout {
    size_t z, xn, wn, total;
};

RouteLayout route_layout(int64_t M, int32_t E)
{
    auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
    RouteLayout L;
    // rows = K slices times tokens, the most that any token count up to M needs
    const int64_t net = (E + 64 * tile_waves(E) - 1) / (64 * tile_waves(E));
    size_t rows = (size_t)(M < 1 ? 1 : M);
    for (int64_t t = 1; t <= 256 && RL_TM * (t - 1) < M; t++) {
        const size_t r = (size_t)(most_slices(t * net) * (RL_TM * t < M ? RL_TM * t : M));
        rows = r > rows ? r : rows;
    }
    L.z = 0;
    L.xn = up(rows * (size_t)E * sizeof(float));
    L.wn = L.xn + up(rows * sizeof(float));
    L.total = L.wn + up(8 * RL_FRAGS * sizeof(float));
    return L;
}

bool al(const void *p, size_t n) { return (uintptr_t)p % n == 0; }

} // namespace
} // namespace spear

using namespace spear;

extern "C" {

size_t spear_route_workspace_size(int64_t M, int32_t E)
{
    if (M < 0 || E < 1 || E > SPEAR_MAX_EXPERTS || M > MAX_TOKENS)
        return 0;
    return route_layout(M, E).total;
}

spear_status spear_route(const spear_bf16 *x, int64_t M, int64_t K, const spear_router *router,
                         float *weights, int32_t *ids, void *workspace, size_t ws_bytes,
                         void *stream)
{
    if (!router || !router->w || !workspace || (M > 0 && (!x || !weights || !ids)))
        return SPEAR_E_NULL;
    const spear_router &r = *router;
    if (M < 0 || M > MAX_TOKENS || K < 32 || K % 32 != 0 || r.E < 1 || r.E > SPEAR_MAX_EXPERTS ||
        r.topk < 1 || r.topk > SPEAR_MAX_TOPK || r.n_group < 1 || r.n_group > SPEAR_MAX_GROUPS ||
        r.E % r.n_group != 0 || r.topk_group < 1 || r.topk_group > r.n_group ||
        (int64_t)r.topk > (int64_t)r.topk_group * (r.E / r.n_group))
        return SPEAR_E_SHAPE;
    if ((r.score != SPEAR_SCORE_SOFTMAX && r.score != SPEAR_SCORE_SIGMOID) ||
        (r.group_best != 1 && r.group_best != 2) || (r.renorm != 0 && r.renorm != 1) || isnan(r.scale))
        return SPEAR_E_ARG;
    if (!al(x, 16) || !al(r.w, 16) || !al(r.bias, 4) || !al(weights, 4) || !al(ids, 4) ||
        !al(workspace, 256))
        return SPEAR_E_ALIGN;
    if (ws_bytes < spear_route_workspace_size(M, r.E))
        return SPEAR_E_WORKSPACE;
    const spear_status st = check_device();
    if (st != SPEAR_OK || M == 0)
        return st;
    const RouteLayout L = route_layout(M, r.E);
    uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
    const int64_t net = (r.E + 64 * tile_waves(r.E) - 1) / (64 * tile_waves(r.E));
    const int64_t stages = (K + 63) / 64, tiles = (M + RL_TM - 1) / RL_TM * net;
    int64_t ks = most_slices(tiles);
    ks = ks > stages / 2 ? (stages / 2 > 1 ? stages / 2 : 1) : ks;    // two stages a slice at least
    const int64_t chains = ((stages + ks - 1) / ks + RL_CHAIN - 1) / RL_CHAIN + 1;
    const RouteArgs a = {x, r.w, r.bias, weights, ids, reinterpret_cast<float *>(ws + L.z),
                         reinterpret_cast<float *>(ws + L.xn), reinterpret_cast<float *>(ws + L.wn), M, K, r.E,
                         r.topk, r.score, r.n_group, r.topk_group, r.group_best, r.renorm, r.scale,
                         (float)(32 + 2 * RL_CHAIN + chains + ks) * 1.1920929e-7f, (int32_t)ks, (int32_t)net};
    const hipStream_t s = (hipStream_t)stream;
    return launch_route(a, s) == hipSuccess ? SPEAR_OK : SPEAR_E_HIP;
}

} // extern "C"
