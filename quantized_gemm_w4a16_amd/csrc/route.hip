// route.hip -- which experts a token takes (spear_route): logits, softmax or
// sigmoid scores, a bias for the choice, groups, top-k and renormalised
// weights (gfx950).
//
//   z_me = sum_k x[m][k] w[e][k], s = softmax(z) or sigmoid(z), c = s + bias;
//   the topk largest c of the kept groups, weights from s.
//
// The choice is that of logits summed in fp64.  Two forms reach it:
//  * fused (few tokens): one workgroup a token sums the logits in fp64 (each
//    bf16 x bf16 product is exact there) and its first wave chooses;
//  * two launches: the logits by bf16 MFMA in fp32, each with a bound of its
//    error, then one wave a token chooses.  Where the bounds leave the order of
//    two candidates open (a few tokens in a hundred), that wave sums the
//    logits in question again in fp64, so the choice is the same as before.
#include <math.h>

#include "spear_internal.hpp"

namespace spear {

namespace {

struct RouteArgs {
    const uint16_t *x, *w;
    const float *bias;
    float *weights;
    int32_t *ids;
    float *z;                                             // [M][E] logits (two launches)
    float *xn, *wn;                                       // [M], [E]: 2-norms of the rows of x and w
    int64_t M, K;
    int32_t E, topk, score, n_group, topk_group, group_best, renorm;
    float scale;
    float zerr;                                           // error of z over xn wn
};

// ------------------------------------------------------------- fp64 reductions
__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        v += __shfl_xor(v, o);
    return v;
}
__device__ __forceinline__ double wave_max(double v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const double u = __shfl_xor(v, o);
        v = u > v ? u : v;
    }
    return v;
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
// One wave, one token; lane l holds experts J l .. J l + J - 1, so that index
// order is (lane, j) order.  z: logits.  RB: each logit is known to within
// zd[j] only; where that leaves the choice open the logits in question are
// summed again in fp64.  A candidate that cannot be chosen is -inf.
template <int J, int RB>
struct Choice {
    const RouteArgs &a;
    const int64_t m;
    const int lane;
    double z[J], s[J], c[J], d[J];                        // logit, score, choice, bound of c's error
    double mx, sum;                                       // softmax: largest logit, sum of exp(z - mx)

    __device__ __forceinline__ Choice(const RouteArgs &a_, int64_t m_, int lane_) : a(a_), m(m_), lane(lane_) {}

    __device__ __forceinline__ int expert(int j) const { return J * lane + j; }
    __device__ __forceinline__ bool real(int j) const { return J * lane + j < a.E; }

    // score and choice of candidate j; zd: bound of its logit's error
    __device__ __forceinline__ void score(int j, double zd)
    {
        const double ninf = -INFINITY;
        if (a.score == SPEAR_SCORE_SOFTMAX) {
            s[j] = real(j) ? exp(z[j] - mx) / sum : 0.0;
            d[j] = 2.5 * zd * s[j];                       // both exp(z) and the sum are off by e^zd at most
        } else {
            s[j] = 1.0 / (1.0 + exp(-z[j]));
            d[j] = 0.25 * zd;
        }
        const double v = a.bias && real(j) ? s[j] + (double)a.bias[expert(j)] : s[j];
        c[j] = real(j) && v == v ? v : ninf;
        if (RB && zd != 0.0)                              // and fp64's own roundings
            d[j] += 1e-15 + (fabs(v) < 1e300 ? 1e-15 * fabs(v) : 0.0);
    }

    __device__ __forceinline__ void softmax_sums()
    {
        double t = -INFINITY;
        bool nan = false;
#pragma unroll
        for (int j = 0; j < J; j++)
            if (real(j)) {
                t = z[j] > t ? z[j] : t;
                nan |= z[j] != z[j];
            }
        mx = __any(nan) ? __builtin_nan("") : wave_max(t);
        double u = 0.0;
#pragma unroll
        for (int j = 0; j < J; j++)
            u += real(j) ? exp(z[j] - mx) : 0.0;
        sum = wave_sum(u);
    }

    // The logits of the candidates in `pick` (bit j of each lane) in fp64, two
    // experts at a time: their loads overlap.
    __device__ void resum(uint32_t pick)
    {
#pragma unroll
        for (int j = 0; j < J; j++) {
            uint64_t todo = __ballot((pick >> j) & 1);
            while (todo) {                                // uniform
                const int l0 = __builtin_ctzll(todo);
                todo &= todo - 1;
                const int l1 = todo ? __builtin_ctzll(todo) : l0;
                todo &= todo - 1;
                const uint16_t *w0 = a.w + (int64_t)(J * l0 + j) * a.K, *w1 = a.w + (int64_t)(J * l1 + j) * a.K;
                double s0 = 0.0, s1 = 0.0;
                for (int64_t k = 8 * lane; k < a.K; k += 512) {
                    const u32x4 xv = ld16(a.x + m * a.K + k);
                    s0 = dot8(xv, ld16(w0 + k), s0);
                    s1 = dot8(xv, ld16(w1 + k), s1);
                }
                s0 = wave_sum(s0);
                s1 = wave_sum(s1);
                if (lane == l0)
                    z[j] = s0;
                else if (lane == l1)
                    z[j] = s1;
            }
        }
    }

    // All logits in fp64.
    __device__ void resum_all()
    {
        uint32_t pick = 0;
#pragma unroll
        for (int j = 0; j < J; j++)
            pick |= real(j) ? 1u << j : 0u;
        resum(pick);
        if (a.score == SPEAR_SCORE_SOFTMAX)
            softmax_sums();
#pragma unroll
        for (int j = 0; j < J; j++)
            score(j, 0.0);
    }

    // The candidates in `pick` in fp64.  Softmax with a bias compares s + bias,
    // which the sum over all experts shifts: there all of them are summed again.
    __device__ void settle(uint32_t pick)
    {
        if (a.score == SPEAR_SCORE_SOFTMAX && a.bias) {
            resum_all();
            return;
        }
        resum(pick);
#pragma unroll
        for (int j = 0; j < J; j++)
            if ((pick >> j) & 1)
                score(j, 0.0);
    }

    // ---- groups: drop the candidates of the groups that are not kept.  sc:
    // one choice an expert, and sd: its bound, in LDS, this wave's own.
    // Returns the kept groups as a bit mask (bit = group).
    __device__ uint64_t groups(double *sc, double *sd, uint32_t *pick)
    {
        const int G = a.n_group, gs = a.E / G;
        const double ninf = -INFINITY;
#pragma unroll
        for (int j = 0; j < J; j++)
            if (real(j)) {
                sc[expert(j)] = c[j];
                if (RB)
                    sd[expert(j)] = d[j];
            }
        wait_lgkmcnt0();
        double b0 = ninf, b1 = ninf, dm = 0.0, t0 = ninf, t1 = ninf;
        if (lane < G)
            for (int i = 0; i < gs; i++) {
                const double v = sc[lane * gs + i];
                b1 = v > b0 ? b0 : (v > b1 ? v : b1);
                b0 = v > b0 ? v : b0;
                if (RB) {
                    const double dv = sd[lane * gs + i], lo = v - dv;
                    dm = dv > dm ? dv : dm;
                    t1 = lo > t0 ? t0 : (lo > t1 ? lo : t1);
                    t0 = lo > t0 ? lo : t0;
                }
            }
        const bool two = a.group_best == 2 && gs > 1;
        double gv = lane < G ? (two ? b0 + b1 : b0) : ninf;
        gv = gv == gv ? gv : ninf;                        // +inf and -inf biases in one group
        int rank = 0;
        for (int g = 0; g < G; g++) {
            const double o = __shfl(gv, g);
            rank += o > gv || (o == gv && g < lane);
        }
        const bool in = lane < G && rank < a.topk_group;
        if (RB) {
            // open: a kept group whose least value does not clear the largest
            // value of the others, and the other way round
            const double ge = two ? 2.0 * dm : dm;
            const double least = wave_max(in ? -(gv - ge) : ninf);          // -(smallest kept)
            const double most = wave_max(lane < G && !in ? gv + ge : ninf);
            uint32_t want = 0;
            if (!(-least > most)) {
                const bool open = lane < G && (in ? !(gv - ge > most) : !(gv + ge < -least));
                const uint64_t og = __ballot(open);
                const double thr = two ? t1 : t0;         // what may be among the group's best
#pragma unroll
                for (int j = 0; j < J; j++) {
                    const int g = real(j) ? expert(j) / gs : 0;
                    const double tg = __shfl(thr, g);
                    if (real(j) && ((og >> g) & 1) && d[j] != 0.0 && c[j] > ninf && !(c[j] + d[j] < tg))
                        want |= 1u << j;
                }
            }
            *pick = want;
        }
        return __ballot(in);
    }

    // ---- top-k by rounds.  Winner t goes to lane t.  Returns the chosen
    // candidates (bit j); the bounds of the choice in *ok (RB).
    int my_id;
    double my_s, total;
    __device__ uint32_t top(bool *ok)
    {
        const double ninf = -INFINITY;
        uint32_t left = 0, chosen = 0;
#pragma unroll
        for (int j = 0; j < J; j++)
            left |= c[j] > ninf ? 1u << j : 0u;
        my_id = -1;
        my_s = total = 0.0;
        double prev = INFINITY;                           // the last winner's choice, less its bound
        bool good = true;
        low = INFINITY;
        for (int t = 0; t < a.topk; t++) {
            double bv = ninf;
            int bj = 0;
#pragma unroll
            for (int j = 0; j < J; j++)
                if (((left >> j) & 1) && c[j] > bv) {
                    bv = c[j];
                    bj = j;
                }
            const double best = wave_max(bv);
            if (best == ninf)
                break;                                    // no candidate is left
            const int wl = __builtin_ctzll(__ballot(bv == best && ((left >> bj) & 1)));
            double bs = 0.0, bd = 0.0;
#pragma unroll
            for (int j = 0; j < J; j++)
                if (bj == j) {
                    bs = s[j];
                    bd = d[j];
                }
            const int id = __shfl(J * lane + bj, wl);
            const double ws = __shfl(bs, wl);
            if (RB) {
                const double wd = __shfl(bd, wl);
                good &= prev > best + wd;
                prev = best - wd;
                low = prev < low ? prev : low;
            }
            if (lane == wl) {
                left &= ~(1u << bj);
                chosen |= 1u << bj;
            }
            total += ws;
            if (lane == t) {
                my_id = id;
                my_s = ws;
            }
        }
        if (RB) {
            double u = ninf;
#pragma unroll
            for (int j = 0; j < J; j++)
                if ((left >> j) & 1)
                    u = c[j] + d[j] > u ? c[j] + d[j] : u;
            const double rest = wave_max(u);
            *ok = good && (rest == ninf || rest < prev);
        }
        return chosen;
    }
    double low;                                           // top(): the least a winner may be

    __device__ void write() const
    {
        if (lane < a.topk) {
            double w = my_id < 0 ? 0.0 : my_s;
            if (a.renorm)
                w = total == 0.0 ? 0.0 : w / total;
            a.ids[m * a.topk + lane] = my_id;
            a.weights[m * a.topk + lane] = my_id < 0 ? 0.f : (float)(w * (double)a.scale);
        }
    }

    // zd: the largest error of a logit of candidate j
    __device__ void run(const float (&zd)[J], double *sc, double *sd)
    {
        bool all = false;                                 // bounds of no use: sum everything again
        if (RB) {
#pragma unroll
            for (int j = 0; j < J; j++)
                all |= real(j) && !(zd[j] < 0.05f && z[j] == z[j]);
            all = __any(all);
        }
        if (all) {
            resum_all();
        } else {
            if (a.score == SPEAR_SCORE_SOFTMAX)
                softmax_sums();
#pragma unroll
            for (int j = 0; j < J; j++)
                score(j, RB ? (double)zd[j] : 0.0);
        }
        if (a.topk_group < a.n_group) {
            uint32_t pick = 0;
            uint64_t kept = groups(sc, sd, &pick);
            if (RB && __any(pick != 0)) {
                settle(pick);
                kept = groups(sc, sd, &pick);
            }
            const int gs = a.E / a.n_group;
#pragma unroll
            for (int j = 0; j < J; j++)
                if (real(j) && !((kept >> (expert(j) / gs)) & 1))
                    c[j] = -INFINITY;
        }
        bool ok = true;
        const uint32_t chosen = top(&ok);
        if (RB && !ok && !all) {
            // every candidate that may be among the best: the winners, and what
            // reaches the least of them
            uint32_t pick = 0;
#pragma unroll
            for (int j = 0; j < J; j++)
                if (c[j] > -INFINITY && d[j] != 0.0 && (((chosen >> j) & 1) || !(c[j] + d[j] < low)))
                    pick |= 1u << j;
            // settle() gives choices of dropped groups back their value: keep them out
            uint32_t out = 0;
#pragma unroll
            for (int j = 0; j < J; j++)
                out |= c[j] == -INFINITY ? 1u << j : 0u;
            if (__any(pick != 0)) {                       // (else exact values that are equal)
                settle(pick);
#pragma unroll
                for (int j = 0; j < J; j++)
                    if ((out >> j) & 1)
                        c[j] = -INFINITY;
                top(&ok);
            }
        }
        write();
    }
};

// ------------------------------------------------------------------ one launch
// One workgroup (16 waves) a token.  Wave w sums the logits of experts w,
// w + 16, ... in fp64, four at a time with their loads in flight together; the
// first wave then chooses.
constexpr int RF_WAVES = 16;

template <int J>
__global__ __launch_bounds__(64 * RF_WAVES) void route_fused_kernel(const RouteArgs a)
{
    __shared__ double s_z[SPEAR_MAX_EXPERTS];
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
    Choice<J, 0> ch(a, m, lane);
    const float zd[J] = {};
#pragma unroll
    for (int j = 0; j < J; j++)
        ch.z[j] = ch.real(j) ? s_z[ch.expert(j)] : 0.0;
    wait_lgkmcnt0();                                      // s_z is read before groups() writes it
    ch.run(zd, s_z, nullptr);
}

// ---------------------------------------------------------------- two launches
// Logits by MFMA: a workgroup of 16 waves takes 16 FT tokens and 64 experts,
// its waves the depth: each contracts K / 16 of it straight from global memory
// (two or four 32-deep steps of loads in flight) and the 16 partial sums are added in
// fp64.  A product passes through at most 32 roundings inside a matrix
// instruction (whatever its order) and one for each further instruction of the
// wave's chain, so the error of a logit is at most (32 + chain + 4) 2^-23
// sum |x w|, and sum |x w| at most the product of the rows' 2-norms, which are
// formed on the way.
constexpr int RL_WAVES = 16;
constexpr int RL_FE = 4;                                  // 16-expert fragments of a workgroup
constexpr int rl_batch(int FT) { return FT == 2 ? 2 : 4; }  // steps loaded at once: 128 registers a lane

__device__ __forceinline__ float sq8(u32x4 v, float acc)
{
#pragma unroll
    for (int q = 0; q < 4; q++)
        acc = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(v[q]), as_bf16x2(v[q]), acc, false);
    return acc;
}

template <int FT>
__global__ __launch_bounds__(64 * RL_WAVES) void route_logits_kernel(const RouteArgs a, int64_t units)
{
    __shared__ f32x4 s_z[RL_WAVES][FT * RL_FE][64];
    __shared__ float s_n[RL_WAVES][(FT + RL_FE) * 16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int lr = lane & 15, lg = lane >> 4;
    const int64_t M = a.M, K = a.K;
    const int E = a.E;
    // an XCD takes a contiguous run of units, the experts fastest, so that the
    // workgroups of one token tile find its rows in their L2
    const int64_t q8 = units / 8, r8 = units % 8, xcd = blockIdx.x % 8;
    const int64_t unit = xcd * q8 + (xcd < r8 ? xcd : r8) + blockIdx.x / 8;
    const int net = (E + 16 * RL_FE - 1) / (16 * RL_FE);
    const int64_t m0 = unit / net * (16 * FT);
    const int e0 = (int)(unit % net) * (16 * RL_FE);
    const int64_t T = K / 32, t0 = wave * T / RL_WAVES, t1 = (wave + 1) * T / RL_WAVES;
    const uint16_t *xr[FT], *wr[RL_FE];
#pragma unroll
    for (int f = 0; f < FT; f++) {
        const int64_t m = m0 + 16 * f + lr;
        xr[f] = a.x + (m < M ? m : M - 1) * K + 8 * lg;
    }
#pragma unroll
    for (int f = 0; f < RL_FE; f++) {
        const int e = e0 + 16 * f + lr;
        wr[f] = a.w + (int64_t)(e < E ? e : E - 1) * K + 8 * lg;
    }
    constexpr int RL_B = rl_batch(FT);
    f32x4 acc[RL_FE][FT];
    float xs[FT], ws[RL_FE];
#pragma unroll
    for (int i = 0; i < RL_FE; i++) {
        ws[i] = 0.f;
#pragma unroll
        for (int f = 0; f < FT; f++)
            acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int f = 0; f < FT; f++)
        xs[f] = 0.f;
    for (int64_t t = t0; t < t1; t += RL_B) {
        u32x4 xv[RL_B][FT], wv[RL_B][RL_FE];
#pragma unroll
        for (int b = 0; b < RL_B; b++) {
            const bool live = t + b < t1;                 // uniform
#pragma unroll
            for (int f = 0; f < FT; f++)
                xv[b][f] = live ? ld16(xr[f] + 32 * (t + b)) : zero4();
#pragma unroll
            for (int f = 0; f < RL_FE; f++)
                wv[b][f] = live ? ld16(wr[f] + 32 * (t + b)) : zero4();
        }
#pragma unroll
        for (int b = 0; b < RL_B; b++) {
#pragma unroll
            for (int i = 0; i < RL_FE; i++) {
                ws[i] = sq8(wv[b][i], ws[i]);
#pragma unroll
                for (int f = 0; f < FT; f++)
                    acc[i][f] = mfma16(wv[b][i], xv[b][f], acc[i][f]);
            }
#pragma unroll
            for (int f = 0; f < FT; f++)
                xs[f] = sq8(xv[b][f], xs[f]);
        }
    }
#pragma unroll
    for (int i = 0; i < RL_FE; i++)
#pragma unroll
        for (int f = 0; f < FT; f++)
            s_z[wave][i * FT + f][lane] = acc[i][f];
#pragma unroll
    for (int f = 0; f < FT + RL_FE; f++) {
        float v = f < FT ? xs[f] : ws[f - FT];
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
        if (lg == 0)
            s_n[wave][16 * f + lr] = v;
    }
    __syncthreads();
    // lane (token lr, lg) of fragment pair (i, f): experts e0 + 16 i + 4 lg + q
    for (int q = tid; q < FT * RL_FE * 64; q += 64 * RL_WAVES) {
        const int p = q >> 6, l = q & 63;
        double s[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
        for (int w = 0; w < RL_WAVES; w++) {
            const f32x4 v = s_z[w][p][l];
#pragma unroll
            for (int i = 0; i < 4; i++)
                s[i] += (double)v[i];
        }
        const int64_t m = m0 + 16 * (p % FT) + (l & 15);
        const int e = e0 + 16 * (p / FT) + 4 * (l >> 4);
        if (m < M) {
            float *z = a.z + m * E + e;
            if (e + 3 < E && E % 4 == 0)
                *reinterpret_cast<f32x4 *>(z) = f32x4{(float)s[0], (float)s[1], (float)s[2], (float)s[3]};
            else
                for (int i = 0; i < 4; i++)
                    if (e + i < E)
                        z[i] = (float)s[i];
        }
    }
    if (tid < (FT + RL_FE) * 16) {
        double n = 0.0;
        for (int w = 0; w < RL_WAVES; w++)
            n += (double)s_n[w][tid];
        const float norm = 1.01f * (float)sqrt(n);
        if (tid < 16 * FT) {
            if (e0 == 0 && m0 + tid < M)
                a.xn[m0 + tid] = norm;
        } else if (m0 == 0 && e0 + tid - 16 * FT < E) {
            a.wn[e0 + tid - 16 * FT] = norm;
        }
    }
}

template <int J>
__global__ __launch_bounds__(256) void route_choose_kernel(const RouteArgs a)
{
    __shared__ double s_c[4][64 * J], s_d[4][64 * J];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t m = (int64_t)blockIdx.x * 4 + wave;
    if (m >= a.M)
        return;
    Choice<J, 1> ch(a, m, lane);
    float zd[J];
    const float xe = a.zerr * a.xn[m];
#pragma unroll
    for (int j = 0; j < J; j++) {
        ch.z[j] = ch.real(j) ? (double)a.z[m * a.E + ch.expert(j)] : 0.0;
        zd[j] = ch.real(j) ? xe * a.wn[ch.expert(j)] : 0.f;
    }
    ch.run(zd, s_c[wave], s_d[wave]);
}

// One launch up to this many tokens, while the router's weights are small
// enough for one CU to read them in the time that a second launch would cost.
constexpr int64_t RF_TOKENS = 64;
constexpr int64_t RF_BYTES = 512 << 10;

bool fused(int64_t M, int32_t E, int64_t K) { return M <= RF_TOKENS && 2 * K * E <= RF_BYTES; }

template <int J>
hipError_t launch_route(const RouteArgs &a, hipStream_t s)
{
    if (fused(a.M, a.E, a.K)) {
        hipLaunchKernelGGL(route_fused_kernel<J>, dim3((unsigned)a.M), dim3(64 * RF_WAVES), 0, s, a);
        return hipGetLastError();
    }
    const int64_t net = (a.E + 16 * RL_FE - 1) / (16 * RL_FE);
    const bool two = a.M > 16;
    const int64_t units = net * ((a.M + (two ? 31 : 15)) / (two ? 32 : 16));
    if (two)
        hipLaunchKernelGGL(route_logits_kernel<2>, dim3((unsigned)units), dim3(64 * RL_WAVES), 0, s, a, units);
    else
        hipLaunchKernelGGL(route_logits_kernel<1>, dim3((unsigned)units), dim3(64 * RL_WAVES), 0, s, a, units);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(route_choose_kernel<J>, dim3((unsigned)((a.M + 3) / 4)), dim3(256), 0, s, a);
    return hipGetLastError();
}

struct RouteLayout {
    size_t z, xn, wn, total;
};

RouteLayout route_layout(int64_t M, int32_t E)
{
    auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
    RouteLayout L;
    const size_t m = (size_t)(M < 1 ? 1 : M);
    L.z = 0;
    L.xn = up(m * (size_t)E * sizeof(float));
    L.wn = L.xn + up(m * sizeof(float));
    L.total = L.wn + up((size_t)E * sizeof(float));
    return L;
}

bool al(const void *p, size_t n) { return (uintptr_t)p % n == 0; }

} // namespace
} // namespace spear

using namespace spear;

extern "C" {

size_t spear_route_workspace_size(int64_t M, int32_t E)
{
    if (M < 0 || E < 1 || E > SPEAR_MAX_EXPERTS || M > ((int64_t)1 << 40))
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
    if (M < 0 || M > 0x7FFFFFFF || K < 32 || K % 32 != 0 || r.E < 1 || r.E > SPEAR_MAX_EXPERTS ||
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
    const int64_t chain = (K / 32 + RL_WAVES - 1) / RL_WAVES;
    const RouteArgs a = {x, r.w, r.bias, weights, ids, reinterpret_cast<float *>(ws + L.z),
                         reinterpret_cast<float *>(ws + L.xn), reinterpret_cast<float *>(ws + L.wn), M, K, r.E,
                         r.topk, r.score, r.n_group, r.topk_group, r.group_best, r.renorm, r.scale,
                         (float)(32 + chain + 4) * 1.1920929e-7f};
    const hipStream_t s = (hipStream_t)stream;
    const hipError_t e = r.E <= 64 ? launch_route<1>(a, s) : r.E <= 128 ? launch_route<2>(a, s)
                         : r.E <= 256 ? launch_route<4>(a, s) : launch_route<8>(a, s);
    return e == hipSuccess ? SPEAR_OK : SPEAR_E_HIP;
}

} // extern "C"
