// route.hip -- which experts a token takes (spear_route): logits in fp64,
// softmax or sigmoid scores, a bias for the choice, groups, top-k and
// renormalised weights (gfx950).
//
//   z_me = sum_k x[m][k] w[e][k], s = softmax(z) or sigmoid(z), c = s + bias;
//   the topk largest c of the kept groups, weights from s.
//
// Each bf16 x bf16 product is exact in fp32 and the sum is carried in fp64, so
// two experts change places only where their logits agree to about 1e-15.
#include <math.h>

#include "spear_internal.hpp"

namespace spear {

namespace {

constexpr int RT_TM = 8;                                  // tokens a wave takes with one expert row
constexpr int RT_EL = SPEAR_MAX_EXPERTS / 64;             // experts a lane holds in the choice

struct RouteArgs {
    const uint16_t *x, *w;
    const float *bias;
    float *weights;
    int32_t *ids;
    double *z;                                            // [M][E] logits
    int64_t M, K;
    int32_t E, topk, score, n_group, topk_group, group_best, renorm;
    float scale;
};

// Logits: one wave takes one expert's row and up to RT_TM tokens.
__global__ __launch_bounds__(256) void route_logits_kernel(const RouteArgs a)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e = (int)blockIdx.x * 4 + wave;
    const int64_t m0 = (int64_t)blockIdx.y * RT_TM;
    if (e >= a.E)
        return;
    double acc[RT_TM];
#pragma unroll
    for (int t = 0; t < RT_TM; t++)
        acc[t] = 0.0;
    for (int64_t k = 8 * lane; k < a.K; k += 512) {
        const u32x4 wv = ld16(a.w + (int64_t)e * a.K + k);
#pragma unroll
        for (int t = 0; t < RT_TM; t++) {
            const int64_t m = m0 + t < a.M ? m0 + t : a.M - 1;
            const u32x4 xv = ld16(a.x + m * a.K + k);
#pragma unroll
            for (int q = 0; q < 4; q++) {
                acc[t] += (double)(__uint_as_float(xv[q] << 16) * __uint_as_float(wv[q] << 16));
                acc[t] += (double)(__uint_as_float(xv[q] & 0xFFFF0000u) *
                                   __uint_as_float(wv[q] & 0xFFFF0000u));
            }
        }
    }
#pragma unroll
    for (int t = 0; t < RT_TM; t++) {
#pragma unroll
        for (int o = 32; o > 0; o >>= 1)
            acc[t] += __shfl_xor(acc[t], o);
        if (lane == 0 && m0 + t < a.M)
            a.z[(m0 + t) * a.E + e] = acc[t];
    }
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

// The choice of one token by one wave.  Lane l holds experts l, l + 64, ...
// A candidate that can never be chosen is -inf (NaN choices become -inf).
__global__ __launch_bounds__(256) void route_choose_kernel(const RouteArgs a)
{
    __shared__ double s_c[4][SPEAR_MAX_EXPERTS];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t m = (int64_t)blockIdx.x * 4 + wave;
    if (m >= a.M)
        return;
    const int E = a.E, G = a.n_group, gs = E / G;
    const double ninf = -INFINITY;
    double s[RT_EL], c[RT_EL];
#pragma unroll
    for (int j = 0; j < RT_EL; j++) {
        const int e = lane + 64 * j;
        s[j] = e < E ? a.z[m * E + e] : ninf;
    }
    if (a.score == SPEAR_SCORE_SOFTMAX) {
        double mx = ninf, sum = 0.0;
        bool nan = false;
#pragma unroll
        for (int j = 0; j < RT_EL; j++) {
            mx = s[j] > mx ? s[j] : mx;
            nan |= s[j] != s[j];
        }
        mx = __any(nan) ? __builtin_nan("") : wave_max(mx);
#pragma unroll
        for (int j = 0; j < RT_EL; j++) {
            s[j] = lane + 64 * j < E ? exp(s[j] - mx) : 0.0;
            sum += s[j];
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1)
            sum += __shfl_xor(sum, o);
#pragma unroll
        for (int j = 0; j < RT_EL; j++)
            s[j] /= sum;
    } else {
#pragma unroll
        for (int j = 0; j < RT_EL; j++)
            s[j] = 1.0 / (1.0 + exp(-s[j]));
    }
#pragma unroll
    for (int j = 0; j < RT_EL; j++) {
        const int e = lane + 64 * j;
        c[j] = ninf;
        if (e < E) {
            const double v = a.bias ? s[j] + (double)a.bias[e] : s[j];
            c[j] = v == v ? v : ninf;
        }
    }
    if (a.topk_group < G) {
        // group g (lane g): the sum of its best one or two choices
#pragma unroll
        for (int j = 0; j < RT_EL; j++)
            s_c[wave][lane + 64 * j] = c[j];
        wait_lgkmcnt0();                                  // this wave's own words
        double b0 = ninf, b1 = ninf;
        if (lane < G)
            for (int i = 0; i < gs; i++) {
                const double v = s_c[wave][lane * gs + i];
                b1 = v > b0 ? b0 : (v > b1 ? v : b1);
                b0 = v > b0 ? v : b0;
            }
        double gv = lane < G ? ((a.group_best == 2 && gs > 1) ? b0 + b1 : b0) : ninf;
        gv = gv == gv ? gv : ninf;                        // +inf and -inf biases in one group
        int rank = 0;
        for (int g = 0; g < G; g++) {
            const double o = __shfl(gv, g);
            rank += o > gv || (o == gv && g < lane);
        }
        const uint64_t kept = __ballot(lane < G && rank < a.topk_group);
#pragma unroll
        for (int j = 0; j < RT_EL; j++) {
            const int e = lane + 64 * j;
            if (e < E && !((kept >> (e / gs)) & 1))
                c[j] = ninf;
        }
    }
    // top-k: the best remaining candidate, round by round
    double wsum = 0.0, mine = 0.0;
    int my_id = -1;
    for (int t = 0; t < a.topk; t++) {
        double bv = ninf, bs = 0.0;
        int be = 0x7FFFFFFF;
#pragma unroll
        for (int j = 0; j < RT_EL; j++)
            if (c[j] > bv) {
                bv = c[j];
                bs = s[j];
                be = lane + 64 * j;
            }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const double ov = __shfl_xor(bv, o), os = __shfl_xor(bs, o);
            const int oe = __shfl_xor(be, o);
            if (ov > bv || (ov == bv && oe < be)) {
                bv = ov;
                bs = os;
                be = oe;
            }
        }
        if (bv == ninf)
            break;                                        // no candidate left (uniform)
#pragma unroll
        for (int j = 0; j < RT_EL; j++)
            if (lane + 64 * j == be)
                c[j] = ninf;
        wsum += bs;
        if (lane == t) {
            my_id = be;
            mine = bs;
        }
    }
    if (lane < a.topk) {
        double w = my_id < 0 ? 0.0 : mine;
        if (a.renorm)
            w = wsum == 0.0 ? 0.0 : w / wsum;
        a.ids[m * a.topk + lane] = my_id;
        a.weights[m * a.topk + lane] = my_id < 0 ? 0.f : (float)(w * (double)a.scale);
    }
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
    return (((size_t)(M < 1 ? 1 : M) * (size_t)E * sizeof(double)) + 255) & ~(size_t)255;
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
    RouteArgs a = {x, r.w, r.bias, weights, ids, reinterpret_cast<double *>(workspace), M, K, r.E,
                   r.topk, r.score, r.n_group, r.topk_group, r.group_best, r.renorm, r.scale};
    const hipStream_t s = (hipStream_t)stream;
    // token groups travel in the grid's y, at most 65535 of them a launch
    const int64_t step = (int64_t)65535 * RT_TM;
    for (int64_t m0 = 0; m0 < M; m0 += step) {
        RouteArgs b = a;
        b.x = x + m0 * K;
        b.z = a.z + m0 * r.E;
        b.M = M - m0 < step ? M - m0 : step;
        hipLaunchKernelGGL(route_logits_kernel,
                           dim3((unsigned)((r.E + 3) / 4), (unsigned)((b.M + RT_TM - 1) / RT_TM)),
                           dim3(256), 0, s, b);
        if (hipGetLastError() != hipSuccess)
            return SPEAR_E_HIP;
    }
    hipLaunchKernelGGL(route_choose_kernel, dim3((unsigned)((M + 3) / 4)), dim3(256), 0, s, a);
    return hipGetLastError() == hipSuccess ? SPEAR_OK : SPEAR_E_HIP;
}

} // extern "C"
