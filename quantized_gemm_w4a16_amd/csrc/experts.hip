// experts.hip -- the routed tokens through their experts' two 4-bit layers
// (spear_w4_experts), gfx950.
//
//   h_mj = act(up_e x_m + b)  (or the gated pair),  e = ids[m][j]
//   y[m] = residual[m] + sum_j weights[m][j] (down_e h_mj + b)
//
// A slot is one (token, choice) pair, slot = topk m + j.  Launches:
//  1. plan: the slots of each expert in ascending order, cut into row tiles;
//  2. up:   each row tile's tokens through its expert's first layer, h by slot;
//  3. down: h through the second layer, fp32 rows by slot;
//  4. join: each token's rows times their weights, in slot order, plus residual.
// No launch waits on another workgroup, and no result depends on an order that
// the hardware chooses: the sums of an output are taken in one fixed order.
#include <string.h>

#include "spear_internal.hpp"

namespace spear {

namespace {

constexpr int XT = 16;                                    // rows of the smallest tile

struct ExpertsLayout {
    size_t hdr, zeros, tiles, list, h, d, total;
    int64_t slots;
};

// Row tiles of bm rows: every expert in use has its slots cut into tiles, the
// last one ragged, so at most slots / bm + (experts in use) of them.
int64_t max_tiles(int64_t slots, int32_t E, int bm) { return slots / bm + (slots < E ? slots : E); }

// Rows of a tile by the slots an expert has on average.
int tile_rows(int64_t slots, int32_t E)
{
    const int64_t per = slots / E;
    return per >= 48 ? 128 : per >= 12 ? 64 : XT;
}

ExpertsLayout experts_layout(int64_t M, int32_t topk, int32_t E, int64_t I, int64_t N)
{
    ExpertsLayout L;
    auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
    L.slots = (M < 1 ? 1 : M) * topk;
    size_t off = 0;
    L.hdr = off;
    off = up(off + 64);
    L.zeros = off;                                        // 256 zero bytes, written by the plan
    off = up(off + 256);
    L.tiles = off;
    off = up(off + (size_t)max_tiles(L.slots, E, XT) * sizeof(Tile));
    L.list = off;
    off = up(off + (size_t)L.slots * 4);
    L.h = off;
    off = up(off + (size_t)L.slots * (size_t)I * 2);
    L.d = off;
    off = up(off + (size_t)L.slots * (size_t)N * 4);
    L.total = off;
    return L;
}

// ---------------------------------------------------------------------- plan
// One workgroup an expert.  Every workgroup counts all slots (LDS counters; a
// count does not depend on the order of its additions), so it knows where its
// own rows and tiles begin, then writes its slots in ascending order by ballot.
__global__ __launch_bounds__(1024) void plan_kernel(const int32_t *__restrict__ ids, int32_t slots, int32_t E,
                                                    int32_t bm, uint32_t *__restrict__ zeros,
                                                    int32_t *__restrict__ ntiles, Tile *__restrict__ tiles,
                                                    int32_t *__restrict__ list)
{
    __shared__ int cnt[SPEAR_MAX_EXPERTS];
    __shared__ int wave_tot[16];
    __shared__ int s_pos, s_tile, s_all;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int e = blockIdx.x;
    for (int i = tid; i < E; i += 1024)
        cnt[i] = 0;
    __syncthreads();
    for (int i = tid; i < slots; i += 1024) {
        const int v = ids[i];
        if (v >= 0 && v < E)
            atomicAdd(&cnt[v], 1);
    }
    __syncthreads();
    if (wave == 0) {
        int pos = 0, tile = 0, all = 0;
        for (int i = lane; i < E; i += 64) {
            const int t = (cnt[i] + bm - 1) / bm;
            all += t;
            if (i < e) {
                pos += cnt[i];
                tile += t;
            }
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            pos += __shfl_xor(pos, o);
            tile += __shfl_xor(tile, o);
            all += __shfl_xor(all, o);
        }
        if (lane == 0) {
            s_pos = pos;
            s_tile = tile;
            s_all = all;
        }
    }
    __syncthreads();
    if (e == 0 && tid == 0)
        *ntiles = s_all;
    if (e == 0 && tid < 64)
        zeros[tid] = 0u;                                  // what the products read past K
    const int mine = cnt[e], pos0 = s_pos, tile0 = s_tile;
    for (int t = tid; t * bm < mine; t += 1024) {
        Tile q;
        q.e = e;
        q.pos = pos0 + t * bm;
        q.cnt = mine - t * bm < bm ? mine - t * bm : bm;
        q.pad = 0;
        tiles[tile0 + t] = q;
    }
    if (mine == 0)
        return;
    int base = pos0;
    for (int c0 = 0; c0 < slots; c0 += 1024) {
        const int i = c0 + tid;
        const bool f = i < slots && ids[i] == e;
        const uint64_t mask = __ballot(f);
        if (lane == 0)
            wave_tot[wave] = __popcll(mask);
        __syncthreads();
        int off = base, total = 0;
        for (int w = 0; w < 16; w++) {
            if (w < wave)
                off += wave_tot[w];
            total += wave_tot[w];
        }
        if (f)
            list[off + __popcll(mask & ((1ull << lane) - 1ull))] = i;
        base += total;
        __syncthreads();
    }
}

// --------------------------------------------------------------- the products
struct GroupArgs {
    const uint16_t *x;        // rows [.][K]: tokens (up) or h by slot (down)
    const uint8_t *packed;    // [E][N][K/2]
    const float *scales;      // [E][N]
    const uint8_t *zeros;     // [E][N] or null
    const float *bias;        // [E][N] or null
    void *out;                // up: h [slots][N or N / 2] bf16; down: [slots][N] fp32
    const int32_t *ntiles;
    const Tile *tiles;
    const int32_t *list;
    int64_t N, K;
    int32_t div;              // a row's source is slot / div (topk for up, 1 for down)
    int32_t act, glu;
    int32_t ncb;              // channel blocks of 64: the grid's fastest index
};

// One wave takes 16 channels of a row tile over all of K.  Lane (c, g) holds
// channel c's 32 codes k = 128 s + 32 g .. + 31 of super-step s as one 16-byte
// load, and the same depths of row c of the tile: 64 bytes.  Rows past the
// tile's end are zero.
template <int UP>
__global__ __launch_bounds__(256) void group_kernel(const GroupArgs a)
{
    const int tile = (int)(blockIdx.x / (uint32_t)a.ncb), cb = (int)(blockIdx.x % (uint32_t)a.ncb);
    if (tile >= *a.ntiles)
        return;
    const Tile q = a.tiles[tile];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int lr = lane & 15, lg = lane >> 4;
    const int64_t N = a.N, K = a.K;
    const int64_t n0 = ((int64_t)cb * 4 + wave) * 16;
    if (n0 >= N)
        return;
    const int64_t nc = n0 + lr < N ? n0 + lr : N - 1;
    const int64_t base = (int64_t)q.e * N;
    const int slot = lr < q.cnt ? a.list[q.pos + lr] : -1;
    const uint16_t *xr = a.x + (int64_t)(slot < 0 ? 0 : slot / a.div) * K;
    const uint8_t *wr = a.packed + (base + nc) * (K / 2);
    f32x4 acc = {0.f, 0.f, 0.f, 0.f}, rs = acc;
    const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    for (int64_t k0 = 0; k0 < K; k0 += 128) {
        const int64_t k = k0 + 32 * lg;
        const bool kv = k < K;
        const u32x4 w = ld16(wr + (kv ? k : 0) / 2);
        u32x4 xv[4];
#pragma unroll
        for (int d = 0; d < 4; d++)
            xv[d] = kv && slot >= 0 ? ld16(xr + k + 8 * d) : zero4();
#pragma unroll
        for (int d = 0; d < 4; d++) {
            acc = mfma16(unpack8(w[d]), xv[d], acc);
            rs = mfma16(ones, xv[d], rs);
        }
    }
    // lane (row lr, lg): channels n0 + 4 lg + i
    if (slot < 0)
        return;
    float t[4], b[4], o[4];
    const int64_t n = n0 + 4 * lg;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int64_t nn = base + (n + i < N ? n + i : N - 1);
        const float zp = a.zeros ? (float)a.zeros[nn] : 8.f;
        t[i] = a.scales[nn] * __builtin_fmaf(-(UNPACK_OFF + zp), rs[0], UNPACK_SCALE * acc[i]);
        b[i] = a.bias ? a.bias[nn] : 0.f;
    }
    if (UP) {
        epi_apply(t, b, a.act, a.glu, o);
        epi_store<0>(a.out, slot, n, a.glu, a.glu ? N / 2 : N, o);
    } else {
        epi_apply(t, b, SPEAR_ACT_NONE, 0, o);
        epi_store<1>(a.out, slot, n, 0, N, o);
    }
}

// ---------------------------------------------------------------------- join
// A thread takes four channels of one token.
struct JoinArgs {
    const float *d;           // [slots][N]
    const int32_t *ids;
    const float *weights;
    const uint16_t *res;
    uint16_t *y;
    int64_t M, N;
    int32_t topk, E;
};

__global__ __launch_bounds__(256) void join_kernel(const JoinArgs a)
{
    const int64_t nq = (a.N + 3) / 4;
    const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (idx >= a.M * nq)
        return;
    const int64_t m = idx / nq, n = 4 * (idx % nq), N = a.N;
    float o[4];
    epi_load_res<0>(a.res, m, n, 0, N, o);
    for (int j = 0; j < a.topk; j++) {
        const int64_t slot = m * a.topk + j;
        const int e = a.ids[slot];
        if (e < 0 || e >= a.E)
            continue;
        const float w = a.weights[slot];
        float v[4];
        epi_load_res<1>(a.d, slot, n, 0, N, v);
#pragma unroll
        for (int i = 0; i < 4; i++)
            o[i] = __builtin_fmaf(w, v[i], o[i]);
    }
    epi_store<0>(a.y, m, n, 0, N, o);
}

bool al(const void *p, size_t n) { return (uintptr_t)p % n == 0; }

} // namespace
} // namespace spear

using namespace spear;

extern "C" {

size_t spear_w4_experts_workspace_size(int64_t M, int32_t topk, int32_t E, int64_t I, int64_t N)
{
    if (M < 0 || topk < 1 || topk > SPEAR_MAX_TOPK || E < 1 || E > SPEAR_MAX_EXPERTS || I < 32 || N < 1 ||
        M > 0x7FFFFFFF / topk || I > ((int64_t)1 << 31) || N > ((int64_t)1 << 31))
        return 0;
    return experts_layout(M, topk, E, I, N).total;
}

spear_status spear_w4_experts(const spear_bf16 *x, int64_t M, const spear_experts *w,
                              const int32_t *ids, const float *weights, int32_t topk,
                              const spear_bf16 *residual, spear_bf16 *y, void *workspace,
                              size_t ws_bytes, void *stream)
{
    if (!w || !w->up || !w->up_scales || !w->down || !w->down_scales || !workspace ||
        (M > 0 && (!x || !ids || !weights || !y)))
        return SPEAR_E_NULL;
    const int64_t K = w->K, I = w->I, N = w->N;
    const int64_t lim = (int64_t)1 << 31;
    if (M < 0 || topk < 1 || topk > SPEAR_MAX_TOPK || w->E < 1 || w->E > SPEAR_MAX_EXPERTS || K < 32 ||
        K % 32 != 0 || I < 32 || I % 32 != 0 || N < 1 || M > 0x7FFFFFFF / topk || K > lim || I > lim || N > lim)
        return SPEAR_E_SHAPE;
    if (w->act < SPEAR_ACT_NONE || w->act > SPEAR_ACT_GELU_TANH || (w->glu != 0 && w->glu != 1))
        return SPEAR_E_ARG;
    if (!al(x, 16) || !al(w->up, 16) || !al(w->down, 16) || !al(w->up_scales, 4) || !al(w->down_scales, 4) ||
        !al(w->up_bias, 4) || !al(w->down_bias, 4) || !al(ids, 4) || !al(weights, 4) || !al(residual, 16) ||
        !al(y, 16) || !al(workspace, 256))
        return SPEAR_E_ALIGN;
    const ExpertsLayout L = experts_layout(M, topk, w->E, I, N);
    if (ws_bytes < L.total)
        return SPEAR_E_WORKSPACE;
    const int64_t NU = w->glu ? 2 * I : I, wide = NU > N ? NU : N;
    const int bm = tile_rows(L.slots, w->E);
    const int64_t nt = max_tiles(L.slots, w->E, bm);
    // grids: row tiles times channel tiles of at least 64, and join quads
    if (nt > 0x7FFFFFFF / ((wide + 63) / 64) || (M * ((N + 3) / 4) + 255) / 256 > 0x7FFFFFFF)
        return SPEAR_E_SHAPE;
    const spear_status st = check_device();
    if (st != SPEAR_OK || M == 0)
        return st;
    const hipStream_t s = (hipStream_t)stream;
    uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
    int32_t *ntiles = reinterpret_cast<int32_t *>(ws + L.hdr);
    Tile *tiles = reinterpret_cast<Tile *>(ws + L.tiles);
    int32_t *list = reinterpret_cast<int32_t *>(ws + L.list);
    hipLaunchKernelGGL(plan_kernel, dim3((unsigned)w->E), dim3(1024), 0, s, ids, (int32_t)L.slots, w->E, bm,
                       reinterpret_cast<uint32_t *>(ws + L.zeros), ntiles, tiles, list);
    if (hipGetLastError() != hipSuccess)
        return SPEAR_E_HIP;
    if (bm == XT) {
        GroupArgs u = {x, w->up, w->up_scales, w->up_zeros, w->up_bias, ws + L.h, ntiles, tiles, list,
                       NU, K, topk, w->act, w->glu, (int32_t)((NU + 63) / 64)};
        hipLaunchKernelGGL(group_kernel<1>, dim3((unsigned)(nt * u.ncb)), dim3(256), 0, s, u);
        if (hipGetLastError() != hipSuccess)
            return SPEAR_E_HIP;
        GroupArgs d = {reinterpret_cast<const uint16_t *>(ws + L.h), w->down, w->down_scales, w->down_zeros,
                       w->down_bias, ws + L.d, ntiles, tiles, list, N, I, 1, SPEAR_ACT_NONE, 0,
                       (int32_t)((N + 63) / 64)};
        hipLaunchKernelGGL(group_kernel<0>, dim3((unsigned)(nt * d.ncb)), dim3(256), 0, s, d);
        if (hipGetLastError() != hipSuccess)
            return SPEAR_E_HIP;
    } else {
        LinearArgs a;
        memset(&a, 0, sizeof a);
        a.ws = ws;
        a.P.zeros = L.zeros;
        a.G.ntiles = ntiles;
        a.G.tiles = tiles;
        a.G.list = list;
        a.x = x;
        a.packed = w->up;
        a.scales = w->up_scales;
        a.zeros = w->up_zeros;
        a.E.bias = w->up_bias;
        a.E.act = w->act;
        a.E.glu = w->glu;
        a.y = ws + L.h;
        a.N = NU;
        a.K = K;
        a.G.div = topk;
        if (launch_gemm_grouped(a, bm, nt, s) != hipSuccess)
            return SPEAR_E_HIP;
        a.x = reinterpret_cast<const uint16_t *>(ws + L.h);
        a.packed = w->down;
        a.scales = w->down_scales;
        a.zeros = w->down_zeros;
        a.E.bias = w->down_bias;
        a.E.act = SPEAR_ACT_NONE;
        a.E.glu = 0;
        a.y = ws + L.d;
        a.out_f32 = 1;
        a.N = N;
        a.K = I;
        a.G.div = 1;
        if (launch_gemm_grouped(a, bm, nt, s) != hipSuccess)
            return SPEAR_E_HIP;
    }
    JoinArgs j = {reinterpret_cast<const float *>(ws + L.d), ids, weights, residual, y, M, N, topk, w->E};
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)((M * ((N + 3) / 4) + 255) / 256)), dim3(256), 0, s, j);
    return hipGetLastError() == hipSuccess ? SPEAR_OK : SPEAR_E_HIP;
}

} // extern "C"
