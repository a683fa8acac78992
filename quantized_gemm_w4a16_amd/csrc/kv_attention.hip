// kv_attention.hip -- attention over the cache of 4 bits (spear_kv4_attention)
// for gfx950.
//
// The rows of a request and a key head are its fresh tokens times the G query
// heads that share the key head, row = token * G + head, in tiles of TILE_ROWS.
// The keys that a tile sees are cut into chunks of whole 64-token steps; a
// (tile, chunk, key head) is a workgroup's item.  One pass over the keys holds a
// row's maximum m, sum l and output o; an item that has its tile's keys to itself
// writes y, the others leave (m, l, o) in the workspace for a second launch.
#include <math.h>

#include "kv4.hpp"

namespace spear {
namespace {

constexpr int STEP = 64;            // keys of a step
constexpr int FEW_ROWS = 16;        // rows of a tile of the kernel for few rows
constexpr int FEW_WAVES = 4;        // its waves, which take the steps of a chunk in turn
constexpr int FEW_LEAST = 4;        // steps of a chunk, at least
constexpr int FEW_ITEMS = 1024;     // items of all key heads that the cut aims at
constexpr float LOG2E = 1.44269504088896340736f;
constexpr float LN2 = 0.69314718055994530942f;

struct AttnArgs {
    const uint16_t *q;
    int64_t qs;
    const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    const int32_t *table, *q_start, *kv_len;
    uint16_t *y;
    float *lse;
    float *part_o, *part_ml;        // [item][key head][row][D], [item][key head][row][2]
    int64_t T, pages, width;
    int32_t B, heads, G, log_p, window;
    int32_t target;                 // items of a key head that the cut aims at; 0: no cut
    int32_t most;                   // items of a key head that there is room for
    float scale;                    // times log2 e
};

// ------------------------------------------------------------------- items
struct Request {
    int64_t row0;                   // its first row of q
    int32_t fresh, kv;              // its rows and keys
    int32_t tiles, base, steps;     // row tiles; the first step that a row sees; steps from there
};

__device__ __forceinline__ Request request_of(const AttnArgs &a, int b, int tile_rows)
{
    Request r;
    const int64_t T = a.T;
    int64_t q0 = a.q_start[b], q1 = a.q_start[b + 1];
    q0 = q0 < 0 ? 0 : (q0 > T ? T : q0);
    q1 = q1 < q0 ? q0 : (q1 > T ? T : q1);
    const int64_t room = a.width << a.log_p;
    int64_t kv = a.kv_len[b];
    kv = kv < 0 ? 0 : (kv > room ? room : kv);
    r.row0 = q0;
    r.fresh = (int32_t)(q1 - q0);
    r.kv = (int32_t)kv;
    r.tiles = (int32_t)(((int64_t)r.fresh * a.G + tile_rows - 1) / tile_rows);
    // the first fresh token stands at kv - fresh
    int32_t lo = a.window ? r.kv - r.fresh - a.window + 1 : 0;
    lo = lo < 0 ? 0 : lo;
    r.base = lo / STEP;
    r.steps = r.kv > lo ? (r.kv + STEP - 1) / STEP - r.base : 0;
    return r;
}

struct Item {
    Request r;
    int32_t b;                      // which request
    int32_t tile, chunk, chunks;    // of its request
    int32_t size;                   // steps of a chunk
    int32_t item;                   // first item of the tile
    bool found;
};

__device__ __forceinline__ int32_t bcast(int32_t v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// The item (or, by_tile, the tile) number `want`.  Every wave forms the sums over
// all requests, 64 at a time.  A chunk has as many steps as make about a.target
// items of a key head; sums are capped at a.most, behind which there is no item.
template <int ROWS>
__device__ Item find_item(const AttnArgs &a, int32_t want, bool by_tile)
{
    const int lane = threadIdx.x & 63;
    Item it;
    it.found = false;
    it.size = 0x7FFFFFFF;
    if (a.target) {
        float work = 0.f;
        for (int b0 = 0; b0 < a.B; b0 += 64) {
            const int b = b0 + lane;
            if (b < a.B) {
                const Request r = request_of(a, b, ROWS);
                work += (float)r.tiles * (float)r.steps;
            }
        }
#pragma unroll
        for (int d = 1; d < 64; d *= 2)
            work += __shfl_xor(work, d);
        const float s = ceilf(work / (float)a.target);
        it.size = s < (float)FEW_LEAST ? FEW_LEAST : (s > 1e9f ? 1000000000 : (int32_t)s);
    }
    int32_t items0 = 0, tiles0 = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        const int b = b0 + lane;
        int32_t chunks = 0, n = 0, tiles = 0;
        Request r = {};
        if (b < a.B) {
            r = request_of(a, b, ROWS);
            chunks = r.steps <= it.size ? 1 : (r.steps + it.size - 1) / it.size;
            tiles = r.tiles < a.most ? r.tiles : a.most;
            const int64_t all = (int64_t)r.tiles * chunks;
            n = all < a.most ? (int32_t)all : a.most;
        }
        // inclusive sums, held below 2^31 by the cap (64 * most < 2^31)
        int32_t ni = n, ti = tiles;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int32_t x = __shfl_up(ni, d), y = __shfl_up(ti, d);
            ni += lane >= d ? x : 0;
            ti += lane >= d ? y : 0;
        }
        const int32_t end = by_tile ? tiles0 + ti : items0 + ni, len = by_tile ? tiles : n;
        const uint64_t hit = __ballot(end > want && end - len <= want);
        if (hit) {
            const int src = __builtin_ctzll(hit);
            const int32_t first_item = bcast(items0 + ni - n, src), first = bcast(end - len, src);
            it.r.row0 = (int64_t)(uint32_t)bcast((int32_t)r.row0, src);
            it.r.fresh = bcast(r.fresh, src);
            it.r.kv = bcast(r.kv, src);
            it.r.tiles = bcast(r.tiles, src);
            it.r.base = bcast(r.base, src);
            it.r.steps = bcast(r.steps, src);
            it.chunks = bcast(chunks, src);
            it.tile = by_tile ? want - first : (want - first) / it.chunks;
            it.chunk = by_tile ? 0 : (want - first) % it.chunks;
            it.item = first_item + it.tile * it.chunks;
            it.b = b0 + src;
            it.found = true;
            return it;
        }
        items0 += bcast(ni, 63);
        tiles0 += bcast(ti, 63);
        items0 = items0 < a.most ? items0 : a.most;
        tiles0 = tiles0 < a.most ? tiles0 : a.most;
    }
    return it;
}

// --------------------------------------------------------------- few rows
// How the D channels of a token's head lie in the operands of the matrix
// instructions: NC chunks of CW channels, of which lane group g (16 lanes) holds
// CW / 4 consecutive ones, eight to a depth step of the instruction.  A group's
// codes are one load of W words, and all of them belong to one block.
template <int D>
struct Lay {
    static constexpr int CW = D % 128 == 0 ? 128 : (D % 64 == 0 ? 64 : 32);
    static constexpr int NC = D / CW;
    static constexpr int W = CW / 32;
    static constexpr int ROW = 2 * D + 32;   // bytes of a V row in LDS: 8 rows start in 8 different 32-byte banks
};

template <int W>
struct Words { uint32_t w[W]; };

template <int W>
__device__ __forceinline__ Words<W> load_words(const uint8_t *p)
{
    Words<W> r;
    if (W == 4) {
        const u32x4 v = ld16(p);
        r.w[0] = v[0];
        r.w[1 % W] = v[1];
        r.w[2 % W] = v[2];
        r.w[3 % W] = v[3];
    } else if (W == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        r.w[0] = v.x;
        r.w[1 % W] = v.y;
    } else
        r.w[0] = *reinterpret_cast<const uint32_t *>(p);
    return r;
}

// A step's codes and scales of one of K and V in the lanes that load them: lane
// (R = lane % 16, g = lane / 16) has the tokens 4R .. 4R + 3 of the step, which
// lie in one page, and a word with their four scales.
template <int D>
struct Part {
    Words<Lay<D>::W> c[Lay<D>::NC][4];
    uint32_t s[Lay<D>::NC];
};

template <int D>
__device__ __forceinline__ void load_part(Part<D> &p, const uint8_t *codes, const uint8_t *scales, int64_t ph, int32_t off,
                                          int log_p, int g)
{
    using L = Lay<D>;
    const uint8_t *c = codes + ((ph << log_p) + off) * (D / 2) + g * (L::CW / 8);
#pragma unroll
    for (int n = 0; n < L::NC; n++) {
#pragma unroll
        for (int i = 0; i < 4; i++)
            p.c[n][i] = load_words<L::W>(c + i * (D / 2) + n * (L::CW / 2));
        const int block = (n * L::CW + g * (L::CW / 4)) / 32;
        p.s[n] = *reinterpret_cast<const uint32_t *>(scales + ((ph * (D / 32) + block) << log_p) + off);
    }
}

__device__ __forceinline__ float scale_of(uint32_t word, int i) { return kv4_scale((word >> (8 * i)) & 255u); }

__device__ __forceinline__ float max_over_groups(float v)
{
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_over_groups(float v)
{
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Lane l of 16 gets column l of the 4 x 16 tile of 16-bit values whose row r the
// lanes 4r .. 4r + 3 point at, 8 bytes each.
__device__ __forceinline__ uint2 read_turned(const void *p)
{
    typedef __attribute__((address_space(3))) s16x4 lds4;
    const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)p);
    return __builtin_bit_cast(uint2, v);
}

__device__ __forceinline__ uint32_t pair_bf16(float lo, float hi)
{
    return (uint32_t)f2bf(lo) | ((uint32_t)f2bf(hi) << 16);
}

// LDS written by this wave is read back by its other lanes: the order of the
// wave's own accesses suffices, the compiler only has to keep it.
__device__ __forceinline__ void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Matrix instructions, with g the group of a lane and n its place in the group:
//   S^T [key][row] = K Q^T  lane: row n, keys 16 g + 4 r + i in acc[i][r]
//   O^T [channel][row] += V^T P^T  lane: row n, channels 16 dt + 4 g + r in o[dt][r]
// Instruction i of the first takes the keys 4R + i, R = 0 .. 15, so that what a
// lane gets of S is what it has to bring of P to the second, whose depth slots
// (g, j) stand for the keys 16 g + 4 (j % 4) + 2 u + j / 4.  V goes through LDS,
// as bf16, to be read column by column.
template <int D>
__global__ __launch_bounds__(64 * FEW_WAVES) void few_rows_kernel(const AttnArgs a)
{
    using L = Lay<D>;
    constexpr int DT = D / 16, NS = L::NC * L::W;
    constexpr int V_BYTES = 32 * L::ROW;
    static_assert(V_BYTES >= 16 * D * 4, "the waves' outputs are joined in the same LDS");
    __shared__ __attribute__((aligned(16))) uint8_t s_v[FEW_WAVES][V_BYTES];
    __shared__ float s_ml[FEW_WAVES][FEW_ROWS][2];

    const int head = blockIdx.x % a.heads;
    const Item it = find_item<FEW_ROWS>(a, (int32_t)(blockIdx.x / a.heads), false);
    if (!it.found)
        return;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, n = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int b = it.b, G = a.G, log_p = a.log_p;
    const int64_t page_mask = (1 << log_p) - 1;

    // this lane's row and the positions it sees, [first, last]
    const int row = it.tile * FEW_ROWS + n;
    const int tok = row / G, qh = row - tok * G;
    const bool real = tok < it.r.fresh;
    const int pos0 = it.r.kv - it.r.fresh;
    const int last = real ? pos0 + tok : -1;
    const int first = a.window && last - a.window + 1 > 0 ? last - a.window + 1 : 0;
    // ... and what the tile's rows see together
    const int tok0 = it.tile * FEW_ROWS / G;
    int tok1 = (it.tile * FEW_ROWS + FEW_ROWS - 1) / G;
    tok1 = tok1 < it.r.fresh ? tok1 : it.r.fresh - 1;
    const int seen1 = pos0 + tok1 + 1;                                     // one past the last
    const int seen0 = a.window && pos0 + tok0 - a.window + 1 > 0 ? pos0 + tok0 - a.window + 1 : 0;
    const int all1 = pos0 + tok0;                                          // every row sees [all0, all1]
    const int all0 = a.window && pos0 + tok1 - a.window + 1 > 0 ? pos0 + tok1 - a.window + 1 : 0;

    int lo = it.r.base + it.chunk * (it.chunks > 1 ? it.size : 0), hi = it.r.base + it.r.steps;
    if (it.chunks > 1 && lo + it.size < hi)
        hi = lo + it.size;
    lo = lo > seen0 / STEP ? lo : seen0 / STEP;
    const int hi_seen = seen1 > 0 ? (seen1 + STEP - 1) / STEP : 0;
    hi = hi < hi_seen ? hi : hi_seen;

    u32x4 qf[NS];
    {
        const uint16_t *qp = a.q + (it.r.row0 + tok) * a.qs + (int64_t)(head * G + qh) * D;
#pragma unroll
        for (int c = 0; c < L::NC; c++)
#pragma unroll
            for (int s = 0; s < L::W; s++)
                qf[c * L::W + s] = real ? ld16(qp + c * L::CW + g * (L::CW / 4) + 8 * s) : zero4();
    }
    f32x4 o[DT];
#pragma unroll
    for (int d = 0; d < DT; d++)
        o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;

    Part<D> kp, vp;
    const int32_t *table = a.table + (int64_t)b * a.width;
    // Page and place of this lane's four tokens of a step.  Steps behind the last
    // read the first page of the cache, and nothing of it is used.
    auto page_of = [&](int step) {
        const int t0 = step * STEP + 4 * n;
        return step < hi && t0 < it.r.kv ? table[t0 >> log_p] : 0;
    };
    int page = page_of(lo + wave);
    bool lost = page < 0 || page >= a.pages;
    int64_t ph = (int64_t)(lost ? 0 : page) * a.heads + head;
    int32_t off = (int32_t)(((lo + wave) * STEP + 4 * n) & page_mask);
    load_part<D>(kp, a.k_codes, a.k_scales, ph, off, log_p, g);
    load_part<D>(vp, a.v_codes, a.v_scales, ph, off, log_p, g);
    int page_next = page_of(lo + wave + FEW_WAVES);

    for (int step = lo + wave; step < hi; step += FEW_WAVES) {
        const int key0 = step * STEP;
        const uint32_t lost16 = (uint32_t)(__ballot(lost) & 0xFFFF);       // bit R: the keys 4R .. 4R + 3
        f32x4 acc[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < L::NC; c++) {
                const float s = scale_of(kp.s[c], i);
#pragma unroll
                for (int w = 0; w < L::W; w++)
                    acc[i] = mfma16(kv4_bf16(kp.c[c][i].w[w], s), qf[c * L::W + w], acc[i]);
            }
        }
        // the next step's keys
        const bool lost_now = lost;
        page = page_next;
        lost = page < 0 || page >= a.pages;
        ph = (int64_t)(lost ? 0 : page) * a.heads + head;
        off = (int32_t)((key0 + FEW_WAVES * STEP + 4 * n) & page_mask);
        load_part<D>(kp, a.k_codes, a.k_scales, ph, off, log_p, g);
        page_next = page_of(step + 2 * FEW_WAVES);

        const bool edge = key0 < all0 || key0 + STEP - 1 > all1 || lost16 != 0;
        float top = -INFINITY;
        if (edge) {
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const int key = key0 + 16 * g + 4 * r + i;
                    const bool sees = key >= first && key <= last && !(lost16 >> (4 * g + r) & 1);
                    acc[i][r] = sees ? acc[i][r] * a.scale : -INFINITY;
                    top = fmaxf(top, acc[i][r]);
                }
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    acc[i][r] *= a.scale;
                    top = fmaxf(top, acc[i][r]);
                }
        }
        top = max_over_groups(top);
        if (__any(top > m)) {
            const float up = fmaxf(m, top);
            const float f = m == up ? 1.f : __builtin_amdgcn_exp2f(m - up);
            m = up;
            l *= f;
#pragma unroll
            for (int d = 0; d < DT; d++)
                o[d] *= f;
        }
        const float m0 = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int r = 0; r < 4; r++) {
                acc[i][r] = __builtin_amdgcn_exp2f(acc[i][r] - m0);
                l += acc[i][r];
            }

        // keys that no row of the tile sees hold anything: their V is zero
        if (key0 < seen0 || key0 + STEP > seen1 || lost16 != 0) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int key = key0 + 4 * n + i;
                if (lost_now || key < seen0 || key >= seen1) {
#pragma unroll
                    for (int c = 0; c < L::NC; c++) {
#pragma unroll
                        for (int w = 0; w < L::W; w++)
                            vp.c[c][i].w[w] = 0;
                        vp.s[c] = (vp.s[c] & ~(255u << (8 * i))) | (127u << (8 * i));
                    }
                }
            }
        }
        // A block of NaN counts for the rows that see its key only; a zero
        // probability would carry it to the others.
        bool nan_here = false;
#pragma unroll
        for (int c = 0; c < L::NC; c++) {
            const uint32_t x = ~vp.s[c];
            nan_here |= ((x - 0x01010101u) & ~x & 0x80808080u) != 0;
        }
        if (__any(nan_here)) {
#pragma unroll
            for (int c = 0; c < L::NC; c++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const bool mine = ((vp.s[c] >> (8 * i)) & 255u) == 255u;
                    uint64_t who = __ballot(mine);
                    while (who) {
                        const int src = __builtin_ctzll(who);
                        who &= who - 1;
                        const int key = key0 + 4 * (src & 15) + i, block = (c * L::CW + (src >> 4) * (L::CW / 4)) / 32;
                        const float add = key >= first && key <= last ? __builtin_nanf("") : 0.f;
#pragma unroll
                        for (int d = 0; d < DT; d++)
                            if (d / 2 == block)
                                o[d] += add;
                    }
                    if (mine) {
#pragma unroll
                        for (int w = 0; w < L::W; w++)
                            vp.c[c][i].w[w] = 0;
                        vp.s[c] = (vp.s[c] & ~(255u << (8 * i))) | (127u << (8 * i));
                    }
                }
        }

        uint8_t *sv = s_v[wave];
#pragma unroll
        for (int u = 0; u < 2; u++) {
            wave_order();
#pragma unroll
            for (int e = 0; e < 2; e++)
#pragma unroll
                for (int c = 0; c < L::NC; c++) {
                    const float s = scale_of(vp.s[c], 2 * u + e);
#pragma unroll
                    for (int w = 0; w < L::W; w++)
                        *reinterpret_cast<u32x4 *>(sv + (e * 16 + n) * L::ROW + 2 * (c * L::CW + g * (L::CW / 4)) + 16 * w) =
                            kv4_bf16(vp.c[c][2 * u + e].w[w], s);
                }
            wave_order();
            // P as a sum of two bf16: V is read once for both, and P's rounding is gone (2^-17)
            u32x4 p_hi, p_lo;
#pragma unroll
            for (int e = 0; e < 2; e++)
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    const float x = acc[2 * u + e][2 * r], z = acc[2 * u + e][2 * r + 1];
                    const uint32_t hi2 = pair_bf16(x, z);
                    p_hi[2 * e + r] = hi2;
                    p_lo[2 * e + r] = pair_bf16(x - __uint_as_float(hi2 << 16), z - __uint_as_float(hi2 & 0xFFFF0000u));
                }
#pragma unroll
            for (int d = 0; d < DT; d++) {
                const uint8_t *at = sv + (4 * g + (n >> 2)) * L::ROW + 32 * d + 8 * (n & 3);
                const uint2 x = read_turned(at), z = read_turned(at + 16 * L::ROW);
                const u32x4 vt = {x.x, x.y, z.x, z.y};
                o[d] = mfma16(vt, p_hi, o[d]);
                o[d] = mfma16(vt, p_lo, o[d]);
            }
        }
        load_part<D>(vp, a.v_codes, a.v_scales, ph, off, log_p, g);
    }

    // ---- the four waves' parts of the chunk
    l = sum_over_groups(l);
    wave_order();
    float *so = reinterpret_cast<float *>(s_v[wave]);                      // [row][D]
#pragma unroll
    for (int d = 0; d < DT; d++)
        *reinterpret_cast<f32x4 *>(so + n * D + 16 * d + 4 * g) = o[d];
    if (g == 0) {
        s_ml[wave][n][0] = m;
        s_ml[wave][n][1] = l;
    }
    __syncthreads();
    const int rows = it.r.fresh * G - it.tile * FEW_ROWS;                  // real rows of the tile
    for (int x = tid; x < 16 * (D / 4); x += 64 * FEW_WAVES) {
        const int r = x / (D / 4), c = 4 * (x % (D / 4));
        if (r >= rows)
            break;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < FEW_WAVES; w++)
            mm = fmaxf(mm, s_ml[w][r][0]);
        const float ref = mm == -INFINITY ? 0.f : mm;
        float ll = 0.f;
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < FEW_WAVES; w++) {
            const float f = __builtin_amdgcn_exp2f(s_ml[w][r][0] - ref);
            ll += f * s_ml[w][r][1];
            sum += f * *reinterpret_cast<const f32x4 *>(reinterpret_cast<const float *>(s_v[w]) + r * D + c);
        }
        if (it.chunks > 1) {
            const int64_t p = ((int64_t)(it.item + it.chunk) * a.heads + head) * FEW_ROWS + r;
            *reinterpret_cast<f32x4 *>(a.part_o + p * D + c) = sum;
            if (c == 0) {
                a.part_ml[2 * p] = mm;
                a.part_ml[2 * p + 1] = ll;
            }
        } else {
            const int rr = it.tile * FEW_ROWS + r;
            const int64_t hrow = (it.r.row0 + rr / G) * ((int64_t)a.heads * G) + head * G + rr % G;
            const float inv = ll == 0.f ? 0.f : 1.f / ll;
            *reinterpret_cast<uint2 *>(a.y + hrow * D + c) =
                make_uint2(pair_bf16(sum[0] * inv, sum[1] * inv), pair_bf16(sum[2] * inv, sum[3] * inv));
            if (c == 0 && a.lse)
                a.lse[hrow] = ll == 0.f ? -INFINITY : (mm + __log2f(ll)) * LN2;
        }
    }
}

// The chunks of a tile joined, in their order; a workgroup takes a tile of a key head.
template <int D, int ROWS>
__global__ __launch_bounds__(256) void join_chunks_kernel(const AttnArgs a)
{
    const int head = blockIdx.x % a.heads;
    const Item it = find_item<ROWS>(a, (int32_t)(blockIdx.x / a.heads), true);
    if (!it.found || it.chunks < 2)
        return;
    const int G = a.G, rows = it.r.fresh * G - it.tile * ROWS;
    const int64_t p0 = ((int64_t)it.item * a.heads + head) * ROWS, next = (int64_t)a.heads * ROWS;
    for (int x = threadIdx.x; x < ROWS * (D / 4); x += 256) {
        const int r = x / (D / 4), c = 4 * (x % (D / 4));
        if (r >= rows)
            break;
        float mm = -INFINITY;
        for (int i = 0; i < it.chunks; i++)
            mm = fmaxf(mm, a.part_ml[2 * (p0 + i * next + r)]);
        const float ref = mm == -INFINITY ? 0.f : mm;
        float ll = 0.f;
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
        for (int i = 0; i < it.chunks; i++) {
            const int64_t p = p0 + i * next + r;
            const float f = __builtin_amdgcn_exp2f(a.part_ml[2 * p] - ref);
            ll += f * a.part_ml[2 * p + 1];
            sum += f * *reinterpret_cast<const f32x4 *>(a.part_o + p * D + c);
        }
        const int rr = it.tile * ROWS + r;
        const int64_t hrow = (it.r.row0 + rr / G) * ((int64_t)a.heads * G) + head * G + rr % G;
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        *reinterpret_cast<uint2 *>(a.y + hrow * D + c) =
            make_uint2(pair_bf16(sum[0] * inv, sum[1] * inv), pair_bf16(sum[2] * inv, sum[3] * inv));
        if (c == 0 && a.lse)
            a.lse[hrow] = ll == 0.f ? -INFINITY : (mm + __log2f(ll)) * LN2;
    }
}

// ------------------------------------------------------------------- host
struct AttnLayout {
    int64_t tiles, items;           // of a key head, at most
    int32_t target;                 // 0: no cut
    size_t part_o, part_ml, total;
};

bool al(const void *p, size_t n) { return (uintptr_t)p % n == 0; }

bool attention_sizes(int64_t T, int32_t B, int64_t max_fresh, int32_t Hq, int32_t heads, int32_t D, int64_t width, int32_t P)
{
    return T >= 0 && T <= SPEAR_MAX_ROWS && B >= 0 && B <= SPEAR_MAX_REQUESTS && max_fresh >= 0 && heads >= 1 &&
           heads <= SPEAR_MAX_HEADS && Hq >= heads && Hq <= SPEAR_MAX_HEADS && Hq % heads == 0 && Hq / heads <= 64 &&
           (D == 64 || D == 96 || D == 128 || D == 192 || D == 256) && P >= 16 && P <= 1024 && (P & (P - 1)) == 0 &&
           width >= 1 && width <= SPEAR_MAX_CONTEXT / P && T * Hq <= (int64_t)1 << 27;
}

AttnLayout attention_layout(int64_t T, int32_t B, int64_t max_fresh, int32_t Hq, int32_t heads, int32_t D)
{
    AttnLayout L;
    const int64_t G = Hq / heads, rows = T * G;
    // tiles of a key head: at most one more a request than its rows fill, and no
    // fewer than all rows fill and requests of max_fresh rows make
    const int64_t more = T < B ? T : B;
    L.tiles = rows / FEW_ROWS + more;
    int64_t least = (rows + FEW_ROWS - 1) / FEW_ROWS;
    const int64_t each = max_fresh > 0 ? (T + max_fresh - 1) / max_fresh : 0;
    least = least > each ? least : each;
    const int64_t cut = (FEW_ITEMS + heads - 1) / heads;
    L.target = least * heads >= FEW_ITEMS ? 0 : (int32_t)cut;
    L.items = L.tiles + (L.target ? cut + 16 : 0);
    // The room of the parts does not depend on max_fresh and grows with T and B, so
    // that a workspace of the largest step serves every other: with a cut, least is
    // below cut and L.tiles below cut + more.
    const int64_t room = (L.tiles < cut + more ? L.tiles : cut + more) + cut + 16;
    L.part_o = 0;
    L.part_ml = (size_t)(room * heads * FEW_ROWS * D) * sizeof(float);
    L.total = L.part_ml + (size_t)(room * heads * FEW_ROWS * 2) * sizeof(float);
    return L;
}

template <int D>
hipError_t launch_attention(const AttnArgs &a, const AttnLayout &L, hipStream_t s)
{
    hipLaunchKernelGGL((few_rows_kernel<D>), dim3((unsigned)(L.items * a.heads)), dim3(64 * FEW_WAVES), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.target)
        return e;
    hipLaunchKernelGGL((join_chunks_kernel<D, FEW_ROWS>), dim3((unsigned)(L.tiles * a.heads)), dim3(256), 0, s, a);
    return hipGetLastError();
}

} // namespace
} // namespace spear

using namespace spear;

extern "C" {

size_t spear_kv4_attention_workspace_size(int64_t T, int32_t B, int64_t max_fresh, int32_t Hq,
                                          int32_t heads, int32_t D, int64_t width, int32_t P)
{
    return attention_sizes(T, B, max_fresh, Hq, heads, D, width, P) ? attention_layout(T, B, max_fresh, Hq, heads, D).total : 0;
}

spear_status spear_kv4_attention(const spear_bf16 *q, int64_t q_stride, int64_t T, int32_t Hq,
                                 const spear_kv4 *kv, const int32_t *table, int64_t width,
                                 const int32_t *q_start, const int32_t *kv_len, int32_t B,
                                 int64_t max_fresh, float scale, int32_t window, spear_bf16 *y,
                                 float *lse, void *workspace, size_t ws_bytes, void *stream)
{
    if (!workspace || (T > 0 && B > 0 && (!q || !table || !q_start || !kv_len || !y)))
        return SPEAR_E_NULL;
    spear_status st = check_kv4(kv);
    if (st != SPEAR_OK)
        return st;
    if (!attention_sizes(T, B, max_fresh, Hq, kv->heads, kv->D, width, kv->P) || window < 0 ||
        window > SPEAR_MAX_CONTEXT || q_stride < (int64_t)Hq * kv->D || q_stride % 8 != 0 ||
        q_stride > ((int64_t)1 << 36) || (q == y && q_stride != (int64_t)Hq * kv->D))
        return SPEAR_E_SHAPE;
    if (!(scale > 0.f) || !isfinite(scale))
        return SPEAR_E_ARG;
    if (!al(q, 16) || !al(y, 16) || !al(table, 4) || !al(q_start, 4) || !al(kv_len, 4) || !al(lse, 4) || !al(workspace, 256))
        return SPEAR_E_ALIGN;
    const AttnLayout L = attention_layout(T, B, max_fresh, Hq, kv->heads, kv->D);
    if (ws_bytes < L.total)
        return SPEAR_E_WORKSPACE;
    st = check_device();
    if (st != SPEAR_OK || T == 0 || B == 0)
        return st;
    uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
    const AttnArgs a = {q, q_stride, kv->k_codes, kv->k_scales, kv->v_codes, kv->v_scales, table, q_start, kv_len, y, lse,
                        reinterpret_cast<float *>(ws + L.part_o), reinterpret_cast<float *>(ws + L.part_ml), T, kv->pages,
                        width, B, kv->heads, Hq / kv->heads, __builtin_ctz(kv->P), window, L.target, (int32_t)L.items,
                        scale * LOG2E};
    const hipStream_t s = (hipStream_t)stream;
    hipError_t e = hipSuccess;
    switch (kv->D) {
    case 64: e = launch_attention<64>(a, L, s); break;
    case 96: e = launch_attention<96>(a, L, s); break;
    case 128: e = launch_attention<128>(a, L, s); break;
    case 192: e = launch_attention<192>(a, L, s); break;
    default: e = launch_attention<256>(a, L, s); break;
    }
    return e == hipSuccess ? SPEAR_OK : SPEAR_E_HIP;
}

} // extern "C"
