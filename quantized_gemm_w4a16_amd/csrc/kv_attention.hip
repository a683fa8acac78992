// kv_attention.hip -- attention over the cache of 4 bits (spear_kv4_attention)
// for gfx950.
//
// The rows of a request and a key head are its fresh tokens times the G query
// heads that share the key head, row = token * G + head, in tiles of TILE_ROWS.
// The keys that a tile sees are cut into chunks of whole 64-token steps; a
// (tile, chunk, key head) is a workgroup's item.  One pass over the keys holds a
// row's maximum m, sum l and output o; an item that has its tile's keys to itself
// writes y, the others leave (m, l, o) in the workspace, to be joined in the
// chunks' order: by the last of them to finish (few rows), or by a second launch.
#include <math.h>

#include "kv4.hpp"

namespace spear {
namespace {

constexpr int STEP = 64;            // keys of a step
constexpr int FEW_ROWS = 16;        // rows of a tile of the kernel for few rows
constexpr int FEW_WAVES = 4;        // its waves, which take the steps of a chunk in turn
constexpr int FEW_ITEMS = 768;      // items of all key heads that the cut aims at: three a CU (wide heads two)
// Steps of a chunk, at least: a join costs as much as some steps, and pays where
// there are CUs without work.  us with 4 / 16: one request of 1021 keys and 8 heads 9.4
// / 11.4, 300 tiles of up to 5 steps 16.5 / 10.7, 450 tiles of up to 25 53 / 43.
constexpr int FEW_LEAST = 4, FEW_LEAST_FULL = 16;
constexpr int FIT_REQUESTS = 256;   // requests of a step whose chunks are made to fit
constexpr int JB = 8;               // chunks whose parts are on their way at once in the join
constexpr int MANY_LEAST = 4;       // steps of its chunks, at least
constexpr float LOG2E = 1.44269504088896340736f;
constexpr float LN2 = 0.69314718055994530942f;

struct AttnArgs {
    const uint16_t *q;
    int64_t qs;
    const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    const int32_t *table, *q_start, *kv_len;
    uint16_t *y;
    float *lse;
    int64_t T, pages, width;
    int32_t B, heads, G, log_p, window;
    float scale;                    // times log2 e
};

// The requests that a kernel takes and how their keys are cut.
struct Cut {
    float *part_o, *part_ml;        // [item][key head][row][D], [item][key head][row][2]
    float *group_ml;                // as part_ml, of groups of chunks
    int32_t rows0, rows1;           // requests of rows0 < rows <= rows1
    int32_t target;                 // items of a key head that the cut aims at; 0: no cut
    int32_t least, least_full;      // steps of a chunk, at least: with few tiles, with a tile a CU
    int32_t most;                   // items of a key head that there is room for
    int32_t fit;                    // chunks are made to fit c.target, or twice that
    uint32_t *count;                // [tile][key head] parts that are done; then [item][key head] chunks of a
                                    // group; all 0 between calls
};
constexpr int64_t COUNTS = 8192;            // tiles of all key heads that a cut may have
constexpr int64_t GROUP_COUNTS = 32768;     // items
static_assert((COUNTS + GROUP_COUNTS) * sizeof(uint32_t) == SPEAR_KV4_COUNTER_BYTES, "the part that a caller zeroes");

// ------------------------------------------------------------------- items
struct Request {
    int32_t row0;                   // its first row of q
    int32_t fresh, kv;              // its rows and keys
    int32_t tiles, base, steps;     // row tiles; the first step that a row sees; steps from there
};

__device__ __forceinline__ Request request_of(const AttnArgs &a, const Cut &c, int b, int tile_rows)
{
    Request r;
    const int32_t T = (int32_t)a.T, room = (int32_t)(a.width << a.log_p);
    int32_t q0 = a.q_start[b], q1 = a.q_start[b + 1];
    q0 = q0 < 0 ? 0 : (q0 > T ? T : q0);
    q1 = q1 < q0 ? q0 : (q1 > T ? T : q1);
    const int32_t kv = a.kv_len[b];
    r.kv = kv < 0 ? 0 : (kv > room ? room : kv);
    r.row0 = q0;
    r.fresh = q1 - q0;
    const int32_t rows = r.fresh * a.G;
    r.tiles = rows > c.rows0 && rows <= c.rows1 ? (rows + tile_rows - 1) / tile_rows : 0;
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
    int32_t number;                 // of the tile, of all requests
    bool found;
};

__device__ __forceinline__ int32_t bcast(int32_t v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// Sums over the lanes up to this one (16 lanes, then the rows of 16 before).
template <int CTRL, int ROWS>
__device__ __forceinline__ int32_t from_lane(int32_t v)
{
    return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int32_t scan64(int32_t v)
{
    v += from_lane<0x111, 0xF>(v);
    v += from_lane<0x112, 0xF>(v);
    v += from_lane<0x114, 0xF>(v);
    v += from_lane<0x118, 0xF>(v);
    v += from_lane<0x142, 0xA>(v);
    return v + from_lane<0x143, 0xC>(v);
}
__device__ __forceinline__ float total64(float v)
{
    v += __int_as_float(from_lane<0x111, 0xF>(__float_as_int(v)));
    v += __int_as_float(from_lane<0x112, 0xF>(__float_as_int(v)));
    v += __int_as_float(from_lane<0x114, 0xF>(__float_as_int(v)));
    v += __int_as_float(from_lane<0x118, 0xF>(__float_as_int(v)));
    v += __int_as_float(from_lane<0x142, 0xA>(__float_as_int(v)));
    v += __int_as_float(from_lane<0x143, 0xC>(__float_as_int(v)));
    return __int_as_float(bcast(__float_as_int(v), 63));
}

// a / b where it is at most 2^22, and a and b less than 2^25: a reciprocal's product is
// off by less than one.
__device__ __forceinline__ int32_t quotient(int32_t a, int32_t b)
{
    const int32_t q = (int32_t)((float)a * __builtin_amdgcn_rcpf((float)b)), r = a - q * b;
    return q + (r >= b) - (r < 0);
}

// Token and query head of the rows of a tile, from a multiplication: with the tile's
// first row `rem` rows into token `tok`, (rem + i) / G for rem + i < 320 and G <= 64 by
// 2^16 / G, cut, plus one (all of them tried).
struct TileRows {
    int32_t tok, rem, by, G;
    __device__ __forceinline__ TileRows(int32_t first, int32_t G)
        : tok(first / G), rem(first - tok * G), by((int32_t)(65536.f * __builtin_amdgcn_rcpf((float)G)) + 1), G(G)
    {
    }
    __device__ __forceinline__ int32_t token(int32_t i) const { return tok + ((rem + i) * by >> 16); }
    __device__ __forceinline__ int32_t head(int32_t i, int32_t token) const { return rem + i - (token - tok) * G; }
};

// The item (or, by_tile, the tile) number `want`.  Every wave forms the sums over
// all requests, 64 at a time.  A chunk has as many steps as make c.target
// items of a key head, or twice as many; sums are capped at c.most, behind which there is no item.
// A tile whose items do not all lie below c.most (rows that q_start gives to more
// than one request) has none, so that its count of chunks ends where it began.
template <int ROWS>
__device__ Item find_item(const AttnArgs &a, const Cut &c, int32_t want, bool by_tile)
{
    const int lane = threadIdx.x & 63;
    Item it;
    it.found = false;
    it.size = 0x7FFFFFFF;
    int32_t uncut = 0;                                    // steps below which a tile stays whole
    Request mine = {};
    if (lane < a.B)
        mine = request_of(a, c, lane, ROWS);
    if (c.target) {
        float work = 0.f, tiles = 0.f;
        for (int b0 = 0; b0 < a.B; b0 += 64) {
            const int b = b0 + lane;
            if (b < a.B) {
                const Request r = b0 ? request_of(a, c, b, ROWS) : mine;
                work += (float)r.tiles * (float)r.steps;
                tiles += (float)r.tiles;
            }
        }
        float s = ceilf(total64(work) / (float)c.target);
        tiles = total64(tiles);
        const float fill = tiles * (float)a.heads * (float)c.least_full * (1.f / 256.f);
        const int32_t least = fill > (float)c.least_full ? c.least_full : (fill < (float)c.least ? c.least : (int32_t)fill);
        uncut = 2 * least;
        s = s < (float)least ? (float)least : s;
        // A tile has whole chunks, so there are more of them than work / s, and the few
        // behind c.target start when the first have ended.  Somewhat longer ones fit, or
        // there are twice as many (48 requests of 300 to 16000 tokens, 32 heads over 8, 128
        // channels 56.8 -> 52.3 us by the former, 256 channels 103 -> 98 by the latter).
        // Not before the kernel for many rows, where it finds little to do (80 rows of 8
        // requests each 67 -> 69 us), and not for many requests, whose walks cost more than
        // it gives (one key head of 128 channels, requests of 300 to 6000 tokens: 307 of them
        // 35 us with and 31 without, 537 62 and 52; of 256 channels 256 of them 48 and 54,
        // 358 70 and 66).
        // So many tiles as 0.6 of what is aimed at hardly fit, and are cut in half at once
        // (us, counted first / at once: 134 requests of 300 to 16000 tokens, 4 heads of 64
        // 50 / 46, of 128 74 / 70; 67 of 2000 to 6000, 8 heads of 128 56 / 61, 81 78 / 75).
        const float s0 = s, most = ceilf(1.4f * s0);
        for (int k = tiles > 0.6f * (float)c.target ? 7 : 0; c.fit && a.B <= FIT_REQUESTS; k++) {
            float n = 0.f;
            for (int b0 = 0; b0 < a.B; b0 += 64) {
                const int b = b0 + lane;
                if (b < a.B) {
                    const Request r = b0 ? request_of(a, c, b, ROWS) : mine;
                    n += (float)r.tiles * ((float)r.steps <= s || r.steps < uncut ? 1.f : ceilf((float)r.steps / s));
                }
            }
            n = total64(n);
            if (n <= (float)c.target)
                break;
            if (s >= most || k == 7) {
                s = ceilf(0.5f * s0);
                s = s < (float)least ? (float)least : s;
                break;
            }
            s = ceilf(s * n / (float)c.target);
            s = s > most ? most : s;
        }
        it.size = s > 1e9f ? 1000000000 : (int32_t)s;
    }
    int32_t items0 = 0, tiles0 = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        const int b = b0 + lane;
        int32_t chunks = 0, n = 0, tiles = 0;
        Request r = {};
        if (b < a.B) {
            r = b0 ? request_of(a, c, b, ROWS) : mine;
            chunks = r.steps <= it.size || r.steps < uncut ? 1 : quotient(r.steps + it.size - 1, it.size);
            tiles = r.tiles < c.most ? r.tiles : c.most;
            const int64_t all = (int64_t)r.tiles * chunks;
            n = all < c.most ? (int32_t)all : c.most;
        }
        // held below 2^31 by the cap (64 * most < 2^31)
        const int32_t ni = scan64(n), ti = scan64(tiles);
        const int32_t end = by_tile ? tiles0 + ti : items0 + ni, len = by_tile ? tiles : n;
        const uint64_t hit = __ballot(end > want && end - len <= want);
        if (hit) {
            const int src = __builtin_ctzll(hit);
            const int32_t first_item = bcast(items0 + ni - n, src), first_tile = bcast(tiles0 + ti - tiles, src);
            it.r.row0 = bcast(r.row0, src);
            it.r.fresh = bcast(r.fresh, src);
            it.r.kv = bcast(r.kv, src);
            it.r.tiles = bcast(r.tiles, src);
            it.r.base = bcast(r.base, src);
            it.r.steps = bcast(r.steps, src);
            it.chunks = bcast(chunks, src);
            it.size = (it.r.steps + it.chunks - 1) / it.chunks;
            it.tile = by_tile ? want - first_tile : (it.chunks < 2 ? want - first_item : quotient(want - first_item, it.chunks));
            it.chunk = by_tile ? 0 : want - first_item - it.tile * it.chunks;
            it.item = first_item + it.tile * it.chunks;
            it.number = first_tile + it.tile;
            it.b = b0 + src;
            it.found = it.chunks < 2 || (it.item <= c.most - it.chunks && (int64_t)(it.number + 1) * a.heads <= COUNTS);
            static_assert(COUNTS + 2 * FEW_ITEMS + 18 * SPEAR_MAX_HEADS <= GROUP_COUNTS, "c.most items of all key heads");
            return it;
        }
        items0 += bcast(ni, 63);
        tiles0 += bcast(ti, 63);
        items0 = items0 < c.most ? items0 : c.most;
        tiles0 = tiles0 < c.most ? tiles0 : c.most;
    }
    return it;
}

// --------------------------------------------------------------- few rows
// How the D channels of a token's head lie in the operands of the matrix
// instructions: NC chunks of CW channels, of which lane group g (16 lanes) holds
// CW / 4 consecutive ones, eight to a depth step of the instruction.  A group's
// codes are W words side by side, and all of them belong to one block; at D = 96
// and 192, to the blocks of the group's first and last word.  (There, three chunks
// of 32 or 64 would have a block each, but loads of 4 or 8 bytes: 48 requests of up
// to 16000 tokens, 32 heads over 8, 99 -> 40 and 111 -> 86 us.)
template <int D>
struct Lay {
    static constexpr int CW = D % 128 == 0 ? 128 : D;
    static constexpr int NC = D / CW;
    static constexpr int W = CW / 32;
    static constexpr bool TWO = W % 3 == 0;
    static constexpr int NS = TWO ? 2 : NC;  // blocks of a group
    static __device__ __forceinline__ int block(int s, int g) { return (g * (CW / 4) + s * (TWO ? CW / 4 - 8 : CW)) / 32; }
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
#pragma unroll
        for (int w = 0; w < W; w++)
            r.w[w] = reinterpret_cast<const uint32_t *>(p)[w];
    return r;
}

// A step's codes and scales of one of K and V in the lanes that load them: lane
// (R = lane % 16, g = lane / 16) has the tokens 4R .. 4R + 3 of the step, which
// lie in one page, and a word with their four scales.
template <int D>
struct Part {
    Words<Lay<D>::W> c[Lay<D>::NC][4];
    uint32_t s[Lay<D>::NS];

    // the four scales of word w of chunk n
    __device__ __forceinline__ uint32_t scales(int n, int w, int g) const
    {
        if (!Lay<D>::TWO)
            return s[n];
        const int third = 3 * w / Lay<D>::W;
        return third == 0 ? s[0] : (third == 2 || g % 2 ? s[Lay<D>::NS - 1] : s[0]);
    }
    // token i's values are finite: its scales are 1
    __device__ __forceinline__ void tame(int i)
    {
#pragma unroll
        for (int n = 0; n < Lay<D>::NS; n++)
            s[n] = (s[n] & ~(255u << (8 * i))) | (127u << (8 * i));
    }
};

template <int D>
__device__ __forceinline__ void load_part(Part<D> &p, const uint8_t *codes, const uint8_t *scales, int64_t ph, int32_t off,
                                          int log_p, int g)
{
    using L = Lay<D>;
    const uint8_t *c = codes + ((ph << log_p) + off) * (D / 2) + g * (L::CW / 8);
    if (D == 64) {
        // a group has a token's 32 bytes at first (turn_part): four loads of 8 bytes a lane
        // take 39 us where these take 32 (48 requests of up to 16000 tokens, 32 heads over 8)
        c = codes + ((ph << log_p) + off + g) * 32;
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const u32x4 v = ld16(c + 8 * i);
            p.c[0][i].w[0] = v[0];
            p.c[0][i].w[1 % L::W] = v[1];
            p.c[0][i + 1].w[0] = v[2];
            p.c[0][i + 1].w[1 % L::W] = v[3];
        }
    } else
#pragma unroll
    for (int n = 0; n < L::NC; n++)
#pragma unroll
        for (int i = 0; i < 4; i++)
            p.c[n][i] = load_words<L::W>(c + i * (D / 2) + n * (L::CW / 2));
#pragma unroll
    for (int n = 0; n < L::NS; n++)
        p.s[n] = *reinterpret_cast<const uint32_t *>(scales + ((ph * (D / 32) + L::block(n, g)) << log_p) + off);
}

// D = 64: from group g's token 4R + g, pieces c[0][0 .. 3] of its channels, to the
// tokens 4R .. 4R + 3, channels 16 g .. 16 g + 15 of each.
__device__ __forceinline__ void swap_halves(uint32_t &a, uint32_t &b)
{
    auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap_rows(uint32_t &a, uint32_t &b)
{
    auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
template <int D>
__device__ __forceinline__ void turn_part(Part<D> &p)
{
    if (D != 64)
        return;
#pragma unroll
    for (int w = 0; w < Lay<D>::W; w++) {
        swap_halves(p.c[0][0].w[w], p.c[0][2].w[w]);
        swap_halves(p.c[0][1].w[w], p.c[0][3].w[w]);
        swap_rows(p.c[0][0].w[w], p.c[0][1].w[w]);
        swap_rows(p.c[0][2].w[w], p.c[0][3].w[w]);
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

// LDS written by this wave is read back by its other lanes: the order of the
// wave's own accesses suffices, the compiler only has to keep it.
__device__ __forceinline__ void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Partial results pass from workgroup to workgroup within a launch: they are
// written through to where every XCD reads, and a workgroup counts itself as done
// only when its stores have returned.  (An agent-scope release would write back
// the whole L2 of the XCD for each.)
__device__ __forceinline__ void store_far(float *p, float x, float y)
{
    const uint64_t v = (uint64_t)__float_as_uint(y) << 32 | __float_as_uint(x);
    __hip_atomic_store(reinterpret_cast<uint64_t *>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 load_far(const float *p)
{
    const uint64_t v = __hip_atomic_load(reinterpret_cast<uint64_t *>(const_cast<float *>(p)), __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
    return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}
__device__ __forceinline__ void stores_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// A row's maximum m is that of its products z = q . k.  Its probabilities are held as
//   2^(scale z - e), e = scale m rounded, by one fma each (scale with log2 e in it),
// and from |e| = FAR on, where e has no bits behind the point (and may lie beyond fp32),
//   2^(scale (z - m)).
constexpr float FAR = 0x1p24f;

// Rounded by itself: never the product of an fma.
__device__ __forceinline__ float scaled(float m, float scale)
{
#pragma clang fp contract(off)
    return m * scale;
}
__device__ __forceinline__ bool is_far(float m, float e) { return (__builtin_fabsf(e) >= FAR) & (__builtin_fabsf(m) < INFINITY); }

// What probabilities held for the maximum m weigh where up >= m is the maximum: where
// neither is far, and where one may be.
__device__ __forceinline__ float part_weight(float m, float up, float scale)
{
    return __builtin_amdgcn_exp2f(scaled(m, scale) - scaled(up, scale));
}
__device__ __forceinline__ float far_weight(float m, float up, float scale)
{
    const float e = scaled(m, scale), e_up = scaled(up, scale);
    const float d = (e - e_up) + ((is_far(m, e) ? __builtin_fmaf(m, scale, -e) : 0.f) -
                                  (is_far(up, e_up) ? __builtin_fmaf(up, scale, -e_up) : 0.f));
    return __builtin_amdgcn_exp2f(d > -INFINITY ? d : (m - up) * scale);
}
// The sum of a part whose maximum is far has its sign set.
__device__ __forceinline__ float marked(float l, float m, float scale) { return is_far(m, scaled(m, scale)) ? -l : l; }

// The part (m2, l2, v) joined to (m, l, sum) where a maximum may be far.
__device__ __forceinline__ void join_far(float &m, float &l, f32x4 &sum, float m2, float l2, f32x4 v, float scale)
{
    const float up = fmaxf(m, m2), ref = up == -INFINITY ? 0.f : up;
    const float f = far_weight(m, ref, scale), w = far_weight(m2, ref, scale);
    l = marked(f * __builtin_fabsf(l) + w * __builtin_fabsf(l2), up, scale);
    sum = f * sum + w * v;
    m = up;
}

// A row's maximum as it goes over the keys (of the lane's row, in all lanes that share it).
struct RowMax {
    float m = -INFINITY;
    float least = -INFINITY;        // m; -INFINITY where it is far: products then lose m first
    float add = 0.f;                // of the fma that makes products exponents

    __device__ __forceinline__ bool takes(float top) const { return __any(top > least); }
    // Products z of which `top` is the row's largest: what was held so far is to be
    // multiplied by the result.
    template <class V, int N>
    __device__ __forceinline__ float take(float top, float scale, V (&z)[N])
    {
        const float up = fmaxf(m, top), e = scaled(up, scale);
        float f = part_weight(m, up, scale);
        const bool now = is_far(up, e), was = least < m;
        add = up == -INFINITY ? 0.f : -e;
        least = up;
        if (__builtin_expect(__any(now | was), 0)) {
            f = far_weight(m, up, scale);
            add = now ? 0.f : add;
            least = now ? -INFINITY : up;
            const float off = now ? up : 0.f;
#pragma unroll
            for (int i = 0; i < N; i++)
                z[i] -= off;
        }
        f = m == up ? 1.f : f;
        m = up;
        return f;
    }
    __device__ __forceinline__ float marked_sum(float l) const { return least < m ? -l : l; }
};

// Four channels from c on of row i of a tile, and with c == 0 its lse.
template <int D>
__device__ __forceinline__ void store_out(const AttnArgs &a, const Item &it, int head, const TileRows &rows, int i, int c, f32x4 sum,
                                          float m, float l)
{
    const int32_t tok = rows.token(i);
    const int64_t hrow = (it.r.row0 + tok) * ((int64_t)a.heads * a.G) + head * a.G + rows.head(i, tok);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<uint2 *>(a.y + hrow * D + c) =
        make_uint2(pair_bf16(sum[0] * inv, sum[1] * inv), pair_bf16(sum[2] * inv, sum[3] * inv));
    if (c == 0 && a.lse) {
        const float e = scaled(m, a.scale), log2_l = __log2f(l);       // (e beyond fp32: without log2 e)
        a.lse[hrow] = l == 0.f ? -INFINITY : (__builtin_fabsf(e) < INFINITY ? (e + log2_l) * LN2 : m * (a.scale * LN2) + log2_l * LN2);
    }
}

// One tile of 16 rows and a chunk of its keys:
//   m' = max(m, max_j s_j), l' = l 2^(m - m') + sum_j 2^(s_j - m'), o likewise,
//   s = scale log2(e) q . k, over 64 keys a wave at a time, the waves' (m, l, o) joined
//   in LDS at the end.
// The cache is read once, a step ahead, straight into registers: K's codes become
// the first product's operand where they were loaded, V's pass through LDS of the
// wave's own, so that no wave waits for another inside the loop.  Requests of one
// token are bound by the cache's bytes (48 requests of up to 16000 tokens, 32 heads
// of 128 over 8: 207 MB in 44 us, 4.7 TB/s), long ones
// cut over the whole chip also by what comes before and after (two of 131000 tokens
// 136 MB in 38 us, of which the plan, the first page and the first keys take 5 and the
// join 8).  Tiles of many rows on few keys are bound by the instructions of a wave: it
// issues a vector one in 8 cycles at most, 430 a step at 128 channels and 730 at 256,
// 3 us (24 requests of up to 150 tokens under a window of 1500, 10 heads of 256 over
// 2: 35 us for 7 steps in a row).
//
// Matrix instructions, with g the group of a lane and n its place in the group:
//   S^T [key][row] = K Q^T  lane: row n, keys 16 g + 4 r + i in acc[i][r]
//   O^T [channel][row] += V^T P^T  lane: row n, channels 16 dt + 4 g + r in o[dt][r]
// Instruction i of the first takes the keys 4R + i, R = 0 .. 15, so that what a
// lane gets of S is what it has to bring of P to the second, whose depth slots
// (g, j) stand for the keys 16 g + 4 (j % 4) + 2 u + j / 4.  V goes through LDS,
// as bf16, to be read column by column.
template <int D>
__global__ __launch_bounds__(64 * FEW_WAVES, D <= 128 ? 3 : 2) void few_rows_kernel(const AttnArgs a, const Cut cut)
{
    using L = Lay<D>;
    constexpr int DT = D / 16, NS = L::NC * L::W;
    constexpr int V_BYTES = 32 * L::ROW;
    static_assert(V_BYTES >= 16 * D * 4, "the waves' outputs are joined in the same LDS");
    __shared__ __attribute__((aligned(16))) uint8_t s_v[FEW_WAVES][V_BYTES];
    __shared__ float s_ml[FEW_WAVES][FEW_ROWS][2];
    __shared__ bool s_last;

    const int head = blockIdx.x % a.heads;
    const Item it = find_item<FEW_ROWS>(a, cut, (int32_t)(blockIdx.x / a.heads), false);
    if (!it.found)
        return;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, n = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int b = it.b, G = a.G, log_p = a.log_p;
    const int64_t page_mask = (1 << log_p) - 1;

    // this lane's row and the positions it sees, [first, last]
    const TileRows tile_rows(it.tile * FEW_ROWS, G);
    const int tok = tile_rows.token(n), qh = tile_rows.head(n, tok);
    const bool real = tok < it.r.fresh;
    const int pos0 = it.r.kv - it.r.fresh;
    const int last = real ? pos0 + tok : -1;
    const int first = a.window && last - a.window + 1 > 0 ? last - a.window + 1 : 0;
    // ... and what the tile's rows see together
    const int tok0 = tile_rows.tok;
    int tok1 = tile_rows.token(FEW_ROWS - 1);
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
        const uint16_t *qp = a.q + (int64_t)(it.r.row0 + tok) * a.qs + (int64_t)(head * G + qh) * D;
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
    RowMax best;
    float l = 0.f;

    Part<D> kp, vp;
    const int32_t *table = a.table + (int64_t)b * a.width;
    // Page and place of this lane's four tokens of a step.  Steps behind the last
    // read the first page of the cache, and nothing of it is used.  What is loaded is
    // first touched a step later: a use of it here would wait for it.
    auto in_step = [&](int step) { return (step < hi) & (step * STEP + 4 * n < it.r.kv); };
    auto page_of = [&](int step) { return (uint32_t)table[in_step(step) ? (step * STEP + 4 * n) >> log_p : 0]; };
    const uint32_t last_page = (uint32_t)a.pages - 1;
    bool lost;
    int64_t ph;
    int32_t off;
    auto place = [&](int step, uint32_t page) {
        const bool in = in_step(step);
        lost = in & (page > last_page);
        ph = (int64_t)((in & !lost) ? page : 0u) * a.heads + head;
        off = (int32_t)((step * STEP + 4 * n) & page_mask);
    };
    // Loads return in the order they are issued, and the waits in the loop are for the
    // order there: page, K, V.
    place(lo + wave, page_of(lo + wave));
    uint32_t page_next = page_of(lo + wave + FEW_WAVES);
    __builtin_amdgcn_sched_barrier(0);
    load_part<D>(kp, a.k_codes, a.k_scales, ph, off, log_p, g);
    __builtin_amdgcn_sched_barrier(0);
    load_part<D>(vp, a.v_codes, a.v_scales, ph, off, log_p, g);
    __builtin_amdgcn_sched_barrier(0);

    for (int step = lo + wave; step < hi; step += FEW_WAVES) {
        const int key0 = step * STEP;
        const uint32_t lost16 = (uint32_t)(__ballot(lost) & 0xFFFF);       // bit R: the keys 4R .. 4R + 3
        f32x4 acc[4];
        turn_part<D>(kp);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < L::NC; c++)
#pragma unroll
                for (int w = 0; w < L::W; w++)
                    acc[i] = mfma16(kv4_bf16(kp.c[c][i].w[w], scale_of(kp.scales(c, w, g), i)), qf[c * L::W + w], acc[i]);
        }
        // the next step's keys
        const bool lost_now = lost;
        place(step + FEW_WAVES, page_next);
        page_next = page_of(step + 2 * FEW_WAVES);
        __builtin_amdgcn_sched_barrier(0);
        load_part<D>(kp, a.k_codes, a.k_scales, ph, off, log_p, g);
        __builtin_amdgcn_sched_barrier(0);

        const bool edge = key0 < all0 || key0 + STEP - 1 > all1 || lost16 != 0;
        float top = -INFINITY;
        if (edge) {
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const int key = key0 + 16 * g + 4 * r + i;
                    const bool sees = key >= first && key <= last && !(lost16 >> (4 * g + r) & 1);
                    acc[i][r] = sees ? acc[i][r] : -INFINITY;
                    top = fmaxf(top, acc[i][r]);
                }
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int r = 0; r < 4; r++)
                    top = fmaxf(top, acc[i][r]);
        }
        top = max_over_groups(top);
        if (best.takes(top)) {
            const float f = best.take(top, a.scale, acc);
            l *= f;
#pragma unroll
            for (int d = 0; d < DT; d++)
                o[d] *= f;
        }
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int r = 0; r < 4; r++) {
                acc[i][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][r], a.scale, best.add));
                l += acc[i][r];
            }

        // keys that no row of the tile sees hold anything: their V is made finite, which
        // probabilities of 0 leave out
        if (key0 < seen0 || key0 + STEP > seen1 || lost16 != 0) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int key = key0 + 4 * n + i;
                if (lost_now || key < seen0 || key >= seen1)
                    vp.tame(i);
            }
        }
        // A block of NaN counts for the rows that see its key only; a zero
        // probability would carry it to the others.
        bool nan_here = false;
#pragma unroll
        for (int c = 0; c < L::NS; c++) {
            const uint32_t x = ~vp.s[c];
            nan_here |= ((x - 0x01010101u) & ~x & 0x80808080u) != 0;
        }
        if (__any(nan_here)) {
#pragma unroll
            for (int c = 0; c < L::NS; c++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const bool mine = ((vp.s[c] >> (8 * i)) & 255u) == 255u;
                    uint64_t who = __ballot(mine);
                    while (who) {
                        const int src = __builtin_ctzll(who);
                        who &= who - 1;
                        const int key = key0 + 4 * (src & 15) + i, block = L::block(c, src >> 4);
                        const float add = key >= first && key <= last ? __builtin_nanf("") : 0.f;
#pragma unroll
                        for (int d = 0; d < DT; d++)
                            if (d / 2 == block)
                                o[d] += add;
                    }
                    if (mine)
                        vp.s[c] = (vp.s[c] & ~(255u << (8 * i))) | (127u << (8 * i));
                }
        }

        uint8_t *sv = s_v[wave];
        turn_part<D>(vp);
#pragma unroll
        for (int u = 0; u < 2; u++) {
            wave_order();
#pragma unroll
            for (int e = 0; e < 2; e++)
#pragma unroll
                for (int c = 0; c < L::NC; c++)
#pragma unroll
                    for (int w = 0; w < L::W; w++)
                        *reinterpret_cast<u32x4 *>(sv + (e * 16 + n) * L::ROW + 2 * (c * L::CW + g * (L::CW / 4)) + 16 * w) =
                            kv4_bf16(vp.c[c][2 * u + e].w[w], scale_of(vp.scales(c, w, g), 2 * u + e));
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
        __builtin_amdgcn_sched_barrier(0);
        load_part<D>(vp, a.v_codes, a.v_scales, ph, off, log_p, g);
        __builtin_amdgcn_sched_barrier(0);
    }

    // ---- the four waves' parts of the chunk
    l = sum_over_groups(l);
    wave_order();
    float *so = reinterpret_cast<float *>(s_v[wave]);                      // [row][D]
#pragma unroll
    for (int d = 0; d < DT; d++)
        *reinterpret_cast<f32x4 *>(so + n * D + 16 * d + 4 * g) = o[d];
    if (g == 0) {
        s_ml[wave][n][0] = best.m;
        s_ml[wave][n][1] = best.marked_sum(l);
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
        float ll = 0.f, least = 0.f;
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < FEW_WAVES; w++)
            least = fminf(least, s_ml[w][r][1]);
#pragma unroll
        for (int w = 0; w < FEW_WAVES; w++) {
            const float f = part_weight(s_ml[w][r][0], ref, a.scale);
            ll += f * s_ml[w][r][1];
            sum += f * *reinterpret_cast<const f32x4 *>(reinterpret_cast<const float *>(s_v[w]) + r * D + c);
        }
        if (__builtin_expect(least < 0.f, 0)) {
            mm = -INFINITY;
            ll = 0.f;
            sum = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma nounroll
            for (int w = 0; w < FEW_WAVES; w++)
                join_far(mm, ll, sum, s_ml[w][r][0], s_ml[w][r][1],
                         *reinterpret_cast<const f32x4 *>(reinterpret_cast<const float *>(s_v[w]) + r * D + c), a.scale);
        }
        if (it.chunks > 1) {
            const int64_t p = ((int64_t)(it.item + it.chunk) * a.heads + head) * FEW_ROWS + r;
            store_far(cut.part_o + p * D + c, sum[0], sum[1]);
            store_far(cut.part_o + p * D + c + 2, sum[2], sum[3]);
            if (c == 0)
                store_far(cut.part_ml + 2 * p, mm, ll);
        } else
            store_out<D>(a, it, head, tile_rows, r, c, sum, mm, __builtin_fabsf(ll));
    }
    if (it.chunks < 2)
        return;

    // ---- the last workgroup to finish joins the chunks, in their order.  A CU takes
    // in some 40 GB/s of them, so many are joined in two steps, by groups of about as
    // many as there are groups (92 chunks: 15 -> 6 us behind the last).
    const int real_rows = rows < FEW_ROWS ? rows : FEW_ROWS, work = real_rows * (D / 4);
    int sharers = 1;                                      // threads that share a row's four channels, a chunk each in turn
    while (2 * sharers * work <= 64 * FEW_WAVES)
        sharers *= 2;
    const int64_t next = (int64_t)a.heads * FEW_ROWS;
    float *s_part = reinterpret_cast<float *>(s_v);                        // [thread][6]
    auto is_last = [&](uint32_t *count, int n) {
        stores_done();
        __syncthreads();
        if (tid == 0) {
            s_last = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)n - 1;
            if (s_last)
                __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        return s_last;
    };
    // n parts, the first of `item`, `by` items apart; into the first of them, or y
    auto join = [&](int item, int by, int n, const float *part_ml, bool to_y) {
        const int64_t p0 = ((int64_t)item * a.heads + head) * FEW_ROWS;
        for (int x0 = 0; x0 < work; x0 += 64 * FEW_WAVES) {
            const int x = x0 + tid % (64 * FEW_WAVES / sharers), sh = tid / (64 * FEW_WAVES / sharers);
            const bool in = x < work;
            const int r = in ? x / (D / 4) : 0, c = in ? 4 * (x % (D / 4)) : 0;
            float mm = -INFINITY, ll = 0.f;
            f32x4 sum = {0.f, 0.f, 0.f, 0.f};
            float least = 0.f;
            for (int i0 = sh; i0 < n; i0 += JB * sharers) {
                float2 ml[JB], lo2[JB], hi2[JB];
#pragma unroll
                for (int j = 0; j < JB; j++) {
                    const int i = i0 + j * sharers < n ? i0 + j * sharers : i0;
                    const int64_t p = p0 + (int64_t)i * by * next + r;
                    ml[j] = load_far(part_ml + 2 * p);
                    lo2[j] = load_far(cut.part_o + p * D + c);
                    hi2[j] = load_far(cut.part_o + p * D + c + 2);
                }
                float up = mm;
#pragma unroll
                for (int j = 0; j < JB; j++) {
                    up = fmaxf(up, ml[j].x);
                    least = fminf(least, ml[j].y);
                }
                const float ref = up == -INFINITY ? 0.f : up, f = part_weight(mm, ref, a.scale);
                ll *= f;
                sum *= f;
                mm = up;
#pragma unroll
                for (int j = 0; j < JB; j++) {
                    // (a part whose weight is 0 counts too: it may hold a NaN)
                    const float w = part_weight(ml[j].x, ref, a.scale);
                    if (i0 + j * sharers < n) {
                        ll += w * ml[j].y;
                        sum += w * f32x4{lo2[j].x, lo2[j].y, hi2[j].x, hi2[j].y};
                    }
                }
            }
            if (__builtin_expect(least < 0.f, 0)) {
                mm = -INFINITY;
                ll = 0.f;
                sum = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma nounroll
                for (int i = sh; i < n; i += sharers) {
                    const int64_t p = p0 + (int64_t)i * by * next + r;
                    const float2 ml = load_far(part_ml + 2 * p), lo2 = load_far(cut.part_o + p * D + c), hi2 = load_far(cut.part_o + p * D + c + 2);
                    join_far(mm, ll, sum, ml.x, ml.y, f32x4{lo2.x, lo2.y, hi2.x, hi2.y}, a.scale);
                }
            }
            if (sharers > 1) {
                __syncthreads();
                s_part[tid * 6] = mm;
                s_part[tid * 6 + 1] = ll;
#pragma unroll
                for (int e = 0; e < 4; e++)
                    s_part[tid * 6 + 2 + e] = sum[e];
                __syncthreads();
                if (sh == 0)
                    for (int j = 1; j < sharers; j++) {
                        const float *o2 = s_part + (tid + j * (64 * FEW_WAVES / sharers)) * 6;
                        const float up = fmaxf(mm, o2[0]), ref = up == -INFINITY ? 0.f : up;
                        if (__builtin_expect(fminf(ll, o2[1]) < 0.f, 0)) {
                            join_far(mm, ll, sum, o2[0], o2[1], f32x4{o2[2], o2[3], o2[4], o2[5]}, a.scale);
                            continue;
                        }
                        const float f = part_weight(mm, ref, a.scale), w = part_weight(o2[0], ref, a.scale);
                        mm = up;
                        ll = f * ll + w * o2[1];
                        sum = f * sum + w * f32x4{o2[2], o2[3], o2[4], o2[5]};
                    }
            }
            if (in && sh == 0) {
                if (to_y)
                    store_out<D>(a, it, head, tile_rows, r, c, sum, mm, __builtin_fabsf(ll));
                else {
                    // a row's m and l, which its other threads may still read, to a place of
                    // their own
                    store_far(cut.part_o + (p0 + r) * D + c, sum[0], sum[1]);
                    store_far(cut.part_o + (p0 + r) * D + c + 2, sum[2], sum[3]);
                    if (c == 0)
                        store_far(cut.group_ml + 2 * (p0 + r), mm, ll);
                }
            }
        }
    };
    int size = it.chunks, groups = 1;
    if (it.chunks > 2 * JB) {
        size = (int)ceilf(__builtin_sqrtf((float)it.chunks));
        groups = (it.chunks + size - 1) / size;
        const int first_chunk = it.chunk / size * size, n = it.chunks - first_chunk < size ? it.chunks - first_chunk : size;
        const int item = it.item + first_chunk;
        if (!is_last(cut.count + COUNTS + (int64_t)item * a.heads + head, n))
            return;
        join(item, 1, n, cut.part_ml, false);
    }
    if (is_last(cut.count + (int64_t)it.number * a.heads + head, groups > 1 ? groups : it.chunks))
        join(it.item, groups > 1 ? size : 1, groups > 1 ? groups : it.chunks, groups > 1 ? cut.group_ml : cut.part_ml, true);
}

// -------------------------------------------------------------- many rows
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// A matrix instruction of 32 x 32 needs 12 wait states before a vector instruction
// reads its result.  Where branches lie between, the compiler has counted the longer
// path only (9 states at D = 192), so they are spent here.
__device__ __forceinline__ void results_there(f32x16 (&z)[1]) { asm volatile("s_nop 11" : "+v"(z[0])); }
__device__ __forceinline__ void results_there(f32x16 (&z)[2]) { asm volatile("s_nop 11" : "+v"(z[0]), "+v"(z[1])); }

__device__ __forceinline__ float max_over_halves(float v)
{
    auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}

// A workgroup's W waves take 32 rows each and share the keys: a step's K and V go
// to LDS as bf16 once, two steps in turn, while the codes of the one after are on
// their way.  With h the half of a lane (lane / 32) and n its place in it:
//   S^T [key][row] = K Q^T          lane: row n, keys 8 (r / 4) + 4 h + r % 4 in s[r]
//   O^T [channel][row] += V^T P^T   lane: row n, channels 8 (r / 4) + 4 h + r % 4
// so that P stays where S was, as in the kernel for few rows.  P is one bf16
// here (off by 2^-8 of its size at most, as y is by its own rounding, and the sum goes over
// many of them): a second term would make half as many matrix instructions more.
// 8192 tokens of a prompt on 16384 keys, 32 heads of 128 over 8: 1.65 TFLOP in 1.75 ms,
// 941 TFLOP/s.  The waves meet at each step, so its matrix instructions (two fifths of
// the time), exponentials and LDS reads hardly overlap; probabilities without
// exponentials take 8 % less, steps without reads of K 13 %, of V 10 %, without the
// staging 25 %.
template <int D, int W>
struct Tiles {
    static constexpr int NB = D / 32, KROW = 2 * D + 16, VROW = D == 96 ? 2 * D : 2 * D + 64;
    // Keys of a step: heads of more than 128 channels take half as many, so that two
    // workgroups fit a CU.
    static constexpr int KT = D <= 128 ? 2 : 1, SK = 32 * KT;
    static constexpr int UNITS = SK * NB, U = (2 * UNITS + 64 * W - 1) / (64 * W);
    static constexpr int BUF = SK * (KROW + VROW);
};

template <int D, int W>
__global__ __launch_bounds__(64 * W, D > 192 ? 1 : 2) void many_rows_kernel(const AttnArgs a, const Cut cut)
{
    using L = Tiles<D, W>;
    constexpr int DT = D / 32, KS = D / 16, ROWS = 32 * W, KT = L::KT, SK = L::SK;
    __shared__ __attribute__((aligned(16))) uint8_t s_kv[2 * L::BUF];      // two buffers of K rows, then V rows
    __shared__ int32_t s_flag[5][2];       // step + 1 if a page of its keys is gone; ... if its V has a block of NaN

    const int head = blockIdx.x % a.heads;
    const Item it = find_item<ROWS>(a, cut, (int32_t)(blockIdx.x / a.heads), false);
    if (!it.found)
        return;
    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, n = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = a.G, log_p = a.log_p;
    const int page_mask = (1 << log_p) - 1;
    const int pos0 = it.r.kv - it.r.fresh, rows = it.r.fresh * G;
    const int32_t *table = a.table + (int64_t)it.b * a.width;
    const int first_row = it.tile * ROWS;
    const TileRows tile_rows(first_row, G);

    // what the rows from r0 up to r1 see together: [s0, s1), and each of them: [e0, e1]
    auto range = [&](int r0, int r1, int &s0, int &s1, int &e0, int &e1) {
        r1 = r1 < rows ? r1 : rows;
        const int t0 = tile_rows.token(r0 - first_row), t1 = tile_rows.token(r1 - 1 - first_row);
        s0 = a.window && pos0 + t0 - a.window + 1 > 0 ? pos0 + t0 - a.window + 1 : 0;
        s1 = r0 < r1 ? pos0 + t1 + 1 : 0;
        e0 = a.window && pos0 + t1 - a.window + 1 > 0 ? pos0 + t1 - a.window + 1 : 0;
        e1 = pos0 + t0;
    };
    int seen0, seen1, x0, x1, mine0, mine1, all0, all1;
    range(it.tile * ROWS, it.tile * ROWS + ROWS, seen0, seen1, x0, x1);
    const int row0 = it.tile * ROWS + 32 * wave, row = row0 + n;
    range(row0, row0 + 32, mine0, mine1, all0, all1);

    int lo = it.r.base + it.chunk * (it.chunks > 1 ? it.size : 0), hi = it.r.base + it.r.steps;
    if (it.chunks > 1 && lo + it.size < hi)
        hi = lo + it.size;
    // from here on in steps of SK keys
    lo *= STEP / SK;
    hi *= STEP / SK;
    lo = lo > seen0 / SK ? lo : seen0 / SK;
    const int hi_seen = seen1 > 0 ? (seen1 + SK - 1) / SK : 0;
    hi = hi < hi_seen ? hi : hi_seen;

    u32x4 qf[KS];
    const int tok = tile_rows.token(row - first_row);
    const int last = row < rows ? pos0 + tok : -1;
    const int first = a.window && last - a.window + 1 > 0 ? last - a.window + 1 : 0;
    {
        const uint16_t *qp = a.q + (int64_t)(it.r.row0 + tok) * a.qs + (int64_t)(head * G + tile_rows.head(row - first_row, tok)) * D + 8 * h;
#pragma unroll
        for (int s = 0; s < KS; s++)
            qf[s] = row < rows ? ld16(qp + 16 * s) : zero4();
    }
    f32x16 o[DT];
    RowMax best;
    float l = 0.f;
#pragma unroll
    for (int d = 0; d < DT; d++)
#pragma unroll
        for (int r = 0; r < 16; r++)
            o[d][r] = 0.f;

    // ---- codes on their way: unit u is a block of 32 channels of a key, of K below
    // UNITS and of V from there on, a wave all of the one or the other
    u32x4 code[L::U];
    uint32_t scales[L::U], page[L::U];
    bool gone[L::U];
    const uint32_t code_page = (uint32_t)a.heads * (D / 2) << log_p, scale_page = (uint32_t)a.heads * L::NB << log_p;
    const uint32_t last_page = (uint32_t)a.pages - 1;
    auto is_v = [&](int i) { return i * 64 * W + 64 * wave >= L::UNITS; };
    auto is_unit = [&](int i) { return 2 * L::UNITS % (64 * W) == 0 || i * 64 * W + 64 * wave < 2 * L::UNITS; };
    auto unit = [&](int i) { return i * 64 * W + tid - (is_v(i) ? L::UNITS : 0); };
    // What is loaded is first touched a step later: a use of it here would wait for it.
    auto real_key = [&](int step, int i) { return (step < hi) & (step * SK + unit(i) / L::NB < it.r.kv); };
    auto find_pages = [&](int step) {
#pragma unroll
        for (int i = 0; i < L::U; i++)
            page[i] = (uint32_t)table[real_key(step, i) ? (step * SK + unit(i) / L::NB) >> log_p : 0];
    };
    auto load = [&](int step) {
#pragma unroll
        for (int i = 0; i < L::U; i++)
            if (is_unit(i)) {
                const int blk = unit(i) % L::NB;
                const uint32_t off = (uint32_t)(step * SK + unit(i) / L::NB) & page_mask;
                const bool in = real_key(step, i);
                gone[i] = in & (page[i] > last_page);
                const uint32_t p = (in & !gone[i]) ? page[i] : 0u;
                code[i] = ld16((is_v(i) ? a.v_codes : a.k_codes) + ((uint64_t)p * code_page +
                               ((((uint32_t)head << log_p) + off) * (D / 2) + 16 * blk)));
                // the scales of four tokens, of which key % 4 is this unit's
                scales[i] = *reinterpret_cast<const uint32_t *>((is_v(i) ? a.v_scales : a.k_scales) +
                                (uint64_t)p * scale_page + ((((uint32_t)head * L::NB + blk) << log_p) + (off & ~3u)));
            }
    };
    // No branch: the stores are spread between matrix instructions.
    auto store = [&](int step) {
#pragma unroll
        for (int i = 0; i < L::U; i++)
            if (is_unit(i)) {
                const int key = unit(i) / L::NB, blk = unit(i) % L::NB, at = step * SK + key;
                const uint32_t byte = (scales[i] >> (8 * (key & 3))) & 255u;
                // keys that no row of the tile sees hold anything: their V is made finite,
                // which probabilities of 0 leave out.  A block of NaN in V is put in by
                // hand, for the rows that see it
                const bool seen = (at >= seen0) & (at < seen1) & !gone[i], nan = seen & (byte == 255u);
                const bool clear = is_v(i) & (!seen | nan), note = is_v(i) ? nan : gone[i];
                s_flag[note ? step & 3 : 4][is_v(i)] = step + 1;
                const float sc = kv4_scale(clear ? 127u : byte);
                // rows of V that start in the same banks take their words in another order
                const int turn = is_v(i) ? key & 1 : 0;
                uint8_t *p = s_kv + (step & 1) * L::BUF + (is_v(i) ? SK * L::KROW + key * L::VROW : key * L::KROW) + 64 * blk;
#pragma unroll
                for (int w = 0; w < 4; w++) {
                    const uint32_t c = turn ? code[i][w ^ 1] : code[i][w];
                    *reinterpret_cast<u32x4 *>(p + ((16 * w) ^ (16 * turn))) = kv4_bf16(c, sc);
                }
            }
    };
    auto scores = [&](int step, f32x16 (&z)[KT]) {
        const uint8_t *sk = s_kv + (step & 1) * L::BUF + n * L::KROW + 16 * h;
#pragma unroll
        for (int kt = 0; kt < KT; kt++) {
#pragma unroll
            for (int r = 0; r < 16; r++)
                z[kt][r] = 0.f;
#pragma unroll
            for (int c = 0; c < KS; c++)
                z[kt] = mfma32(ld16(sk + 32 * kt * L::KROW + 32 * c), qf[c], z[kt]);
        }
        results_there(z);
    };

    if (tid < 8)
        s_flag[tid >> 1][tid & 1] = 0;
    if (lo < hi) {
        find_pages(lo);
        load(lo);
        find_pages(lo + 1);
        __syncthreads();
        store(lo);
        load(lo + 1);
        find_pages(lo + 2);
        __syncthreads();
    }

    // The next step's K and V go to LDS while this one's probabilities are formed and
    // used: the compiler spreads them between the matrix instructions.
    for (int step = lo; step < hi; step++) {
        const int key0 = step * SK;
        f32x16 s[KT];
        scores(step, s);
        uint64_t lost = 0;
        if (__builtin_amdgcn_readfirstlane(s_flag[step & 3][0]) == step + 1) {
            const int key = key0 + lane;
            lost = __ballot(lane < SK && key < it.r.kv && (uint32_t)table[key >> log_p] > last_page);
        }
        if (key0 < all0 || key0 + SK - 1 > all1 || lost != 0) {
            const int f = first - key0 - 4 * h, e = last - key0 - 4 * h;
            const uint64_t gone4 = lost >> (4 * h);
#pragma unroll
            for (int kt = 0; kt < KT; kt++)
#pragma unroll
                for (int r = 0; r < 16; r++) {
                    const int k = 32 * kt + 8 * (r / 4) + r % 4;
                    s[kt][r] = k >= f && k <= e && !(gone4 >> k & 1) ? s[kt][r] : -INFINITY;
                }
        }
        float top = s[0][0];
#pragma unroll
        for (int r = 1; r < 16 * KT; r++)
            top = fmaxf(top, s[r / 16][r % 16]);
        top = max_over_halves(top);
        if (best.takes(top)) {
            const float f = best.take(top, a.scale, s);
            l *= f;
#pragma unroll
            for (int d = 0; d < DT; d++)
                o[d] *= f;
        }
        u32x4 p[KT][2];
#pragma unroll
        for (int kt = 0; kt < KT; kt++) {
#pragma unroll
            for (int r = 0; r < 16; r++) {
                s[kt][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kt][r], a.scale, best.add));
                l += s[kt][r];
            }
#pragma unroll
            for (int r = 0; r < 8; r++)
                p[kt][r / 4][r % 4] = pair_bf16(s[kt][2 * r], s[kt][2 * r + 1]);
        }
        store(step + 1);
        load(step + 2);
        find_pages(step + 3);
        const uint8_t *sv = s_kv + (step & 1) * L::BUF + SK * L::KROW + (4 * h + ((lane & 15) >> 2)) * L::VROW +
                            32 * ((lane >> 4) & 1) + 8 * (lane & 3);
#pragma unroll
        for (int u = 0; u < 2 * KT; u++)
#pragma unroll
            for (int d = 0; d < DT; d++) {
                const uint8_t *at = sv + 16 * u * L::VROW + 64 * d;
                const uint2 x = read_turned(at), y = read_turned(at + 8 * L::VROW);
                o[d] = mfma32(u32x4{x.x, x.y, y.x, y.y}, p[u / 2][u % 2], o[d]);
            }
        const int32_t nan = __builtin_amdgcn_readfirstlane(s_flag[step & 3][1]);
        if (nan == step + 1) {
            // blocks of NaN in V, for the rows that see their keys
            const int key = key0 + lane;
            const uint32_t p = lane < SK && key < it.r.kv ? (uint32_t)table[key >> log_p] : 0xFFFFFFFFu;
#pragma unroll
            for (int blk = 0; blk < L::NB; blk++) {
                const uint64_t sat = (uint64_t)(p > last_page ? 0u : p) * scale_page +
                                     ((((uint32_t)head * L::NB + blk) << log_p) + (key & page_mask));
                uint64_t who = __ballot(p <= last_page && a.v_scales[sat] == 255);
                while (who) {
                    const int k = key0 + __builtin_ctzll(who);
                    who &= who - 1;
                    o[blk] += k >= first && k <= last ? __builtin_nanf("") : 0.f;
                }
            }
        }
        __syncthreads();
    }

    auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
    l = __uint_as_float(x[0]) + __uint_as_float(x[1]);
    if (row >= rows)
        return;
    const int64_t p = ((int64_t)(it.item + it.chunk) * a.heads + head) * ROWS + (row - it.tile * ROWS);
#pragma unroll
    for (int d = 0; d < DT; d++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
            const f32x4 v = {o[d][4 * r], o[d][4 * r + 1], o[d][4 * r + 2], o[d][4 * r + 3]};
            const int c = 32 * d + 8 * r + 4 * h;
            if (it.chunks > 1)
                *reinterpret_cast<f32x4 *>(cut.part_o + p * D + c) = v;
            else
                store_out<D>(a, it, head, tile_rows, row - first_row, c, v, best.m, l);
        }
    if (it.chunks > 1 && h == 0) {
        cut.part_ml[2 * p] = best.m;
        cut.part_ml[2 * p + 1] = best.marked_sum(l);
    }
}

// The chunks of a tile of many rows joined, in their order: a wave takes JOIN rows,
// whose channels it splits by four; the lanes left over share the chunks.  Bound by
// the parts' round trips: 256 rows of 32 heads of 128 over 8 in 8 chunks, 33 MB, 10 us.
constexpr int JOIN = 4;

template <int D, int ROWS>
__global__ __launch_bounds__(256, 3) void join_chunks_kernel(const AttnArgs a, const Cut cut)
{
    constexpr int Q = D / 4, S = Q <= 32 ? (Q <= 16 ? 4 : 2) : 1;
    const int head = blockIdx.x % a.heads;
    const Item it = find_item<ROWS>(a, cut, (int32_t)(blockIdx.x / a.heads), true);
    if (!it.found || it.chunks < 2)
        return;
    const int lane = threadIdx.x & 63, q = lane % (64 / S), sh = lane / (64 / S);
    const int r0 = (blockIdx.y * 4 + (threadIdx.x >> 6)) * JOIN, rows = it.r.fresh * a.G - it.tile * ROWS;
    const int64_t p0 = ((int64_t)it.item * a.heads + head) * ROWS, next = (int64_t)a.heads * ROWS;
    if (r0 >= rows)
        return;
    const int c = 4 * (q < Q ? q : 0);
    const TileRows tile_rows(it.tile * ROWS, a.G);
    float mm[JOIN], ll[JOIN];
    f32x4 sum[JOIN];
    float least = 0.f;
#pragma unroll
    for (int r = 0; r < JOIN; r++) {
        mm[r] = -INFINITY;
        ll[r] = 0.f;
        sum[r] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    for (int i0 = sh; i0 < it.chunks; i0 += 4 * S) {
        float2 ml[4][JOIN];
        f32x4 v[4][JOIN];
#pragma unroll
        for (int j = 0; j < 4; j++)
#pragma unroll
            for (int r = 0; r < JOIN; r++) {
                const int i = i0 + j * S < it.chunks ? i0 + j * S : i0;
                const int64_t p = p0 + i * next + (r0 + r < rows ? r0 + r : r0);
                ml[j][r] = *reinterpret_cast<const float2 *>(cut.part_ml + 2 * p);
                v[j][r] = *reinterpret_cast<const f32x4 *>(cut.part_o + p * D + c);
            }
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (i0 + j * S < it.chunks)
#pragma unroll
                for (int r = 0; r < JOIN; r++) {
                    const float up = fmaxf(mm[r], ml[j][r].x), ref = up == -INFINITY ? 0.f : up;
                    const float f = part_weight(mm[r], ref, a.scale), w = part_weight(ml[j][r].x, ref, a.scale);
                    least = fminf(least, ml[j][r].y);
                    mm[r] = up;
                    ll[r] = f * ll[r] + w * ml[j][r].y;
                    sum[r] = f * sum[r] + w * v[j][r];
                }
    }
    const bool far = __any(least < 0.f);
    if (__builtin_expect(far, 0))
#pragma unroll
        for (int r = 0; r < JOIN; r++) {
            float m = -INFINITY, l = 0.f;
            f32x4 o = {0.f, 0.f, 0.f, 0.f};
            least = 0.f;
#pragma nounroll
            for (int i = sh; i < it.chunks; i += S) {
                const int64_t p = p0 + i * next + (r0 + r < rows ? r0 + r : r0);
                const float2 ml = *reinterpret_cast<const float2 *>(cut.part_ml + 2 * p);
                least = fminf(least, ml.y);
                join_far(m, l, o, ml.x, ml.y, *reinterpret_cast<const f32x4 *>(cut.part_o + p * D + c), a.scale);
            }
            if (least < 0.f) {                            // (the other rows keep their bits)
                mm[r] = m;
                ll[r] = l;
                sum[r] = o;
            }
        }
    auto across = [&](auto weight) {
#pragma unroll
        for (int d = 64 / S; d < 64; d *= 2)
#pragma unroll
            for (int r = 0; r < JOIN; r++) {
                const float m2 = __shfl_xor(mm[r], d), l2 = __shfl_xor(ll[r], d);
                const float up = fmaxf(mm[r], m2), ref = up == -INFINITY ? 0.f : up;
                const float f = weight(mm[r], ref, a.scale), w = weight(m2, ref, a.scale);
                mm[r] = up;
                // the same order in both lanes
                const float x = f * __builtin_fabsf(ll[r]), y = w * __builtin_fabsf(l2);
                ll[r] = x + y;
#pragma unroll
                for (int e = 0; e < 4; e++)
                    sum[r][e] = f * sum[r][e] + w * __shfl_xor(sum[r][e], d);
            }
    };
    if (__builtin_expect(far, 0))
        across(far_weight);
    else
        across(part_weight);
    if (sh == 0 && q < Q)
#pragma unroll
        for (int r = 0; r < JOIN; r++)
            if (r0 + r < rows && r0 + r < ROWS)
                store_out<D>(a, it, head, tile_rows, r0 + r, c, sum[r], mm[r], __builtin_fabsf(ll[r]));
}

// ------------------------------------------------------------------- host
struct AttnLayout {
    int64_t tiles[2], items[2];     // of a key head, at most: kernel for few rows, for many
    int32_t target[2];              // 0: no cut; -1: no launch
    int32_t limit;                  // rows of a request up to which the kernel for few takes it
    int32_t wide;                   // eight waves a workgroup
    size_t part_o[2], part_ml[2], group_ml, total;
};

bool al(const void *p, size_t n) { return (uintptr_t)p % n == 0; }

bool attention_sizes(int64_t T, int32_t B, int64_t max_fresh, int32_t Hq, int32_t heads, int32_t D, int64_t width, int32_t P)
{
    return T >= 0 && T <= SPEAR_MAX_ROWS && B >= 0 && B <= SPEAR_MAX_REQUESTS && max_fresh >= 0 && heads >= 1 &&
           heads <= SPEAR_MAX_HEADS && Hq >= heads && Hq <= SPEAR_MAX_HEADS && Hq % heads == 0 && Hq / heads <= 64 &&
           (D == 64 || D == 96 || D == 128 || D == 192 || D == 256) && P >= 16 && P <= 1024 && (P & (P - 1)) == 0 &&
           width >= 1 && width <= SPEAR_MAX_CONTEXT / P && T * Hq <= (int64_t)1 << 27;
}

// Steps whose requests have up to FEW_ROWS_ALL rows take the kernel for few rows, which
// spreads them over more workgroups without a second launch, and so do steps of few rows
// and keys (all heads).  us, few / both: 48 requests on up to 8000 keys, one token of a
// group of 64 of 128 channels 34 / 48, of 256 54 / 127; 64 rows, 8 heads of 256 199 /
// 577, 4 of 128 62 / 77; 128 rows, 4 of 128 107 / 88.  It does not pay for 64 rows, 4
// heads of 64, 52 / 46, and, since every workgroup walks the requests, for a thousand of
// them with 64 rows each on up to 400 keys, 8 heads of 128, 549 / 498 (40 rows 396 / 467,
// heads of 256 1015 / 1213, 300 requests on up to 1000 keys 146 / 167).  300 rows of a
// prompt, 16 heads over 8, 17 / 26; 1000 rows 24 / 38; 64 rows on 8192 keys, 32 over 8,
// 34 / 40 (2^24 rows x keys); 256 rows on 8192 107 / 62.  The keys are what the table has
// room for; an entry wider than the lengths takes both.
// Where a step takes both, requests of up to FEW_LIMIT rows take the one for few, and
// those of one token, whose G rows are up to 64.
constexpr int FEW_ROWS_ALL = 64;
constexpr int FEW_LIMIT = 32;
constexpr int64_t FEW_WORK = (int64_t)1 << 24;
// Eight waves a workgroup, which share the staging of a step's keys, if requests fill
// them (1024 rows a key head on 8192 keys 187 -> 166 us; 80 rows 52 -> 70).
constexpr int WIDE_ROWS = 256;

AttnLayout attention_layout(int64_t T, int32_t B, int64_t max_fresh, int32_t Hq, int32_t heads, int32_t D, int64_t keys)
{
    AttnLayout L;
    const int64_t G = Hq / heads, rows = T * G, requests = T < B ? T : B;
    max_fresh = max_fresh < T ? max_fresh : T;
    const bool both = T > 0 && max_fresh * G > FEW_ROWS_ALL && rows * heads > FEW_WORK / (keys < 1 ? 1 : keys);
    const int64_t limit = G > FEW_LIMIT ? G : FEW_LIMIT, of_few = (limit + FEW_ROWS - 1) / FEW_ROWS;     // tiles of a request
    L.limit = both ? (int32_t)limit : 0x7FFFFFFF;         // (one kernel alone takes all)
    L.wide = D <= 128 && max_fresh * G >= WIDE_ROWS;
    const int many = 32 * (L.wide ? 8 : 4);
    const int resident = L.wide || D > 192 ? 256 : 512;   // workgroups of the kernel for many rows
    size_t off = SPEAR_KV4_COUNTER_BYTES;                 // first, whatever the sizes: calls of all sizes share it
    for (int k = 0; k < 2; k++) {
        const int tile = k ? many : FEW_ROWS, goal = k ? resident : (D > 128 ? 512 : FEW_ITEMS);
        const int64_t cut = (goal + heads - 1) / heads, most_cut = ((k ? 512 : FEW_ITEMS) + heads - 1) / heads;
        // tiles of a key head: at most one more a request than its rows fill (few
        // rows: at most what a request may have; many: of the requests that can have
        // more than limit rows), and no fewer than all rows fill and requests of
        // max_fresh rows make
        const int64_t longer = rows / (limit + 1), more = k && longer < requests ? longer : requests;
        int64_t tiles = rows / tile + more, least = (rows + tile - 1) / tile;
        const int64_t each = max_fresh > 0 ? (T + max_fresh - 1) / max_fresh : 0;
        least = least > each ? least : each;
        if (!k && both) {
            const int64_t few = more * of_few;
            tiles = tiles < few ? tiles : few;
            least = 0;
        }
        L.target[k] = k && !both ? -1 : (least * heads >= goal || tiles * heads > COUNTS ? 0 : (int32_t)cut);
        L.tiles[k] = tiles;
        L.items[k] = tiles + (L.target[k] ? (k || both ? cut : 2 * cut) + 16 : 0);
        // The room of the parts does not depend on max_fresh and grows with T and B,
        // so that a workspace of the largest step serves every other.  Where there are
        // parts, tiles * heads <= COUNTS, and rows fill up to most_cut tiles, or (few rows,
        // before the other kernel) of_few a request, one of which `more` counts.
        const int64_t fill = k ? rows / 128 : rows / FEW_ROWS, behind = more * (of_few - 1);
        const int64_t full = !k && behind > most_cut ? behind : most_cut;
        const int64_t extra = (k ? most_cut : 2 * most_cut) + 16;
        const int64_t parts = ((fill < full ? fill : full) + more + extra) * heads, most_parts = COUNTS + extra * heads;
        // (so few rows have no request for the kernel for many)
        const int64_t room_rows = k && rows <= FEW_ROWS_ALL ? 0 : (parts < most_parts ? parts : most_parts) * (k ? 256 : FEW_ROWS);
        L.part_o[k] = off;
        off += (size_t)(room_rows * D) * sizeof(float);
        L.part_ml[k] = off;
        off += (size_t)(room_rows * 2) * sizeof(float);
        if (!k) {
            L.group_ml = off;
            off += (size_t)(room_rows * 2) * sizeof(float);
        }
    }
    L.total = off;
    return L;
}

template <int D, int W>
hipError_t launch_many(const AttnArgs &a, const Cut &c, const AttnLayout &L, hipStream_t s)
{
    constexpr int ROWS = 32 * W;
    hipLaunchKernelGGL((many_rows_kernel<D, W>), dim3((unsigned)(L.items[1] * a.heads)), dim3(64 * W), 0, s, a, c);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !c.target)
        return e;
    hipLaunchKernelGGL((join_chunks_kernel<D, ROWS>), dim3((unsigned)(L.tiles[1] * a.heads), ROWS / (4 * JOIN)), dim3(256), 0, s, a, c);
    return hipGetLastError();
}

template <int D>
hipError_t launch_attention(const AttnArgs &a, const AttnLayout &L, uint8_t *ws, hipStream_t s)
{
    Cut c[2];
    for (int k = 0; k < 2; k++)
        c[k] = {reinterpret_cast<float *>(ws + L.part_o[k]), reinterpret_cast<float *>(ws + L.part_ml[k]),
                reinterpret_cast<float *>(ws + L.group_ml), k ? L.limit : 0, k ? 0x7FFFFFFF : L.limit, L.target[k], k ? MANY_LEAST : FEW_LEAST,
                k ? MANY_LEAST : FEW_LEAST_FULL, (int32_t)L.items[k], L.target[1] < 0,
                reinterpret_cast<uint32_t *>(ws)};
    hipLaunchKernelGGL((few_rows_kernel<D>), dim3((unsigned)(L.items[0] * a.heads)), dim3(64 * FEW_WAVES), 0, s, a, c[0]);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || L.target[1] < 0)
        return e;
    if constexpr (D <= 128)
        if (L.wide)
            return launch_many<D, 8>(a, c[1], L, s);
    return launch_many<D, 4>(a, c[1], L, s);
}

} // namespace
} // namespace spear

using namespace spear;

extern "C" {

size_t spear_kv4_attention_workspace_size(int64_t T, int32_t B, int64_t max_fresh, int32_t Hq,
                                          int32_t heads, int32_t D, int64_t width, int32_t P)
{
    return attention_sizes(T, B, max_fresh, Hq, heads, D, width, P) ? attention_layout(T, B, max_fresh, Hq, heads, D, width * P).total : 0;
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
    if (!(scale > 0.f) || !isfinite(scale * LOG2E))
        return SPEAR_E_ARG;
    if (!al(q, 16) || !al(y, 16) || !al(table, 4) || !al(q_start, 4) || !al(kv_len, 4) || !al(lse, 4) || !al(workspace, 256))
        return SPEAR_E_ALIGN;
    max_fresh = max_fresh < T ? max_fresh : T;
    const AttnLayout L = attention_layout(T, B, max_fresh, Hq, kv->heads, kv->D,
                                          window && window + max_fresh < width * kv->P ? window + max_fresh : width * kv->P);
    if (ws_bytes < L.total)
        return SPEAR_E_WORKSPACE;
    st = check_device();
    if (st != SPEAR_OK || T == 0 || B == 0)
        return st;
    uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
    const AttnArgs a = {q, q_stride, kv->k_codes, kv->k_scales, kv->v_codes, kv->v_scales, table, q_start, kv_len, y, lse,
                        T, kv->pages, width, B, kv->heads, Hq / kv->heads, __builtin_ctz(kv->P), window, scale * LOG2E};
    const hipStream_t s = (hipStream_t)stream;
    hipError_t e = hipSuccess;
    switch (kv->D) {
    case 64: e = launch_attention<64>(a, L, ws, s); break;
    case 96: e = launch_attention<96>(a, L, ws, s); break;
    case 128: e = launch_attention<128>(a, L, ws, s); break;
    case 192: e = launch_attention<192>(a, L, ws, s); break;
    default: e = launch_attention<256>(a, L, ws, s); break;
    }
    return e == hipSuccess ? SPEAR_OK : SPEAR_E_HIP;
}

} // extern "C"
