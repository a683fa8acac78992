// experts.hip -- the routed tokens through their experts' two 4-bit layers
// (spear_w4_experts), gfx950.
//
//   h_mj = act(up_e x_m + b)  (or the gated pair),  e = ids[m][j]
//   y[m] = residual[m] + sum_j weights[m][j] (down_e h_mj + b)
//
// A slot is one (token, choice) pair, slot = topk m + j.  Few slots take two
// launches (below); else:
//  1. plan: the slots of each expert in ascending order, cut into row tiles;
//  2. up:   each row tile's tokens through its expert's first layer, h by slot;
//  3. down: h through the second layer, fp32 rows by slot;
//  4. join: each token's rows times their weights, in slot order, plus residual.
// h is held in bf16, what the second layer's matrix instructions take (as fp32 it
// would be two words there, twice the instructions and twice the rows' LDS); its
// rounding, 2^-8 at most, is why outputs differ from fp32 throughout by more than
// their own.
// No launch waits on another workgroup, and no result depends on an order that
// the hardware chooses: the sums of an output are taken in one fixed order.
#include <string.h>
#include <type_traits>

#include "spear_internal.hpp"

namespace spear {

namespace {

constexpr int XT = 16;                                    // rows of the smallest tile
constexpr int64_t MAX_SLOTS = 1 << 30;
constexpr int64_t MAX_CHANNELS = 1 << 25;                 // I and N: a row tile's blocks fit one launch

struct ExpertsLayout {
    size_t hdr, zeros, tiles, list, h, d, total;
    int64_t slots;
};

// Row tiles of bm rows: every expert in use has its slots cut into tiles, the
// last one ragged, so at most slots / bm + (experts in use) of them.
int64_t max_tiles(int64_t slots, int32_t E, int bm) { return slots / bm + (slots < E ? slots : E); }

// Rows of a tile by the slots an expert has on average; slots without an expert
// here count too, the ids being on the device, so a device that holds an eighth of
// the experts takes the tiles of eight times its load.  Whole calls, us with 16
// / 64 rows (32 rows are behind one of them everywhere):
//   32 experts 2048 -> 2 x 1408 -> 2048:  12 slots 59 / 62, 16: 63 / 65, 20: 74 / 68
//    8 experts 4096 -> 2 x 4096 -> 4096:  12 slots 70 / 72, 16: 83 / 75, 20: 92 / 76
// and with 64 / 128 rows, where 128 need long enough rows to fill their pipeline:
//   the first:                            256 slots 280 / 332, 768: 729 / 761, 1024: 959 / 999
//   the second:                           128 slots 195 / 216, 320: 372 / 368, 1024: 1058 / 1002
//    8 experts 4096 -> 2 x 8192 -> 4096:  256 slots 611 / 632, 320: 699 / 671, 1024: 2081 / 1781
int tile_rows(int64_t slots, int32_t E, int64_t K, int64_t I)
{
    const int64_t per = slots / E, depth = K < I ? K : I;
    return per < 16 ? XT : per * depth < 320 * 4096 ? 64 : 128;
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
// Bound by the round trips of its two passes over the ids: 4 to 5 us up to 1200
// slots, 11.6 us for 8192 of 8 experts, and in proportion from there.
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
    int32_t ncb;              // channel blocks: the grid's fastest index
    const int32_t *ids;       // few slots: the blocks' own plan
    int32_t slots, E;
    int32_t tile0;            // the launch's first row tile
};

struct JoinArgs {
    const float *d;           // [slots][N]
    const int32_t *ids;
    const float *weights;
    const uint16_t *res;
    uint16_t *y;
    int64_t M, N;
    int32_t topk, E;
};

// All of the arguments in one batch at entry (fetched where they are used, each
// batch is a round trip before the first load).
__device__ __forceinline__ void pin_group_args(const GroupArgs &a)
{
    pin_arg(a.x); pin_arg(a.packed); pin_arg(a.scales); pin_arg(a.zeros); pin_arg(a.bias);
    pin_arg(a.out); pin_arg(a.ntiles); pin_arg(a.tiles); pin_arg(a.list); pin_arg(a.N); pin_arg(a.K);
    pin_arg(a.div); pin_arg(a.act); pin_arg(a.glu); pin_arg(a.ncb); pin_arg(a.ids); pin_arg(a.slots);
    pin_arg(a.E); pin_arg(a.tile0);
}

// Up to this many slots, two launches: the products make their own plan, the
// second joins.  us with two / four launches, 2048 -> 2 x 1024 -> 2048: 8 slots of
// 64 experts 18.8 / 21.8, 12: 24.7 / 25.4, 16: 27.3 / 25.4, 24: 35.7 / 30.4; of 16
// experts 12: 24.9 / 25.5, 16: 24.3 / 24.8, 24: 26.8 / 25.1; of 8 experts 16: 19.7 /
// 22.1, 32: 22.1 / 21.8.
constexpr int FEW_SLOTS = 16;

// What depths past K read: zeros (16 bytes a lane of 16).
__device__ __align__(256) static uint8_t g_zeros[256];

// The streaming product: a workgroup of NW waves takes a row tile of up to BM
// rows and 16 NW channels, wave w 16 of them over all of K.  Weights go from
// memory to registers, RING - 1 chunks of SC depths (SC / 128 16-byte loads a
// lane) ahead of the one in use, and are unpacked once for all the tile's rows;
// the rows go by DMA to RING LDS buffers a chunk deep (2 SC bytes a row, its
// 16-byte pieces swizzled by row % 16 on the way; zeros past K), with one
// barrier a chunk.  Lane (c, g) holds channel c's 32 codes k = 128 s + 32 g .. + 31 of
// step s as one load, and reads the same depths of its token row as four.  The
// rows' sums, which remove the unpacking's offset, are shared out over the
// waves by depth and meet in LDS.  16-row tiles are bound by the weights' way in
// (16 tokens, 8 of 64 experts, 2048 -> 2 x 1024: 33 us for 119 MB, 3.6 TB/s).  In
// 64-row tiles the weights' loads become FLAT ones (their row variants share the
// pointers by reference), which count as LDS reads too, so each chunk waits for
// all that is in flight; that round trip and the LDS reads, every wave all the
// rows and one at a time, bound them (300 tokens, 4 of 32, 2048 -> 2 x 1408: 48 us
// for 94 MB).  With global loads in their place the waits hold as counted, but it
// measured slower: 61 us, and 58 with the LDS reads four at a time (84 registers
// instead of 64).  Rows past the tile's end repeat the last one and are
// not stored: an output depends on its own row alone.
// PLAN 1 (few slots): no plan was launched.  The block's tile is an expert, or
// with fewer slots than experts a slot whose expert no earlier slot has; each
// wave finds that expert's slots in ids by a ballot.
template <int BM, int NW, int UP, int PLAN, int RING, int SC>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(1))) void stream_kernel(const GroupArgs a)
{
    constexpr int NF = BM / 16, NS = SC / 128;            // fragments; steps of a chunk
    constexpr int RB = 2 * SC, RI = 1024 / RB;            // bytes of a row's chunk; rows a DMA takes
    constexpr int NI = BM / (RI * NW), NP = 4 * NS / NW;  // row DMAs, and depth pieces of the sums, a wave
    static_assert(NI * RI * NW == BM && NP * NW == 4 * NS, "rows and depth pieces over waves");
    static_assert(RING == 2 || RING == 4, "one LDS object a buffer");
    __shared__ __attribute__((aligned(16))) uint8_t s_x0[BM * RB], s_x1[BM * RB];
    __shared__ __attribute__((aligned(16))) uint8_t s_x2[RING > 2 ? BM * RB : 16], s_x3[RING > 2 ? BM * RB : 16];
    __shared__ float s_rs[NW][BM];
    uint8_t *const ring[4] = {s_x0, s_x1, s_x2, s_x3};
    pin_group_args(a);
    const int tile = a.tile0 + (int)(blockIdx.x / (uint32_t)a.ncb), cb = (int)(blockIdx.x % (uint32_t)a.ncb);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, lg = lane >> 4;
    Tile q;
    uint64_t mine = 0;                                    // PLAN: the expert's slots
    if constexpr (PLAN != 0) {
        static_assert(FEW_SLOTS <= BM, "an expert's slots are one tile");
        const int id = lane < a.slots ? a.ids[lane] : -1;
        const int e = a.slots < a.E ? __builtin_amdgcn_readlane(id, tile) : tile;
        mine = __ballot(id == e && lane < a.slots);
        if (e < 0 || e >= a.E || mine == 0 || (a.slots < a.E && __builtin_ctzll(mine) != tile))
            return;
        q = {e, 0, (int)__popcll(mine), 0};
    } else {
        q = a.tiles[tile];                                // (the table has room for every block)
        if (tile >= *a.ntiles)
            return;
    }
    auto slot_of = [&](int r) __attribute__((always_inline)) {
        if constexpr (PLAN != 0) {
            uint64_t m = mine;                            // the r-th set bit
            for (int i = 0; i < r; i++)
                m &= m - 1;
            return (int)__builtin_ctzll(m);
        } else {
            return a.list[q.pos + r];
        }
    };
    const int64_t N = a.N, K = a.K;
    const int64_t n0 = ((int64_t)cb * NW + wave) * 16;
    const int64_t base = (int64_t)q.e * N;
    const int64_t C = (K + SC - 1) / SC;
    // The epilogue's operands, without branches.  Their lines are cold, a round
    // trip of 2 to 3 us: with registers to spare (16-row tiles) they are loaded
    // ahead of the stream, else in one go behind it.
    constexpr bool EARLY = BM == 16;
    float sc[4], b[4];
    uint32_t zr[4];
    auto operands = [&]() __attribute__((always_inline)) {
        const int64_t n = n0 + 4 * lg;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int64_t nn = n + i < N ? n + i : N - 1;
            sc[i] = a.scales[base + nn];
            zr[i] = load_zero_byte(a.zeros ? a.zeros + base : nullptr, a.scales + base, nn);
        }
        epi_load_bias(a.bias ? a.bias + base : nullptr, a.scales + base, n, N, b);
    };
    const uint8_t *const wr = a.packed + (base + (n0 + lr < N ? n0 + lr : N - 1)) * (K / 2) + 16 * lg;
    auto load_w = [&](int64_t c, u32x4 (&w)[NS]) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < NS; t++) {
            // past K: the row's first codes, which meet zeros
            const bool in = SC * c + 128 * t + 32 * lg < K;
            w[t] = ld16(in ? wr + (SC * c + 128 * t) / 2 : wr - 16 * lg);
        }
    };
    u32x4 w[RING][NS];
#pragma unroll
    for (int j = 0; j < RING; j++)
        load_w(j < C ? j : C - 1, w[j]);
    if constexpr (EARLY)
        operands();
    // DMA i of a wave fills 1 KB: RI rows from RI (wave + NW i) on, lane l the
    // piece p ^ (row % 16) of row l / (64 / RI), p = l % (64 / RI)
    const uint16_t *xs[NI];
    int xk[NI];
#pragma unroll
    for (int i = 0; i < NI; i++) {
        const int r = RI * (wave + NW * i) + (RI > 1 ? lane / (64 / RI) : 0);
        const int rr = r < q.cnt ? r : q.cnt - 1;
        xk[i] = 8 * ((lane % (64 / RI)) ^ row_turn(r & 15));
        xs[i] = a.x + (int64_t)(slot_of(rr) / a.div) * K + xk[i];
    }
    auto issue_x = [&](int64_t c, uint8_t *buf) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NI; i++) {
            const void *src = SC * c + xk[i] < K ? (const void *)(xs[i] + SC * c) : (const void *)(g_zeros + 16 * lr);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                             (__attribute__((address_space(3))) void *)(buf + 1024 * (wave + NW * i)),
                                             16, 0, 0);
        }
    };
#pragma unroll
    for (int j = 0; j < RING; j++)
        issue_x(j < C ? j : C - 1, ring[j]);

    f32x4 acc[NF], rs[NF];
#pragma unroll
    for (int f = 0; f < NF; f++)
        acc[f] = rs[f] = f32x4{0.f, 0.f, 0.f, 0.f};
    const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    // LDS pieces of row lr for depths 8 (16 t + 4 lg + d): 16 t + ((4 lg + d) ^ lr)
    int xo[4];
#pragma unroll
    for (int d = 0; d < 4; d++)
        xo[d] = lr * RB + (((4 * lg + d) ^ row_turn(lr)) << 4);
    // All steps of a chunk, past K with zero rows, and then this wave's share of
    // the rows' sums.  No branch: it would leave weight loads pending where
    // paths meet, and the compiler would wait for everything there; and after a
    // matrix instruction and a taken branch this toolchain can leave out the
    // wait states before its result is read.  FR: fragments taken.
    auto use = [&](auto FR, const uint8_t *buf, const u32x4 (&w)[NS]) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < NS; t++)
#pragma unroll
            for (int d = 0; d < 4; d++) {
                const u32x4 wv = unpack8(w[t][d]);
#pragma unroll
                for (int f = 0; f < decltype(FR)::value; f++)
                    acc[f] = mfma16(wv, *reinterpret_cast<const u32x4 *>(buf + xo[d] + 256 * t + 16 * RB * f), acc[f]);
            }
#pragma unroll
        for (int i = 0; i < NP; i++) {
            const int p = wave + NW * i;                  // piece 4 t + d
            const int off = lr * RB + 256 * (p >> 2) + (((4 * lg + (p & 3)) ^ row_turn(lr)) << 4);
#pragma unroll
            for (int f = 0; f < decltype(FR)::value; f++)
                rs[f] = mfma16(ones, *reinterpret_cast<const u32x4 *>(buf + off + 16 * RB * f), rs[f]);
        }
    };
    auto run = [&](auto FR) __attribute__((always_inline)) {
        // Younger than the rows of the next chunk: its weights, and the further chunks.
        constexpr int WAIT = NS + (RING - 2) * (NI + NS);
        static_assert(WAIT < 64, "vmcnt");
        wait_vmcnt<0>();
        read_barrier();
        int64_t c = 0;
        for (; c + 2 * RING <= C; c += RING) {
#pragma unroll
            for (int j = 0; j < RING; j++) {
                use(FR, ring[j], w[j]);
                wait_vmcnt<WAIT>();                       // this wave's rows of the next chunk
                read_barrier();                           // every wave's; chunk c + j free
                issue_x(c + j + RING, ring[j]);
                __builtin_amdgcn_sched_barrier(0);        // keeps the order the wait counts on
                load_w(c + j + RING, w[j]);
            }
        }
        // the last RING .. 2 RING - 1 chunks (fewer where K is short)
        wait_vmcnt<0>();
        read_barrier();
#pragma unroll
        for (int j = 0; j < RING; j++)
            if (c + j < C) {
                use(FR, ring[j], w[j]);
                if (j < RING - 1 && c + j + RING < C) {
                    read_barrier();
                    issue_x(c + j + RING, ring[j]);
                    load_w(c + j + RING, w[j]);
                }
            }
        if (c + RING < C) {
            wait_vmcnt<0>();
            read_barrier();
#pragma unroll
            for (int j = 0; j < RING - 1; j++)
                if (c + RING + j < C)
                    use(FR, ring[j], w[j]);
        }
        if constexpr (!EARLY)
            operands();
        int32_t slot[NF];
#pragma unroll
        for (int f = 0; f < decltype(FR)::value; f++) {
            slot[f] = slot_of(16 * f + lr < q.cnt ? 16 * f + lr : 0);
            if (lg == 0)
                s_rs[wave][16 * f + lr] = rs[f][0];
        }
        __syncthreads();
        // lane (row lr of fragment f, lg): channels n0 + 4 lg + i
#pragma unroll
        for (int f = 0; f < decltype(FR)::value; f++) {
            const int r = 16 * f + lr;
            float sum = 0.f;
#pragma unroll
            for (int v = 0; v < NW; v++)
                sum += s_rs[v][r];
            float t[4], bb[4], o[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                t[i] = sc[i] * __builtin_fmaf(-(UNPACK_OFF + zero_point(a.zeros, zr[i])), sum,
                                              UNPACK_SCALE * acc[f][i]);
                bb[i] = a.bias ? b[i] : 0.f;
            }
            epi_apply(t, bb, UP ? a.act : SPEAR_ACT_NONE, UP ? a.glu : 0, o);
            if (r < q.cnt)
                epi_store<(UP ? 0 : 1)>(a.out, slot[f], n0 + 4 * lg, UP ? a.glu : 0, UP && a.glu ? N / 2 : N, o);
        }
    };
    const int nf = (q.cnt + 15) / 16;                     // fragments in use
    if constexpr (NF == 4) {
        if (nf == 3)
            run(std::integral_constant<int, 3>());
        else if (nf == 2)
            run(std::integral_constant<int, 2>());
        else if (nf == 1)
            run(std::integral_constant<int, 1>());
        else
            run(std::integral_constant<int, 4>());
    } else {
        static_assert(NF == 1, "fragments of a tile");
        run(std::integral_constant<int, 1>());
    }
}

template <int BM, int NW, int UP, int PLAN, int RING, int SC>
hipError_t launch_stream_t(GroupArgs a, int64_t tiles, hipStream_t s)
{
    a.ncb = (int32_t)((a.N + 16 * NW - 1) / (16 * NW));
    const int64_t most = MAX_BLOCKS > a.ncb ? MAX_BLOCKS / a.ncb : 1;    // tiles a launch
    for (int64_t t = 0; t < tiles; t += most) {
        a.tile0 = (int32_t)t;
        const int64_t n = tiles - t < most ? tiles - t : most;
        hipLaunchKernelGGL((stream_kernel<BM, NW, UP, PLAN, RING, SC>), dim3((unsigned)(n * a.ncb)), dim3(64 * NW), 0,
                           s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

// 64 rows: 8 waves of 16 channels and 256 depths a chunk (300 tokens, 32 experts,
// first product: 48 us; 512 depths 57, 32 channels a wave 58, 16 waves 61).  16
// rows: two buffers of 512 depths with a plan (16 tokens, 64 experts: 31 us, four
// buffers 43, whose registers leave half the workgroups a CU), four without one
// (a few workgroups a CU at most, where depth in flight is all there is).
template <int UP>
hipError_t launch_stream(const GroupArgs &a, int bm, int64_t tiles, hipStream_t s)
{
    return bm == 64 ? launch_stream_t<64, 8, UP, 0, 2, 256>(a, tiles, s)
                    : launch_stream_t<16, 4, UP, 0, 2, 512>(a, tiles, s);
}

// ------------------------------------------------- few slots: down and join
// One launch for the second layer and the join: a workgroup takes 16 output
// channels, its 8 waves the experts in use (a wave an expert at a time, its 16
// channels of weights straight to registers, the rows of h from L2), each
// slot's sums go to LDS, and after one barrier a thread takes one channel of a
// token over its slots in order, as the join does.  With at most four experts
// in use two waves share one by depth.  Bound by its chain of round trips (one
// token, 8 experts, 1024 -> 2048: 8.3 us for 8.4 MB).
struct FewArgs {
    GroupArgs g;              // the second layer: x is h by slot
    JoinArgs j;
};
constexpr int FW_WAVES = 8;
constexpr int FW_B = 8;                                   // 128-deep steps loaded at once

__global__ __launch_bounds__(64 * FW_WAVES) void few_down_kernel(const FewArgs a)
{
    __shared__ float s_d[2][FEW_SLOTS][17];
    pin_group_args(a.g);
    pin_arg(a.j.weights); pin_arg(a.j.res); pin_arg(a.j.y); pin_arg(a.j.M); pin_arg(a.j.topk);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lr = lane & 15, lg = lane >> 4;
    const int64_t N = a.g.N, K = a.g.K, n0 = (int64_t)blockIdx.x * 16;
    const int slots = a.g.slots, E = a.g.E;
    int id = lane < slots ? a.g.ids[lane] : -1;           // lane: a slot's expert
    id = id >= 0 && id < E ? id : -1;
    const float wt = lane < slots ? a.j.weights[lane] : 0.f;
    int jobs = 0;                                         // experts in use
    for (int s = 0; s < slots; s++) {
        const int e = __builtin_amdgcn_readlane(id, s);
        jobs += e >= 0 && __builtin_ctzll(__ballot(id == e)) == s;
    }
    const int topk = a.j.topk, M = (int)a.j.M;
    const int64_t rn = n0 + (tid & 15);                   // the join's first residual, ahead of the stream
    const float res0 = a.j.res && (tid >> 4) < M && rn < N ? bf16f(a.j.res[(int64_t)(tid >> 4) * N + rn]) : 0.f;
    const int parts = 2 * jobs <= FW_WAVES ? 2 : 1, part = wave % parts;
    const int64_t S = (K + 127) / 128, t0 = part * S / parts, t1 = (part + 1) * S / parts;
    const int64_t nc = n0 + lr < N ? n0 + lr : N - 1;
    const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    for (int s = 0, job = 0; s < slots; s++) {
        const int e = __builtin_amdgcn_readlane(id, s);
        uint64_t rows = __ballot(id == e);                // the expert's slots
        if (e < 0 || __builtin_ctzll(rows) != s)
            continue;
        if (job++ % (FW_WAVES / parts) != wave / parts)
            continue;
        const int64_t base = (int64_t)e * N;
        const uint8_t *wr = a.g.packed + (base + nc) * (K / 2) + 16 * lg;
        float sc[4], b[4];
        uint32_t zr[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int64_t nn = n0 + 4 * lg + i < N ? n0 + 4 * lg + i : N - 1;
            sc[i] = a.g.scales[base + nn];
            zr[i] = load_zero_byte(a.g.zeros ? a.g.zeros + base : nullptr, a.g.scales + base, nn);
        }
        epi_load_bias(a.g.bias ? a.g.bias + base : nullptr, a.g.scales + base, n0 + 4 * lg, N, b);
        const float bf = a.g.bias && part == 0 ? 1.f : 0.f;
        int slot = -1;                                // lane row lr: the lr-th of them
        for (int i = 0; i < FEW_SLOTS && rows; i++) {
            if (lr == i)
                slot = __builtin_ctzll(rows);
            rows &= rows - 1;
        }
        const uint16_t *hr = a.g.x + (int64_t)(slot < 0 ? 0 : slot) * K + 32 * lg;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f}, rs = acc;
        for (int64_t t = t0; t < t1; t += FW_B) {
            u32x4 w[FW_B], xv[FW_B][4];
#pragma unroll
            for (int i = 0; i < FW_B; i++) {
                const int64_t k = 128 * (t + i);
                const bool kv = t + i < t1 && k + 32 * lg < K;
                w[i] = ld16(kv ? wr + k / 2 : wr - 16 * lg);
#pragma unroll
                for (int d = 0; d < 4; d++)
                    xv[i][d] = kv && slot >= 0 ? ld16(hr + k + 8 * d) : zero4();
            }
#pragma unroll
            for (int i = 0; i < FW_B; i++)
#pragma unroll
                for (int d = 0; d < 4; d++) {
                    acc = mfma16(unpack8(w[i][d]), xv[i][d], acc);
                    rs = mfma16(ones, xv[i][d], rs);
                }
        }
        if (slot >= 0) {
#pragma unroll
            for (int i = 0; i < 4; i++)
                s_d[part][slot][4 * lg + i] =
                    sc[i] * __builtin_fmaf(-(UNPACK_OFF + zero_point(a.g.zeros, zr[i])), rs[0],
                                           UNPACK_SCALE * acc[i]) + (bf != 0.f ? b[i] : 0.f);
        }
    }
    __syncthreads();
    // thread: channel tid % 16 of token tid / 16 (every lane shuffles)
    static_assert(16 * FEW_SLOTS <= 64 * FW_WAVES, "a thread an output");
    const int m = tid >> 4;
    const bool in = m < M && rn < N;
    float o = res0;
    for (int j = 0; j < topk; j++) {
        const int slot = m < M ? m * topk + j : 0;
        const int e = __shfl(id, slot);
        const float ws = __shfl(wt, slot);
        if (in && e >= 0) {
            const float d = parts == 2 ? s_d[0][slot][tid & 15] + s_d[1][slot][tid & 15] : s_d[0][slot][tid & 15];
            o = __builtin_fmaf(ws, d, o);
        }
    }
    if (in)
        a.j.y[m * N + rn] = f2bf(o);
}

// ---------------------------------------------------------------------- join
// A thread takes four channels of one token.  4096 tokens x 4096 channels, two
// slots each, residual: 40 us for 201 MB, 5.0 TB/s, what a copy reaches.  Few tokens
// are bound by round trips, so JB slots' rows are in flight at once (16 tokens x 8
// slots: 4 us).
constexpr int JB = 8;

__global__ __launch_bounds__(256) void join_kernel(const JoinArgs a)
{
    const int64_t nq = (a.N + 3) / 4, N = a.N, step = (int64_t)gridDim.x * 256;
    for (int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x; idx < a.M * nq; idx += step) {
        const int64_t m = idx / nq, n = 4 * (idx % nq);
        float o[4];
        epi_load_res<0>(a.res, m, n, 0, N, o);
        // JB slots' loads in flight at once; a slot without an expert has an
        // unwritten row, whose values are dropped
        for (int j0 = 0; j0 < a.topk; j0 += JB) {
            float v[JB][4], w[JB];
            int e[JB];
#pragma unroll
            for (int j = 0; j < JB; j++) {
                const int64_t slot = m * a.topk + (j0 + j < a.topk ? j0 + j : a.topk - 1);
                e[j] = j0 + j < a.topk ? a.ids[slot] : -1;
                w[j] = a.weights[slot];
                epi_load_res<1>(a.d, slot, n, 0, N, v[j]);
            }
#pragma unroll
            for (int j = 0; j < JB; j++)
                if (e[j] >= 0 && e[j] < a.E) {
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        o[i] = __builtin_fmaf(w[j], v[j][i], o[i]);
                }
        }
        epi_store<0>(a.y, m, n, 0, N, o);
    }
}
constexpr int64_t JOIN_BLOCKS = 1 << 22;                  // most of a launch (2^32 threads are too many)

bool al(const void *p, size_t n) { return (uintptr_t)p % n == 0; }

} // namespace
} // namespace spear

using namespace spear;

extern "C" {

size_t spear_w4_experts_workspace_size(int64_t M, int32_t topk, int32_t E, int64_t I, int64_t N)
{
    if (M < 0 || topk < 1 || topk > SPEAR_MAX_TOPK || E < 1 || E > SPEAR_MAX_EXPERTS || I < 32 || I % 32 != 0 || N < 1 ||
        M > MAX_SLOTS / topk || I > MAX_CHANNELS || N > MAX_CHANNELS)
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
    if (M < 0 || topk < 1 || topk > SPEAR_MAX_TOPK || w->E < 1 || w->E > SPEAR_MAX_EXPERTS || K < 32 ||
        K % 32 != 0 || I < 32 || I % 32 != 0 || N < 1 || M > MAX_SLOTS / topk || K > ((int64_t)1 << 31) ||
        I > MAX_CHANNELS || N > MAX_CHANNELS)
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
    const int64_t NU = w->glu ? 2 * I : I;
    const int bm = tile_rows(L.slots, w->E, K, I);
    const int64_t nt = max_tiles(L.slots, w->E, bm);
    const spear_status st = check_device();
    if (st != SPEAR_OK || M == 0)
        return st;
    const hipStream_t s = (hipStream_t)stream;
    uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
    int32_t *ntiles = reinterpret_cast<int32_t *>(ws + L.hdr);
    Tile *tiles = reinterpret_cast<Tile *>(ws + L.tiles);
    int32_t *list = reinterpret_cast<int32_t *>(ws + L.list);
    if (L.slots <= FEW_SLOTS) {
        GroupArgs u = {x, w->up, w->up_scales, w->up_zeros, w->up_bias, ws + L.h, nullptr, nullptr, nullptr,
                       NU, K, topk, w->act, w->glu, 0, ids, (int32_t)L.slots, w->E};
        const int64_t blocks = L.slots < w->E ? L.slots : w->E;
        if (launch_stream_t<16, 4, 1, 1, 4, 512>(u, blocks, s) != hipSuccess)
            return SPEAR_E_HIP;
        const FewArgs f = {{reinterpret_cast<const uint16_t *>(ws + L.h), w->down, w->down_scales, w->down_zeros,
                            w->down_bias, nullptr, nullptr, nullptr, nullptr, N, I, 1, SPEAR_ACT_NONE, 0, 0, ids,
                            (int32_t)L.slots, w->E},
                           {nullptr, ids, weights, residual, y, M, N, topk, w->E}};
        hipLaunchKernelGGL(few_down_kernel, dim3((unsigned)((N + 15) / 16)), dim3(64 * FW_WAVES), 0, s, f);
        return hipGetLastError() == hipSuccess ? SPEAR_OK : SPEAR_E_HIP;
    }
    hipLaunchKernelGGL(plan_kernel, dim3((unsigned)w->E), dim3(1024), 0, s, ids, (int32_t)L.slots, w->E, bm,
                       reinterpret_cast<uint32_t *>(ws + L.zeros), ntiles, tiles, list);
    if (hipGetLastError() != hipSuccess)
        return SPEAR_E_HIP;
    if (bm <= 64) {
        const GroupArgs u = {x, w->up, w->up_scales, w->up_zeros, w->up_bias, ws + L.h, ntiles, tiles, list,
                             NU, K, topk, w->act, w->glu, 0, ids, 0, w->E};
        if (launch_stream<1>(u, bm, nt, s) != hipSuccess)
            return SPEAR_E_HIP;
        const GroupArgs d = {reinterpret_cast<const uint16_t *>(ws + L.h), w->down, w->down_scales, w->down_zeros,
                             w->down_bias, ws + L.d, ntiles, tiles, list, N, I, 1, SPEAR_ACT_NONE, 0, 0, ids, 0, w->E};
        if (launch_stream<0>(d, bm, nt, s) != hipSuccess)
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
        if (launch_gemm_grouped(a, nt, s) != hipSuccess)
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
        if (launch_gemm_grouped(a, nt, s) != hipSuccess)
            return SPEAR_E_HIP;
    }
    JoinArgs j = {reinterpret_cast<const float *>(ws + L.d), ids, weights, residual, y, M, N, topk, w->E};
    const int64_t jb = (M * ((N + 3) / 4) + 255) / 256;
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)(jb < JOIN_BLOCKS ? jb : JOIN_BLOCKS)), dim3(256), 0, s, j);
    return hipGetLastError() == hipSuccess ? SPEAR_OK : SPEAR_E_HIP;
}

} // extern "C"
