// spear_internal.hpp -- device helpers, workspace layout and launcher
// declarations shared by the translation units of libspear (gfx950 only).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/spear.h"

namespace spear {

// ---------------------------------------------------------------- vector types
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// One bf16 MFMA, 16x16 output, 32-deep.  Operand layout (wave64): lane l holds
// row (l % 16) of A and column (l % 16) of B, each for the 8 consecutive depth
// positions 8*(l / 16) .. +7; the result lane l holds rows 4*(l / 16) .. +3 of
// column (l % 16).  Any permutation of the depth positions applied to both
// operands alike leaves the result unchanged.
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// One packed word (8 codes; nibble position p holds code (0,2,4,6,1,3,5,7)[p])
// -> bf16 pairs holding 1 + u/16 exactly: the nibble becomes the top 4 of the 7
// mantissa bits of a value in [1, 2).  Pair p takes nibble positions (p, p + 4),
// i.e. codes (2p, 2p + 1): the pairs come out in natural order, as the
// activations' bf16 pairs lie.  The epilogue removes the offset and the zero point:
// 16 sum x (1 + u/16) - (16 + z) sum x = sum x (u - z).  Keeping the nibble in
// the high mantissa bits keeps that offset small (16 sum x).
__device__ __forceinline__ u32x4 unpack8(uint32_t w)
{
    // The mask and the exponent bits go through registers so that each output
    // is one shift and one v_and_or_b32 (two literals cannot share one VOP3).
    uint32_t m, c;
    asm("s_mov_b32 %0, 0x780078" : "=s"(m));
    asm("v_mov_b32 %0, 0x3f803f80" : "=v"(c));
    u32x4 r;
    r[0] = ((w << 3) & m) | c;
    r[1] = ((w >> 1) & m) | c;
    r[2] = ((w >> 5) & m) | c;
    r[3] = ((w >> 9) & m) | c;
    return r;
}

// Scale of the unpacked value and the offset it carries: unpacked = (OFF + u) / SCALE.
constexpr float UNPACK_SCALE = 16.0f;
constexpr float UNPACK_OFF = 16.0f;

__device__ __forceinline__ u32x4 ld16(const void *p)
{
    return *reinterpret_cast<const u32x4 *>(p);
}

__device__ __forceinline__ u32x4 zero4()
{
    u32x4 z = {0u, 0u, 0u, 0u};
    return z;
}

__device__ __forceinline__ float bf16f(uint16_t h)
{
    return __uint_as_float((uint32_t)h << 16);
}

// fp32 -> bf16 bits, round to nearest even (finite values).
__device__ __forceinline__ uint16_t f2bf(float f)
{
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}

__device__ __forceinline__ bf16x2 as_bf16x2(uint32_t v)
{
    // element-wise bit casts of vector lanes miscompile with this toolchain;
    // copy through a scalar instead
    bf16x2 r;
    __builtin_memcpy(&r, &v, sizeof r);
    return r;
}

// sum of the 8 bf16 in d (fp32 accumulate, two per dot2).
__device__ __forceinline__ float sum8(u32x4 d, float acc)
{
    const bf16x2 one = {(__bf16)1.0f, (__bf16)1.0f};
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const uint32_t t = d[e];
        acc = __builtin_amdgcn_fdot2_f32_bf16(as_bf16x2(t), one, acc, false);
    }
    return acc;
}

// Zero points are read without a branch (a load under a branch makes the
// compiler wait for every outstanding load where the branch ends): with no
// zero points the byte is read from the scales array, which is always valid
// and at least N bytes long, and replaced by 8 where it is used.
__device__ __forceinline__ uint32_t load_zero_byte(const uint8_t *zeros, const float *scales,
                                                   int64_t n)
{
    const uint8_t *p = zeros ? zeros : reinterpret_cast<const uint8_t *>(scales);
    return p[n];
}
__device__ __forceinline__ float zero_point(const uint8_t *zeros, uint32_t raw)
{
    return zeros ? (float)raw : 8.f;
}

// ------------------------------------------------------------ workspace layout
// Header: 64 uint32 counters, all zero between calls.
enum {
    HDR_TIMEOUTS = 4,  // bounded waits that expired (cleared by the host query)
    HDR_WORDS = 64
};

constexpr int DEC_WAVES = 4;        // decode workgroup: 4 waves split its K range
constexpr int DEC_SW_MAX = 8;       // 128-deep super-steps per decode wave, at most
constexpr int DEC_LDS_MAX = 81920;  // LDS bytes of staged activations (M + 1 rows), at most
// Launch epoch of the fused decode: 64-bit counters, one per 128-byte line so
// that the per-workgroup claims do not queue behind each other on one address.
constexpr int EPOCH_CTRS = 64;
constexpr int EPOCH_STRIDE = 128;

constexpr int PROD_BYTES = 8192;  // bytes of A an EC producer workgroup reads, about
constexpr int MAX_PROD = 32;      // at most this many EC producer workgroups
constexpr int PROD_WORDS = 4096;  // above 8 tokens: partial words an epilogue loads, at most
constexpr int PROD_CHUNK = 4;     // producer partials a consumer wave loads per batch
constexpr int PRE_SLOTS = 512;    // EC pre-pass: (token group, K slice) partial slots, at most
                                  // (fewer than PRE_GROUPS groups, about 256 workgroups)
// Decode's own EC pre-pass: K slices, at most (2048 -> 16384 pair at one token and
// 8192 -> 2048 at 16, us: 4 slices 13.0 and 17.4, 8: 13.4 and 15.0, 16: 16.0 and 15.6).
constexpr int FEW_SLICES = 8;
constexpr int FEW_RANK = 64;      // ... and padded rank, at most
constexpr int PRE_GROUPS = 128;   // EC pre-pass: token groups below which K is split

struct WsLayout {
    size_t hdr, epoch, zeros, splitp, pu, pz, vhi, vlo, vtag, active, preu, prez, gpart, total;
    size_t idx;         // semi-fused prefill: the active-token list [mpad], then its count
    int64_t nslot;      // producers that pu and pz have room for
    int64_t ncg, ksplit, spw, nprod, prod_k, rpad, mpad;
};

WsLayout ws_layout(int64_t M, int64_t N, int64_t K, int32_t r);

// ------------------------------------------------------------- kernel params
// Offsets (bytes) of the workspace regions the decode kernels use.  A decode
// call's layout holds only small regions ahead of them (the host checks that
// they fit 32 bits).
struct DecOffsets {
    uint32_t hdr, epoch, splitp, pu, pz, vhi, vlo, active;
};

// The epilogue after the layer (spear_w4_linear_epilogue): one 64-byte line.
struct EpiArgs {
    const float *bias;      // [N] or null
    const void *res;        // [M][N or N / 2] of the output's type, or null
    int32_t act;            // SPEAR_ACT_*
    int32_t glu;            // 1: channels 2i and 2i + 1 make output channel i
    int32_t on;             // host side: the call has an epilogue
    int32_t few;            // decode with the EC's pre-pass before it: K slices of the partials
    // Partials of A x [few][16][rpad] and of the gate logit [few][16][2 halves],
    // 64-bit words as in the fused exchange, whose place they take.  Their upper
    // half is zero, the tag of no launch: whatever layout another call's token
    // count gives the workspace, none takes them for its own.
    uint32_t *fu, *fz;
};

// A row tile of a grouped product: rows list[pos .. pos + cnt) through expert e.
struct Tile {
    int32_t e, pos, cnt, pad;
};

// A grouped product (spear_w4_experts): the weights of every expert one after
// the other, and the row tiles that a launch before wrote.
struct GrpArgs {
    const int32_t *ntiles;  // row tiles in use (the grid has room for the most there can be)
    const Tile *tiles;
    const int32_t *list;    // slots by expert
    int32_t div;            // a row's source is slot / div
    uint32_t base8;         // the launch's first block, in eights (an XCD each)
};

// Blocks of one launch of a product over row tiles, at most: more take several
// launches (a launch holds less than 2^32 threads).
constexpr int64_t MAX_BLOCKS = 1 << 20;

struct LinearArgs {
    // The leading block (212 bytes, four 64-byte lines) is what the decode
    // kernels load at entry.  Each further 64-byte line of arguments a kernel
    // loads adds about 0.35 us to its launch (measured in graph replay: 3.1 us
    // for one line, 3.9 us for four, 5.0 us for eight), so the fields they use
    // come first and no wider than they need to be.
    const uint16_t *x;
    const uint8_t *packed;
    const float *scales;
    const uint8_t *zeros;
    const uint16_t *A, *B, *wg;
    void *y;
    uint8_t *ws;
    float *g_out;
    int32_t *idx_out;
    int32_t *nact_out;
    int64_t M, N, K;
    double thr;      // logit(tau) for the hard gate
    float b;
    int32_t hard;
    int32_t r, rpad;
    int32_t ncg, ksplit, spw, nprod, prod_k;   // decode: channel groups, K ranges, EC producers
    uint32_t wait_limit;
    int32_t out_f32;
    int32_t gate_h;  // vector gate: hidden width (0: scalar gate only)
    float alpha;
    DecOffsets D;
    uint32_t grid;   // the launch's workgroups (gridDim's hidden argument sits in a line of its own)
    // The prefill kernels load the leading block and this one (bytes 0 to 359,
    // six lines): the vector gate MLP, the prefill tiling and the offsets of the
    // workspace regions they use (64-bit: a prefill workspace may pass 4 GiB).
    const float *gw1, *gc1, *gw2, *gc2;   // vector gate MLP (gate_h > 0)
    int32_t pre_ks;  // EC pre-pass: K slices per token group
    int32_t g_bm;    // MFMA GEMM: tokens per tile (64 or 128)
    int32_t g_bn;    // MFMA GEMM: channels per tile (64 with 64-token tiles, else 256)
    int32_t g_ks;    // MFMA GEMM: K slices per tile (partials reduced by a second launch)
    int32_t npre;    // K-split GEMM with the EC pre-pass in its launch: leading pre-pass blocks
    int64_t mpad;
    struct {
        size_t hdr, zeros, vhi, vlo, vtag, active, preu, prez, gpart, idx;
    } P;
    // The kernels with an epilogue load this line too, the grouped ones the next.
    alignas(64) EpiArgs E;
    GrpArgs G;
    // Host side only.
    WsLayout L;
};
static_assert(offsetof(LinearArgs, gw1) == 216 && offsetof(LinearArgs, D) == 180 &&
                  offsetof(LinearArgs, grid) == 212 && offsetof(LinearArgs, E) == 384,
              "the decode kernels' leading block");

// Swizzle of rows staged in LDS for MFMA operands: the 16-byte pieces of row r
// swap places by piece ^ row_turn(r % 16).  A 16-byte LDS read serves its lanes
// in groups of 16: 0-3, 12-15, 20-23 and 24-27 together, then 4-7, 8-11, 16-19
// and 28-31, and so on.  Lane 16 g + r reads piece 4 g + d of row r, so a group
// holds rows 0-3 and 12-15 of one g and the other rows of the next, and with a
// turn by r itself the two halves meet in the same banks; this turn keeps all 16
// apart (bank conflicts counted: 46 % of the LDS cycles before, none after).
__host__ __device__ __forceinline__ int row_turn(int r)
{
    const int q = r >> 2;
    return (r & 3) | ((q == 0 ? 0 : q == 3 ? 1 : q + 1) << 2);
}

// Byte offset in a row of packed weights (K / 2 bytes) of what the GEMM stages
// for its 32-deep piece c (0..3) of the 128-deep stage st.  Past K the piece's
// last one inside K, or the row's first where none is (K < 128): finite values
// that meet zero activations, and always inside the row.
__host__ __device__ __forceinline__ int64_t w_piece(int64_t K, int c) { return 32 * c < K ? c : 0; }
__host__ __device__ __forceinline__ int64_t w_last_stage(int64_t K, int c)
{
    return (K - 32 * w_piece(K, c) + 127) / 128 - 1;
}
__host__ __device__ __forceinline__ int64_t w_offset(int64_t K, int c, int64_t st)
{
    const int64_t last = w_last_stage(K, c);
    return 16 * w_piece(K, c) + 64 * (st < last ? st : last);
}

// Explicit counter waits (gfx9 s_waitcnt encoding: vmcnt bits 3:0 and 15:14,
// expcnt 6:4, lgkmcnt 11:8) and a barrier without the fence of
// __syncthreads, for code that orders its memory operations itself.
template <int N>
__device__ __forceinline__ void wait_vmcnt()
{
    static_assert(N >= 0 && N < 64, "vmcnt");
    __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | 0x70 | 0xF00);
}
__device__ __forceinline__ void wait_lgkmcnt0() { __builtin_amdgcn_s_waitcnt(0xC07F); }
// The barrier waits for this wave's LDS reads: a buffer that the waves have read
// is written again behind it, and a read still in flight could return what
// another wave writes.  (As asm that clobbers memory the wait cost the large GEMM
// 2 %; a test takes the assembly for reads that the compiler moves past it.)
__device__ __forceinline__ void read_barrier()
{
    wait_lgkmcnt0();
    __builtin_amdgcn_s_barrier();
}

// Load the arguments a kernel uses at entry, in one batch.  The compiler
// otherwise fetches fields of a large argument struct lazily, in several
// batches that each cost a memory round trip before the first data load can
// be issued; and each 64-byte line of arguments loaded costs about 0.35 us a
// launch, so each kernel family loads only the leading lines it uses.
template <typename T>
__device__ __forceinline__ void pin_arg(const T &v)
{
    static_assert(sizeof(T) == 4 || sizeof(T) == 8, "scalar argument");
    if constexpr (sizeof(T) == 8)
        asm volatile("" ::"s"(__builtin_bit_cast(uint64_t, v)));
    else
        asm volatile("" ::"s"(__builtin_bit_cast(uint32_t, v)));
}


// The decode kernels' arguments: the leading block only (the vector gate's
// weights are loaded where that path needs them).
__device__ __forceinline__ void pin_dec_args(const LinearArgs &a)
{
    pin_arg(a.x); pin_arg(a.packed); pin_arg(a.scales); pin_arg(a.zeros); pin_arg(a.A);
    pin_arg(a.B); pin_arg(a.wg); pin_arg(a.y); pin_arg(a.ws); pin_arg(a.g_out);
    pin_arg(a.idx_out); pin_arg(a.nact_out); pin_arg(a.M); pin_arg(a.N); pin_arg(a.K);
    pin_arg(a.thr); pin_arg(a.b); pin_arg(a.hard); pin_arg(a.r); pin_arg(a.rpad);
    pin_arg(a.ncg); pin_arg(a.ksplit); pin_arg(a.spw); pin_arg(a.nprod); pin_arg(a.prod_k);
    pin_arg(a.wait_limit); pin_arg(a.out_f32); pin_arg(a.gate_h); pin_arg(a.alpha);
    pin_arg(a.D.hdr); pin_arg(a.D.epoch); pin_arg(a.D.splitp); pin_arg(a.D.pu);
    pin_arg(a.D.pz); pin_arg(a.D.vhi); pin_arg(a.D.vlo); pin_arg(a.D.active); pin_arg(a.grid);
}

// The prefill kernels' arguments: the leading block and the prefill block.
__device__ __forceinline__ void pin_pre_args(const LinearArgs &a)
{
    pin_dec_args(a);
    pin_arg(a.gw1); pin_arg(a.gc1); pin_arg(a.gw2); pin_arg(a.gc2);
    pin_arg(a.pre_ks); pin_arg(a.g_bm); pin_arg(a.g_bn); pin_arg(a.g_ks); pin_arg(a.npre);
    pin_arg(a.mpad);
    pin_arg(a.P.hdr); pin_arg(a.P.zeros); pin_arg(a.P.vhi); pin_arg(a.P.vlo); pin_arg(a.P.vtag);
    pin_arg(a.P.active); pin_arg(a.P.preu); pin_arg(a.P.prez); pin_arg(a.P.gpart); pin_arg(a.P.idx);
}

// The epilogue's arguments.
__device__ __forceinline__ void pin_epi_args(const LinearArgs &a)
{
    pin_arg(a.E.bias); pin_arg(a.E.res); pin_arg(a.E.act); pin_arg(a.E.glu); pin_arg(a.E.few);
    pin_arg(a.E.fu); pin_arg(a.E.fz);
}

__device__ __forceinline__ void pin_grp_args(const LinearArgs &a)
{
    pin_arg(a.G.ntiles); pin_arg(a.G.tiles); pin_arg(a.G.list); pin_arg(a.G.div); pin_arg(a.G.base8);
}

// ------------------------------------------------------------------ epilogue
// act(t), the activation a whole launch shares (uniform branch).  expf and
// erfcf in fp32: the activation of a value near zero keeps its relative
// accuracy (t is multiplied on, never subtracted).  silu of a large negative t
// is t / inf = -0, as is the limit; gelu_tanh is written as t sigmoid(2 q),
// q = sqrt(2 / pi) (t + 0.044715 t^3), which equals t / 2 (1 + tanh q) without
// the cancellation of 1 + tanh at negative t.
__device__ __forceinline__ float apply_act(float t, int act)
{
    switch (act) {
    case SPEAR_ACT_RELU:
        return t > 0.f ? t : (t != t ? t : 0.f);
    case SPEAR_ACT_SILU:
        return t == -__builtin_inff() ? 0.f : t / (1.f + expf(-t));
    case SPEAR_ACT_GELU:
        return t == -__builtin_inff() ? 0.f : 0.5f * t * erfcf(-0.70710678118654752f * t);
    case SPEAR_ACT_GELU_TANH: {
        const float q = 1.5957691216057308f * __builtin_fmaf(0.044715f * t * t, t, t);
        return t == -__builtin_inff() ? 0.f : t / (1.f + expf(-q));
    }
    default:
        return t;
    }
}

// Four consecutive channels of one token, before and after the epilogue: t
// holds the layer's outputs n .. n + 3, b their biases (zero without).  With
// the gated pair o[0] and o[1] are output channels n / 2 and n / 2 + 1.
__device__ __forceinline__ void epi_apply(const float (&t)[4], const float (&b)[4], int act, int glu,
                                          float (&o)[4])
{
    if (glu) {
        o[0] = apply_act(t[0] + b[0], act) * (t[1] + b[1]);
        o[1] = apply_act(t[2] + b[2], act) * (t[3] + b[3]);
        o[2] = o[3] = 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++)
            o[i] = apply_act(t[i] + b[i], act);
    }
}

// Biases of channels n .. n + 3 (clamped to N - 1), raw; read without a branch
// from the scales when there is no bias, and then replaced by zeros by the caller.
__device__ __forceinline__ void epi_load_bias(const float *bias, const float *scales, int64_t n, int64_t N,
                                              float (&raw)[4])
{
    const float *p = bias ? bias : scales;
#pragma unroll
    for (int i = 0; i < 4; i++)
        raw[i] = p[n + i < N ? n + i : N - 1];
}

// Residual of the outputs of channels n .. n + 3 of token m, as fp32 (zero
// where there is none or the channel is past the end).  NO = output channels.
template <int OUT_F32>
__device__ __forceinline__ void epi_load_res(const void *res, int64_t m, int64_t n, int glu, int64_t NO,
                                             float (&r)[4])
{
    const int cnt = glu ? 2 : 4;
    const int64_t no = glu ? n >> 1 : n;
    r[0] = r[1] = r[2] = r[3] = 0.f;
    if (!res || no >= NO)
        return;
    if (no + cnt <= NO && NO % cnt == 0) {               // a whole, aligned vector
        if (OUT_F32) {
            const float *p = reinterpret_cast<const float *>(res) + m * NO + no;
            if (cnt == 4) {
                const f32x4 v = *reinterpret_cast<const f32x4 *>(p);
                r[0] = v[0];
                r[1] = v[1];
                r[2] = v[2];
                r[3] = v[3];
            } else {
                const float2 v = *reinterpret_cast<const float2 *>(p);
                r[0] = v.x;
                r[1] = v.y;
            }
        } else {
            const uint16_t *p = reinterpret_cast<const uint16_t *>(res) + m * NO + no;
            uint2 v = make_uint2(0u, 0u);
            if (cnt == 4)
                v = *reinterpret_cast<const uint2 *>(p);
            else
                v.x = *reinterpret_cast<const uint32_t *>(p);
            r[0] = __uint_as_float(v.x << 16);
            r[1] = __uint_as_float(v.x & 0xFFFF0000u);
            r[2] = __uint_as_float(v.y << 16);
            r[3] = __uint_as_float(v.y & 0xFFFF0000u);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; i++)
        if (i < cnt && no + i < NO)
            r[i] = OUT_F32 ? reinterpret_cast<const float *>(res)[m * NO + no + i]
                           : bf16f(reinterpret_cast<const uint16_t *>(res)[m * NO + no + i]);
}

// Store the outputs of channels n .. n + 3 of token m.
template <int OUT_F32>
__device__ __forceinline__ void epi_store(void *yv, int64_t m, int64_t n, int glu, int64_t NO,
                                          const float (&o)[4])
{
    const int cnt = glu ? 2 : 4;
    const int64_t no = glu ? n >> 1 : n;
    const bool vec = no + cnt <= NO && NO % cnt == 0;    // a whole, aligned vector
    if (OUT_F32) {
        float *y = reinterpret_cast<float *>(yv) + m * NO + no;
        if (vec && cnt == 4)
            *reinterpret_cast<f32x4 *>(y) = f32x4{o[0], o[1], o[2], o[3]};
        else if (vec)
            *reinterpret_cast<float2 *>(y) = make_float2(o[0], o[1]);
        else
            for (int i = 0; i < cnt; i++)
                if (no + i < NO)
                    y[i] = o[i];
    } else {
        uint16_t *y = reinterpret_cast<uint16_t *>(yv) + m * NO + no;
        const uint32_t w0 = (uint32_t)f2bf(o[0]) | ((uint32_t)f2bf(o[1]) << 16);
        const uint32_t w1 = (uint32_t)f2bf(o[2]) | ((uint32_t)f2bf(o[3]) << 16);
        if (vec && cnt == 4)
            *reinterpret_cast<uint2 *>(y) = make_uint2(w0, w1);
        else if (vec)
            *reinterpret_cast<uint32_t *>(y) = w0;
        else
            for (int i = 0; i < cnt; i++)
                if (no + i < NO)
                    y[i] = f2bf(o[i]);
    }
}

// ---------------------------------------------- tagged cross-workgroup exchange
// One atomic add per workgroup.  Block b claims on counter b % EPOCH_CTRS and
// a launch adds exactly 2^32 to every counter: the first block of each class
// adds 2^32 - (n - 1), the n - 1 others of the class 1 each, and block 0 adds
// 2^32 to the counters no block of a small grid uses.  Between launches all
// counters hold the same multiple of 2^32, so every block of a launch reads the
// same upper half whatever the order of the adds.  G is the launch's grid size.
__device__ __forceinline__ uint64_t epoch_claim(const LinearArgs &a, uint32_t G)
{
    uint8_t *base = a.ws + a.D.epoch;
    const uint32_t bid = blockIdx.x, c = bid % EPOCH_CTRS;
    uint64_t add = 1;
    if (bid < EPOCH_CTRS)
        add = (1ull << 32) - ((G - 1 - c) / EPOCH_CTRS + 1) + 1;
    if (bid == 0)
        for (uint32_t cc = G; cc < EPOCH_CTRS; cc++)
            __hip_atomic_fetch_add(reinterpret_cast<uint64_t *>(base + (size_t)cc * EPOCH_STRIDE),
                                   1ull << 32, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return __hip_atomic_fetch_add(reinterpret_cast<uint64_t *>(base + (size_t)c * EPOCH_STRIDE), add,
                                  __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Tag of the launch (a zeroed workspace holds tag 0, which no launch uses).
__device__ __forceinline__ uint32_t epoch_tag(uint64_t claimed) { return (uint32_t)(claimed >> 32) + 1u; }

// A zero the compiler cannot see through.  The epoch claim returns into two
// registers long before its value is used; with a literal zero on the other
// path the tag arithmetic is folded (or hoisted) to right behind the atomic,
// and a dead low half lets its register be reused, and each of these makes the
// wave wait for the atomic and every older load there.  Adding this opaque
// zero at the use keeps the arithmetic, and both registers, where they belong.
__device__ __forceinline__ uint64_t opaque_zero64()
{
    uint32_t lo, hi;
    asm volatile("v_mov_b32 %0, 0" : "=v"(lo));
    asm volatile("v_mov_b32 %0, 0" : "=v"(hi));
    return ((uint64_t)hi << 32) | lo;
}

__device__ __forceinline__ void store_tagged(uint64_t *p, uint32_t bits, uint32_t tag)
{
    __hip_atomic_store(p, ((uint64_t)tag << 32) | bits, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t load_tagged(const uint64_t *p)
{
    return __hip_atomic_load(const_cast<uint64_t *>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}


// Host: SPEAR_OK on a gfx950 device, cached per device (api.hip).
spear_status check_device();

hipError_t launch_pack(const void *codes, int32_t kind, int64_t N, int64_t K, uint8_t *packed,
                       int32_t *bad, hipStream_t s);
hipError_t launch_gate(const uint16_t *x, int64_t M, int64_t K, const uint16_t *wg, float b,
                       double thr, int32_t hard, float *g, int32_t *idx, int32_t *nact,
                       hipStream_t s);
hipError_t launch_compact(const int32_t *flags, int64_t M, int32_t *idx, int32_t *nact,
                          hipStream_t s, int32_t *idx2 = nullptr, int32_t *nact2 = nullptr);
hipError_t launch_zero(void *p, size_t bytes, hipStream_t s);
hipError_t launch_stream_read(const void *p, size_t bytes, uint32_t *sink, hipStream_t s);
hipError_t launch_decode(const LinearArgs &a, int ec_mode, hipStream_t s);
hipError_t launch_decode_epi(const LinearArgs &a, int ec_mode, hipStream_t s);
hipError_t launch_prepass(const LinearArgs &a, hipStream_t s);
hipError_t launch_gemm(const LinearArgs &a, int ec_on, int force_large, hipStream_t s);
// Grouped: a.G's row tiles of 128 rows, at most max_tiles of them.
hipError_t launch_gemm_grouped(const LinearArgs &a, int64_t max_tiles, hipStream_t s);
hipError_t launch_ec_apply(const LinearArgs &a, hipStream_t s);

} // namespace spear
