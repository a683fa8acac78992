// kv_step.hip -- the plan of a serving step, rotary positions, and the cache of
// 4 bits written and read (spear_kv4_plan, spear_rope, spear_rope_kv4_write,
// spear_kv4_read, spear_rope_frequencies) for gfx950.
#include <float.h>
#include <math.h>

#include "kv4.hpp"

namespace spear {
namespace {

bool al(const void *p, size_t n) { return (uintptr_t)p % n == 0; }

// ----------------------------------------------------------------------- plan
// q_start = prefix sum of the fresh tokens, kv_len = cached + fresh, and the pages
// taken = ceil(kv_len / P) - ceil(cached / P), again summed up in front of each
// request.  Every workgroup forms the same sums over the requests (eight at most a
// thread) and takes its share of the new pages and of the rows; the first writes
// what there is one of.  Nothing that a workgroup reads is written by another:
// a row whose page is new computes the page from the free list.  Bound by round trips
// (lengths, then the table or the free list): one request 4.1 us, 256 requests of
// up to 535 tokens 5.4 us, in one launch.
constexpr int PL_THREADS = 512;
constexpr int PL_MOST = SPEAR_MAX_REQUESTS / PL_THREADS;

struct PlanArgs {
    const int32_t *cached, *fresh;
    int32_t *table;
    const int32_t *free_pages, *n_free;
    spear_kv4_step out;
    int64_t width, n_pages, T;
    int32_t B, log_p;
};

// Sum of v over the lower threads of the workgroup, and over all of them.
__device__ int64_t before_me(int64_t v, int64_t *total, int64_t *s_wave)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t incl = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int64_t o = __shfl_up(incl, d);
        incl += lane >= d ? o : 0;
    }
    if (lane == 63)
        s_wave[wave] = incl;
    __syncthreads();
    int64_t base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < PL_THREADS / 64; w++) {
        base += w < wave ? s_wave[w] : 0;
        all += s_wave[w];
    }
    __syncthreads();
    *total = all;
    return base + incl - v;
}

// The last index of a[0 .. n), ascending, whose value is at most v (a[0] <= v).
__device__ int last_at_most(const int32_t *a, int n, int32_t v)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= v)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ __launch_bounds__(PL_THREADS) void plan_step_kernel(const PlanArgs a)
{
    __shared__ int64_t s_wave[PL_THREADS / 64];
    __shared__ int32_t s_start[SPEAR_MAX_REQUESTS], s_taken[SPEAR_MAX_REQUESTS], s_cached[SPEAR_MAX_REQUESTS];
    const int tid = threadIdx.x, B = a.B, lp = a.log_p;
    const int per = (B + PL_THREADS - 1) / PL_THREADS, first = tid * per;
    const int64_t P1 = (1 << lp) - 1, width = a.width;
    const bool writer = blockIdx.x == 0;

    int32_t fresh[PL_MOST], cached[PL_MOST];
    int64_t sum = 0;
#pragma unroll
    for (int j = 0; j < PL_MOST; j++) {
        const int i = first + j;
        const bool in = j < per && i < B;
        const int32_t f = in ? a.fresh[i] : 0, c = in ? a.cached[i] : 0;
        fresh[j] = f < 0 ? 0 : (f > a.T ? (int32_t)a.T : f);
        cached[j] = c < 0 ? 0 : c;
        sum += fresh[j];
    }
    int64_t nf = a.n_free[0];
    nf = nf < 0 ? 0 : (nf > a.n_pages ? a.n_pages : nf);
    int64_t all;
    int64_t start = before_me(sum, &all, s_wave);
    const int32_t rows = (int32_t)(all < a.T ? all : a.T);

    int64_t takes = 0, beyond = 0;
#pragma unroll
    for (int j = 0; j < PL_MOST; j++) {
        const int i = first + j;
        const int64_t s0 = start < a.T ? start : a.T;
        start += fresh[j];
        const int64_t s1 = start < a.T ? start : a.T;
        if (j < per && i < B) {
            const int64_t kv = (int64_t)cached[j] + (s1 - s0);
            const int64_t held = ((int64_t)cached[j] + P1) >> lp, full = (kv + P1) >> lp;
            s_start[i] = (int32_t)s0;
            s_cached[i] = cached[j];
            fresh[j] = (int32_t)((full < width ? full : width) - (held < width ? held : width));   // pages taken
            takes += fresh[j];
            beyond += full > (held > width ? held : width) ? full - (held > width ? held : width) : 0;
            if (writer) {
                a.out.q_start[i] = (int32_t)s0;
                a.out.kv_len[i] = (int32_t)(kv < 0x7FFFFFFF ? kv : 0x7FFFFFFF);
            }
        } else
            fresh[j] = 0;
    }
    int64_t wanted, over;
    int64_t taken = before_me(takes, &wanted, s_wave);
    before_me(beyond, &over, s_wave);
#pragma unroll
    for (int j = 0; j < PL_MOST; j++)
        if (j < per && first + j < B) {
            s_taken[first + j] = (int32_t)taken;
            taken += fresh[j];
        }
    if (writer && tid == 0) {
        a.out.q_start[B] = rows;
        a.out.n_left[0] = (int32_t)(nf > wanted ? nf - wanted : 0);
        a.out.status[0] = (int32_t)(wanted > nf ? wanted - nf : 0);
        a.out.status[1] = (int32_t)over;
    }
    __syncthreads();

    const int64_t me = (int64_t)blockIdx.x * PL_THREADS + tid, step = (int64_t)gridDim.x * PL_THREADS;
    for (int64_t k = me; k < wanted; k += step) {
        const int i = last_at_most(s_taken, B, (int32_t)k);
        const int64_t held = ((int64_t)s_cached[i] + P1) >> lp;
        a.table[i * width + held + (k - s_taken[i])] = k < nf ? a.free_pages[nf - 1 - k] : -1;
    }
    for (int64_t t = me; t < a.T; t += step) {
        int32_t pos = 0;
        int64_t slot = -1;
        if (t < rows) {
            const int i = last_at_most(s_start, B, (int32_t)t);
            const int64_t p = (int64_t)s_cached[i] + (t - s_start[i]), j = p >> lp;
            const int64_t held = ((int64_t)s_cached[i] + P1) >> lp;
            pos = (int32_t)p;
            if (j < width) {
                int32_t page;
                if (j >= held) {
                    const int64_t k = s_taken[i] + (j - held);
                    page = k < nf ? a.free_pages[nf - 1 - k] : -1;
                } else
                    page = a.table[i * width + j];
                slot = page < 0 ? -1 : ((int64_t)page << lp) + (p & P1);
            }
        }
        a.out.positions[t] = pos;
        a.out.slots[t] = slot;
    }
}

// ----------------------------------------------------------- rotation and write
struct RopeArgs {
    const uint16_t *q, *k, *v;
    uint16_t *y;
    int64_t qs, ks, vs, ys;          // elements from row to row
    const int32_t *pos;
    const int64_t *slots;
    const double *freqs;             // NULL: nothing is rotated
    double scale;
    uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    int64_t places, T;               // pages * P; rows
    int32_t Hq, Hkv, D, rot, layout, log_p;
};

// The fp32 that rounds on to fewer bits as x does: the bits that fp32 has no room
// for go into its last one (a tie stays a tie only if it is one).
__device__ __forceinline__ float keep_odd(double x)
{
    const uint64_t b = __double_as_longlong(x);
    const uint32_t lo = (uint32_t)b;
    const uint32_t kept = (lo & 0xE0000000u) | ((lo & 0x1FFFFFFFu) ? 0x20000000u : 0u);
    return (float)__longlong_as_double((b & 0xFFFFFFFF00000000ull) | kept);
}

// The first 16 bits of x, rounded towards 0, of which its product with a bf16 is exact.
__device__ __forceinline__ float high_term(double x) { return __uint_as_float(__float_as_uint((float)x) & 0xFFFFFF00u); }

template <int CTRL>
__device__ __forceinline__ uint32_t quad(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

// The largest of the quad's lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t v)
{
    uint32_t o = quad<0xB1>(v);                          // lanes 1 0 3 2
    v = o > v ? o : v;
    o = quad<0x4E>(v);                                   // lanes 2 3 0 1
    return o > v ? o : v;
}

// The exponent of a block whose largest magnitude has the bits `top`, plus 127: a
// mantissa of 1.75 or more carries into it.
__device__ __forceinline__ uint32_t block_exponent(uint32_t top)
{
    const int e = (int)((top + 0x200000u) >> 23) - 2;
    return e < 2 ? 2u : (e > 252 ? 252u : (uint32_t)e);
}

__device__ __forceinline__ uint32_t codes8(const float (&f)[8], uint32_t e)
{
    const float s = kv4_scale(e);
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[0], f[1], s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[2], f[3], s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[4], f[5], s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[6], f[7], s, 3);
}

// The largest magnitude's bits among eight channels and those that the quad's other
// lanes hold of their block.
__device__ __forceinline__ uint32_t top8(const float (&f)[8])
{
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const uint32_t b = __float_as_uint(f[j]) & 0x7FFFFFFFu;
        top = b > top ? b : top;
    }
    return quad_max(top);
}

// Eight channels of a block of 32 whose largest magnitude has the bits `top` -> the
// eight codes; *byte the block's scale.
__device__ __forceinline__ uint32_t hold8(const float (&f)[8], uint32_t top, uint32_t *byte)
{
    const uint32_t e = block_exponent(top);
    *byte = top >= 0x7F800000u ? 255u : e;               // a NaN or an infinity
    return codes8(f, e);
}

// A workgroup takes up to N * (256 / (D / 8)) heads of a row; without the cache,
// then of the row gridDim.x further on, whose channels are on their way while it
// works on this one (6000 rows of 24 heads of 256: 28.7 -> 25.2 us; with the cache
// the loop's registers halve the workgroups of a CU, and 8192 rows of 32 + 8 + 8 heads
// of 128 take 68 us, without it 40).  Bound by bytes (24.1 us, 147 MB) and, with the
// cache, as much by vector instructions (38 us, 177 MB): the terms of a factor are
// formed once a row, not by every thread (25.5 and 41 us).  A thread has eight
// channels (16 bytes) of up to N heads, always the same channels.  The row is staged
// in LDS, where a channel finds its partner whatever rot is; all reads of a head come
// before its writes (a row may be rotated in place).
//
// Angles, cosines and sines are fp64: at position 2^20 an fp32 angle is off by
// 2^-5.  q is rotated in fp32 with the factors in two terms, of which the first
// has 16 bits, so that its products with bf16 are exact: x c0 + p s0 is rounded
// once.  The second terms, 2^-15 of the first at most, are rounded to 2^-40, and the
// product, the sum and the join of theirs to 2^-39: r = (x c0 + p s0) + (x c1 + p s1) is
// off by 2^-23 |r| + 2^-37 |m| (|x| + |p|) before its rounding to bf16.  k, whose values next to a border of e2m1 would
// fall on the other side, is rotated in fp64.  (Two heads a thread without the cache:
// four waves a SIMD, as launch_rope counts on, are 128 registers; left to itself the
// compiler takes 131.)
template <int N, bool KV>
__global__ __launch_bounds__(256, N == 2 && !KV ? 4 : 1) void rope_kernel(const RopeArgs a)
{
    __shared__ u32x4 s_x[N][256];
    __shared__ double2 s_cs[KV ? 128 : 1];
    __shared__ f32x4 s_cf[128];                           // cosine and sine in two terms each
    const int tid = threadIdx.x, D = a.D, cph = D / 8, hpi = 256 / cph;
    const int hl = tid / cph, c = tid - hl * cph;
    const int heads = a.Hq + (KV ? 2 * a.Hkv : 0), h0 = blockIdx.y * (hpi * N) + hl;
    const int n = a.rot / 2;
    const bool pairs = a.layout == SPEAR_ROPE_PAIRS, turn = a.freqs && 8 * c < a.rot;
    // (half) the frequency of a channel; of none behind rot
    auto place = [&](int e) { return e < n ? e : (e < a.rot ? e - n : 0); };
    u32x4 x[N];
    int64_t slot = -1;
    int32_t pos = 0;
    const double freq = a.freqs && tid < n ? a.freqs[tid] : 0.0;
    auto load = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int h = h0 + i * hpi;
            if (hl < hpi && h < heads) {
                const uint16_t *p = h < a.Hq ? a.q + t * a.qs + (int64_t)h * D
                                    : h < a.Hq + a.Hkv ? a.k + t * a.ks + (int64_t)(h - a.Hq) * D
                                                       : a.v + t * a.vs + (int64_t)(h - a.Hq - a.Hkv) * D;
                x[i] = ld16(p + 8 * c);
            }
        }
        if (KV)
            slot = a.slots[t];
        if (a.freqs && tid < n)
            pos = a.pos[t];
    };
    load(blockIdx.x);
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        if (a.freqs && tid < n) {
            double s, co;
            sincos((double)pos * freq, &s, &co);
            co *= a.scale;
            s *= a.scale;
            const float c0 = high_term(co), s0 = high_term(s);
            s_cf[tid] = f32x4{c0, (float)(co - (double)c0), s0, (float)(s - (double)s0)};
            if (KV)
                s_cs[tid] = make_double2(co, s);
        }
#pragma unroll
        for (int i = 0; i < N; i++)
            s_x[i][tid] = x[i];
        const bool there = KV && slot >= 0 && slot < a.places;
        const int64_t page = slot >> a.log_p, off = slot & ((1 << a.log_p) - 1);
        __syncthreads();
        if (!KV && t + gridDim.x < a.T)
            load(t + gridDim.x);

        // y_j = x_j c_j + p_j s_j for the channels below rot, p_j the partner, negative for
        // the first of a pair
        f32x4 cs[8];
        int at = 8 * c;                                   // (half) the first partner
        if (turn) {
            if (pairs) {
#pragma unroll
                for (int j = 0; j < 8; j += 2)
                    cs[j] = cs[j + 1] = s_cf[4 * c + j / 2 < n ? 4 * c + j / 2 : 0];
            } else
#pragma unroll
                for (int j = 0; j < 8; j++)
                    cs[j] = s_cf[place(8 * c + j)];
            at += 8 * c >= n ? -n : n;
        }
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int h = h0 + i * hpi;
            if (hl >= hpi || h >= heads)
                continue;
            const bool is_q = h < a.Hq, is_v = KV && h >= a.Hq + a.Hkv;
            const u32x4 own = s_x[i][tid];
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; j++)
                f[j] = bf16f((uint16_t)(own[j >> 1] >> (16 * (j & 1))));
            const uint16_t *row = reinterpret_cast<const uint16_t *>(&s_x[i][hl * cph]);
            // the rotated channels in fp64, from what LDS holds (e0 is opaque: no
            // register is to hold these addresses all along)
            auto anew = [&](auto factors, auto rounded) {
                int e0 = 8 * c;
                asm volatile("" : "+v"(e0));
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const int e = e0 + j;
                    if (e < a.rot) {
                        const bool second = pairs ? e & 1 : e >= n;
                        const int step = pairs ? 1 : n;
                        const double2 d = factors(pairs ? e >> 1 : place(e));
                        const double other = (double)bf16f(row[second ? e - step : e + step]) * d.y;
                        f[j] = rounded((double)bf16f(row[e]) * d.x + (second ? other : -other));
                    }
                }
            };
            if (turn && !is_v) {
                float p[8];
                if (pairs) {
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        p[j] = j & 1 ? f[j ^ 1] : -f[j ^ 1];
                } else if (n % 8 == 0) {                  // the partners lie in one chunk, as the channels do
                    const u32x4 v = *reinterpret_cast<const u32x4 *>(row + at);
                    const uint32_t sign = at > 8 * c ? 0x80008000u : 0u;
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        p[j] = bf16f((uint16_t)((v[j >> 1] ^ sign) >> (16 * (j & 1))));
                } else {
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const int e = 8 * c + j;
                        const float v = bf16f(row[e < n ? e + n : (e < a.rot ? e - n : e)]);
                        p[j] = e < n ? -v : v;
                    }
                }
                if (is_q) {
                    float top = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const float r = __builtin_fmaf(f[j], cs[j][0], p[j] * cs[j][2]) + __builtin_fmaf(f[j], cs[j][1], p[j] * cs[j][3]);
                        top = __builtin_elementwise_maximum(top, __builtin_fabsf(r));       // (a NaN stays)
                        f[j] = 8 * c + j < a.rot ? r : f[j];
                    }
                    // An infinity times a second term of 0 or of the other sign is a NaN that the
                    // formula has not, and a product beyond fp32 may be on its way to less: such
                    // channels are formed anew in fp64.
                    if (!(top < INFINITY))
                        anew([&](int at_cs) {
                            const f32x4 w = s_cf[at_cs];
                            return make_double2((double)w[0] + (double)w[1], (double)w[2] + (double)w[3]);
                        }, [](double r) { return (float)r; });
                } else if (KV) {
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const int e = 8 * c + j;
                        const double2 d = s_cs[pairs ? (e < a.rot ? e >> 1 : 0) : place(e)];
                        const double r = (double)f[j] * d.x + (double)p[j] * d.y;
                        f[j] = e < a.rot ? keep_odd(r) : f[j];
                    }
                }
            }
            if (is_q) {
                u32x4 o;
#pragma unroll
                for (int j = 0; j < 4; j++)
                    o[j] = pair_bf16(f[2 * j], f[2 * j + 1]);
                *reinterpret_cast<u32x4 *>(a.y + t * a.ys + (int64_t)h * D + 8 * c) = o;
            } else if (KV && there) {
                uint32_t top = top8(f);
                if (top == 0x7F800000u && !is_v) {        // (of the quad) a key beyond fp32 is held as the largest
                    if (turn)
                        anew([&](int at_cs) { return s_cs[at_cs]; }, [](double r) {
                            const float k = keep_odd(r);
                            return __builtin_fabsf(k) == INFINITY && __builtin_fabs(r) < INFINITY ? __builtin_copysignf(FLT_MAX, k) : k;
                        });
                    top = top8(f);
                }
                uint32_t byte;
                const uint32_t codes = hold8(f, top, &byte);
                const int64_t ph = page * a.Hkv + (h - a.Hq - (is_v ? a.Hkv : 0));
                uint8_t *cp = is_v ? a.v_codes : a.k_codes, *sp = is_v ? a.v_scales : a.k_scales;
                *reinterpret_cast<uint32_t *>(cp + (((ph << a.log_p) + off) * (D / 2) + 4 * c)) = codes;
                if ((c & 3) == 0)
                    sp[((ph * (D / 32) + (c >> 2)) << a.log_p) + off] = (uint8_t)byte;
            }
        }
        if (KV)
            return;
        __syncthreads();                                  // the row has been read: the next one takes its place
    }
}

// Workgroups that run at once, of up to two heads a thread and of more (us from cold
// memory with 1280 / 1024 / 768 of them: 8192 rows of 32 heads of 128 31.9 / 26.2 / 26.7,
// 3500 of 16 heads of 192 12.2 / 10.6 / 11.5; three heads a thread, 6000 rows of 24 heads
// of 256, 29.7 / 31.1 / 29.0).
constexpr int64_t ROPE_BLOCKS_2 = 1024, ROPE_BLOCKS_4 = 768;

template <bool KV>
hipError_t launch_rope(const RopeArgs &a, int64_t T, hipStream_t s)
{
    const int heads = a.Hq + (KV ? 2 * a.Hkv : 0), hpi = 256 / (a.D / 8);
    // few rows: more workgroups, a head a thread; else as many as a row has, up to four
    const int n = T * heads <= (int64_t)hpi * 2048 ? 1 : (heads + hpi - 1) / hpi;
    const int64_t parts = (heads + hpi * (n < 4 ? n : 4) - 1) / (hpi * (n < 4 ? n : 4)), most = (n <= 2 ? ROPE_BLOCKS_2 : ROPE_BLOCKS_4) / parts;
    const dim3 grid((unsigned)(!KV && most < T ? (most < 1 ? 1 : most) : T), (unsigned)parts);
    switch (n) {
    case 1: hipLaunchKernelGGL((rope_kernel<1, KV>), grid, dim3(256), 0, s, a); break;
    case 2: hipLaunchKernelGGL((rope_kernel<2, KV>), grid, dim3(256), 0, s, a); break;
    case 3: hipLaunchKernelGGL((rope_kernel<3, KV>), grid, dim3(256), 0, s, a); break;
    default: hipLaunchKernelGGL((rope_kernel<4, KV>), grid, dim3(256), 0, s, a); break;
    }
    return hipGetLastError();
}

// A thread takes eight channels, 4 bytes of codes to 16 of bf16, and J of them at once,
// whose dependent loads (slot, then codes and scale) are then on their way together; a
// workgroup takes the channels of `rows` rows.  Bound by what it writes (8192 rows of 8
// heads of 128, k and v: 43 MB in 10.4 us; one at a time 11.3).
template <int J>
__global__ __launch_bounds__(256) void read_kernel(const spear_kv4 kv, const int64_t *slots, int64_t T, int rows, int log_p,
                                                   uint16_t *k, uint16_t *v)
{
    uint16_t *out = blockIdx.y ? v : k;
    const uint8_t *codes = blockIdx.y ? kv.v_codes : kv.k_codes, *scales = blockIdx.y ? kv.v_scales : kv.k_scales;
    if (!out)
        return;
    const uint32_t cph = kv.D / 8, row = kv.heads * cph;  // of a head; of a row
    const int64_t t0 = (int64_t)blockIdx.x * rows;
    const uint32_t n = row * (uint32_t)(T - t0 < rows ? T - t0 : rows);
    out += 8 * t0 * row;
    for (uint32_t i0 = threadIdx.x; i0 < n; i0 += 256 * J) {
        uint32_t w[J], byte[J];
        bool there[J];
#pragma unroll
        for (int j = 0; j < J; j++) {
            const uint32_t i = i0 + 256 * j < n ? i0 + 256 * j : i0, t = i / row, in_row = i - t * row;
            const uint32_t h = in_row / cph, c = in_row - h * cph;
            const int64_t slot = slots[t0 + t];
            there[j] = slot >= 0 && slot < kv.pages * kv.P;
            const int64_t at = there[j] ? slot : 0, ph = (at >> log_p) * kv.heads + h, off = at & (kv.P - 1);
            w[j] = *reinterpret_cast<const uint32_t *>(codes + (((ph << log_p) + off) * (kv.D / 2) + 4 * c));
            byte[j] = scales[((ph * (kv.D / 32) + (c >> 2)) << log_p) + off];
        }
#pragma unroll
        for (int j = 0; j < J; j++)
            if (i0 + 256 * j < n)
                *reinterpret_cast<u32x4 *>(out + 8 * (int64_t)(i0 + 256 * j)) = there[j] ? kv4_bf16(w[j], kv4_scale(byte[j])) : zero4();
    }
}

spear_status check_rotation(const spear_rotation *r, int32_t D)
{
    if (!r->freqs)
        return SPEAR_E_NULL;
    if (r->rot < 2 || r->rot > D || r->rot % 2 != 0)
        return SPEAR_E_SHAPE;
    // within fp32's range with room for the second terms (2^-40 of the first) and for sums
    const double m = fabs(r->scale);
    if ((r->layout != SPEAR_ROPE_HALF && r->layout != SPEAR_ROPE_PAIRS) || !(m == 0.0 || (m >= 0x1p-100 && m <= 0x1p100)))
        return SPEAR_E_ARG;
    return al(r->freqs, 8) ? SPEAR_OK : SPEAR_E_ALIGN;
}

bool bad_stride(int64_t stride, int64_t row) { return stride < row || stride % 8 != 0 || stride > ((int64_t)1 << 36); }

} // namespace

spear_status check_kv4(const spear_kv4 *kv)
{
    if (!kv || !kv->k_codes || !kv->k_scales || !kv->v_codes || !kv->v_scales)
        return SPEAR_E_NULL;
    if (kv->pages < 1 || kv->pages > 0x7FFFFFFF || kv->heads < 1 || kv->heads > SPEAR_MAX_HEADS ||
        (kv->D != 64 && kv->D != 96 && kv->D != 128 && kv->D != 192 && kv->D != 256) || kv->P < 16 || kv->P > 1024 ||
        (kv->P & (kv->P - 1)) != 0)
        return SPEAR_E_SHAPE;
    return al(kv->k_codes, 16) && al(kv->k_scales, 16) && al(kv->v_codes, 16) && al(kv->v_scales, 16) ? SPEAR_OK
                                                                                                     : SPEAR_E_ALIGN;
}

} // namespace spear

using namespace spear;

extern "C" {

spear_status spear_kv4_plan(const int32_t *cached, const int32_t *fresh, int32_t B, int32_t *table,
                            int64_t width, const int32_t *free_pages, int64_t n_pages,
                            const int32_t *n_free, int64_t T, int32_t P,
                            const spear_kv4_step *step, void *stream)
{
    if (!step || !step->q_start || !step->n_left || !step->status || !n_free ||
        (B > 0 && (!cached || !fresh || !table || !step->kv_len)) || (n_pages > 0 && !free_pages) ||
        (T > 0 && (!step->positions || !step->slots)))
        return SPEAR_E_NULL;
    if (B < 0 || B > SPEAR_MAX_REQUESTS || T < 0 || T > SPEAR_MAX_ROWS || P < 16 || P > 1024 || (P & (P - 1)) != 0 ||
        width < 1 || width > SPEAR_MAX_CONTEXT / P || n_pages < 0 || n_pages > 0x7FFFFFFF)
        return SPEAR_E_SHAPE;
    if (!al(cached, 4) || !al(fresh, 4) || !al(table, 4) || !al(free_pages, 4) || !al(n_free, 4) ||
        !al(step->q_start, 4) || !al(step->kv_len, 4) || !al(step->positions, 4) || !al(step->slots, 8) ||
        !al(step->n_left, 4) || !al(step->status, 4))
        return SPEAR_E_ALIGN;
    if (step->n_left == n_free || (B > 0 && (step->kv_len == cached || step->kv_len == fresh)))
        return SPEAR_E_ARG;
    const spear_status st = check_device();
    if (st != SPEAR_OK)
        return st;
    const PlanArgs a = {cached, fresh, table, free_pages, n_free, *step, width, n_pages, T, B, __builtin_ctz(P)};
    const int64_t want = (T + PL_THREADS - 1) / PL_THREADS;
    hipLaunchKernelGGL(plan_step_kernel, dim3((unsigned)(want < 1 ? 1 : (want > 256 ? 256 : want))), dim3(PL_THREADS), 0,
                       (hipStream_t)stream, a);
    return hipGetLastError() == hipSuccess ? SPEAR_OK : SPEAR_E_HIP;
}

spear_status spear_rope_frequencies(int32_t rot, double base, int32_t kind, double factor,
                                    double original, double low, double high, double *freqs)
{
    if (!freqs)
        return SPEAR_E_NULL;
    if (rot < 2 || rot > 256 || rot % 2 != 0 || (kind == SPEAR_ROPE_BASE && rot < 4))
        return SPEAR_E_SHAPE;
    if (kind < SPEAR_ROPE_PLAIN || kind > SPEAR_ROPE_PARTS || !(base > 1.0) || !isfinite(base) || !(factor > 0.0) ||
        !isfinite(factor) ||
        (kind == SPEAR_ROPE_PARTS && (!(original > 0.0) || !isfinite(original) || !(low < high) || !isfinite(low) ||
                                      !isfinite(high))))
        return SPEAR_E_ARG;
    const double b = kind == SPEAR_ROPE_BASE ? base * pow(factor, (double)rot / (rot - 2)) : base;
    for (int i = 0; i < rot / 2; i++) {
        double f = pow(b, -2.0 * i / rot);
        if (kind == SPEAR_ROPE_LINEAR)
            f /= factor;
        if (kind == SPEAR_ROPE_PARTS) {
            double g = (original * f / (2.0 * M_PI) - low) / (high - low);
            g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
            f = (1.0 - g) * f / factor + g * f;
        }
        freqs[i] = f;
    }
    return SPEAR_OK;
}

spear_status spear_rope(const spear_bf16 *x, int64_t x_stride, int64_t T, int32_t H, int32_t D,
                        const int32_t *positions, const spear_rotation *rope, spear_bf16 *y,
                        int64_t y_stride, void *stream)
{
    if (!rope || (T > 0 && (!x || !positions || !y)))
        return SPEAR_E_NULL;
    if (T < 0 || T > SPEAR_MAX_ROWS || H < 1 || H > SPEAR_MAX_HEADS || D < 8 || D > 256 || D % 8 != 0 ||
        bad_stride(x_stride, (int64_t)H * D) || bad_stride(y_stride, (int64_t)H * D) || (x == y && x_stride != y_stride))
        return SPEAR_E_SHAPE;
    spear_status st = check_rotation(rope, D);
    if (st != SPEAR_OK)
        return st;
    if (!al(x, 16) || !al(y, 16) || !al(positions, 4))
        return SPEAR_E_ALIGN;
    st = check_device();
    if (st != SPEAR_OK || T == 0)
        return st;
    RopeArgs a = {};
    a.q = x;
    a.qs = x_stride;
    a.y = y;
    a.ys = y_stride;
    a.pos = positions;
    a.freqs = rope->freqs;
    a.scale = rope->scale;
    a.rot = rope->rot;
    a.layout = rope->layout;
    a.Hq = H;
    a.D = D;
    a.T = T;
    return launch_rope<false>(a, T, (hipStream_t)stream) == hipSuccess ? SPEAR_OK : SPEAR_E_HIP;
}

spear_status spear_rope_kv4_write(const spear_bf16 *q, int64_t q_stride, const spear_bf16 *k,
                                  int64_t k_stride, const spear_bf16 *v, int64_t v_stride,
                                  int64_t T, int32_t Hq, const int32_t *positions,
                                  const int64_t *slots, const spear_rotation *rope,
                                  const spear_kv4 *kv, spear_bf16 *q_out, int64_t q_out_stride,
                                  void *stream)
{
    if (T > 0 && (!q || !k || !v || !slots || !q_out || (rope && !positions)))
        return SPEAR_E_NULL;
    spear_status st = check_kv4(kv);
    if (st != SPEAR_OK)
        return st;
    const int64_t kvr = (int64_t)kv->heads * kv->D;
    if (T < 0 || T > SPEAR_MAX_ROWS || Hq < 1 || Hq > SPEAR_MAX_HEADS || bad_stride(q_stride, (int64_t)Hq * kv->D) ||
        bad_stride(q_out_stride, (int64_t)Hq * kv->D) || bad_stride(k_stride, kvr) || bad_stride(v_stride, kvr) ||
        (q == q_out && q_stride != q_out_stride))
        return SPEAR_E_SHAPE;
    if (rope) {
        st = check_rotation(rope, kv->D);
        if (st != SPEAR_OK)
            return st;
    }
    if (!al(q, 16) || !al(k, 16) || !al(v, 16) || !al(q_out, 16) || !al(positions, 4) || !al(slots, 8))
        return SPEAR_E_ALIGN;
    st = check_device();
    if (st != SPEAR_OK || T == 0)
        return st;
    RopeArgs a = {q, k, v, q_out, q_stride, k_stride, v_stride, q_out_stride, positions, slots, rope ? rope->freqs : nullptr,
                  rope ? rope->scale : 1.0, kv->k_codes, kv->k_scales, kv->v_codes, kv->v_scales, kv->pages * kv->P, T, Hq,
                  kv->heads, kv->D, rope ? rope->rot : 0, rope ? rope->layout : 0, __builtin_ctz(kv->P)};
    return launch_rope<true>(a, T, (hipStream_t)stream) == hipSuccess ? SPEAR_OK : SPEAR_E_HIP;
}

spear_status spear_kv4_read(const spear_kv4 *kv, const int64_t *slots, int64_t T, spear_bf16 *k,
                            spear_bf16 *v, void *stream)
{
    if (T > 0 && !slots)
        return SPEAR_E_NULL;
    spear_status st = check_kv4(kv);
    if (st != SPEAR_OK)
        return st;
    if (T < 0 || T > SPEAR_MAX_ROWS)
        return SPEAR_E_SHAPE;
    if (!al(slots, 8) || !al(k, 16) || !al(v, 16))
        return SPEAR_E_ALIGN;
    st = check_device();
    if (st != SPEAR_OK || T == 0 || (!k && !v))
        return st;
    // four of them at once where that leaves 512 workgroups
    const int64_t row = (int64_t)kv->heads * (kv->D / 8);
    const int each = T * row >= 256 * 1024 ? 4 : 1;
    const int rows = 256 * each > row ? (int)(256 * each / row) : 1;
    const dim3 grid((unsigned)((T + rows - 1) / rows), 2);
    if (each == 4)
        hipLaunchKernelGGL((read_kernel<4>), grid, dim3(256), 0, (hipStream_t)stream, *kv, slots, T, rows, __builtin_ctz(kv->P), k, v);
    else
        hipLaunchKernelGGL((read_kernel<1>), grid, dim3(256), 0, (hipStream_t)stream, *kv, slots, T, rows, __builtin_ctz(kv->P), k, v);
    return hipGetLastError() == hipSuccess ? SPEAR_OK : SPEAR_E_HIP;
}

} // extern "C"
