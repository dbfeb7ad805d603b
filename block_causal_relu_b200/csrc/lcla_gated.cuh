// lcla_gated.cuh -- device code of the gated recurrence (lcla_gated_* in
// include/lcla.h).
//
// Per (batch entry, head), with a fp32 state S [value][key]:
//   S_t = e^{g_t} S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t.
// In tiles of 32 tokens, G the running sum of g inside the tile (inclusive),
// G_C its last value, S0 the state before the tile:
//   o_t / scale = e^{G_t} S0 q_t + sum_{s <= t} e^{G_t - G_s} (q_t . k_s) v_s
//   S1          = e^{G_C} S0 + sum_s (e^{G_C - G_s} v_s) k_s^T
// With R_t the gradient of the loss by S_t divided by scale, R_t = e^{g_{t+1}}
// R_{t+1} + do_t q_t^T, the gradients are the same sums:
//   dq = scale S_t^T do_t   the recurrence with (query, key, value) = (do, v, k);
//   dk = scale R_t^T v_t    the reversed one with (v, do, q);
//   dv = scale R_t k_t      the reversed one with (k, q, do).
// The reversed recurrence runs through the tiles from the last one, with
//   o_s / scale = e^{G_C - G_s} R q_s + sum_{t >= s} e^{G_t - G_s} (q_s . k_t) v_t
//   R           <- e^{G_C} R + sum_t (e^{G_t} v_t) k_t^T.
//
// All exponents are differences of G taken in one tile.  G is summed in double
// and kept as a whole part and a fraction in fp32, so that a difference is
// exact to 2^-24 however strong the decays of the tokens before it are.
//
// One warp owns 32 rows (values) of one head's state in registers, as the
// accumulator of 16x8 matrix instructions, and walks the tiles of a segment
// alone; at head dim 64 the two warps of a head share the tiles.  The layout of
// an accumulator is also that of an operand, so neither the state nor the
// weighted scores pass through shared memory.
#ifndef LCLA_GATED_CUH
#define LCLA_GATED_CUH

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "lcla_f32x2.cuh"

namespace lcla {
namespace gated {

constexpr int TILE = 32;           // tokens per tile
constexpr int WARPS = 4;           // warps per block: 4 heads at d = 32, 2 at d = 64
constexpr int THREADS = WARPS * 32;
constexpr float RESET = -1000.f;   // a log decay below this counts as this: e^-1000 is zero in fp32, e^1000 infinite

// ---------------------------------------------------------------- operands
// A pair is two neighbouring entries of the contraction index in one lane.  In<T> holds them as given: one bf16x2
// register, or the two tf32 terms of each float.  Co<T> holds computed fp32 values (states, weighted scores and weighted
// values): three bf16 terms of 8 bits each, which keep all 24 bits, or two tf32 terms (22 bits).  With two bf16 terms
// some bf16 outputs were a step beside the fp32 result's rounding (480p forward: 1.1e-4 from plain fp32 in the 2-norm and
// 211 us; with three 3.9e-5, which other orders of the sums leave, and 243 us).
constexpr int TERMS = 3;
template <typename T>
struct In;
template <>
struct In<__nv_bfloat16> {
    uint32_t u;
};
template <>
struct In<float> {
    uint32_t h[2], l[2];
};
template <typename T>
struct Co {
    uint32_t u[TERMS];
};
template <>
struct Co<float> {
    uint32_t h[2], l[2];
};

__device__ __forceinline__ uint32_t pack_bf16(float x, float y)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
    return r;
}
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
// The nearest tf32 value (an infinity stays one; the rest of a NaN that this turns into a zero is a NaN).  Two integer
// instructions: the conversion instruction takes longer (fp32 480p-like forward at d = 32: 261 us with it, 235 without).
__device__ __forceinline__ uint32_t tf32(float x) { return (__float_as_uint(x) + 0x1000u) & 0xffffe000u; }
__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void split(Co<__nv_bfloat16> &o, float2 v)
{
#pragma unroll
    for (int i = 0; i < TERMS; ++i) {
        o.u[i] = pack_bf16(v.x, v.y);
        if (i + 1 < TERMS) v = fma2(make_float2(lo_f(o.u[i]), hi_f(o.u[i])), both(-1.f), v);
    }
}
template <typename P>
__device__ __forceinline__ void split_tf32(P &o, float2 v)
{
    o.h[0] = tf32(v.x);
    o.h[1] = tf32(v.y);
    // the rest has at most 13 significant bits of either sign; the matrix unit takes the first 11, which leaves 2^-23
    const float2 l = fma2(make_float2(__uint_as_float(o.h[0]), __uint_as_float(o.h[1])), both(-1.f), v);
    o.l[0] = __float_as_uint(l.x);
    o.l[1] = __float_as_uint(l.y);
}
__device__ __forceinline__ void split(Co<float> &o, float2 v) { split_tf32(o, v); }
__device__ __forceinline__ float2 value(const In<__nv_bfloat16> &p) { return make_float2(lo_f(p.u), hi_f(p.u)); }
__device__ __forceinline__ float2 value(const In<float> &p)
{
    return make_float2(__uint_as_float(p.h[0]) + __uint_as_float(p.l[0]),
                       __uint_as_float(p.h[1]) + __uint_as_float(p.l[1]));
}

// ZERO: the sum starts from zero, which needs no registers to be cleared.
template <bool ZERO>
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    if (ZERO)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%10,%10,%10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <bool ZERO>
__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    if (ZERO)
        asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%10,%10,%10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// c (+)= A B over 16 entries of the contraction, in STEPS instructions: products of the terms of A and B, the smallest
// first.  A's pairs: (row l/4, k 0-7), (row l/4 + 8, k 0-7), (row l/4, k 8-15), (row l/4 + 8, k 8-15); B's: (k 0-7),
// (k 8-15) of column l/4.  Callers take one step of several products in turn, so that no instruction waits for the one
// before it.
template <typename T, bool COMPUTED>   // whether one of the factors is a Co
struct Steps {
    static constexpr int N = sizeof(T) == 2 ? (COMPUTED ? TERMS : 1) : 6;
};
template <bool ZERO>
__device__ __forceinline__ void mma(int, float (&c)[4], const In<__nv_bfloat16> (&a)[4], const In<__nv_bfloat16> &b0,
                                    const In<__nv_bfloat16> &b1)
{
    mma_bf16<ZERO>(c, a[0].u, a[1].u, a[2].u, a[3].u, b0.u, b1.u);
}
template <bool ZERO>
__device__ __forceinline__ void mma(int step, float (&c)[4], const Co<__nv_bfloat16> (&a)[4],
                                    const In<__nv_bfloat16> &b0, const In<__nv_bfloat16> &b1)
{
    const int i = TERMS - 1 - step;
    mma_bf16<ZERO>(c, a[0].u[i], a[1].u[i], a[2].u[i], a[3].u[i], b0.u, b1.u);
}
template <bool ZERO>
__device__ __forceinline__ void mma(int step, float (&c)[4], const In<__nv_bfloat16> (&a)[4],
                                    const Co<__nv_bfloat16> &b0, const Co<__nv_bfloat16> &b1)
{
    const int i = TERMS - 1 - step;
    mma_bf16<ZERO>(c, a[0].u, a[1].u, a[2].u, a[3].u, b0.u[i], b1.u[i]);
}
// A tf32 instruction contracts 8 entries: its slots 0-3 take the first of each pair, slots 4-7 the second.
template <bool ZERO, typename PA, typename PB>
__device__ __forceinline__ void mma_split(int step, float (&c)[4], const PA (&a)[4], const PB &b0, const PB &b1)
{
    switch (step) {
    case 0: return mma_tf32<ZERO>(c, a[0].l[0], a[1].l[0], a[0].l[1], a[1].l[1], b0.h[0], b0.h[1]);
    case 1: return mma_tf32<false>(c, a[2].l[0], a[3].l[0], a[2].l[1], a[3].l[1], b1.h[0], b1.h[1]);
    case 2: return mma_tf32<false>(c, a[0].h[0], a[1].h[0], a[0].h[1], a[1].h[1], b0.l[0], b0.l[1]);
    case 3: return mma_tf32<false>(c, a[2].h[0], a[3].h[0], a[2].h[1], a[3].h[1], b1.l[0], b1.l[1]);
    case 4: return mma_tf32<false>(c, a[0].h[0], a[1].h[0], a[0].h[1], a[1].h[1], b0.h[0], b0.h[1]);
    default: return mma_tf32<false>(c, a[2].h[0], a[3].h[0], a[2].h[1], a[3].h[1], b1.h[0], b1.h[1]);
    }
}
template <bool ZERO>
__device__ __forceinline__ void mma(int step, float (&c)[4], const In<float> (&a)[4], const In<float> &b0,
                                    const In<float> &b1)
{
    mma_split<ZERO>(step, c, a, b0, b1);
}
template <bool ZERO>
__device__ __forceinline__ void mma(int step, float (&c)[4], const Co<float> (&a)[4], const In<float> &b0,
                                    const In<float> &b1)
{
    mma_split<ZERO>(step, c, a, b0, b1);
}
template <bool ZERO>
__device__ __forceinline__ void mma(int step, float (&c)[4], const In<float> (&a)[4], const Co<float> &b0,
                                    const Co<float> &b1)
{
    mma_split<ZERO>(step, c, a, b0, b1);
}

// -------------------------------------------------------- tiles in shared memory
// A tile holds 32 token rows of one head, d entries each.  16-byte pieces are swapped inside a row by the row's number,
// so that the 8 rows that a matrix load touches fall on different banks.
template <typename T, int D>
struct Tile {
    static constexpr int RB = D * (int)sizeof(T);   // bytes of a row: 64, 128 or 256
    static constexpr int BYTES = TILE * RB;
    static constexpr int PIECES = RB / 16;

    __device__ static __forceinline__ uint32_t at(int row, int piece)
    {
        const int key = RB == 64 ? (row >> 1) & 3 : row & 7;
        return row * RB + ((piece ^ key) << 4);
    }
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ float lds(uint32_t addr)
{
    float r;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(r) : "r"(addr) : "memory");
    return r;
}
__device__ __forceinline__ float2 lds2(uint32_t addr)
{
    float2 r;
    asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(r.x), "=f"(r.y) : "r"(addr) : "memory");
    return r;
}
__device__ __forceinline__ void lds4(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3)
{
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t lds_u(uint32_t addr)
{
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(addr) : "memory");
    return r;
}

// A operand: rows 16 m + [0, 16) of the tile, entries 16 ks + [0, 16).
template <int D>
__device__ __forceinline__ void load_a(In<__nv_bfloat16> (&a)[4], uint32_t tile, int m, int ks, int lane)
{
    const int row = 16 * m + (lane & 15), piece = 2 * ks + (lane >> 4);
    ldsm4(tile + Tile<__nv_bfloat16, D>::at(row, piece), a[0].u, a[1].u, a[2].u, a[3].u);
}
template <int D>
__device__ __forceinline__ void load_a(In<float> (&a)[4], uint32_t tile, int m, int ks, int lane)
{
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const int row = 16 * m + (lane >> 2) + 8 * (p & 1), col = 16 * ks + 8 * (p >> 1) + 2 * (lane & 3);
        const float2 v = lds2(tile + Tile<float, D>::at(row, col >> 2) + 4 * (col & 3));
        split_tf32(a[p], v);
    }
}
// B operands of two column tiles: columns are the rows 16 sb + [0, 16) of the tile, contraction over 16 ks + [0, 16).
template <int D>
__device__ __forceinline__ void load_b(In<__nv_bfloat16> (&b)[2][2], uint32_t tile, int sb, int ks, int lane)
{
    const int row = 16 * sb + (lane & 7) + 8 * (lane >> 4), piece = 2 * ks + ((lane >> 3) & 1);
    ldsm4(tile + Tile<__nv_bfloat16, D>::at(row, piece), b[0][0].u, b[0][1].u, b[1][0].u, b[1][1].u);
}
template <int D>
__device__ __forceinline__ void load_b(In<float> (&b)[2][2], uint32_t tile, int sb, int ks, int lane)
{
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int row = 16 * sb + 8 * n + (lane >> 2), col = 16 * ks + 8 * p + 2 * (lane & 3);
            const float2 v = lds2(tile + Tile<float, D>::at(row, col >> 2) + 4 * (col & 3));
            split_tf32(b[n][p], v);
        }
}
// Transposed: contraction over the rows 16 sb + [0, 16), entries 16 fb + [0, 16) as columns; t[fh][kh] holds entry
// 16 fb + 8 fh + l/4 of the rows 16 sb + 8 kh + 2 (l%4) + {0, 1}.
template <int D>
__device__ __forceinline__ void load_t(In<__nv_bfloat16> (&t)[2][2], uint32_t tile, int sb, int fb, int lane)
{
    const int row = 16 * sb + (lane & 15), piece = 2 * fb + (lane >> 4);
    ldsm4t(tile + Tile<__nv_bfloat16, D>::at(row, piece), t[0][0].u, t[0][1].u, t[1][0].u, t[1][1].u);
}
template <int D>
__device__ __forceinline__ void load_t(In<float> (&t)[2][2], uint32_t tile, int sb, int fb, int lane)
{
#pragma unroll
    for (int fh = 0; fh < 2; ++fh)
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) {
            const int row = 16 * sb + 8 * kh + 2 * (lane & 3), col = 16 * fb + 8 * fh + (lane >> 2);
            const float x = lds(tile + Tile<float, D>::at(row, col >> 2) + 4 * (col & 3));
            const float y = lds(tile + Tile<float, D>::at(row + 1, col >> 2) + 4 * (col & 3));
            split_tf32(t[fh][kh], make_float2(x, y));
        }
}

// ------------------------------------------------------------------ work
// One recurrence of a launch: the forward, or one of the gradient's three.
struct Role {
    const void *q, *k, *v;   // query, key, value [B, N, H, d]
    const void *x;           // dot: the tensor whose rows meet the output's, or NULL
    void *out;
    float *dot;              // [d / 32][B, H, N]: sign * <x, out> over each 32 entries; in a strong tile with the carried
                             // state's part of out alone
    float *norm;             // [d / 32][B, H, tiles]: sum of squares of the state before a strong tile, 32 rows each, or
                             // -1 where the tile is mild
    const float *state;      // state before each segment [nseg][B, H, d, d], or of the whole call (nseg = 1), or NULL (zero)
    float *state_end;        // nseg = 1: the state after the last token, or NULL
    float sign;
    bool rev;                // the reversed recurrence
    bool transposed;         // `state` lies [key][value]
};

struct Work {
    const float *g;          // [B, N, H]
    int B, H, N, nseg, seg_tiles;   // segments of seg_tiles tiles
    float scale;
};

// Weights of a tile, per warp, in shared memory.
struct Weights {
    float whole[TILE];       // whole part and fraction of -G / ln 2 (of G / ln 2 in the reversed recurrence)
    float frac[TILE];
    float in[TILE];          // weight of the carried state in each token's output
    float out[TILE];         // weight of each token in the next state
};

__device__ __forceinline__ float bounded(float g) { return g < RESET ? RESET : g > -RESET ? -RESET : g; }

// Nearest whole number and the rest of |x| < 2^31, by adding 1.5 * 2^52 to it.
__device__ __forceinline__ void whole_and_rest(double x, float &whole, float &rest)
{
    const double t = x + 6755399441055744.0;
    whole = (float)__double2loint(t);
    rest = (float)(x - (t - 6755399441055744.0));
}

// 2^(whole + rest), |rest| <= 1/2, within an fp32 rounding or two: the Taylor polynomial of degree 7 of 2^rest, whose
// remainder (ln 2 / 2)^8 / 8! is 5e-9, times an exact power.  A state of many tiles ago has been multiplied by as many
// decays: the 2^-22 of the approximate instruction would add up (measured: 1e-6 of the state over 145 segments).
__device__ __forceinline__ float exact_ex2(float whole, float rest)
{
    float p = 1.5252734e-5f;
    p = fmaf(p, rest, 1.5403530e-4f);
    p = fmaf(p, rest, 1.3333558e-3f);
    p = fmaf(p, rest, 9.6181291e-3f);
    p = fmaf(p, rest, 5.5504109e-2f);
    p = fmaf(p, rest, 2.4022651e-1f);
    p = fmaf(p, rest, 6.9314718e-1f);
    return fmaf(p, rest, 1.f) * ex2(whole);
}

// Reads one log decay per lane; returns the decay of the whole tile and, in lane 31's `total`, its G / ln 2.
__device__ __forceinline__ float tile_weights(Weights *w, float g, bool rev, int lane, double &total)
{
    double G = (double)bounded(g) * 1.4426950408889634;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, G, o);
        if (lane >= o) G += up;
    }
    total = G;
    float a, b;
    whole_and_rest(G, a, b);
    const float ea = __shfl_sync(0xffffffffu, a, 31), eb = __shfl_sync(0xffffffffu, b, 31);
    const float fromstart = ex2(a + b), toend = ex2((ea - a) + (eb - b));
    __syncwarp();                          // the previous tile's weights have been read
    w->whole[lane] = rev ? a : -a;
    w->frac[lane] = rev ? b : -b;
    w->in[lane] = rev ? toend : fromstart;
    w->out[lane] = rev ? fromstart : toend;
    __syncwarp();
    return exact_ex2(ea, eb);
}

// Whether a tile is strong, for the gates' gradient: it keeps less than e^-3 of a state, or one of its tokens less than
// e^-1.  Lanes hold the log decays, lane 31 in `total` the tile's G / ln 2.
__device__ __forceinline__ bool strong_tile(float g, double total, int lane)
{
    return __any_sync(0xffffffffu, g < -1.f || (lane == 31 && total < -3.0 * 1.4426950408889634));
}

template <int NS>
__device__ __forceinline__ void group_sync(int group)
{
    if (NS == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * NS) : "memory");
}

template <int NS>
__device__ __forceinline__ bool group_any(int group, bool x)
{
    if (NS == 1) return __any_sync(0xffffffffu, x);
    int any;
    asm volatile("{.reg .pred p, q; setp.ne.u32 p, %1, 0; bar.red.or.pred q, %2, %3, p; selp.s32 %0, 1, 0, q;}"
                 : "=r"(any)
                 : "r"((unsigned)x), "r"(1 + group), "n"(32 * NS)
                 : "memory");
    return any != 0;
}

// The warps of a head copy 32 token rows of it into a tile; rows past N are filled with zeros.  `p` is the thread's own
// first 16 bytes of the tile, `live` the rows before N.
template <typename T, int D>
__device__ __forceinline__ void copy_tile(uint32_t tile, const char *p, size_t row_bytes, int live, int tid)
{
    using L = Tile<T, D>;
    constexpr int NT = D;                                  // threads of a head: 32 per 32 entries
    constexpr int RPI = NT / L::PIECES;                    // rows per step
    const int piece = tid % L::PIECES, r0 = tid / L::PIECES;
    if (live >= TILE) {
#pragma unroll
        for (int r = 0; r < TILE; r += RPI, p += RPI * row_bytes)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tile + L::at(r0 + r, piece)), "l"(p) : "memory");
        return;
    }
    const char *const first = p - (size_t)r0 * row_bytes;   // the tile's first row is before N
#pragma unroll
    for (int r = 0; r < TILE; r += RPI, p += RPI * row_bytes) {
        const bool on = r0 + r < live;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tile + L::at(r0 + r, piece)),
                     "l"(on ? p : first), "r"(on ? 16 : 0)
                     : "memory");
    }
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void wait_copies()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

// The warp's 32 values of all tokens of a tile, transposed: [16-token block][16-value block][half][token half].  `flip`
// exchanges the token blocks, so that a direction known only at run time needs no register chosen at run time.
template <typename T>
using Values = In<T>[2][2][2][2];
template <typename T, int D>
__device__ __forceinline__ void load_values(Values<T> &v, uint32_t vt, bool flip, int slab, int lane)
{
#pragma unroll
    for (int sb = 0; sb < 2; ++sb)
#pragma unroll
        for (int m = 0; m < 2; ++m) load_t<D>(v[sb][m], vt, flip ? 1 - sb : sb, 2 * slab + m, lane);
}

// A masked score is a zero that still meets its value in the matrix units, and 0 times a NaN or an infinity would reach
// the outputs of tokens that do not see that value.  not_finite: whether the warp's 32 values of a tile hold one (0 times
// it is a NaN).  take_out: such values become zeros in the tile; returns the first token of each (lane: entry), in the
// recurrence's direction.  put_back: the outputs of the tokens from there on, and the value's row of the state, become NaNs.
template <typename T, int D>
__device__ __forceinline__ bool not_finite(uint32_t vt, int slab, int lane)
{
    constexpr int PIECES = 32 * (int)sizeof(T) / 16;      // of a row's 32 values
    uint32_t z[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int at = 32 * i + lane;
        uint32_t u[4];
        lds4(vt + Tile<T, D>::at(at / PIECES, slab * PIECES + at % PIECES), u[0], u[1], u[2], u[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (sizeof(T) == 2) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(z[j]) : "r"(u[j]), "r"(0u));
            else z[j] = __float_as_uint(fmaf(__uint_as_float(u[j]), 0.f, __uint_as_float(z[j])));
        }
    }
    const uint32_t any = (z[0] | z[1]) | (z[2] | z[3]);
    return __any_sync(0xffffffffu, (any & (sizeof(T) == 2 ? 0x7fff7fffu : 0x7fffffffu)) != 0);
}
template <typename T, int D>
__device__ __forceinline__ int take_out(uint32_t vt, bool rev, int slab, int lane)
{
    int first = rev ? -1 : TILE;
    for (int i = 0; i < TILE; ++i) {
        const int row = rev ? i : TILE - 1 - i, byte = (32 * slab + lane) * (int)sizeof(T);
        const uint32_t at = vt + Tile<T, D>::at(row, byte >> 4) + (byte & 15);
        if (sizeof(T) == 4) {
            if (!isfinite(lds(at))) {
                first = row;
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(0u) : "memory");
            }
        } else {
            uint16_t u;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(u) : "r"(at) : "memory");
            if ((u & 0x7f80u) == 0x7f80u) {
                first = row;
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((uint16_t)0) : "memory");
            }
        }
    }
    __syncwarp();
    return first;
}
__device__ __forceinline__ void put_nan(float *p) { *p = __uint_as_float(0x7fffffffu); }
__device__ __forceinline__ void put_nan(__nv_bfloat16 *p) { *reinterpret_cast<unsigned short *>(p) = 0x7fff; }
// `out`: the warp's 32 entries of the tile's first token; dot: its first token's, or NULL.
template <typename T, int D>
__device__ __forceinline__ void put_back(float (&S)[2][D / 8][4], T *out, size_t row, float *dot, int first, int live,
                                         bool rev, int lane)
{
    __syncwarp();                              // after the other lanes' writes to the same places
    const int from = rev ? 0 : first, to = min(rev ? first + 1 : TILE, live);
    for (int t = from; t < to; ++t) put_nan(out + t * row + lane);
    if (dot && (rev ? lane <= (int)__reduce_max_sync(0xffffffffu, first) : lane >= (int)__reduce_min_sync(0xffffffffu, first)) &&
        lane < live)
        put_nan(dot + lane);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int f = __shfl_sync(0xffffffffu, first, 16 * m + 8 * h + (lane >> 2));
            if (f >= 0 && f < TILE)
#pragma unroll
                for (int e = 0; e < D / 8; ++e) {
                    put_nan(&S[m][e][2 * h]);
                    put_nan(&S[m][e][2 * h + 1]);
                }
        }
}

// S <- decay S + sum over the tile's tokens of (weight v) k^T, for the warp's 32 values and all keys.  Each tile's
// sum starts from zero and meets the state in one rounded multiply-add: the matrix units cut off low bits as they
// accumulate, which a long sum in them would collect.  LATER: the tiles come from the other end, S <- S + decay sum.
template <typename T, int D, bool LATER = false>
__device__ __forceinline__ void update(float (&S)[2][D / 8][4], uint32_t kt, const Values<T> &v, bool flip,
                                       const Weights *w, float decay, int lane)
{
    Co<T> a[2][2][4];                                // [value block][token block]
#pragma unroll
    for (int sb = 0; sb < 2; ++sb)
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) {
            const int row = 16 * (flip ? 1 - sb : sb) + 8 * kh + 2 * (lane & 3);
            const float2 u = *reinterpret_cast<const float2 *>(&w->out[row]);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int fh = 0; fh < 2; ++fh) split(a[m][sb][2 * kh + fh], mul2(value(v[sb][m][fh][kh]), u));
        }
#pragma unroll
    for (int e = 0; e < D / 16; ++e) {                   // 16 keys: four sums side by side
        In<T> k[2][2][2];
        float c[2][2][4];
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) load_t<D>(k[sb], kt, flip ? 1 - sb : sb, e, lane);
#pragma unroll
        for (int sb = 0; sb < 2; ++sb)
#pragma unroll
            for (int i = 0; i < Steps<T, true>::N; ++i)
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        if (sb == 0 && i == 0) mma<true>(i, c[m][n], a[m][sb], k[sb][n][0], k[sb][n][1]);
                        else mma<false>(i, c[m][n], a[m][sb], k[sb][n][0], k[sb][n][1]);
                    }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                float(&st)[4] = S[m][2 * e + n];
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const float2 old = make_float2(st[i], st[i + 1]), sum = make_float2(c[m][n][i], c[m][n][i + 1]);
                    const float2 r = LATER ? fma2(sum, both(decay), old) : fma2(old, both(decay), sum);
                    st[i] = r.x;
                    st[i + 1] = r.y;
                }
            }
    }
}

// The warp's rows of a [d][d] state in global memory.
template <int D>
__device__ __forceinline__ void read_state(float (&S)[2][D / 8][4], const float *p, bool transposed, int slab, int lane)
{
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = 32 * slab + 16 * m + 8 * h + (lane >> 2), e = 8 * n + 2 * (lane & 3);
                float2 v = make_float2(0.f, 0.f);
                if (p) {
                    if (transposed) v = make_float2(p[e * D + c], p[(e + 1) * D + c]);
                    else v = *reinterpret_cast<const float2 *>(p + c * D + e);
                }
                S[m][n][2 * h] = v.x;
                S[m][n][2 * h + 1] = v.y;
            }
}
template <int D>
__device__ __forceinline__ void write_state(const float (&S)[2][D / 8][4], float *p, int slab, int lane)
{
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = 32 * slab + 16 * m + 8 * h + (lane >> 2), e = 8 * n + 2 * (lane & 3);
                *reinterpret_cast<float2 *>(p + c * D + e) = make_float2(S[m][n][2 * h], S[m][n][2 * h + 1]);
            }
}

template <typename T>
__device__ __forceinline__ void write_rows(T *out, size_t row, const float (&acc)[4][4], int t, int N, int lane);

// Two rows (t, t + 8) of 32 outputs.  A lane holds two neighbouring entries of each of four 8-entry tiles; fp32 stores
// them as they are (a quad fills 32 bytes).
template <>
__device__ __forceinline__ void write_rows<float>(float *out, size_t row, const float (&acc)[4][4], int t, int N,
                                                  int lane)
{
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (t + 8 * h < N)
#pragma unroll
            for (int n = 0; n < 4; ++n)
                *reinterpret_cast<float2 *>(out + (size_t)(8 * h) * row + 8 * n + 2 * (lane & 3)) =
                    make_float2(acc[n][2 * h], acc[n][2 * h + 1]);
}
// bf16: neighbouring lanes swap one register, so that each stores 8 bytes and a quad fills 32.
template <>
__device__ __forceinline__ void write_rows<__nv_bfloat16>(__nv_bfloat16 *out, size_t row, const float (&acc)[4][4],
                                                          int t, int N, int lane)
{
    const bool odd = lane & 1;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < 4; n += 2) {
            const uint32_t a = pack_bf16(acc[n][2 * h], acc[n][2 * h + 1]);
            const uint32_t b = pack_bf16(acc[n + 1][2 * h], acc[n + 1][2 * h + 1]);
            const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
            // even lanes keep tile n, odd lanes tile n + 1
            const uint2 v = odd ? make_uint2(got, b) : make_uint2(a, got);
            if (t + 8 * h < N)
                *reinterpret_cast<uint2 *>(out + (size_t)(8 * h) * row + 8 * (n + odd) + 4 * ((lane & 3) >> 1)) = v;
        }
}

enum Direction { FORWARD, REVERSED, EITHER };   // EITHER: the role says which, so that both run the same instructions

// One recurrence over one segment of one head.  A value that is not finite leaves the state so to the segment's end: there
// it is looked for, and where it is found (true) the segment has to run once more with CAREFUL, which takes such values
// out of their tiles.  (Looking in each tile cost 2 to 9 %.)
template <typename T, int D, Direction DIR, bool DOT, int STAGES, bool CAREFUL>
__device__ __forceinline__ bool recur(const Work &w, const Role &r, int b, int h, int seg, int group, int slab, int lane,
                                      uint32_t ring, Weights *wt)
{
    using L = Tile<T, D>;
    constexpr int NS = D / 32, TENSORS = DOT ? 4 : 3, STAGE = TENSORS * L::BYTES;
    const int tiles = (w.N + TILE - 1) / TILE;
    const int first = seg * w.seg_tiles, n = min(w.seg_tiles, tiles - first);
    if (n <= 0) return false;
    const bool rev = DIR == EITHER ? r.rev : DIR == REVERSED;
    const size_t row = (size_t)w.H * D, row_bytes = row * sizeof(T);
    const size_t at = (size_t)b * w.N * row + (size_t)h * D;
    const float *gp = w.g + (size_t)b * w.N * w.H + h;
    const int tid = slab * 32 + lane;
    auto tile_at = [&](int i) { return (rev ? first + n - 1 - i : first + i) * TILE; };
    // the thread's 16 bytes of the next tile to copy, and the way to the one after it
    const size_t own = (at + (size_t)(tile_at(0) + tid / L::PIECES) * row) * sizeof(T) + tid % L::PIECES * 16;
    const char *src[4] = {(const char *)r.q + own, (const char *)r.k + own, (const char *)r.v + own,
                          DOT ? (const char *)r.x + own : nullptr};
    const long long step = (rev ? -TILE : TILE) * (long long)row_bytes;
    auto load = [&](int i) {
        if (i < n) {
            const uint32_t s = ring + (i % STAGES) * STAGE;
#pragma unroll
            for (int j = 0; j < TENSORS; ++j) {
                copy_tile<T, D>(s + j * L::BYTES, src[j], row_bytes, w.N - tile_at(i), tid);
                src[j] += step;
            }
        }
        commit();
    };
    T *out = (T *)r.out + at + 32 * slab;
    auto load_g = [&](int i) {
        const int t = i < n ? tile_at(i) + lane : w.N;
        return t < w.N ? gp[(size_t)t * w.H] : 0.f;
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) load(i);
    float g = load_g(0);

    // The inputs above were there before the call; the states come from the kernel before this one.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float S[2][D / 8][4];
    const float *st = r.state;
    if (st) st += (((size_t)(w.nseg > 1 ? seg : 0) * w.B + b) * w.H + h) * D * D;
    read_state<D>(S, st, DIR != FORWARD && r.transposed, slab, lane);

    for (int i = 0; i < n; ++i) {
        const float gnext = load_g(i + 1);
        double total;
        const float decay = tile_weights(wt, g, rev, lane, total);
        const bool strong = DOT && strong_tile(g, total, lane);
        g = gnext;
        wait_copies<STAGES - 2>();
        group_sync<NS>(group);               // this tile has landed for every warp, and the last one's slot is free
        load(i + STAGES - 1);
        const uint32_t qt = ring + (i % STAGES) * STAGE, kt = qt + L::BYTES, vt = kt + L::BYTES, xt = vt + L::BYTES;
        const int t0 = tile_at(i);
        const bool bad = CAREFUL && not_finite<T, D>(vt, slab, lane);
        const int nan_from = bad ? take_out<T, D>(vt, rev, slab, lane) : 0;

        // Query rows are taken 16 at a time, the block that sees one key block (itself) first: acc[m] holds the rows
        // from 16 block(m) on.
        auto block = [&](int m) { return rev ? 1 - m : m; };
        // the carried state's part of the outputs
        float acc[2][4][4];
        In<T> q[2][D / 16][4];
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            load_a<D>(q[0][ks], qt, block(0), ks, lane);
            load_a<D>(q[1][ks], qt, block(1), ks, lane);
            Co<T> s[4][2];
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float(&x)[4] = S[c >> 1][2 * ks + e];
                    split(s[c][e], make_float2(x[2 * (c & 1)], x[2 * (c & 1) + 1]));
                }
#pragma unroll
            for (int j = 0; j < Steps<T, true>::N; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        if (ks == 0 && j == 0) mma<true>(j, acc[m][c], q[m][ks], s[c][0], s[c][1]);
                        else mma<false>(j, acc[m][c], q[m][ks], s[c][0], s[c][1]);
                    }
        }
        // <x, out> over the warp's entries of a row: block m, rows l/4 + 8 hh
        auto dot = [&](int m, int hh) {
            float s = 0.f;
            const int rr = 16 * block(m) + 8 * hh + (lane >> 2);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int col = 32 * slab + 8 * c + 2 * (lane & 3);
                float2 x;
                if (sizeof(T) == 4) {
                    x = lds2(xt + L::at(rr, col >> 2) + 4 * (col & 3));
                } else {
                    const uint32_t u = lds_u(xt + L::at(rr, col >> 3) + 2 * (col & 7));
                    x = make_float2(lo_f(u), hi_f(u));
                }
                s = fmaf(x.x, acc[m][c][2 * hh], s);
                s = fmaf(x.y, acc[m][c][2 * hh + 1], s);
            }
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            return s + __shfl_xor_sync(0xffffffffu, s, 2);
        };
        auto put_dot = [&](int m, int hh, float s) {
            const int t = t0 + 16 * block(m) + 8 * hh + (lane >> 2);
            if ((lane & 3) == 0 && t < w.N) r.dot[(((size_t)slab * w.B + b) * w.H + h) * w.N + t] = r.sign * s;
        };
        // A strong tile: the dots of the carried state's part, and that state's norm.  In one place, so that the products
        // below are not split by branches.
        float norm = -1.f;
        if (strong) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const float in = wt->in[16 * block(m) + 8 * hh + (lane >> 2)] * w.scale;
                    put_dot(m, hh, dot(m, hh) * in);
                }
            float2 sq = both(0.f);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int c = 0; c < D / 8; ++c)
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {
                        const float2 x = make_float2(S[m][c][j], S[m][c][j + 1]);
                        sq = fma2(x, x, sq);
                    }
            norm = sq.x + sq.y;
#pragma unroll
            for (int o = 16; o; o >>= 1) norm += __shfl_xor_sync(0xffffffffu, norm, o);
        }
        if (DOT && lane == 0) r.norm[(((size_t)slab * w.B + b) * w.H + h) * tiles + t0 / TILE] = norm;
        // the tile's own part
        Values<T> v;
        load_values<T, D>(v, vt, rev, slab, lane);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int row0 = 16 * block(m);
            float2 gw[2], gf[2];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int t = row0 + 8 * hh + (lane >> 2);
                gw[hh] = both(-wt->whole[t]);
                gf[hh] = both(-wt->frac[t]);
                const float2 wi = both(wt->in[t]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float2 r = mul2(make_float2(acc[m][c][2 * hh], acc[m][c][2 * hh + 1]), wi);
                    acc[m][c][2 * hh] = r.x;
                    acc[m][c][2 * hh + 1] = r.y;
                }
            }
#pragma unroll
            for (int j = 0; j <= m; ++j) {
                const int sb = block(j);
                float sc[2][4];
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    In<T> k[2][2];
                    load_b<D>(k, kt, sb, ks, lane);
#pragma unroll
                    for (int i = 0; i < Steps<T, false>::N; ++i)
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt) {
                            if (ks == 0 && i == 0) mma<true>(i, sc[nt], q[m][ks], k[nt][0], k[nt][1]);
                            else mma<false>(i, sc[nt], q[m][ks], k[nt][0], k[nt][1]);
                        }
                }
                Co<T> p[4];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const int s = 16 * sb + 8 * nt + 2 * (lane & 3);
                    const float2 kw = *reinterpret_cast<const float2 *>(&wt->whole[s]);
                    const float2 kf = *reinterpret_cast<const float2 *>(&wt->frac[s]);
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const float2 e = add2(add2(gw[hh], kw), add2(gf[hh], kf));
                        float2 x = mul2(make_float2(sc[nt][2 * hh], sc[nt][2 * hh + 1]), make_float2(ex2(e.x), ex2(e.y)));
                        if (j == m) {          // key minus query, inside the block
                            const int ahead = 8 * (nt - hh) + 2 * (lane & 3) - (lane >> 2);
                            x.x = (rev ? ahead >= 0 : ahead <= 0) ? x.x : 0.f;
                            x.y = (rev ? ahead >= -1 : ahead <= -1) ? x.y : 0.f;
                        }
                        split(p[2 * nt + hh], x);
                    }
                }
#pragma unroll
                for (int i = 0; i < Steps<T, true>::N; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) mma<false>(i, acc[m][c], p, v[j][c >> 1][c & 1][0], v[j][c >> 1][c & 1][1]);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    const float2 r = mul2(make_float2(acc[m][c][j], acc[m][c][j + 1]), both(w.scale));
                    acc[m][c][j] = r.x;
                    acc[m][c][j + 1] = r.y;
                }
            if (DOT) {
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const float s = dot(m, hh);
                    if (!strong) put_dot(m, hh, s);
                }
            }
            const int t = t0 + row0 + (lane >> 2);
            write_rows<T>(out + (size_t)t * row, row, acc[m], t, w.N, lane);
        }
        if (bad)
            put_back<T, D>(S, out + (size_t)t0 * row, row,
                           DOT && !strong ? r.dot + (((size_t)slab * w.B + b) * w.H + h) * w.N + t0 : nullptr, nan_from,
                           w.N - t0, rev, lane);
        if (i + 1 < n || r.state_end) update<T, D>(S, kt, v, rev, wt, decay, lane);
    }
    wait_copies<0>();
    if (!CAREFUL) {
        float2 z = both(0.f);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < D / 8; ++e)
#pragma unroll
                for (int j = 0; j < 4; j += 2) z = fma2(make_float2(S[m][e][j], S[m][e][j + 1]), both(0.f), z);
        bool bad = ((__float_as_uint(z.x) | __float_as_uint(z.y)) & 0x7fffffffu) != 0;
        if (!r.state_end) bad |= not_finite<T, D>(ring + ((n - 1) % STAGES) * STAGE + 2 * L::BYTES, slab, lane);
        if (group_any<NS>(group, bad)) return true;
    }
    if (r.state_end) write_state<D>(S, r.state_end + ((size_t)b * w.H + h) * D * D, slab, lane);
    return false;
}

// What a segment adds to the state, from zero, and its decay.  The tiles are taken against the recurrence's direction,
// each with the decay of those after it: the last ones read here are the first that the recurrence reads, and still in L2.
template <typename T, int D, int STAGES>
__device__ __forceinline__ void total(const Work &w, const void *key, const void *val, float *part, float *decays, bool rev,
                                      int b, int h, int seg, int group, int slab, int lane, uint32_t ring, Weights *wt)
{
    using L = Tile<T, D>;
    constexpr int NS = D / 32, STAGE = 2 * L::BYTES;
    const int tiles = (w.N + TILE - 1) / TILE;
    const int first = seg * w.seg_tiles, n = min(w.seg_tiles, tiles - first);
    const size_t row = (size_t)w.H * D, row_bytes = row * sizeof(T);
    const size_t at = (size_t)b * w.N * row + (size_t)h * D;
    const float *gp = w.g + (size_t)b * w.N * w.H + h;
    const int tid = slab * 32 + lane;
    auto tile_at = [&](int i) { return (rev ? first + i : first + n - 1 - i) * TILE; };
    const size_t own = (at + (size_t)(tile_at(0) + tid / L::PIECES) * row) * sizeof(T) + tid % L::PIECES * 16;
    const char *kp = (const char *)key + own, *vp = (const char *)val + own;
    const long long step = (rev ? TILE : -TILE) * (long long)row_bytes;
    auto load = [&](int i) {
        if (i < n) {
            const uint32_t s = ring + (i % STAGES) * STAGE;
            copy_tile<T, D>(s, kp, row_bytes, w.N - tile_at(i), tid);
            copy_tile<T, D>(s + L::BYTES, vp, row_bytes, w.N - tile_at(i), tid);
            kp += step;
            vp += step;
        }
        commit();
    };
    auto load_g = [&](int i) {
        const int t = i < n ? tile_at(i) + lane : w.N;
        return t < w.N ? gp[(size_t)t * w.H] : 0.f;
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) load(i);
    float g = load_g(0);
    float S[2][D / 8][4] = {};
    double sum = 0.0;
    float after = 1.f;
    for (int i = 0; i < n; ++i) {
        const float gnext = load_g(i + 1);
        double t;
        const float decay = tile_weights(wt, g, rev, lane, t);
        sum += t;
        g = gnext;
        wait_copies<STAGES - 2>();
        group_sync<NS>(group);
        load(i + STAGES - 1);
        const uint32_t kt = ring + (i % STAGES) * STAGE;
        Values<T> v;
        load_values<T, D>(v, kt + L::BYTES, false, slab, lane);
        update<T, D, true>(S, kt, v, false, wt, after, lane);
        after *= decay;
    }
    wait_copies<0>();
    const size_t at_s = ((size_t)seg * w.B + b) * w.H + h;
    write_state<D>(S, part + at_s * D * D, slab, lane);
    if (decays && slab == 0 && lane == 31) decays[at_s] = (float)exp2(sum);
}

}  // namespace gated
}  // namespace lcla

#endif
