// lcla_rope.cu -- rotary tables on the device (lcla_rotary_tables) and the
// per-head RMS norm of queries and keys with the rotation in the same pass,
// forward and gradient (lcla_qk_norm_rope, lcla_qk_norm_rope_backward).
//
// Tables.  cos/sin[n][p] = amp * cos/sin(pos_a(n) * f_p).  A frequency is kept
// as a 64-bit fraction of a revolution, so that the product with an integer
// position, taken modulo 2^64, is the reduced angle of that fraction without any
// rounding.  The fraction itself is within 2^-64 (host, long double), which a
// position of 2^36 makes 2^-28 of a revolution.
//
// Norm and rotation.  A row is one head of one token:
//   n = x * rsqrt(mean(x^2) + eps) * w,   y = R n   on the first rd entries,
// with R the rotation of interleaved pairs (2p, 2p+1) or of half-layout pairs
// (p, p + rd/2).  Gradient, with m = R^T gy, r = rsqrt(mean(x^2) + eps):
//   gx = r (w m) - x r^3 mean(w m x),   gw = sum over rows of m x r.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "lcla.h"
#include "lcla_f32x2.cuh"
#include "lcla_host.h"

namespace {

using namespace lcla;
using namespace lcla::host;

// ------------------------------------------------------------------ tables
constexpr int kMaxPairs = 128;
constexpr int kMaxAxes = 3;
constexpr long long kMaxIndex = 1ll << 36;   // where a frequency's 2^-64 is 2e-8 of an angle
constexpr int kTabThreads = 256;
constexpr int kTabTokens = 4;      // tokens per thread

// Division of 0 <= n < 2^31 by a constant (Granlund and Montgomery, "Division by Invariant Integers using
// Multiplication"): n / d = (high 32 bits of n m, plus n) >> s.
struct Divisor {
    unsigned d, m, s;
};
Divisor make_divisor(unsigned d)
{
    unsigned s = 0;
    while ((1ull << s) < d) ++s;
    return Divisor{d, (unsigned)((((1ull << s) - d) << 32) / d + 1), s};
}
__device__ __forceinline__ unsigned divide(unsigned n, const Divisor &d) { return (__umulhi(n, d.m) + n) >> d.s; }

struct TabPlan {
    unsigned long long freq[kMaxPairs];   // revolutions per position, times 2^64
    unsigned char axis[kMaxPairs];
    long long first;
    long long extent[kMaxAxes];           // extent[a]: how far axis a counts (a >= 1)
    Divisor by[kMaxAxes];                 // the same as divisors, where they and all indices are below 2^31
    bool narrow;
    int axes, pairs, N;
    float amp;
};

// sin and cos of r * 2 pi / 2^64 for |r| <= 2^61, an eighth of a turn: the Taylor polynomials of degree 9 and 10,
// whose remainders (pi/4)^11/11! and (pi/4)^12/12! lie below 2e-9.
__device__ __forceinline__ void sincos_eighth(long long r, float &s, float &c)
{
    const float x = __ll2float_rn(r) * 3.4061215800865545e-19f;   // 2 pi / 2^64
    const float y = x * x;
    s = fmaf(y, fmaf(y, fmaf(y, 2.7557319e-6f, -1.9841270e-4f), 8.3333333e-3f), -1.6666667e-1f);
    s = fmaf(x * y, s, x);
    c = fmaf(y, fmaf(y, fmaf(y, fmaf(y, -2.7557319e-7f, 2.4801587e-5f), -1.3888889e-3f), 4.1666667e-2f), -0.5f);
    c = fmaf(y, c, 1.f);
}

// Bound by the integer and conversion instructions it issues, 48 for an entry of both tables: the minute-scale latent's
// 108.6 MB in 28 us (a first version with divisions and shared-memory reads for every four entries took 57; 32-bit
// positions and two 32-bit conversions instead of a 64-bit one changed nothing).  A thread keeps VEC entries'
// frequencies in registers and writes them for kTabTokens tokens; a block covers 256 / (pairs / VEC) tokens at a time.
template <int VEC>
__global__ void __launch_bounds__(kTabThreads)
rotary_tables_k(const __grid_constant__ TabPlan p, const long long *__restrict__ positions, float *__restrict__ cosv,
                float *__restrict__ sinv)
{
    const int groups = p.pairs / VEC, rows = kTabThreads / groups;
    const int row = threadIdx.x / groups, j = (threadIdx.x - row * groups) * VEC;
    if (row >= rows) return;
    unsigned long long freq[VEC];
    int axis[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        freq[i] = p.freq[j + i];
        axis[i] = p.axis[j + i];
    }
    const int n0 = (int)((long long)blockIdx.x * rows * kTabTokens) + row;
    unsigned long long given[kTabTokens][kMaxAxes];
    if (positions) {
#pragma unroll
        for (int k = 0; k < kTabTokens; ++k)
#pragma unroll
            for (int a = 0; a < kMaxAxes; ++a)
                given[k][a] = a < p.axes ? (unsigned long long)positions[(size_t)a * p.N + min(n0 + k * rows, p.N - 1)] : 0;
    }
#pragma unroll
    for (int k = 0; k < kTabTokens; ++k) {
        const int n = n0 + k * rows;
        if (n >= p.N) return;
        unsigned long long pos[kMaxAxes] = {0, 0, 0};
        if (positions) {
#pragma unroll
            for (int a = 0; a < kMaxAxes; ++a) pos[a] = given[k][a];
        } else if (p.narrow) {
            unsigned m = (unsigned)(p.first + n);
#pragma unroll
            for (int a = kMaxAxes - 1; a > 0; --a)
                if (a < p.axes) {
                    const unsigned q = divide(m, p.by[a]);
                    pos[a] = m - q * p.by[a].d;
                    m = q;
                }
            pos[0] = m;
        } else {
            long long m = p.first + n;
#pragma unroll
            for (int a = kMaxAxes - 1; a > 0; --a)
                if (a < p.axes) {
                    const long long q = m / p.extent[a];
                    pos[a] = (unsigned long long)(m - q * p.extent[a]);
                    m = q;
                }
            pos[0] = (unsigned long long)m;
        }
        float c[VEC], s[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const unsigned long long turn = (axis[i] == 0 ? pos[0] : axis[i] == 1 ? pos[1] : pos[2]) * freq[i];
            // the nearest quarter turn, and what is left
            const unsigned high = (unsigned)(turn >> 32), quad = (high + 0x20000000u) >> 30;
            const unsigned left = high - (quad << 30);
            float sn, cs;
            sincos_eighth((long long)(((unsigned long long)left << 32) | (unsigned)turn), sn, cs);
            const unsigned x = __float_as_uint((quad & 1) ? sn : cs), y = __float_as_uint((quad & 1) ? cs : sn);
            c[i] = __uint_as_float(x ^ (((quad + 1) << 30) & 0x80000000u)) * p.amp;   // quarters 1 and 2
            s[i] = __uint_as_float(y ^ ((quad << 30) & 0x80000000u)) * p.amp;         // quarters 2 and 3
        }
        const size_t at = (size_t)n * p.pairs + j;
        if (VEC == 4) {
            *reinterpret_cast<float4 *>(cosv + at) = make_float4(c[0], c[VEC > 1], c[VEC / 2], c[VEC - 1]);
            *reinterpret_cast<float4 *>(sinv + at) = make_float4(s[0], s[VEC > 1], s[VEC / 2], s[VEC - 1]);
        } else {
            cosv[at] = c[0];
            sinv[at] = s[0];
        }
    }
}

// ------------------------------------------------------- norm and rotation
constexpr int kVec = 8;            // entries of a row per lane
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kReads = 5;          // reads of a unit of the forward

struct View {                      // rows of one tensor: token t, head h at p + t * ld + h * d
    const void *p;
    long long ld;
};

struct NormArgs {
    View x[2], gy[2];              // 0: queries, 1: keys
    void *y[2];
    long long ldy[2];
    const float *w[2];
    const float *cosv, *sinv;
    const long long *positions;
    float *part;                   // gradient: [ctas][d] per side, queries' CTAs first
    long long T;                   // tokens, B * N
    int N, P, d, rd, heads[2], units[2], ctas[2];
    int span[2];                   // gradient: reads that a warp takes of a token at a time
    float eps, inv_d;
};

// A lane's 8 entries of a row as two pairs of even and two of odd ones, for packed arithmetic.
struct Eight {
    float2 e[2], o[2];             // e[j] = entries 4j, 4j + 2; o[j] = entries 4j + 1, 4j + 3
};
__device__ __forceinline__ Eight zeros() { return Eight{{both(0.f), both(0.f)}, {both(0.f), both(0.f)}}; }
__device__ __forceinline__ float total(const Eight &a)
{
    const float2 s = add2(add2(a.e[0], a.e[1]), add2(a.o[0], a.o[1]));
    return s.x + s.y;
}
__device__ __forceinline__ Eight times(const Eight &a, const Eight &b)
{
    return Eight{{mul2(a.e[0], b.e[0]), mul2(a.e[1], b.e[1])}, {mul2(a.o[0], b.o[0]), mul2(a.o[1], b.o[1])}};
}
__device__ __forceinline__ Eight times(const Eight &a, float s)
{
    const float2 b = both(s);
    return Eight{{mul2(a.e[0], b), mul2(a.e[1], b)}, {mul2(a.o[0], b), mul2(a.o[1], b)}};
}
__device__ __forceinline__ Eight plus_times(const Eight &a, const Eight &b, const Eight &c)   // a b + c
{
    return Eight{{fma2(a.e[0], b.e[0], c.e[0]), fma2(a.e[1], b.e[1], c.e[1])},
                 {fma2(a.o[0], b.o[0], c.o[0]), fma2(a.o[1], b.o[1], c.o[1])}};
}
__device__ __forceinline__ Eight plus_times(const Eight &a, float s, const Eight &c)
{
    const float2 b = both(s);
    return Eight{{fma2(a.e[0], b, c.e[0]), fma2(a.e[1], b, c.e[1])}, {fma2(a.o[0], b, c.o[0]), fma2(a.o[1], b, c.o[1])}};
}

// The same entries as they lie in memory.
template <typename T>
struct Raw {
    static constexpr int WORDS = 2 * (int)sizeof(T);
    uint32_t w[WORDS];
    __device__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < WORDS; i += 4) {
            const uint4 u = reinterpret_cast<const uint4 *>(p)[i / 4];
            w[i] = u.x; w[i + 1] = u.y; w[i + 2] = u.z; w[i + 3] = u.w;
        }
    }
    __device__ void store(T *p) const
    {
#pragma unroll
        for (int i = 0; i < WORDS; i += 4) reinterpret_cast<uint4 *>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
    __device__ void zero()
    {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0;
    }
    __device__ Raw from_lane(int lane) const   // every lane of the warp takes part
    {
        Raw r;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) r.w[i] = __shfl_sync(0xffffffffu, w[i], lane);
        return r;
    }
    __device__ Eight get() const
    {
        Eight x;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (sizeof(T) == 2) {
                const uint32_t a = w[2 * j], b = w[2 * j + 1];
                x.e[j] = make_float2(__uint_as_float(a << 16), __uint_as_float(b << 16));
                x.o[j] = make_float2(__uint_as_float(a & 0xffff0000u), __uint_as_float(b & 0xffff0000u));
            } else {
                const uint32_t *v = w + (4 * j) % WORDS;
                x.e[j] = make_float2(__uint_as_float(v[0]), __uint_as_float(v[2]));
                x.o[j] = make_float2(__uint_as_float(v[1]), __uint_as_float(v[3]));
            }
        }
        return x;
    }
    __device__ void set(const Eight &x)
    {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (sizeof(T) == 2) {
                w[2 * j] = pack(x.e[j].x, x.o[j].x);
                w[2 * j + 1] = pack(x.e[j].y, x.o[j].y);
            } else {
                uint32_t *v = w + (4 * j) % WORDS;
                v[0] = __float_as_uint(x.e[j].x);
                v[1] = __float_as_uint(x.o[j].x);
                v[2] = __float_as_uint(x.e[j].y);
                v[3] = __float_as_uint(x.o[j].y);
            }
        }
    }
    __device__ static uint32_t pack(float lo, float hi)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

// Entries [at, at + 8) of a fp32 array, or `fill` without it.
__device__ __forceinline__ Eight eight_of(const float *p, int at, bool on, float fill)
{
    float v[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = fill;
    if (p && on) {
        const float4 a = reinterpret_cast<const float4 *>(p + at)[0], b = reinterpret_cast<const float4 *>(p + at)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    return Eight{{make_float2(v[0], v[2]), make_float2(v[4], v[6])}, {make_float2(v[1], v[3]), make_float2(v[5], v[7])}};
}

// Each entry of R x (or R^T x) is c x + s x', x' the other entry of its pair: in the same lane (interleaved) or in lane
// `partner` (half layout).  c and s serve all rows of a token.
template <bool HALF>
struct Turn {
    Eight c, s;

    __device__ static int partner(const NormArgs &a, int l, int lane)
    {
        const int per = a.rd / 2 / kVec;            // lanes per half
        return !HALF || kVec * l >= a.rd ? lane : l >= per ? lane - per : lane + per;
    }
    // sign +1: R, -1: R^T
    __device__ void load(const NormArgs &a, long long token, int l, float sign)
    {
        long long row = a.positions ? a.positions[token] : (unsigned)token % (unsigned)a.N;
        row = row < 0 ? 0 : row >= a.P ? a.P - 1 : row;   // a bad position reads a wrong row, never out of bounds
        const int hp = a.rd / 2;
        const float *pc = a.cosv + row * hp, *ps = a.sinv + row * hp;
        if (HALF) {
            const bool on = kVec * l < a.rd, second = kVec * l >= hp;
            const int p0 = second ? kVec * l - hp : kVec * l;
            c = eight_of(pc, p0, on, 1.f);
            s = times(eight_of(ps, p0, on, 0.f), second ? sign : -sign);
        } else {
            const int p0 = kVec / 2 * l;
            float4 u = make_float4(1.f, 1.f, 1.f, 1.f), v = make_float4(0.f, 0.f, 0.f, 0.f);
            if ((hp & 3) == 0) {                          // whole 16-byte pieces of aligned table rows
                if (p0 < hp) {
                    u = *reinterpret_cast<const float4 *>(pc + p0);
                    v = *reinterpret_cast<const float4 *>(ps + p0);
                }
            } else {
                if (p0 < hp) { u.x = pc[p0]; v.x = ps[p0]; }
                if (p0 + 1 < hp) { u.y = pc[p0 + 1]; v.y = ps[p0 + 1]; }
                if (p0 + 2 < hp) { u.z = pc[p0 + 2]; v.z = ps[p0 + 2]; }
                if (p0 + 3 < hp) { u.w = pc[p0 + 3]; v.w = ps[p0 + 3]; }
            }
            c.e[0] = c.o[0] = make_float2(u.x, u.y);
            c.e[1] = c.o[1] = make_float2(u.z, u.w);
            s.o[0] = make_float2(sign * v.x, sign * v.y);
            s.o[1] = make_float2(sign * v.z, sign * v.w);
            s.e[0] = make_float2(-s.o[0].x, -s.o[0].y);
            s.e[1] = make_float2(-s.o[1].x, -s.o[1].y);
        }
    }
};
// The other entries of the pairs.
template <bool HALF, typename T>
__device__ __forceinline__ Eight others(const Raw<T> &r, const Eight &x, int partner)
{
    if (HALF) return r.from_lane(partner).get();
    return Eight{{x.o[0], x.o[1]}, {x.e[0], x.e[1]}};
}

template <int G>
__device__ __forceinline__ float row_sum(float v)   // over the G lanes of a row
{
#pragma unroll
    for (int o = G / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Bound by HBM (x read, y written).  G lanes hold a row, 8 entries (16 bytes of bf16) each, so a warp reads 32 / G
// consecutive heads of a token at once.  A unit is U such reads of one token and side: the rotation's factors, times
// the weight, are made once for all of them, and the U reads are in flight together.
template <typename T, int G, bool HALF, int U>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 3)
qk_norm_rope_k(const __grid_constant__ NormArgs a)
{
    constexpr int R = 32 / G;
    const int lane = threadIdx.x & 31, l = lane % G, sub = lane / G;
    const unsigned unit = blockIdx.x * kWarps + (threadIdx.x >> 5), per = a.units[0] + a.units[1];
    const long long token = unit / per;
    if (token >= a.T) return;
    int part = (int)(unit % per);
    const int side = part >= a.units[0];
    if (side) part -= a.units[0];
    const int H = a.heads[side], h0 = part * U * R + sub;
    const bool in = kVec * l < a.d;
    const T *x = static_cast<const T *>(a.x[side].p) + token * a.x[side].ld + kVec * l + (size_t)h0 * a.d;
    T *y = static_cast<T *>(a.y[side]) + token * a.ldy[side] + kVec * l + (size_t)h0 * a.d;
    Raw<T> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        raw[u].zero();
        if (in && h0 + u * R < H) raw[u].load(x + u * R * a.d);
    }
    const int other = Turn<HALF>::partner(a, l, lane);
    Turn<HALF> t;
    t.load(a, token, l, 1.f);
    const float *w = a.w[side];
    if (w) {   // the factor of an entry's partner carries the partner's weight
        const int lp = l + other - lane;
        const Eight mine = eight_of(w, kVec * l, in, 1.f);
        const Eight its = HALF ? eight_of(w, kVec * lp, in, 1.f) : Eight{{mine.o[0], mine.o[1]}, {mine.e[0], mine.e[1]}};
        t.c = times(t.c, mine);
        t.s = times(t.s, its);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Eight v = raw[u].get();
        const float r = rsqrtf(fmaf(row_sum<G>(total(times(v, v))), a.inv_d, a.eps));
        const Eight o = times(plus_times(v, t.c, times(others<HALF>(raw[u], v, other), t.s)), r);
        Raw<T> res;
        res.set(o);
        if (in && h0 + u * R < H) res.store(y + u * R * a.d);
    }
}

// Bound by HBM (x and gy read, gx written).  CTAs take one side each and stride over its visits, so that the weight's
// gradient gathers in registers; a CTA leaves one [d] partial, and qk_norm_weight_grad_k adds those in a fixed order.
// A visit is a run of `span` units of one token, a unit U reads of 32 / G heads in flight together.  A training batch at
// d = 64 (252 MB) takes 54 us so: each warp loads and computes in turn, and issuing its 30 M warp instructions alone takes
// about half of that.  Measured and dropped: the next unit's reads held in registers meanwhile (60 us: it spills), a ring of
// reads in shared memory per warp (68 us: more instructions).  A unit is of one token, so few heads leave most of it idle:
// 300000 tokens of 1 + 1 heads, d = 32, take 618 us (the forward 330) where HBM would take 23 (18).
template <typename T>
struct Back {
    static constexpr int READS = sizeof(T) == 2 ? 5 : 3;   // what 128 registers hold
};

template <typename T, int G, bool HALF>
__global__ void __launch_bounds__(kThreads, 2)
qk_norm_rope_backward_k(const __grid_constant__ NormArgs a)
{
    constexpr int R = 32 / G, U = Back<T>::READS;
    __shared__ float red[kWarps][G * kVec];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, l = lane % G, sub = lane / G;
    const int side = (int)blockIdx.x >= a.ctas[0];
    const int cta = side ? (int)blockIdx.x - a.ctas[0] : (int)blockIdx.x;
    const int H = a.heads[side];
    const bool in = kVec * l < a.d;
    const Eight w = eight_of(a.w[side], kVec * l, in, 1.f);
    Eight gw = zeros();
    const int other = Turn<HALF>::partner(a, l, lane);
    const unsigned span = a.span[side], per_token = (a.units[side] + span - 1) / span;
    const long long visits = a.T * per_token, step = (long long)a.ctas[side] * kWarps;
    for (long long visit = (long long)cta * kWarps + wid; visit < visits; visit += step) {
        const unsigned first = (unsigned)visit % per_token * span;
        const long long token = (unsigned)visit / per_token;
        Turn<HALF> t;
        t.load(a, token, l, -1.f);
        const T *x = static_cast<const T *>(a.x[side].p) + token * a.x[side].ld + kVec * l;
        const T *gy = static_cast<const T *>(a.gy[side].p) + token * a.gy[side].ld + kVec * l;
        T *gx = static_cast<T *>(a.y[side]) + token * a.ldy[side] + kVec * l;
        const int last = min((int)(first + span) * U * R, H);
        for (int h0 = (int)first * U * R + sub; h0 - sub < last; h0 += U * R) {
            Raw<T> rx[U], rg[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                rx[u].zero();
                rg[u].zero();
                if (in && h0 + u * R < H) {
                    rx[u].load(x + (h0 + u * R) * a.d);
                    rg[u].load(gy + (h0 + u * R) * a.d);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Eight v = rx[u].get(), g = rg[u].get();
                const Eight m = plus_times(g, t.c, times(others<HALF>(rg[u], g, other), t.s));
                const Eight mx = times(m, v), wm = times(m, w);
                const float ss = row_sum<G>(total(times(v, v))), dot = row_sum<G>(total(times(mx, w)));
                const bool live = h0 + u * R < H;            // rows past the last head add nothing, whatever eps is
                const float r = live ? rsqrtf(fmaf(ss, a.inv_d, a.eps)) : 0.f;
                gw = plus_times(mx, r, gw);
                const Eight o = times(plus_times(v, -(dot * a.inv_d * r * r), wm), r);
                Raw<T> res;
                res.set(o);
                if (in && live) res.store(gx + (h0 + u * R) * a.d);
            }
        }
    }
    if (!a.part) return;
    const float mine[kVec] = {gw.e[0].x, gw.o[0].x, gw.e[0].y, gw.o[0].y, gw.e[1].x, gw.o[1].x, gw.e[1].y, gw.o[1].y};
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        float s = mine[j];
#pragma unroll
        for (int o = G; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (sub == 0) red[wid][kVec * l + j] = s;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.d; i += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) s += red[k][i];
        a.part[(size_t)blockIdx.x * a.d + i] = s;
    }
}

// One block per side and 32 entries of d: its 32 warps each add every 32nd of the CTAs' partials, in double.
constexpr int kSumThreads = 1024;
constexpr int kBwdCtas = 148 * 2;    // CTAs of the gradient: what is resident at once
__global__ void __launch_bounds__(kSumThreads)
qk_norm_weight_grad_k(const float *__restrict__ part, int d, int ctas_q, int ctas_k, float *gwq, float *gwk)
{
    constexpr int W = kSumThreads / 32, PER = (kBwdCtas + W - 1) / W;
    __shared__ double red[W][33];
    const int side = blockIdx.y, lane = threadIdx.x & 31, wid = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
    float *gw = side ? gwk : gwq;
    if (!gw) return;
    const float *p = part + (side ? (size_t)ctas_q * d : 0);
    const int n = side ? ctas_k : ctas_q, at = i < d ? i : d - 1;
    float v[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) v[k] = wid + k * W < n ? p[(size_t)(wid + k * W) * d + at] : 0.f;
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < PER; ++k) s += v[k];
    red[wid][lane] = s;
    __syncthreads();
    if (wid != 0) return;
#pragma unroll 8
    for (int k = 1; k < W; ++k) s += red[k][lane];
    if (i < d) gw[i] = (float)s;
}

// ----------------------------------------------------------------- host

constexpr long long kMaxUnits = 0xfffffff0ll;   // the kernels count units in 32 bits, rounded up to whole blocks

int lanes_per_row(int d)            // the power of two that holds d / 8 lanes
{
    int g = 4;
    while (g * kVec < d) g *= 2;
    return g;
}

template <typename T, bool HALF, int U>
void launch_norm(const NormArgs &a, int G, unsigned grid, cudaStream_t st)
{
    switch (G) {
    case 4: qk_norm_rope_k<T, 4, HALF, U><<<grid, kThreads, 0, st>>>(a); break;
    case 8: qk_norm_rope_k<T, 8, HALF, U><<<grid, kThreads, 0, st>>>(a); break;
    case 16: qk_norm_rope_k<T, 16, HALF, U><<<grid, kThreads, 0, st>>>(a); break;
    default: qk_norm_rope_k<T, 32, HALF, U><<<grid, kThreads, 0, st>>>(a);
    }
}
template <typename T>
void launch_norm(const NormArgs &a, int G, bool half, int U, unsigned grid, cudaStream_t st)
{
    if (half) U == 1 ? launch_norm<T, true, 1>(a, G, grid, st) : launch_norm<T, true, kReads>(a, G, grid, st);
    else U == 1 ? launch_norm<T, false, 1>(a, G, grid, st) : launch_norm<T, false, kReads>(a, G, grid, st);
}

template <typename T, bool HALF>
void launch_norm_backward(const NormArgs &a, int G, unsigned grid, cudaStream_t st)
{
    switch (G) {
    case 4: qk_norm_rope_backward_k<T, 4, HALF><<<grid, kThreads, 0, st>>>(a); break;
    case 8: qk_norm_rope_backward_k<T, 8, HALF><<<grid, kThreads, 0, st>>>(a); break;
    case 16: qk_norm_rope_backward_k<T, 16, HALF><<<grid, kThreads, 0, st>>>(a); break;
    default: qk_norm_rope_backward_k<T, 32, HALF><<<grid, kThreads, 0, st>>>(a);
    }
}

// Units of U reads per token, on each side.  Several 16-byte reads a lane in flight keep HBM busy (480p, 587 MB:
// 106 us with 3, 100 us with 5, 104 us with 9); a call with too few rows to fill the SMs that way takes U = 1, which
// has the shorter chain.  Measured with 1 and 5, 70 + 70 heads of d = 32, by tokens: 1 2.5 and 2.7 us, 64 2.9 and 3.3, 256
// (4608 reads) 3.3 and 3.5, 400 4.3 and 4.1, 1000 6.8 and 5.1.
int set_units(NormArgs &a, int G)
{
    const int R = 32 / G;
    const long long reads = a.T * ((a.heads[0] + R - 1) / R + (a.heads[1] + R - 1) / R);
    const int U = reads < 148 * 32 ? 1 : kReads;
    for (int s = 0; s < 2; ++s) a.units[s] = (a.heads[s] + R * U - 1) / (R * U);
    return U;
}

int check_norm(int B, int N, int H, int Hk, int d, int rd, int half, int P, const void *positions, float eps, int dtype)
{
    if (B < 1 || N < 0 || H < 1 || Hk < 0 || P < (N > 0) || d < 1 || rd < 0 || rd > d || (rd & 1)) return LCLA_ERR_INVALID_ARG;
    if (dtype != LCLA_BF16 && dtype != LCLA_F32) return LCLA_ERR_INVALID_ARG;
    if (half != 0 && half != 1) return LCLA_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !isfinite(eps)) return LCLA_ERR_INVALID_ARG;
    if (!positions && P < N) return LCLA_ERR_INVALID_ARG;
    if ((d % kVec) != 0 || d > 256) return LCLA_ERR_UNSUPPORTED;
    if (half && (rd % (2 * kVec)) != 0) return LCLA_ERR_UNSUPPORTED;
    if ((long long)B * N > (1ll << 30) || H > 65536 || Hk > 65536) return LCLA_ERR_UNSUPPORTED;
    if ((long long)B * N * (H + Hk) > (1ll << 36)) return LCLA_ERR_UNSUPPORTED;
    return LCLA_OK;
}

// One tensor of [T] tokens whose rows of `width` entries lie `ld` entries apart.
struct Span {
    const void *p;
    long long ld;
    size_t width, bytes, esz;
};

int make_span(Span *s, const void *p, long long ld, long long T, int heads, int d, size_t esz)
{
    const size_t width = (size_t)heads * d;
    *s = Span{p, ld, width * esz, T && heads ? ((size_t)(T - 1) * ld + width) * esz : 0, esz};
    if (!heads || !T) return LCLA_OK;
    if (!p || ld < (long long)width || ld > (1ll << 32)) return LCLA_ERR_INVALID_ARG;
    if (misaligned(p) || (ld * esz) % 16 != 0) return LCLA_ERR_MISALIGNED;
    return LCLA_OK;
}

// Whether two tensors share bytes.  Two windows of the columns of one buffer (the same ld) are told apart.
bool spans_meet(const Span &a, const Span &b)
{
    if (!overlaps(a.p, a.bytes, b.p, b.bytes)) return false;
    if (a.ld != b.ld || a.ld == 0) return true;
    const size_t ld = (size_t)a.ld * a.esz;
    const uintptr_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
    const size_t off = pa < pb ? (pb - pa) % ld : (ld - (pa - pb) % ld) % ld;   // b's column, counted from a's
    return off < a.width || off + b.width > ld;
}
bool same_span(const Span &a, const Span &b) { return a.p == b.p && a.ld == b.ld && a.width == b.width; }
Span flat(const void *p, size_t bytes) { return Span{p, 0, bytes, p ? bytes : 0, 1}; }

}  // namespace

extern "C" {

int lcla_rotary_tables(const long long *positions, long long first, int N, int axes, const int *axis_dims,
                       const int *axis_extents, double theta, int scaling, double factor, double original_len,
                       double beta_fast, double beta_slow, float *rope_cos, float *rope_sin, void *stream)
{
    if (N < 0 || axes < 1 || axes > kMaxAxes || !axis_dims) return LCLA_ERR_INVALID_ARG;
    if (!(theta >= 1.0) || !isfinite(theta)) return LCLA_ERR_INVALID_ARG;
    if (scaling < LCLA_ROPE_NONE || scaling > LCLA_ROPE_YARN) return LCLA_ERR_INVALID_ARG;
    if (scaling != LCLA_ROPE_NONE && (!(factor >= 1.0) || !isfinite(factor))) return LCLA_ERR_INVALID_ARG;
    if (scaling == LCLA_ROPE_YARN && (!(original_len > 0.0) || !isfinite(original_len) || !(beta_slow >= 0.0) ||
                                      !(beta_fast > beta_slow) || !isfinite(beta_fast)))
        return LCLA_ERR_INVALID_ARG;
    TabPlan p = {};
    const long double two_pi = 6.283185307179586476925286766559L, per_radian = 18446744073709551616.0L / two_pi;
    for (int a = 0; a < axes; ++a) {
        const int D = axis_dims[a];
        if (D < 2 || (D & 1)) return LCLA_ERR_INVALID_ARG;
        if (p.pairs + D / 2 > kMaxPairs) return LCLA_ERR_UNSUPPORTED;
        if (scaling == LCLA_ROPE_NTK && D == 2) return LCLA_ERR_INVALID_ARG;   // its exponent D / (D - 2)
        // theta^(-2j/D) from a few powers, since powl takes 0.2 us: every 8th, the fourth and the first, and products of at
        // most four of them, within 7 roundings of 64 bits
        const long double base =
            scaling == LCLA_ROPE_NTK ? (long double)theta * powl(factor, (long double)D / (D - 2)) : (long double)theta;
        auto power = [&](int j) { return powl(base, -2.0L * j / D); };
        long double low[8] = {1.0L, D > 2 ? power(1) : 1.0L}, high = 1.0L;
        low[2] = low[1] * low[1];
        low[3] = low[2] * low[1];
        low[4] = D > 8 ? power(4) : 1.0L;
        for (int j = 5; j < 8; ++j) low[j] = low[4] * low[j - 4];
        for (int j = 0; j < D / 2; ++j) {
            if (j > 0 && j % 8 == 0) high = power(j);
            long double f = high * low[j % 8];
            if (scaling == LCLA_ROPE_LINEAR) f /= factor;
            if (scaling == LCLA_ROPE_YARN) {
                const long double turns = original_len * f / two_pi;
                long double keep = (turns - beta_slow) / ((long double)beta_fast - beta_slow);
                keep = keep < 0.0L ? 0.0L : keep > 1.0L ? 1.0L : keep;
                f = f * keep + f / factor * (1.0L - keep);
            }
            p.freq[p.pairs] = (unsigned long long)(long long)(f * per_radian + 0.5L);
            p.axis[p.pairs++] = (unsigned char)a;
        }
        p.extent[a] = 1;
        if (a > 0 && !positions) {
            if (!axis_extents || axis_extents[a - 1] < 1) return LCLA_ERR_INVALID_ARG;
            p.extent[a] = axis_extents[a - 1];
        }
        p.by[a] = make_divisor((unsigned)p.extent[a]);
    }
    if (N > (1 << 30) || first < 0 || first > kMaxIndex - N) return LCLA_ERR_UNSUPPORTED;
    if (N == 0) return LCLA_OK;
    if (!rope_cos || !rope_sin) return LCLA_ERR_INVALID_ARG;
    if (misaligned(rope_cos) || misaligned(rope_sin) || ((uintptr_t)positions & 7u)) return LCLA_ERR_MISALIGNED;
    const size_t nt = (size_t)N * p.pairs * sizeof(float), np = (size_t)axes * N * sizeof(long long);
    if (overlaps(rope_cos, nt, rope_sin, nt) || overlaps(positions, np, rope_cos, nt) ||
        overlaps(positions, np, rope_sin, nt))
        return LCLA_ERR_INVALID_ARG;
    p.first = first;
    p.axes = axes;
    p.N = N;
    p.amp = scaling == LCLA_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.f;
    p.narrow = first + N <= 0x7fffffffLL;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int vec = p.pairs % 4 == 0 ? 4 : 1, tokens = kTabThreads / (p.pairs / vec) * kTabTokens;
    const unsigned grid = (unsigned)((N + (long long)tokens - 1) / tokens);
    if (vec == 4) rotary_tables_k<4><<<grid, kTabThreads, 0, st>>>(p, positions, rope_cos, rope_sin);
    else rotary_tables_k<1><<<grid, kTabThreads, 0, st>>>(p, positions, rope_cos, rope_sin);
    return launched();
}

int lcla_qk_norm_rope(const void *q, long long ldq, const void *k, long long ldk, int B, int N, int H, int Hk, int d,
                      const float *q_weight, const float *k_weight, float eps, const float *rope_cos,
                      const float *rope_sin, int table_rows, int rotary_dims, int half_layout,
                      const long long *positions, void *q_out, long long ldq_out, void *k_out, long long ldk_out,
                      int dtype, void *stream)
{
    int rc = check_norm(B, N, H, Hk, d, rotary_dims, half_layout, table_rows, positions, eps, dtype);
    if (rc != LCLA_OK) return rc;
    const size_t esz = dtype == LCLA_BF16 ? 2 : 4;
    const long long T = (long long)B * N;
    if (T == 0) return LCLA_OK;
    Span in[2], out[2];
    const void *ptr[4] = {q, k, q_out, k_out};
    const long long ld[4] = {ldq, ldk, ldq_out, ldk_out};
    for (int i = 0; i < 4; ++i)
        if ((rc = make_span(i < 2 ? &in[i] : &out[i - 2], ptr[i], ld[i], T, (i & 1) ? Hk : H, d, esz)) != LCLA_OK)
            return rc;
    if (rotary_dims > 0 && (!rope_cos || !rope_sin)) return LCLA_ERR_INVALID_ARG;
    if (misaligned(rope_cos) || misaligned(rope_sin) || misaligned(q_weight) || misaligned(k_weight) ||
        ((uintptr_t)positions & 7u))
        return LCLA_ERR_MISALIGNED;
    const size_t ntab = (size_t)table_rows * (rotary_dims / 2) * 4;
    const Span reads[] = {flat(rope_cos, ntab), flat(rope_sin, ntab), flat(q_weight, (size_t)d * 4),
                          flat(k_weight, (size_t)d * 4), flat(positions, (size_t)T * 8)};
    for (int i = 0; i < 2; ++i) {
        for (const Span &r : reads)
            if (spans_meet(out[i], r)) return LCLA_ERR_INVALID_ARG;
        for (int j = 0; j < 2; ++j)   // in place: the same rows, which a lane group reads before it writes them
            if (spans_meet(out[i], in[j]) && !(i == j && same_span(out[i], in[i]))) return LCLA_ERR_INVALID_ARG;
    }
    if (spans_meet(out[0], out[1])) return LCLA_ERR_INVALID_ARG;
    NormArgs a = {};
    a.x[0] = View{q, ldq};
    a.x[1] = View{k, ldk};
    a.y[0] = q_out;
    a.y[1] = k_out;
    a.ldy[0] = ldq_out;
    a.ldy[1] = ldk_out;
    a.w[0] = q_weight;
    a.w[1] = k_weight;
    a.cosv = rope_cos;
    a.sinv = rope_sin;
    a.positions = positions;
    a.T = T;
    a.N = N; a.P = table_rows; a.d = d; a.rd = rotary_dims;
    a.heads[0] = H; a.heads[1] = Hk;
    a.eps = eps;
    a.inv_d = 1.f / d;
    const int G = lanes_per_row(d), U = set_units(a, G);
    const long long units = T * (a.units[0] + a.units[1]);
    if (units > kMaxUnits) return LCLA_ERR_UNSUPPORTED;
    const unsigned grid = (unsigned)((units + kWarps - 1) / kWarps);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == LCLA_BF16) launch_norm<__nv_bfloat16>(a, G, half_layout != 0, U, grid, st);
    else launch_norm<float>(a, G, half_layout != 0, U, grid, st);
    return launched();
}

size_t lcla_qk_norm_rope_backward_workspace_bytes(int d)
{
    return d < 1 || d > 256 || (d % kVec) ? 0 : (size_t)kBwdCtas * d * sizeof(float);
}

int lcla_qk_norm_rope_backward(const void *dq_out, long long lddq_out, const void *dk_out, long long lddk_out,
                               const void *q, long long ldq, const void *k, long long ldk, int B, int N, int H, int Hk,
                               int d, const float *q_weight, const float *k_weight, float eps, const float *rope_cos,
                               const float *rope_sin, int table_rows, int rotary_dims, int half_layout,
                               const long long *positions, void *dq, long long lddq, void *dk, long long lddk,
                               float *dq_weight, float *dk_weight, int dtype, void *workspace, size_t workspace_bytes,
                               void *stream)
{
    int rc = check_norm(B, N, H, Hk, d, rotary_dims, half_layout, table_rows, positions, eps, dtype);
    if (rc != LCLA_OK) return rc;
    if ((dq_weight && !q_weight) || (dk_weight && (!k_weight || !Hk))) return LCLA_ERR_INVALID_ARG;
    const size_t esz = dtype == LCLA_BF16 ? 2 : 4;
    const long long T = (long long)B * N;
    const bool want = dq_weight || dk_weight;
    const size_t need = lcla_qk_norm_rope_backward_workspace_bytes(d);
    Span in[4], out[2];
    const void *ptr[6] = {q, k, dq_out, dk_out, dq, dk};
    const long long ld[6] = {ldq, ldk, lddq_out, lddk_out, lddq, lddk};
    for (int i = 0; i < 6; ++i)
        if ((rc = make_span(i < 4 ? &in[i] : &out[i - 4], ptr[i], ld[i], T, (i & 1) ? Hk : H, d, esz)) != LCLA_OK)
            return rc;
    if (T > 0 && rotary_dims > 0 && (!rope_cos || !rope_sin)) return LCLA_ERR_INVALID_ARG;
    if (misaligned(rope_cos) || misaligned(rope_sin) || misaligned(q_weight) || misaligned(k_weight) ||
        misaligned(dq_weight) || misaligned(dk_weight) || misaligned(workspace) || ((uintptr_t)positions & 7u))
        return LCLA_ERR_MISALIGNED;
    if (want && (!workspace || workspace_bytes < need)) return LCLA_ERR_WORKSPACE;
    const size_t ntab = (size_t)table_rows * (rotary_dims / 2) * 4, nw = (size_t)d * 4;
    const Span reads[] = {in[0], in[1], in[2], in[3], flat(rope_cos, ntab), flat(rope_sin, ntab), flat(q_weight, nw),
                          flat(k_weight, nw), flat(positions, (size_t)T * 8)};
    const Span writes[] = {out[0], out[1], flat(dq_weight, nw), flat(dk_weight, nw),
                           flat(want ? workspace : nullptr, need)};
    for (int i = 0; i < 5; ++i) {
        // dq may take the place of its own incoming gradient, dk of its own
        for (int j = 0; j < 9; ++j)
            if (spans_meet(writes[i], reads[j]) && !(i < 2 && j == i + 2 && same_span(writes[i], reads[j])))
                return LCLA_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (spans_meet(writes[i], writes[j])) return LCLA_ERR_INVALID_ARG;
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    NormArgs a = {};
    a.x[0] = View{q, ldq};
    a.x[1] = View{k, ldk};
    a.gy[0] = View{dq_out, lddq_out};
    a.gy[1] = View{dk_out, lddk_out};
    a.y[0] = dq;
    a.y[1] = dk;
    a.ldy[0] = lddq;
    a.ldy[1] = lddk;
    a.w[0] = q_weight;
    a.w[1] = k_weight;
    a.cosv = rope_cos;
    a.sinv = rope_sin;
    a.positions = positions;
    a.part = want ? static_cast<float *>(workspace) : nullptr;
    a.T = T;
    a.N = N; a.P = table_rows; a.d = d; a.rd = rotary_dims;
    a.heads[0] = H; a.heads[1] = Hk;
    a.eps = eps;
    a.inv_d = 1.f / d;
    if (T > 0) {
        const int G = lanes_per_row(d), R = 32 / G, U = dtype == LCLA_BF16 ? Back<__nv_bfloat16>::READS : Back<float>::READS;
        for (int s = 0; s < 2; ++s) {
            a.units[s] = (a.heads[s] + R * U - 1) / (R * U);
            a.span[s] = T >= kBwdCtas * kWarps && a.units[s] ? a.units[s] : 1;   // whole tokens, if every warp has one
        }
        // the CTAs are dealt out between queries and keys by their reads
        const long long uq = T * a.units[0], uk = T * a.units[1];
        if (uq > kMaxUnits || uk > kMaxUnits) return LCLA_ERR_UNSUPPORTED;
        const long long all = uq + uk, full = (all + kWarps - 1) / kWarps + 1;
        const int ctas = (int)(full < kBwdCtas ? (full < 2 ? 2 : full) : kBwdCtas);
        a.ctas[1] = uk ? (int)((double)ctas * uk / all) : 0;
        if (uk && a.ctas[1] < 1) a.ctas[1] = 1;
        a.ctas[0] = ctas - a.ctas[1];
        const bool half = half_layout != 0;
        if (dtype == LCLA_BF16)
            half ? launch_norm_backward<__nv_bfloat16, true>(a, G, ctas, st)
                 : launch_norm_backward<__nv_bfloat16, false>(a, G, ctas, st);
        else
            half ? launch_norm_backward<float, true>(a, G, ctas, st) : launch_norm_backward<float, false>(a, G, ctas, st);
    }
    if (want)
        qk_norm_weight_grad_k<<<dim3((d + 31) / 32, 2), kSumThreads, 0, st>>>(static_cast<float *>(workspace), d,
                                                                          a.ctas[0], a.ctas[1], dq_weight, dk_weight);
    return launched();
}

}  // extern "C"
