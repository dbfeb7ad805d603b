// lcla_rope.cu -- rotary tables on the device (lcla_rotary_tables) and the
// per-head RMS norm of queries and keys with the rotation in the same pass,
// forward and gradient (lcla_qk_norm_rope, lcla_qk_norm_rope_backward).
//
// Tables.  cos/sin[n][p] = amp * cos/sin(pos_a(n) * f_p).  A frequency is kept
// as a 64-bit fraction of a revolution, so that the product with an integer
// position, taken modulo 2^64, is the reduced angle without any rounding
// however far the position is.
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
#include "lcla_host.h"

namespace {

using namespace lcla::host;

// ------------------------------------------------------------------ tables
constexpr int kMaxPairs = 128;
constexpr int kMaxAxes = 3;
constexpr int kTabThreads = 256;
constexpr int kTabVec = 4;         // consecutive table entries per thread

struct TabPlan {
    unsigned long long freq[kMaxPairs];   // revolutions per position, times 2^64
    unsigned char axis[kMaxPairs];
    long long first;
    long long extent[kMaxAxes];           // extent[a]: how far axis a counts (a >= 1)
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

__device__ __forceinline__ unsigned long long token_position(const TabPlan &p, const long long *positions, int a, int n)
{
    if (positions) return (unsigned long long)positions[(size_t)a * p.N + n];
    const long long at = p.first + n;
    if (p.axes == 1) return (unsigned long long)at;
    if ((unsigned long long)at < (1ull << 31)) {   // 32-bit divisions: a third of the cost of 64-bit ones
        unsigned m = (unsigned)at;
        for (int i = p.axes - 1; i > a; --i) m /= (unsigned)p.extent[i];
        return a ? m % (unsigned)p.extent[a] : m;
    }
    long long m = at;
    for (int i = p.axes - 1; i > a; --i) m /= p.extent[i];
    return (unsigned long long)(a ? m % p.extent[a] : m);
}

// One thread writes four consecutive entries of both tables, 16 bytes each.
__global__ void __launch_bounds__(kTabThreads)
rotary_tables_k(const __grid_constant__ TabPlan p, const long long *__restrict__ positions, float *__restrict__ cosv,
                float *__restrict__ sinv)
{
    __shared__ unsigned long long freq[kMaxPairs];   // threads of a warp want different entries
    __shared__ unsigned char axis[kMaxPairs];
    for (int i = threadIdx.x; i < p.pairs; i += kTabThreads) {
        freq[i] = p.freq[i];
        axis[i] = p.axis[i];
    }
    __syncthreads();
    const long long total = (long long)p.N * p.pairs;
    const long long at = ((long long)blockIdx.x * kTabThreads + threadIdx.x) * kTabVec;
    if (at >= total) return;
    int n = (int)(at / p.pairs), j = (int)(at - (long long)n * p.pairs);
    int a = -1;
    unsigned long long pos = 0;
    float c[kTabVec], s[kTabVec];
#pragma unroll
    for (int i = 0; i < kTabVec; ++i) {
        if (at + i < total) {
            if (axis[j] != a) {
                a = axis[j];
                pos = token_position(p, positions, a, n);
            }
            const unsigned long long turn = pos * freq[j];
            const unsigned quad = (unsigned)((turn + (1ull << 61)) >> 62);
            float sn, cs;
            sincos_eighth((long long)(turn - ((unsigned long long)quad << 62)), sn, cs);
            const float x = (quad & 1) ? -sn : cs, y = (quad & 1) ? cs : sn;
            c[i] = ((quad & 2) ? -x : x) * p.amp;
            s[i] = ((quad & 2) ? -y : y) * p.amp;
            if (++j == p.pairs) {
                j = 0;
                ++n;
                a = -1;
            }
        }
    }
    if (at + kTabVec <= total) {
        *reinterpret_cast<float4 *>(cosv + at) = make_float4(c[0], c[1], c[2], c[3]);
        *reinterpret_cast<float4 *>(sinv + at) = make_float4(s[0], s[1], s[2], s[3]);
    } else {
#pragma unroll
        for (int i = 0; i < kTabVec; ++i)
            if (at + i < total) {
                cosv[at + i] = c[i];
                sinv[at + i] = s[i];
            }
    }
}

// ------------------------------------------------------- norm and rotation
constexpr int kVec = 8;            // entries of a row per lane
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

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
    float eps, inv_d;
};

template <typename T>
struct Row8;
template <>
struct Row8<float> {
    float4 a, b;
    __device__ void load(const float *p)
    {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ void get(float (&x)[kVec]) const
    {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};
template <>
struct Row8<__nv_bfloat16> {
    uint4 u;
    __device__ void load(const __nv_bfloat16 *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ void get(float (&x)[kVec]) const
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
};
__device__ __forceinline__ void store8(float *p, const float (&x)[kVec])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[kVec])
{
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// The rotation of a lane's entries [8 l, 8 l + 8): its factors, kept for all rows of a token.
template <bool HALF>
struct Turn {
    static constexpr int NF = HALF ? kVec : kVec / 2;
    float c[NF], s[NF];
    int partner;        // HALF: the lane that holds the other entry of each pair
    bool on;            // HALF: this lane's entries are turned

    __device__ void load(const NormArgs &a, long long token, int l, int lane)
    {
        long long row = a.positions ? a.positions[token] : (unsigned)token % (unsigned)a.N;
        row = row < 0 ? 0 : row >= a.P ? a.P - 1 : row;   // a bad position reads a wrong row, never out of bounds
        const int hp = a.rd / 2;
        const float *pc = a.cosv + row * hp, *ps = a.sinv + row * hp;
        partner = lane;
        if (HALF) {
            const int at = kVec * l, per = hp / kVec;     // lanes per half
            on = at < a.rd;
            const bool second = l >= per;
            const int p0 = second ? at - hp : at;
            if (on) partner = second ? lane - per : lane + per;
#pragma unroll
            for (int j = 0; j < NF; j += 4) {
                const float4 u = on ? *reinterpret_cast<const float4 *>(pc + p0 + j) : make_float4(1.f, 1.f, 1.f, 1.f);
                const float4 v = on ? *reinterpret_cast<const float4 *>(ps + p0 + j) : make_float4(0.f, 0.f, 0.f, 0.f);
                c[j] = u.x; c[j + 1] = u.y; c[j + 2] = u.z; c[j + 3] = u.w;
                // first half: x c - x' s; second half: x c + x' s
                s[j] = second ? v.x : -v.x;
                s[j + 1] = second ? v.y : -v.y;
                s[j + 2] = second ? v.z : -v.z;
                s[j + 3] = second ? v.w : -v.w;
            }
        } else {
            const int p0 = NF * l;
            on = 2 * p0 < a.rd;
            if ((hp & 3) == 0) {                          // whole 16-byte pieces of aligned table rows
                const float4 u = on ? *reinterpret_cast<const float4 *>(pc + p0) : make_float4(1.f, 1.f, 1.f, 1.f);
                const float4 v = on ? *reinterpret_cast<const float4 *>(ps + p0) : make_float4(0.f, 0.f, 0.f, 0.f);
                c[0] = u.x; c[1] = u.y; c[2] = u.z; c[3] = u.w;
                s[0] = v.x; s[1] = v.y; s[2] = v.z; s[3] = v.w;
            } else {
#pragma unroll
                for (int j = 0; j < NF; ++j) {
                    c[j] = p0 + j < hp ? pc[p0 + j] : 1.f;
                    s[j] = p0 + j < hp ? ps[p0 + j] : 0.f;
                }
            }
        }
    }
    // SIGN +1: R x, -1: R^T x.  Every lane of the warp takes part.
    template <int SIGN>
    __device__ void apply(float (&x)[kVec]) const
    {
        if (HALF) {
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const float o = __shfl_sync(0xffffffffu, x[j], partner);
                x[j] = fmaf(x[j], c[j % NF], SIGN * s[j % NF] * o);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kVec / 2; ++j) {
                const float u = x[2 * j], v = x[2 * j + 1], sj = SIGN * s[j];
                x[2 * j] = fmaf(u, c[j], -v * sj);
                x[2 * j + 1] = fmaf(v, c[j], u * sj);
            }
        }
    }
};

template <int G>
__device__ __forceinline__ float row_sum(float v)   // over the G lanes of a row
{
#pragma unroll
    for (int o = G / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ void load_weight(const float *w, bool on, int l, float (&x)[kVec])
{
#pragma unroll
    for (int j = 0; j < kVec; ++j) x[j] = (w && on) ? w[kVec * l + j] : 1.f;
}

// Bound by HBM (x read, y written).  G lanes hold a row, 8 entries (16 bytes of bf16) each, so a warp reads 32 / G
// consecutive heads of a token at once.  A unit is U such reads of one token and side: the rotation factors and the
// weight are loaded once for all of them, and the U reads are in flight together.
template <typename T, int G, bool HALF, int U>
__global__ void __launch_bounds__(kThreads)
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
    const T *x = static_cast<const T *>(a.x[side].p) + token * a.x[side].ld + kVec * l;
    T *y = static_cast<T *>(a.y[side]) + token * a.ldy[side] + kVec * l;
    Row8<T> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        raw[u].zero();
        if (in && h0 + u * R < H) raw[u].load(x + (size_t)(h0 + u * R) * a.d);
    }
    float w[kVec];
    load_weight(a.w[side], in, l, w);
    Turn<HALF> turn;
    turn.load(a, token, l, lane);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float v[kVec], ss = 0.f;
        raw[u].get(v);
#pragma unroll
        for (int j = 0; j < kVec; ++j) ss = fmaf(v[j], v[j], ss);
        const float r = rsqrtf(fmaf(row_sum<G>(ss), a.inv_d, a.eps));
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = v[j] * r * w[j];
        turn.template apply<1>(v);
        if (in && h0 + u * R < H) store8(y + (size_t)(h0 + u * R) * a.d, v);
    }
}

// Bound by HBM (x and gy read, gx written).  CTAs take one side each and stride over its units, so that the weight's
// gradient gathers in registers; a CTA leaves one [d] partial, and qk_norm_weight_grad_k adds those in a fixed order.
template <typename T, int G, bool HALF, int U>
__global__ void __launch_bounds__(kThreads)
qk_norm_rope_backward_k(const __grid_constant__ NormArgs a)
{
    constexpr int R = 32 / G;
    __shared__ float red[kWarps][G * kVec];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, l = lane % G, sub = lane / G;
    const int side = (int)blockIdx.x >= a.ctas[0];
    const int cta = side ? (int)blockIdx.x - a.ctas[0] : (int)blockIdx.x;
    const int H = a.heads[side], per = a.units[side];
    const bool in = kVec * l < a.d;
    float w[kVec], gw[kVec];
    load_weight(a.w[side], in, l, w);
#pragma unroll
    for (int j = 0; j < kVec; ++j) gw[j] = 0.f;
    const long long units = a.T * per, step = (long long)a.ctas[side] * kWarps;
    for (long long unit = (long long)cta * kWarps + wid; unit < units; unit += step) {
        const long long token = (unsigned)unit / (unsigned)per;
        const int h0 = (int)((unsigned)unit % (unsigned)per) * U * R + sub;
        const T *x = static_cast<const T *>(a.x[side].p) + token * a.x[side].ld + kVec * l;
        const T *gy = static_cast<const T *>(a.gy[side].p) + token * a.gy[side].ld + kVec * l;
        T *gx = static_cast<T *>(a.y[side]) + token * a.ldy[side] + kVec * l;
        Row8<T> rx[U], rg[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            rx[u].zero();
            rg[u].zero();
            if (in && h0 + u * R < H) {
                rx[u].load(x + (size_t)(h0 + u * R) * a.d);
                rg[u].load(gy + (size_t)(h0 + u * R) * a.d);
            }
        }
        Turn<HALF> turn;
        turn.load(a, token, l, lane);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[kVec], m[kVec], ss = 0.f, dot = 0.f;
            rx[u].get(v);
            rg[u].get(m);
            turn.template apply<-1>(m);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                ss = fmaf(v[j], v[j], ss);
                dot = fmaf(m[j] * w[j], v[j], dot);
            }
            ss = row_sum<G>(ss);
            dot = row_sum<G>(dot);
            const bool live = h0 + u * R < H;            // rows past the last head add nothing, whatever eps is
            const float r = live ? rsqrtf(fmaf(ss, a.inv_d, a.eps)) : 0.f;
            const float t = dot * a.inv_d * r * r;
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                gw[j] = fmaf(m[j] * r, v[j], gw[j]);
                v[j] = r * fmaf(-v[j], t, m[j] * w[j]);
            }
            if (in && live) store8(gx + (size_t)(h0 + u * R) * a.d, v);
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
#pragma unroll
        for (int o = G; o < 32; o <<= 1) gw[j] += __shfl_xor_sync(0xffffffffu, gw[j], o);
        if (sub == 0) red[wid][kVec * l + j] = gw[j];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.d; i += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) s += red[k][i];
        a.part[(size_t)blockIdx.x * a.d + i] = s;
    }
}

// One block per side and 32 entries of d; its 8 warps each add an eighth of the CTAs' partials, in double.
__global__ void __launch_bounds__(kThreads)
qk_norm_weight_grad_k(const float *__restrict__ part, int d, int ctas_q, int ctas_k, float *gwq, float *gwk)
{
    __shared__ double red[kWarps][32];
    const int side = blockIdx.y, lane = threadIdx.x & 31, wid = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
    float *gw = side ? gwk : gwq;
    if (!gw) return;
    const float *p = part + (side ? (size_t)ctas_q * d : 0);
    const int n = side ? ctas_k : ctas_q;
    double s = 0.0;
    if (i < d)
        for (int c = wid; c < n; c += kWarps) s += p[(size_t)c * d + i];
    red[wid][lane] = s;
    __syncthreads();
    if (wid == 0 && i < d) {
#pragma unroll
        for (int k = 1; k < kWarps; ++k) s += red[k][lane];
        gw[i] = (float)s;
    }
}

// ----------------------------------------------------------------- host
constexpr int kBwdCtas = 148 * 4;   // resident at once: 4 blocks of 256 threads on each SM

constexpr long long kMaxUnits = 0xfffffff0ll;   // the kernels count units in 32 bits, rounded up to whole blocks

int lanes_per_row(int d)            // the power of two that holds d / 8 lanes
{
    int g = 4;
    while (g * kVec < d) g *= 2;
    return g;
}

template <typename T, bool HALF, int U>
void launch_norm(const NormArgs &a, int G, bool back, unsigned grid, cudaStream_t st)
{
    switch (G) {
#define LCLA_G(g)                                                                                  \
    case g:                                                                                        \
        if (back) qk_norm_rope_backward_k<T, g, HALF, U><<<grid, kThreads, 0, st>>>(a);            \
        else qk_norm_rope_k<T, g, HALF, U><<<grid, kThreads, 0, st>>>(a);                          \
        break;
        LCLA_G(4) LCLA_G(8) LCLA_G(16) LCLA_G(32)
#undef LCLA_G
    }
}

template <typename T>
void launch_norm(const NormArgs &a, int G, bool half, int U, bool back, unsigned grid, cudaStream_t st)
{
    if (half) U == 1 ? launch_norm<T, true, 1>(a, G, back, grid, st) : launch_norm<T, true, 3>(a, G, back, grid, st);
    else U == 1 ? launch_norm<T, false, 1>(a, G, back, grid, st) : launch_norm<T, false, 3>(a, G, back, grid, st);
}

// Units of U reads per token, on each side.  U = 3 keeps three 16-byte reads a lane in flight; a call with too few
// rows to fill the SMs that way takes U = 1, which has the shorter chain.
int set_units(NormArgs &a, int G)
{
    const int R = 32 / G;
    const long long reads = a.T * ((a.heads[0] + R - 1) / R + (a.heads[1] + R - 1) / R);
    const int U = reads < 148 * 32 ? 1 : 3;
    for (int s = 0; s < 2; ++s) a.units[s] = (a.heads[s] + R * U - 1) / (R * U);
    return U;
}

int check_norm(int B, int N, int H, int Hk, int d, int rd, int half, int P, const void *positions, float eps, int dtype)
{
    if (B < 1 || N < 0 || H < 1 || Hk < 0 || P < 1 || d < 1 || rd < 0 || rd > d || (rd & 1)) return LCLA_ERR_INVALID_ARG;
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
    const double two_pi = 6.283185307179586476925;
    for (int a = 0; a < axes; ++a) {
        const int D = axis_dims[a];
        if (D < 2 || (D & 1)) return LCLA_ERR_INVALID_ARG;
        if (p.pairs + D / 2 > kMaxPairs) return LCLA_ERR_UNSUPPORTED;
        if (scaling == LCLA_ROPE_NTK && D == 2) return LCLA_ERR_INVALID_ARG;   // its exponent D / (D - 2)
        const double base = scaling == LCLA_ROPE_NTK ? theta * pow(factor, (double)D / (D - 2)) : theta;
        for (int j = 0; j < D / 2; ++j) {
            double f = pow(base, -2.0 * j / D);
            if (scaling == LCLA_ROPE_LINEAR) f /= factor;
            if (scaling == LCLA_ROPE_YARN) {
                const double turns = original_len * f / two_pi;
                double keep = (turns - beta_slow) / (beta_fast - beta_slow);
                keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
                f = f * keep + f / factor * (1.0 - keep);
            }
            p.freq[p.pairs] = (unsigned long long)ldexp(f / two_pi, 64);
            p.axis[p.pairs++] = (unsigned char)a;
        }
        p.extent[a] = 1;
        if (a > 0 && !positions) {
            if (!axis_extents || axis_extents[a - 1] < 1) return LCLA_ERR_INVALID_ARG;
            p.extent[a] = axis_extents[a - 1];
        }
    }
    if (N > (1 << 30) || first < 0 || first > (1ll << 60)) return LCLA_ERR_UNSUPPORTED;
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
    const long long threads = ((long long)N * p.pairs + kTabVec - 1) / kTabVec;
    rotary_tables_k<<<(unsigned)((threads + kTabThreads - 1) / kTabThreads), kTabThreads, 0,
                      reinterpret_cast<cudaStream_t>(stream)>>>(p, positions, rope_cos, rope_sin);
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
    if (dtype == LCLA_BF16) launch_norm<__nv_bfloat16>(a, G, half_layout != 0, U, false, grid, st);
    else launch_norm<float>(a, G, half_layout != 0, U, false, grid, st);
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
        const int G = lanes_per_row(d), U = set_units(a, G);
        // the CTAs are dealt out between queries and keys by their units
        const long long uq = T * a.units[0], uk = T * a.units[1];
        if (uq > kMaxUnits || uk > kMaxUnits) return LCLA_ERR_UNSUPPORTED;
        const long long total = uq + uk, full = (total + kWarps - 1) / kWarps + 1;
        const int ctas = (int)(full < kBwdCtas ? (full < 2 ? 2 : full) : kBwdCtas);
        a.ctas[1] = uk ? (int)((double)ctas * uk / total) : 0;
        if (uk && a.ctas[1] < 1) a.ctas[1] = 1;
        a.ctas[0] = ctas - a.ctas[1];
        if (dtype == LCLA_BF16) launch_norm<__nv_bfloat16>(a, G, half_layout != 0, U, true, ctas, st);
        else launch_norm<float>(a, G, half_layout != 0, U, true, ctas, st);
    }
    if (want)
        qk_norm_weight_grad_k<<<dim3((d + 31) / 32, 2), kThreads, 0, st>>>(static_cast<float *>(workspace), d,
                                                                          a.ctas[0], a.ctas[1], dq_weight, dk_weight);
    return launched();
}

}  // extern "C"
