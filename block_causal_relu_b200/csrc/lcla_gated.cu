// lcla_gated.cu -- the gated recurrence: kernels, plan and entry points
// (lcla_gated_forward, lcla_gated_step, lcla_gated_backward).
//
// A sequence is cut into segments of whole 32-token tiles so that the heads of
// a call fill the SMs.  With more than one segment, gated_totals_k first leaves
// what each segment adds to the state and gated_scan_k turns those into the
// state before each segment; the recurrence then runs in all segments at once.
// The gradient always runs both directions that way, its three recurrences
// side by side in one launch.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "lcla.h"
#include "lcla_gated.cuh"
#include "lcla_host.h"

namespace {

using namespace lcla::host;
using namespace lcla::gated;

constexpr int kSms = 148;

// ---------------------------------------------------------------- kernels
struct Place {
    int b, h, seg, role, group, slab, lane;
    bool live;
};
template <int D>
__device__ __forceinline__ Place place(int H, int roles)
{
    constexpr int NS = D / 32, G = WARPS / NS;
    const int hg = (H + G - 1) / G, warp = threadIdx.x >> 5;
    Place p;
    p.role = blockIdx.x % roles;
    const int u = blockIdx.x / roles;
    p.seg = u / hg;
    p.group = warp / NS;
    p.slab = warp % NS;
    p.h = (u % hg) * G + p.group;
    p.b = blockIdx.y;
    p.lane = threadIdx.x & 31;
    p.live = p.h < H;
    return p;
}

template <typename T, int D, int TENSORS, int STAGES>
struct Smem {
    static constexpr int NS = D / 32, G = WARPS / NS;
    static constexpr int RING = STAGES * TENSORS * Tile<T, D>::BYTES;
    static constexpr int BYTES = G * RING + WARPS * (int)sizeof(Weights);
};
extern __shared__ __align__(128) unsigned char smem[];

// The block's ring of one head and its warp's weights.
template <typename S>
__device__ __forceinline__ uint32_t ring_of(const Place &p)
{
    return (uint32_t)__cvta_generic_to_shared(smem) + p.group * S::RING;
}
template <typename S>
__device__ __forceinline__ Weights *weights_of()
{
    return reinterpret_cast<Weights *>(smem + S::G * S::RING) + (threadIdx.x >> 5);
}

template <typename T, int D>
struct Ring {   // tiles in flight per head: what keeps three blocks (two of fp32 at d = 64) on an SM
    static constexpr int MAIN = sizeof(T) * D >= 256 ? 2 : 3;
    static constexpr int TOTAL = sizeof(T) * D >= 256 ? 3 : 4;
};

template <typename T, int D>
__global__ void __launch_bounds__(THREADS, 3) gated_forward_k(const __grid_constant__ Work w, const __grid_constant__ Role r)
{
    using S = Smem<T, D, 3, Ring<T, D>::MAIN>;
    const Place p = place<D>(w.H, 1);
    if (!p.live) return;
    recur<T, D, false, false, false, 2, 2, 3, Ring<T, D>::MAIN>(w, r, p.b, p.h, p.seg, p.group, p.slab, p.lane,
                                                               ring_of<S>(p), weights_of<S>());
}

struct Roles {
    Role r[3];
};

template <typename T, int D>
__global__ void __launch_bounds__(THREADS, 3) gated_backward_k(const __grid_constant__ Work w, const __grid_constant__ Roles rs)
{
    constexpr int ST = Ring<T, D>::MAIN;
    using S = Smem<T, D, 4, ST>;
    const Place p = place<D>(w.H, 3);
    if (!p.live) return;
    if (p.role == 0)
        recur<T, D, false, true, true, 3, 3, 3, ST>(w, rs.r[0], p.b, p.h, p.seg, p.group, p.slab, p.lane, ring_of<S>(p),
                                                    weights_of<S>());
    else if (p.role == 1)
        recur<T, D, true, true, true, 3, 3, 3, ST>(w, rs.r[1], p.b, p.h, p.seg, p.group, p.slab, p.lane, ring_of<S>(p),
                                                   weights_of<S>());
    else
        recur<T, D, true, false, false, 2, 2, 2, ST>(w, rs.r[2], p.b, p.h, p.seg, p.group, p.slab, p.lane, ring_of<S>(p),
                                                     weights_of<S>());
}

struct Totals {
    const void *key[2], *val[2];
    float *part[2], *decays;
};

template <typename T, int D>
__global__ void __launch_bounds__(THREADS, 3) gated_totals_k(const __grid_constant__ Work w, const __grid_constant__ Totals t,
                                                             int roles)
{
    constexpr int ST = Ring<T, D>::TOTAL;
    using S = Smem<T, D, 2, ST>;
    const Place p = place<D>(w.H, roles);
    if (!p.live) return;
    if (p.role == 0)
        total<T, D, false, ST>(w, t.key[0], t.val[0], t.part[0], t.decays, p.b, p.h, p.seg, p.group, p.slab, p.lane,
                               ring_of<S>(p), weights_of<S>());
    else
        total<T, D, true, ST>(w, t.key[1], t.val[1], t.part[1], nullptr, p.b, p.h, p.seg, p.group, p.slab, p.lane,
                              ring_of<S>(p), weights_of<S>());
}

struct Scan {
    float *part[2];            // in: what each segment adds; out: the state before it (reversed: after it)
    const float *decays;
    const float *init[2];      // [B, H, d, d] or NULL (zero)
    float *last[2], *last2[2]; // the state after all segments, or NULL
    float init_scale[2], last_scale[2];
    int nseg, BH, n4;          // n4: float4s of a state
};

// One thread per float4 of a state; the segments' values are read 8 at a time ahead of the chain.
__global__ void __launch_bounds__(128) gated_scan_k(const __grid_constant__ Scan s)
{
    const int i = blockIdx.x * 128 + threadIdx.x, dir = blockIdx.y;
    const int all = s.BH * s.n4;
    if (i >= all) return;
    const int bh = i / s.n4;
    float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
    if (s.init[dir]) {
        c = reinterpret_cast<const float4 *>(s.init[dir])[i];
        const float m = s.init_scale[dir];
        c.x *= m; c.y *= m; c.z *= m; c.w *= m;
    }
    float4 *part = reinterpret_cast<float4 *>(s.part[dir]);
    constexpr int U = 8;
    for (int k0 = 0; k0 < s.nseg; k0 += U) {
        float4 v[U];
        float d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = dir ? s.nseg - 1 - (k0 + u) : k0 + u;
            if (k0 + u < s.nseg) {
                v[u] = part[(size_t)k * all + i];
                d[u] = s.decays[(size_t)k * s.BH + bh];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = dir ? s.nseg - 1 - (k0 + u) : k0 + u;
            if (k0 + u < s.nseg) {
                part[(size_t)k * all + i] = c;
                c.x = fmaf(c.x, d[u], v[u].x);
                c.y = fmaf(c.y, d[u], v[u].y);
                c.z = fmaf(c.z, d[u], v[u].z);
                c.w = fmaf(c.w, d[u], v[u].w);
            }
        }
    }
    if (s.last2[dir]) reinterpret_cast<float4 *>(s.last2[dir])[i] = c;
    if (s.last[dir]) {
        const float m = s.last_scale[dir];
        reinterpret_cast<float4 *>(s.last[dir])[i] = make_float4(c.x * m, c.y * m, c.z * m, c.w * m);
    }
}

struct GradGate {
    const float *g;
    const float *dot;          // [planes][B, H, N]
    const float *before;       // [nseg + 1][B, H, d, d]: the state before each segment, and after the last
    const float *after;        // [nseg][B, H, d, d]: its gradient after each segment, over scale
    float *dg;
    int B, H, N, nseg, seg_tiles, planes, n4;
    float scale;
};

// dg_t = <S, R> at the segment's end + the sum over the segment's tokens from t on of <q, dq> - <k, dk>.  The sum over
// all later tokens would be the same number, as a difference of two long sums that nearly cancel; starting again at
// each segment's end keeps it to 32-bit accuracy.  One warp per segment of a head.
__global__ void __launch_bounds__(128) gated_dgate_k(const __grid_constant__ GradGate p)
{
    const int lane = threadIdx.x & 31;
    const long long u = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int BH = p.B * p.H;
    if (u >= (long long)BH * p.nseg) return;
    const int bh = (int)(u % BH), seg = (int)(u / BH), b = bh / p.H, h = bh % p.H;
    const int t0 = seg * p.seg_tiles * TILE, t1 = min(p.N, t0 + p.seg_tiles * TILE);
    if (t0 >= t1) return;
    const float4 *S = reinterpret_cast<const float4 *>(p.before) + ((size_t)(seg + 1) * BH + bh) * p.n4;
    const float4 *R = reinterpret_cast<const float4 *>(p.after) + ((size_t)seg * BH + bh) * p.n4;
    float y = 0.f;
    for (int i = lane; i < p.n4; i += 32) {
        const float4 x = S[i], z = R[i];
        y = fmaf(x.x, z.x, fmaf(x.y, z.y, fmaf(x.z, z.z, fmaf(x.w, z.w, y))));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    double carry = (double)y * p.scale;
    const size_t plane = (size_t)BH * p.N;
    const float *dot = p.dot + (size_t)bh * p.N;
    for (int t = t1 - 1 - lane;; t -= 32) {          // lane 0 has the latest token
        float d = 0.f, g = 0.f;
        if (t >= t0) {
            for (int k = 0; k < p.planes; ++k) d += dot[k * plane + t];
            g = p.g[((size_t)b * p.N + t) * p.H + h];
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float up = __shfl_up_sync(0xffffffffu, d, o);
            if (lane >= o) d += up;
        }
        if (t >= t0) p.dg[((size_t)b * p.N + t) * p.H + h] = g < RESET ? 0.f : (float)(carry + d);
        carry += __shfl_sync(0xffffffffu, d, 31);
        if (__shfl_sync(0xffffffffu, t, 31) <= t0) break;
    }
}

// A few tokens against the state: read once, kept in registers, written once.  One block per head; D / 4 lanes hold a
// row of the state, four entries each.
template <typename T, int D>
__global__ void __launch_bounds__(THREADS)
gated_short_k(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v, const float *__restrict__ g,
              int H, int N, float scale, const float *state_in, T *__restrict__ out, float *state_out)
{
    constexpr int LPR = D / 4, RPI = THREADS / LPR, R = D / RPI;   // lanes per row, rows per step, rows per thread
    const int bh = blockIdx.x, b = bh / H, h = bh % H;
    const int l = threadIdx.x % LPR, c0 = threadIdx.x / LPR;
    float4 S[R];
    const size_t st = (size_t)bh * D * D + 4 * l;
#pragma unroll
    for (int i = 0; i < R; ++i)
        S[i] = state_in ? *reinterpret_cast<const float4 *>(state_in + st + (size_t)(c0 + i * RPI) * D)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int t = 0; t < N; ++t) {
        const size_t tok = (size_t)b * N + t, row = (tok * H + h) * D;
        const float gt = g[tok * H + h];
        const float a = expf(gt < RESET ? RESET : gt);
        float kk[4], qq[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            kk[j] = (float)k[row + 4 * l + j];
            qq[j] = (float)q[row + 4 * l + j];
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float vv = (float)v[row + c0 + i * RPI];
            S[i].x = fmaf(S[i].x, a, vv * kk[0]);
            S[i].y = fmaf(S[i].y, a, vv * kk[1]);
            S[i].z = fmaf(S[i].z, a, vv * kk[2]);
            S[i].w = fmaf(S[i].w, a, vv * kk[3]);
            float o = fmaf(S[i].x, qq[0], fmaf(S[i].y, qq[1], fmaf(S[i].z, qq[2], S[i].w * qq[3])));
#pragma unroll
            for (int m = LPR / 2; m; m >>= 1) o += __shfl_xor_sync(0xffffffffu, o, m);
            if (l == 0) out[row + c0 + i * RPI] = (T)(o * scale);
        }
    }
    if (state_out)
#pragma unroll
        for (int i = 0; i < R; ++i) *reinterpret_cast<float4 *>(state_out + st + (size_t)(c0 + i * RPI) * D) = S[i];
}

// ------------------------------------------------------------------- plan
constexpr size_t kAlign = 256;
size_t round_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

constexpr int kShort = 16;         // calls of up to this many tokens take gated_short_k

struct Plan {
    int nseg, seg_tiles;
    size_t before, after, decays, dot, bytes;   // workspace offsets
};

Plan make_plan(int B, int H, int N, int d, int dtype, bool backward)
{
    Plan p = {};
    if (N == 0 || (!backward && N <= kShort)) return p;
    const int tiles = (N + TILE - 1) / TILE, ns = d / 32;
    const long long warps = (long long)B * H * ns;
    long long nseg = ((long long)kSms * 12 + warps - 1) / warps;
    const int min_tiles = backward ? 4 : 8;
    if (nseg > tiles / min_tiles) nseg = tiles / min_tiles;
    if (nseg < 1) nseg = 1;
    p.seg_tiles = (int)((tiles + nseg - 1) / nseg);
    if (backward && p.seg_tiles > 32) p.seg_tiles = 32;
    p.nseg = (tiles + p.seg_tiles - 1) / p.seg_tiles;
    const size_t slice = (size_t)B * H * d * d * sizeof(float);
    size_t at = 0;
    if (p.nseg > 1 || backward) {
        p.before = at;
        at += round_up((p.nseg + 1) * slice);
        p.decays = at;
        at += round_up((size_t)p.nseg * B * H * sizeof(float));
    }
    if (backward) {
        p.after = at;
        at += round_up(p.nseg * slice);
        p.dot = at;
        at += round_up((size_t)2 * ns * B * H * N * sizeof(float));
    }
    p.bytes = at;
    return p;
}

int check_shape(int B, int H, int N, int d, int dtype)
{
    if (B < 1 || H < 1 || N < 0 || d < 1 || (d & 1)) return LCLA_ERR_INVALID_ARG;
    if (dtype != LCLA_BF16 && dtype != LCLA_F32) return LCLA_ERR_INVALID_ARG;
    if (d != 32 && d != 64) return LCLA_ERR_UNSUPPORTED;
    if (N > (1 << 30) || B > 65535 || H > 65535) return LCLA_ERR_UNSUPPORTED;
    // the state kernels count float4s of all heads' states, and the others blocks, in 32 bits
    if ((long long)B * H * d * d / 4 > 0x7ffffff0LL) return LCLA_ERR_UNSUPPORTED;
    if ((long long)((N + 31) / 32) * H * 3 > 0x7fffffffLL) return LCLA_ERR_UNSUPPORTED;
    return LCLA_OK;
}

template <typename F>
void set_smem(F *kernel, int bytes)
{
    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int D>
unsigned blocks(const Work &w, int roles)
{
    constexpr int G = WARPS / (D / 32);
    return (unsigned)((long long)w.nseg * ((w.H + G - 1) / G) * roles);
}

template <typename T, int D>
void launch_totals(const Work &w, const Totals &t, int roles, cudaStream_t st)
{
    using S = Smem<T, D, 2, Ring<T, D>::TOTAL>;
    set_smem(gated_totals_k<T, D>, S::BYTES);
    gated_totals_k<T, D><<<dim3(blocks<D>(w, roles), w.B), THREADS, S::BYTES, st>>>(w, t, roles);
}

void launch_scan(const Scan &s, int dirs, cudaStream_t st)
{
    gated_scan_k<<<dim3((s.BH * s.n4 + 127) / 128, dirs), 128, 0, st>>>(s);
}

template <typename T, int D>
int run_forward(const void *q, const void *k, const void *v, const Work &w, const Plan &p, const float *state_in,
                void *out, float *state_out, unsigned char *ws, cudaStream_t st)
{
    if (w.N <= kShort) {
        gated_short_k<T, D><<<w.B * w.H, THREADS, 0, st>>>((const T *)q, (const T *)k, (const T *)v, w.g, w.H, w.N,
                                                           w.scale, state_in, (T *)out, state_out);
        return launched();
    }
    Role r = {};
    r.q = q; r.k = k; r.v = v; r.out = out;
    r.state = state_in;
    r.state_end = state_out;
    if (w.nseg > 1) {
        Totals t = {};
        float *before = reinterpret_cast<float *>(ws + p.before);
        t.key[0] = k; t.val[0] = v;
        t.part[0] = before;
        t.decays = reinterpret_cast<float *>(ws + p.decays);
        launch_totals<T, D>(w, t, 1, st);
        Scan s = {};
        s.part[0] = before;
        s.decays = t.decays;
        s.init[0] = state_in;
        s.last[0] = state_out;
        s.init_scale[0] = s.last_scale[0] = 1.f;
        s.nseg = w.nseg; s.BH = w.B * w.H; s.n4 = D * D / 4;
        launch_scan(s, 1, st);
        r.state = before;
        r.state_end = nullptr;
    }
    using S = Smem<T, D, 3, Ring<T, D>::MAIN>;
    set_smem(gated_forward_k<T, D>, S::BYTES);
    gated_forward_k<T, D><<<dim3(blocks<D>(w, 1), w.B), THREADS, S::BYTES, st>>>(w, r);
    return launched();
}

template <typename T, int D>
int run_backward(const void *dout, const void *q, const void *k, const void *v, const Work &w, const Plan &p,
                 const float *state_in, const float *dstate_out, void *dq, void *dk, void *dv, float *dg,
                 float *dstate_in, unsigned char *ws, cudaStream_t st)
{
    float *before = reinterpret_cast<float *>(ws + p.before), *after = reinterpret_cast<float *>(ws + p.after);
    float *dot = reinterpret_cast<float *>(ws + p.dot);
    const int BH = w.B * w.H, ns = D / 32;
    Totals t = {};
    t.key[0] = k; t.val[0] = v; t.part[0] = before;
    t.key[1] = q; t.val[1] = dout; t.part[1] = after;
    t.decays = reinterpret_cast<float *>(ws + p.decays);
    launch_totals<T, D>(w, t, 2, st);
    Scan s = {};
    s.part[0] = before; s.part[1] = after;
    s.decays = t.decays;
    s.init[0] = state_in; s.init[1] = dstate_out;
    s.last2[0] = before + (size_t)w.nseg * BH * D * D;
    s.last[1] = dstate_in;
    s.init_scale[0] = s.last_scale[0] = 1.f;
    s.init_scale[1] = 1.f / w.scale;
    s.last_scale[1] = w.scale;
    s.nseg = w.nseg; s.BH = BH; s.n4 = D * D / 4;
    launch_scan(s, 2, st);
    const size_t plane = (size_t)BH * w.N;
    Roles rs = {};
    // recur reads the state of segment `seg` also where there is only one
    rs.r[0].q = dout; rs.r[0].k = v; rs.r[0].v = k; rs.r[0].x = q; rs.r[0].out = dq;
    rs.r[0].state = before; rs.r[0].dot = dot; rs.r[0].sign = 1.f;
    rs.r[1].q = v; rs.r[1].k = dout; rs.r[1].v = q; rs.r[1].x = k; rs.r[1].out = dk;
    rs.r[1].state = after; rs.r[1].dot = dot + ns * plane; rs.r[1].sign = -1.f;
    rs.r[2].q = k; rs.r[2].k = q; rs.r[2].v = dout; rs.r[2].out = dv;
    rs.r[2].state = after;
    using S = Smem<T, D, 4, Ring<T, D>::MAIN>;
    set_smem(gated_backward_k<T, D>, S::BYTES);
    gated_backward_k<T, D><<<dim3(blocks<D>(w, 3), w.B), THREADS, S::BYTES, st>>>(w, rs);
    GradGate gg = {};
    gg.g = w.g; gg.dot = dot; gg.before = before; gg.after = after; gg.dg = dg;
    gg.B = w.B; gg.H = w.H; gg.N = w.N; gg.nseg = w.nseg; gg.seg_tiles = w.seg_tiles;
    gg.planes = 2 * ns; gg.n4 = D * D / 4;
    gg.scale = w.scale;
    const long long units = (long long)BH * w.nseg;
    gated_dgate_k<<<(unsigned)((units + 3) / 4), 128, 0, st>>>(gg);
    return launched();
}

struct Range {
    const void *p;
    size_t n;
};
bool any_overlap(const Range &w, const Range *reads, int n)
{
    for (int i = 0; i < n; ++i)
        if (overlaps(w.p, w.n, reads[i].p, reads[i].n)) return true;
    return false;
}

// the gates are read and written one by one, so any slice of tokens serves
bool misaligned4(const void *p) { return ((uintptr_t)p & 3u) != 0; }

// scale is divided by where a carried gradient meets the recurrence
bool bad_scale(float s) { return !isfinite(s) || !(fabsf(s) >= 1e-18f) || fabsf(s) > 1e18f; }

int forward_impl(const void *q, const void *k, const void *v, const float *g, int B, int H, int N, int d, float scale,
                 const float *state_in, void *out, float *state_out, int dtype, void *ws, size_t ws_bytes, void *stream)
{
    const int rc = check_shape(B, H, N, d, dtype);
    if (rc != LCLA_OK) return rc;
    if (bad_scale(scale)) return LCLA_ERR_INVALID_ARG;
    const size_t esz = dtype == LCLA_BF16 ? 2 : 4, ns = (size_t)B * H * d * d * sizeof(float);
    if (misaligned(state_in) || misaligned(state_out)) return LCLA_ERR_MISALIGNED;
    if (state_in != state_out && overlaps(state_in, ns, state_out, ns)) return LCLA_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0) {
        if (!state_out || state_out == state_in) return LCLA_OK;
        const cudaError_t e = state_in ? cudaMemcpyAsync(state_out, state_in, ns, cudaMemcpyDeviceToDevice, st)
                                       : cudaMemsetAsync(state_out, 0, ns, st);
        return e == cudaSuccess ? LCLA_OK : LCLA_ERR_CUDA;
    }
    if (!q || !k || !v || !g || !out) return LCLA_ERR_INVALID_ARG;
    if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned4(g) || misaligned(out) || misaligned(ws))
        return LCLA_ERR_MISALIGNED;
    const Plan p = make_plan(B, H, N, d, dtype, false);
    if (p.bytes && (!ws || ws_bytes < p.bytes)) return LCLA_ERR_WORKSPACE;
    const size_t nio = (size_t)B * N * H * d * esz, ng = (size_t)B * N * H * sizeof(float);
    const Range reads[] = {{q, nio}, {k, nio}, {v, nio}, {g, ng}, {state_in, ns}};
    const Range o = {out, nio}, s = {state_out, ns}, w = {p.bytes ? ws : nullptr, p.bytes};
    if (any_overlap(o, reads, 5) || any_overlap(s, reads, 4) || any_overlap(w, reads, 5) ||
        overlaps(o.p, o.n, s.p, s.n) || overlaps(o.p, o.n, w.p, w.n) || overlaps(s.p, s.n, w.p, w.n))
        return LCLA_ERR_INVALID_ARG;
    const Work wk = {g, B, H, N, p.nseg, p.seg_tiles, scale};
    unsigned char *wp = static_cast<unsigned char *>(ws);
    if (dtype == LCLA_BF16)
        return d == 32 ? run_forward<__nv_bfloat16, 32>(q, k, v, wk, p, state_in, out, state_out, wp, st)
                       : run_forward<__nv_bfloat16, 64>(q, k, v, wk, p, state_in, out, state_out, wp, st);
    return d == 32 ? run_forward<float, 32>(q, k, v, wk, p, state_in, out, state_out, wp, st)
                   : run_forward<float, 64>(q, k, v, wk, p, state_in, out, state_out, wp, st);
}

}  // namespace

extern "C" {

size_t lcla_gated_forward_workspace_bytes(int B, int H, int N, int d, int dtype)
{
    return check_shape(B, H, N, d, dtype) == LCLA_OK ? make_plan(B, H, N, d, dtype, false).bytes : 0;
}

size_t lcla_gated_backward_workspace_bytes(int B, int H, int N, int d, int dtype)
{
    return check_shape(B, H, N, d, dtype) == LCLA_OK ? make_plan(B, H, N, d, dtype, true).bytes : 0;
}

int lcla_gated_forward(const void *q, const void *k, const void *v, const float *g, int B, int H, int N, int d,
                       float scale, const float *state_in, void *out, float *state_out, int dtype, void *workspace,
                       size_t workspace_bytes, void *stream)
{
    return forward_impl(q, k, v, g, B, H, N, d, scale, state_in, out, state_out, dtype, workspace, workspace_bytes,
                        stream);
}

int lcla_gated_step(const void *q, const void *k, const void *v, const float *g, int B, int H, int L, int d, float scale,
                    float *state, int save, void *out, int dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    const int rc = check_shape(B, H, L, d, dtype);
    if (rc != LCLA_OK) return rc;
    if (!state) return LCLA_ERR_INVALID_ARG;
    return forward_impl(q, k, v, g, B, H, L, d, scale, state, out, save ? state : nullptr, dtype, workspace,
                        workspace_bytes, stream);
}

int lcla_gated_backward(const void *dout, const void *q, const void *k, const void *v, const float *g, int B, int H,
                        int N, int d, float scale, const float *state_in, const float *dstate_out, void *dq, void *dk,
                        void *dv, float *dg, float *dstate_in, int dtype, void *workspace, size_t workspace_bytes,
                        void *stream)
{
    const int rc = check_shape(B, H, N, d, dtype);
    if (rc != LCLA_OK) return rc;
    if (bad_scale(scale)) return LCLA_ERR_INVALID_ARG;
    const size_t esz = dtype == LCLA_BF16 ? 2 : 4, ns = (size_t)B * H * d * d * sizeof(float);
    if (misaligned(state_in) || misaligned(dstate_out) || misaligned(dstate_in)) return LCLA_ERR_MISALIGNED;
    if (dstate_in != dstate_out && overlaps(dstate_in, ns, dstate_out, ns)) return LCLA_ERR_INVALID_ARG;
    if (overlaps(dstate_in, ns, state_in, ns)) return LCLA_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0) {
        if (!dstate_in || dstate_in == dstate_out) return LCLA_OK;
        const cudaError_t e = dstate_out ? cudaMemcpyAsync(dstate_in, dstate_out, ns, cudaMemcpyDeviceToDevice, st)
                                         : cudaMemsetAsync(dstate_in, 0, ns, st);
        return e == cudaSuccess ? LCLA_OK : LCLA_ERR_CUDA;
    }
    if (!dout || !q || !k || !v || !g || !dq || !dk || !dv || !dg) return LCLA_ERR_INVALID_ARG;
    const void *ptrs[] = {dout, q, k, v, dq, dk, dv, workspace};
    for (const void *x : ptrs)
        if (misaligned(x)) return LCLA_ERR_MISALIGNED;
    if (misaligned4(g) || misaligned4(dg)) return LCLA_ERR_MISALIGNED;
    const Plan p = make_plan(B, H, N, d, dtype, true);
    if (!workspace || workspace_bytes < p.bytes) return LCLA_ERR_WORKSPACE;
    const size_t nio = (size_t)B * N * H * d * esz, ng = (size_t)B * N * H * sizeof(float);
    const Range reads[] = {{dout, nio}, {q, nio}, {k, nio}, {v, nio}, {g, ng}, {state_in, ns}, {dstate_out, ns}};
    const Range writes[] = {{dq, nio}, {dk, nio}, {dv, nio}, {dg, ng}, {workspace, p.bytes}, {dstate_in, ns}};
    for (int i = 0; i < 6; ++i) {
        if (any_overlap(writes[i], reads, i == 5 ? 5 : 7)) return LCLA_ERR_INVALID_ARG;
        if (any_overlap(writes[i], writes, i)) return LCLA_ERR_INVALID_ARG;
    }
    const Work wk = {g, B, H, N, p.nseg, p.seg_tiles, scale};
    unsigned char *wp = static_cast<unsigned char *>(workspace);
    if (dtype == LCLA_BF16)
        return d == 32 ? run_backward<__nv_bfloat16, 32>(dout, q, k, v, wk, p, state_in, dstate_out, dq, dk, dv, dg,
                                                         dstate_in, wp, st)
                       : run_backward<__nv_bfloat16, 64>(dout, q, k, v, wk, p, state_in, dstate_out, dq, dk, dv, dg,
                                                         dstate_in, wp, st);
    return d == 32 ? run_backward<float, 32>(dout, q, k, v, wk, p, state_in, dstate_out, dq, dk, dv, dg, dstate_in, wp, st)
                   : run_backward<float, 64>(dout, q, k, v, wk, p, state_in, dstate_out, dq, dk, dv, dg, dstate_in, wp,
                                             st);
}

}  // extern "C"
