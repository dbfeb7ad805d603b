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
// Kernels of a call after its first are launched while the one before them drains (launch_after); they read what it
// wrote only after this.  Every kernel of a call waits so, hence each starts after all before its predecessor.
__device__ __forceinline__ void after_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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

// Blocks of a kernel on an SM, which bounds its registers, and tiles in flight per head.  Measured on the forward at
// d = 32 (bf16, 480p, passes back to back): 3 blocks 224 us with 2 tiles in flight and 241 with 3, 2 blocks 252, 4 blocks
// 268 (they spill); at d = 64: 2 blocks and 3 tiles 346, 2 tiles 343, 4 tiles 336 (the gradient 343, 342, 344), 3 blocks and
// 2 tiles 430.
template <typename T, int D>
struct Shape {
    static constexpr int BLOCKS = sizeof(T) == 2 ? (D == 32 ? 3 : 2) : 2;
    static constexpr int STAGES = sizeof(T) == 2 && D == 64 ? 3 : 2;
    static constexpr int QK_STAGES = 2;
    static constexpr int TOTAL_BLOCKS = BLOCKS;
    static constexpr int TOTAL_STAGES = 3;
};

// The block's recurrences, of ROLES side by side.
template <typename T, int D, Direction DIR, bool DOT, int STAGES, int ROLES, bool CAREFUL>
__device__ __forceinline__ bool run_block(const Work &w, const Role *roles)
{
    using S = Smem<T, D, DOT ? 4 : 3, STAGES>;
    const Place p = place<D>(w.H, ROLES);
    return p.live && recur<T, D, DIR, DOT, STAGES, CAREFUL>(w, roles[p.role], p.b, p.h, p.seg, p.group, p.slab, p.lane,
                                                            ring_of<S>(p), weights_of<S>());
}
// Once more, where a value was not finite.  Not inlined, so that the first run has the registers to itself.
template <typename T, int D, Direction DIR, bool DOT, int STAGES, int ROLES>
__device__ __noinline__ void run_again(const Work &w, const Role *roles)
{
    run_block<T, D, DIR, DOT, STAGES, ROLES, true>(w, roles);
}
template <typename T, int D, Direction DIR, bool DOT, int STAGES, int ROLES>
__device__ __forceinline__ void run(const Work &w, const Role *roles)
{
    if (run_block<T, D, DIR, DOT, STAGES, ROLES, false>(w, roles)) run_again<T, D, DIR, DOT, STAGES, ROLES>(w, roles);
}

// Bound by matrix instructions and issue slots together (144 mma.sync, about 7 cycles each beside other work, and some
// 870 other instructions per tile and head at d = 32): 480p (70 heads, 32760 tokens, 587 MB) 168 us.  fp32 at d = 64: latency
// (255 registers, with spills, and 6 tf32 products where bf16 has 1 to 3: 6 us a tile step of one block).
template <typename T, int D>
__global__ void __launch_bounds__(THREADS, (Shape<T, D>::BLOCKS))
gated_forward_k(const __grid_constant__ Work w, const __grid_constant__ Role r)
{
    run<T, D, FORWARD, false, Shape<T, D>::STAGES, 1>(w, &r);
}

// dq and dk side by side: the same instructions for both directions, since two unrolled bodies together overflow the
// instruction cache (measured at d = 64: warps waited for instructions 2.3 of 6 cycles with three bodies in a launch).
// Bound as the forward: 2 x 4680 tokens, 35 heads, d = 64, bf16 179 us, dv 83 us.
struct Roles {
    Role r[2];
};

template <typename T, int D>
__global__ void __launch_bounds__(THREADS, (Shape<T, D>::BLOCKS))
gated_backward_qk_k(const __grid_constant__ Work w, const __grid_constant__ Roles rs)
{
    run<T, D, EITHER, true, Shape<T, D>::QK_STAGES, 2>(w, rs.r);
}

template <typename T, int D>
__global__ void __launch_bounds__(THREADS, (Shape<T, D>::BLOCKS))
gated_backward_v_k(const __grid_constant__ Work w, const __grid_constant__ Role r)
{
    run<T, D, REVERSED, false, Shape<T, D>::STAGES, 1>(w, &r);
}

// What each segment adds to the state (forward: k, v; gradient: also q, do reversed).  Bound as the forward, by 48
// mma.sync of three terms per tile and head at d = 32: 480p (294 MB) 70 us, its loads alone 49.
struct Totals {
    const void *key[2], *val[2];
    float *part[2], *decays;
};

template <typename T, int D>
__global__ void __launch_bounds__(THREADS, (Shape<T, D>::TOTAL_BLOCKS))
gated_totals_k(const __grid_constant__ Work w, const __grid_constant__ Totals t, int roles)
{
    constexpr int ST = Shape<T, D>::TOTAL_STAGES;
    using S = Smem<T, D, 2, ST>;
    const Place p = place<D>(w.H, roles);
    if (!p.live) return;
    total<T, D, ST>(w, t.key[p.role], t.val[p.role], t.part[p.role], p.role ? nullptr : t.decays, p.role == 1, p.b,
                       p.h, p.seg, p.group, p.slab, p.lane, ring_of<S>(p), weights_of<S>());
}

struct Scan {
    float *part[2];            // in: what each segment adds; out: the state before it (reversed: after it)
    const float *decays;
    const float *init[2];      // [B, H, d, d] or NULL (zero)
    float *last[2], *last2[2]; // the state after all segments, or NULL
    float init_scale[2], last_scale[2];
    int nseg, BH, n4;          // n4: float4s of a state
};

// One lane per float4 of a state, the segments dealt out in runs of SCAN_RUN over the block's warps.  Bound by latency:
// a warp reads its run at once, the runs' sums and decays meet in shared memory, and each warp then carries the state
// through its run (47 segments at d = 64: 9.4 us with one thread for all of them, 8 read ahead of the chain).
constexpr int SCAN_WARPS = 8, SCAN_RUN = 8;      // warps at most: as many as there are runs
__device__ __forceinline__ float4 decayed_plus(const float4 &c, float d, const float4 &v)
{
    return make_float4(fmaf(c.x, d, v.x), fmaf(c.y, d, v.y), fmaf(c.z, d, v.z), fmaf(c.w, d, v.w));
}
__global__ void __launch_bounds__(SCAN_WARPS * 32) gated_scan_k(const __grid_constant__ Scan s)
{
    __shared__ float4 sums[SCAN_WARPS][32];
    __shared__ float decays[SCAN_WARPS][32];
    after_launch_before();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, dir = blockIdx.y;
    const int i = blockIdx.x * 32 + lane, all = s.BH * s.n4, bh = i / s.n4;      // n4 is a multiple of 32
    float4 carry = make_float4(0.f, 0.f, 0.f, 0.f);
    if (s.init[dir]) {
        const float4 c = reinterpret_cast<const float4 *>(s.init[dir])[i];
        const float m = s.init_scale[dir];
        carry = make_float4(c.x * m, c.y * m, c.z * m, c.w * m);
    }
    float4 *part = reinterpret_cast<float4 *>(s.part[dir]);
    auto at = [&](int k) { return dir ? s.nseg - 1 - k : k; };
    for (int first = 0; first < s.nseg; first += warps * SCAN_RUN) {
        const int k0 = first + warp * SCAN_RUN;
        float4 v[SCAN_RUN];
        float d[SCAN_RUN];
#pragma unroll
        for (int u = 0; u < SCAN_RUN; ++u) {            // loads without branches go out together
            const int k = at(min(k0 + u, s.nseg - 1));
            v[u] = part[(size_t)k * all + i];
            d[u] = s.decays[(size_t)k * s.BH + bh];
        }
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        float decay = 1.f;
#pragma unroll
        for (int u = 0; u < SCAN_RUN; ++u)
            if (k0 + u < s.nseg) {
                sum = decayed_plus(sum, d[u], v[u]);
                decay *= d[u];
            }
        sums[warp][lane] = sum;
        decays[warp][lane] = decay;
        __syncthreads();
        float4 c = carry;
#pragma unroll
        for (int w = 0; w < SCAN_WARPS; ++w) {
            if (w == warp) c = carry;
            if (w < warps) carry = decayed_plus(carry, decays[w][lane], sums[w][lane]);
        }
#pragma unroll
        for (int u = 0; u < SCAN_RUN; ++u)
            if (k0 + u < s.nseg) {
                part[(size_t)at(k0 + u) * all + i] = c;
                c = decayed_plus(c, d[u], v[u]);
            }
        __syncthreads();                                // the sums have been read
    }
    if (warp != 0) return;
    if (s.last2[dir]) reinterpret_cast<float4 *>(s.last2[dir])[i] = carry;
    if (s.last[dir]) {
        const float m = s.last_scale[dir];
        reinterpret_cast<float4 *>(s.last[dir])[i] = make_float4(carry.x * m, carry.y * m, carry.z * m, carry.w * m);
    }
}

struct GradGate {
    const void *q, *k, *v, *dout;
    float *dot;                // [planes][B, H, N]: as the roles left them, queries' planes first
    const float *norm;         // [planes][B, H, tiles]
    float *up, *down, *most;   // [B, H, tiles], strong tiles: sum of A, sum of B, the bound of X
    const float *before;       // [nseg + 1][B, H, d, d]: the state before each segment, and after the last
    const float *after;        // [nseg][B, H, d, d]: its gradient after each segment, over scale
    float *dg;
    Work w;
    bool carried;              // a state came in before the first token
};

// Two neighbouring entries of one token's row in global memory, or zeros.
__device__ __forceinline__ In<__nv_bfloat16> pair_of(const __nv_bfloat16 *p, bool on)
{
    return In<__nv_bfloat16>{on ? *reinterpret_cast<const uint32_t *>(p) : 0u};
}
__device__ __forceinline__ In<float> pair_of(const float *p, bool on)
{
    In<float> r;
    split_tf32(r, on ? *reinterpret_cast<const float2 *>(p) : make_float2(0.f, 0.f));
    return r;
}

// Products of a tile's rows a_u . b_s for the 16x16 blocks (0,0), (1,0) and (1,1), whose first rows lie at a and b.
template <typename T, int D>
__device__ __forceinline__ void tile_scores(float (&c)[3][2][4], const T *a, const T *b, size_t row, int live, int lane)
{
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        In<T> fa[2][4], fb[2][2][2];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int u = 16 * m + 8 * (p & 1) + (lane >> 2), e = 16 * ks + 8 * (p >> 1) + 2 * (lane & 3);
                fa[m][p] = pair_of(a + u * row + e, u < live);
                const int s = 16 * m + 8 * (p >> 1) + (lane >> 2), f = 16 * ks + 8 * (p & 1) + 2 * (lane & 3);
                fb[m][p >> 1][p & 1] = pair_of(b + s * row + f, s < live);
            }
#pragma unroll
        for (int i = 0; i < Steps<T, false>::N; ++i)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                if (ks == 0 && i == 0) {
                    mma<true>(i, c[0][n], fa[0], fb[0][n][0], fb[0][n][1]);
                    mma<true>(i, c[1][n], fa[1], fb[0][n][0], fb[0][n][1]);
                    mma<true>(i, c[2][n], fa[1], fb[1][n][0], fb[1][n][1]);
                } else {
                    mma<false>(i, c[0][n], fa[0], fb[0][n][0], fb[0][n][1]);
                    mma<false>(i, c[1][n], fa[1], fb[0][n][0], fb[0][n][1]);
                    mma<false>(i, c[2][n], fa[1], fb[1][n][0], fb[1][n][1]);
                }
            }
    }
}

// In lane t: the sum of M[u][s] over s < t <= u inside the tile, M[u][s] = e^{G_u - G_s} (q_u . k_s) (do_u . v_s).
constexpr int kPairRow = TILE + 1;
template <typename T, int D>
__device__ __forceinline__ float tile_pairs(const GradGate &p, size_t at, size_t row, int live, const Weights *wt,
                                            float *M, int lane)
{
    float qk[3][2][4], dv[3][2][4];
    tile_scores<T, D>(qk, (const T *)p.q + at, (const T *)p.k + at, row, live, lane);
    tile_scores<T, D>(dv, (const T *)p.dout + at, (const T *)p.v + at, row, live, lane);
    __syncwarp();                              // the last tile's sums have been read
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int u = 16 * (i > 0) + 8 * (j >> 1) + (lane >> 2);
                const int s = 16 * (i > 1) + 8 * n + 2 * (lane & 3) + (j & 1);
                const float e = (wt->whole[s] - wt->whole[u]) + (wt->frac[s] - wt->frac[u]);
                M[u * kPairRow + s] = qk[i][n][j] * dv[i][n][j] * ex2(e);
            }
    __syncwarp();
    float x[TILE], sum = 0.f;
#pragma unroll
    for (int s = 0; s < TILE; ++s) x[s] = M[lane * kPairRow + s];
#pragma unroll
    for (int s = 0; s < TILE; ++s) {           // row `lane`: M[u][t] becomes the sum over s < t
        M[lane * kPairRow + s] = sum;
        sum += s < lane ? x[s] : 0.f;
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < TILE; ++u) x[u] = M[u * kPairRow + lane];
    sum = 0.f;
#pragma unroll
    for (int u = TILE - 1; u >= 0; --u) sum += u >= lane ? x[u] : 0.f;
    return sum;
}

// dg_t is scale times the sum of M[u][s] (above) over all pairs s < t <= u of the sequence, the carried state and the
// carried gradient counting as tokens at its ends.  The value at a segment's end is <S, R>; from a token to the one before
// it the sum changes by <q, dq> - <k, dk>.  Where a state decays much between two tokens those terms cancel to less than
// their own roundings, and a running sum would carry the roundings of later tokens to ones that they cannot reach.  So
// tiles go by their decay (strong_tile):
//   mild: the running sum;
//   strong: with D the value after the tile, A_u and B_s the carried states' parts of <q_u, dq_u> and <k_s, dk_s>, and X
//     the pairs around the whole tile,
//       X = D - sum of all B_s, no larger than decay |S before| |R after|,
//       dg_t = X + sum over u >= t of A_u + sum over s < t of B_s + the pairs inside the tile,
//     each a sum over pairs of dg_t alone, and nothing at all across a decay that is zero.
// What errors are left, beside 2^-17 of the magnitudes of dg_t's own pairs: in a mild tile 2^-22 of the terms of the mild
// tiles after it; in X the same of the pairs around the tile's end, never more than its bound (so a single gate of g < -3
// among mild ones has the roundings of its neighbours, 2^-22 e^-g of itself).
// gated_dgate_strong_k, a warp per tile, does what a strong one needs and leaves its part of dg in the first plane;
// gated_dgate_k, a block per segment of a head (at most 32 tiles), takes D through the segment.  Bound by latency: 2 x 4680
// tokens, 35 heads, d = 64, bf16, 6 % of the tiles strong, 16 and 14 us from cold caches; all of them strong 65 us more.
template <typename T, int D>
__global__ void __launch_bounds__(THREADS) gated_dgate_strong_k(const __grid_constant__ GradGate p)
{
    constexpr int PLANES = D / 32;
    __shared__ Weights weights[WARPS];
    __shared__ float pairs[WARPS][TILE * kPairRow];
    after_launch_before();
    const Work &w = p.w;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, BH = w.B * w.H, tiles = (w.N + TILE - 1) / TILE;
    const size_t nplane = (size_t)BH * tiles, unit = (size_t)blockIdx.x * WARPS + warp;
    if (unit >= nplane || p.norm[unit] == -1.f) return;
    const int tile = (int)(unit % tiles), bh = (int)(unit / tiles), b = bh / w.H, h = bh % w.H;
    const int t0 = tile * TILE, t = t0 + lane, u = min(t, w.N - 1);
    const size_t plane = (size_t)BH * w.N, row = (size_t)w.H * D;
    float *dot = p.dot + (size_t)bh * w.N + u;
    float g = w.g[((size_t)b * w.N + u) * w.H + h], A = 0.f, B = 0.f;
#pragma unroll
    for (int k = 0; k < PLANES; ++k) {
        A += dot[k * plane];
        B -= dot[(PLANES + k) * plane];        // <k, dk>, which its planes hold negated
    }
    if (t >= w.N) A = B = g = 0.f;
    double total;
    const float decay = tile_weights(&weights[warp], g, false, lane, total);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {         // sums from each token on, and up to each token
        const float later = __shfl_down_sync(0xffffffffu, A, o), earlier = __shfl_up_sync(0xffffffffu, B, o);
        if (lane + o < 32) A += later;
        if (lane >= o) B += earlier;
    }
    if (lane == 0) p.up[unit] = A;
    if (lane == 31) {
        float sq = 0.f, rq = 0.f;
#pragma unroll
        for (int k = 0; k < PLANES; ++k) {
            sq += p.norm[k * nplane + unit];
            rq += p.norm[(PLANES + k) * nplane + unit];
        }
        p.down[unit] = B;
        // 1.001: the bound's own roundings
        p.most[unit] = decay == 0.f ? 0.f : 1.001f * decay * fabsf(w.scale) * sqrtf(sq) * sqrtf(rq);
    }
    const float pair = tile_pairs<T, D>(p, ((size_t)b * w.N + t0) * row + (size_t)h * D, row, min(TILE, w.N - t0),
                                        &weights[warp], pairs[warp], lane);
    const float before = __shfl_up_sync(0xffffffffu, B, 1);
    // nothing passes a reset: X is zero too
    if (t < w.N) *dot = g < RESET ? 0.f : A + (lane ? before : 0.f) + w.scale * pair;
}

constexpr int kGateTiles = 32;     // tiles of a segment at most
template <int D>
__global__ void __launch_bounds__(THREADS) gated_dgate_k(const __grid_constant__ GradGate p)
{
    constexpr int PLANES = 2 * (D / 32), N4 = D * D / 4, PER = kGateTiles / WARPS;
    __shared__ float ends[WARPS], up[kGateTiles], down[kGateTiles], most[kGateTiles];   // most < 0: a mild tile
    after_launch_before();
    const Work &w = p.w;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, BH = w.B * w.H, tiles = (w.N + TILE - 1) / TILE;
    const int bh = (int)(blockIdx.x % (unsigned)BH), seg = (int)(blockIdx.x / (unsigned)BH), b = bh / w.H, h = bh % w.H;
    const int first = seg * w.seg_tiles, n = min(w.seg_tiles, tiles - first), end = first + n - 1;
    const size_t plane = (size_t)BH * w.N;
    const float *dot = p.dot + (size_t)bh * w.N;
    float own[PER], rest[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {            // loads without branches go out together
        const int t = (end - (warp + WARPS * i)) * TILE + lane, u = min(max(t, 0), w.N - 1);
        own[i] = dot[u];
        rest[i] = 0.f;
#pragma unroll
        for (int k = 1; k < PLANES; ++k) rest[i] += dot[k * plane + u];
        if (t >= w.N) own[i] = rest[i] = 0.f;
    }
    if (warp == 0 && lane < n) {
        const size_t at = (size_t)bh * tiles + end - lane;
        const bool strong = p.norm[at] != -1.f;
        up[lane] = p.up[at];                   // of a mild tile: replaced below
        down[lane] = p.down[at];
        most[lane] = strong ? p.most[at] : -1.f;
    }
    const float4 *S = reinterpret_cast<const float4 *>(p.before) + ((size_t)(seg + 1) * BH + bh) * N4;
    const float4 *R = reinterpret_cast<const float4 *>(p.after) + ((size_t)seg * BH + bh) * N4;
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < N4 / THREADS; ++i) {
        const float4 x = S[threadIdx.x + i * THREADS], z = R[threadIdx.x + i * THREADS];
        y = fmaf(x.x, z.x, fmaf(x.y, z.y, fmaf(x.z, z.z, fmaf(x.w, z.w, y))));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (lane == 0) ends[warp] = y;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int k = warp + WARPS * i;
        if (k < n && most[k] < 0.f) {
            float x = own[i] + rest[i];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float later = __shfl_down_sync(0xffffffffu, x, o);
                if (lane + o < 32) x += later;
            }
            own[i] = x;
            if (lane == 0) up[k] = x;
        }
    }
    __syncthreads();
    double after = 0.0;                        // the value after a tile
#pragma unroll
    for (int k = 0; k < WARPS; ++k) after += ends[k];
    after *= w.scale;
#pragma unroll
    for (int k = 0; k < kGateTiles; ++k)
        if (k < n) {
            const float m = most[k];
            double X = after;
            if (!(m < 0.f)) {
                X = m == 0.f ? 0.0 : after - down[k];
                X = X > m ? m : X < -m ? -m : X;           // a NaN stays one
            }
            const int t = (end - k) * TILE + lane;
            if (k % WARPS == warp && t < w.N)
                p.dg[((size_t)b * w.N + t) * w.H + h] = t == 0 && !p.carried ? 0.f : (float)(X + own[k / WARPS]);
            after = X + up[k];
        }
}

// A few tokens against the state: read once, kept in registers, written once.  One block per head; D / 4 lanes hold a
// row of the state, four entries each.  Bound by HBM: one token of 64 streams of 35 heads at d = 64 (74 MB) 14 us
// from cold caches, 10 with the states in L2.
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
        const float a = expf(bounded(gt));
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

// Calls of a few tokens take gated_short_k, whose time grows with each of them, longer ones the tiles.  Measured in
// microseconds with the states in L2, tokens by tokens / tiles: bf16, 1 stream x 8 heads, d = 32: 1 token 2.0 / 3.9, 2 2.7 /
// 4.1, 4 3.7 / 4.2, 5 4.1 / 4.1, 8 5.7 / 4.1; 8 x 35, d = 64: 4 5.8 / 5.8, 8 9.4 / 5.8; 64 x 35, d = 64: 1 9.7 / 25.8, 4 18.4
// / 26.0, 6 25.6 / 26.6, 8 32.0 / 26.6; fp32, 8 x 35, d = 64: 4 5.7 / 9.6, 8 9.0 / 9.6, 12 12.5 / 9.6.
bool is_short(int N, int dtype) { return N <= (dtype == LCLA_BF16 ? 4 : 8); }

struct Plan {
    int nseg, seg_tiles;
    size_t before, after, decays, dot, norm, sums, bytes;   // workspace offsets
};

// Microseconds of a tile step of the forward's recurrence with one block on an SM, whose warps wait for one instruction
// after another, and with as many as fit, which keep the matrix units and issue slots busy.
struct StepTime {
    double one, full;
    int blocks;
};
StepTime step_time(int d, int dtype)
{
    if (dtype == LCLA_BF16)
        return d == 32 ? StepTime{1.3, 3.0, Shape<__nv_bfloat16, 32>::BLOCKS} : StepTime{1.9, 3.0, Shape<__nv_bfloat16, 64>::BLOCKS};
    return d == 32 ? StepTime{3.0, 4.6, Shape<float, 32>::BLOCKS} : StepTime{7.0, 8.6, Shape<float, 64>::BLOCKS};
}

// A kernel of n blocks over segments of ts tiles; each block spends about 1.5 steps on its start and end.
double kernel_time(long long n, long long ts, const StepTime &t)
{
    const long long cap = (long long)kSms * t.blocks, rounds = n / cap, rest = n % cap;
    double steps = rounds * t.full;
    if (rest) steps += t.one + (t.full - t.one) * ((rest + kSms - 1) / kSms - 1) / (t.blocks - 1);
    return steps * (ts + 1.5);
}

// How many segments: the cheapest by this estimate.  Over 15 problems of 10 to 1024 tiles, each also run with 1 to 128
// segments, its choice was the fastest or within 2.1 us of it.  Its constants are of bf16 kernels with two terms: estimates
// above 80 us are 14 % low to 4 % high (bf16, d = 64 gradient of 2 x 35 heads: 147 tiles in 8 segments 306 us estimated, 346
// measured; 10 tiles in 4 segments 44 and 57, in one 90 measured), and constants fitted again chose worse in one problem of
// the 15.  A step of the totals costs half of the forward's, one of dq and dk 1.4 times; the scan and the launches 6 us and
// more with each segment.
Plan make_plan(int B, int H, int N, int d, int dtype, bool backward)
{
    Plan p = {};
    if (N == 0 || (!backward && is_short(N, dtype))) return p;
    const int tiles = (N + TILE - 1) / TILE, ns = d / 32, G = WARPS / ns;
    const long long per_seg = (long long)((H + G - 1) / G) * B;
    const StepTime t = step_time(d, dtype);
    double best = 1e30;
    p.nseg = 1;
    p.seg_tiles = tiles;
    auto consider = [&](long long ts) {
        if (ts < 1 || ts > tiles || (backward && ts > kGateTiles)) return;
        const long long nseg = (tiles + ts - 1) / ts, b = nseg * per_seg;
        double cost = kernel_time(b, ts, t);
        if (backward) cost += 1.4 * kernel_time(2 * b, ts, t) + 0.5 * kernel_time(2 * b, ts, t) + 4.0;
        else if (nseg > 1) cost += 0.5 * kernel_time(b, ts, t);
        if (backward || nseg > 1) cost += 6.0 + 0.08 * nseg;
        if (cost < best) {
            best = cost;
            p.nseg = (int)nseg;
            p.seg_tiles = (int)ts;
        }
    };
    consider(tiles);
    for (long long ts = 1; ts <= 64; ++ts) consider(ts);
    for (long long c = 1; c <= 16; ++c) {       // segments that fill c rounds of resident blocks
        const long long nseg = c * kSms * t.blocks / per_seg;
        if (nseg > 1) consider((tiles + nseg - 1) / nseg);
    }
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
        p.norm = at;
        at += round_up((size_t)2 * ns * B * H * tiles * sizeof(float));
        p.sums = at;
        at += round_up((size_t)3 * B * H * tiles * sizeof(float));
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
    if ((long long)((N + 31) / 32) * H * 2 > 0x7fffffffLL) return LCLA_ERR_UNSUPPORTED;
    // and the gate gradient's blocks, one per head and segment of at most kGateTiles tiles
    if ((long long)B * H * ((N + 31) / 32) > 0x7fffffffLL) return LCLA_ERR_UNSUPPORTED;
    return LCLA_OK;
}

template <typename F>
void set_smem(F *kernel, int bytes)
{
    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename... KArgs, typename... Args>
void launch_after(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t st, const Args &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
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
    using S = Smem<T, D, 2, Shape<T, D>::TOTAL_STAGES>;
    set_smem(gated_totals_k<T, D>, S::BYTES);
    gated_totals_k<T, D><<<dim3(blocks<D>(w, roles), w.B), THREADS, S::BYTES, st>>>(w, t, roles);
}

void launch_scan(const Scan &s, int dirs, cudaStream_t st)
{
    const int runs = (s.nseg + SCAN_RUN - 1) / SCAN_RUN;
    launch_after(gated_scan_k, dim3(s.BH * (s.n4 / 32), dirs), 32 * (runs < SCAN_WARPS ? runs : SCAN_WARPS), 0, st, s);
}

template <typename T, int D>
int run_forward(const void *q, const void *k, const void *v, const Work &w, const Plan &p, const float *state_in,
                void *out, float *state_out, unsigned char *ws, cudaStream_t st)
{
    if (is_short(w.N, sizeof(T) == 2 ? LCLA_BF16 : LCLA_F32)) {
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
    using S = Smem<T, D, 3, Shape<T, D>::STAGES>;
    auto kernel = gated_forward_k<T, D>;
    set_smem(kernel, S::BYTES);
    const dim3 grid(blocks<D>(w, 1), w.B);
    if (w.nseg > 1) launch_after(kernel, grid, THREADS, S::BYTES, st, w, r);
    else kernel<<<grid, THREADS, S::BYTES, st>>>(w, r);
    return launched();
}

template <typename T, int D>
int run_backward(const void *dout, const void *q, const void *k, const void *v, const Work &w, const Plan &p,
                 const float *state_in, const float *dstate_out, void *dq, void *dk, void *dv, float *dg,
                 float *dstate_in, unsigned char *ws, cudaStream_t st)
{
    float *before = reinterpret_cast<float *>(ws + p.before), *after = reinterpret_cast<float *>(ws + p.after);
    float *dot = reinterpret_cast<float *>(ws + p.dot), *norm = reinterpret_cast<float *>(ws + p.norm);
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
    const size_t plane = (size_t)BH * w.N, nplane = (size_t)BH * ((w.N + TILE - 1) / TILE);
    Roles rs = {};
    // recur reads the state of segment `seg` also where there is only one
    Role &rq = rs.r[0], &rk = rs.r[1], rv = {};
    rq.q = dout; rq.k = v; rq.v = k; rq.x = q; rq.out = dq;
    rq.state = before; rq.transposed = true; rq.dot = dot; rq.norm = norm; rq.sign = 1.f;
    rk.q = v; rk.k = dout; rk.v = q; rk.x = k; rk.out = dk;
    rk.state = after; rk.transposed = true; rk.dot = dot + ns * plane; rk.norm = norm + ns * nplane;
    rk.sign = -1.f;
    rk.rev = true;
    rv.q = k; rv.k = q; rv.v = dout; rv.out = dv;
    rv.state = after; rv.rev = true;
    using S4 = Smem<T, D, 4, Shape<T, D>::QK_STAGES>;
    set_smem(gated_backward_qk_k<T, D>, S4::BYTES);
    launch_after(gated_backward_qk_k<T, D>, dim3(blocks<D>(w, 2), w.B), THREADS, S4::BYTES, st, w, rs);
    using S3 = Smem<T, D, 3, Shape<T, D>::STAGES>;
    set_smem(gated_backward_v_k<T, D>, S3::BYTES);
    launch_after(gated_backward_v_k<T, D>, dim3(blocks<D>(w, 1), w.B), THREADS, S3::BYTES, st, w, rv);
    GradGate gg = {};
    gg.q = q; gg.k = k; gg.v = v; gg.dout = dout;
    gg.dot = dot; gg.norm = norm; gg.before = before; gg.after = after; gg.dg = dg;
    gg.up = reinterpret_cast<float *>(ws + p.sums);
    gg.down = gg.up + nplane;
    gg.most = gg.down + nplane;
    gg.w = w;
    gg.carried = state_in != nullptr;
    launch_after(gated_dgate_strong_k<T, D>, dim3((unsigned)((nplane + WARPS - 1) / WARPS)), THREADS, 0, st, gg);
    launch_after(gated_dgate_k<D>, dim3((unsigned)((long long)BH * w.nseg)), THREADS, 0, st, gg);
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
