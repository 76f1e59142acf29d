// Norm of queries and keys with the position rotation, and its gradient.  A head
// v of D channels becomes u = v r g, r = (sum v^2 / D + eps)^-1/2, and each pair
// (a, b) of u is turned by the angle t of its token's position:
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t).
// Backward, with du = dy turned by -t, w = g du and h = v r:
//   dg = sum du h,   dx = r (w - h sum(w h) / D) = r w - v r^3 sum(w v) / D,
// so that one sweep over a head gives both of its sums, and dx needs nothing
// that is not at hand.
//
// DRAM bounds both directions: each element is read once and written once, and
// a turn's cosine and sine serve every head of the token.  A group of lanes
// holds a head (each lane a vector of its first half and the matching one of its
// second, where the partners of the split pairing are), so a warp takes
// 32 / lanes heads at a time and joins a head's sum by shuffles.
#include <algorithm>
#include <cmath>

#include "map_ops.h"
#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {

using namespace maps;
using dev::grid_dependency_wait;
using dev::grid_launch_dependents;

constexpr int kQkSms = 152;
constexpr int kQkThreads = 256;
constexpr int kQkWarps = kQkThreads / 32;
constexpr int kQkMaxD = 256;
constexpr int kQkBlocks = 4 * kQkSms;   // most CTAs of a gradient call, each with a row of partial sums

struct QkArgs {
    View x, y, dy;              // forward: x -> y; gradient: x, dy -> y
    const float *gq, *gk;
    const int *pos;             // null: the pixel's place
    float *part;                // gradient: [blocks][D] partial sums, or null
    unsigned tokens, HW, W;
    int x_px, y_px, dy_px;      // bytes of a pixel
    int x_joined, y_joined, dy_joined;
    int q_heads, k_heads, D;
    int lanes;                  // lanes of a head's group
    int chunks;                 // runs of heads a token is cut into, for calls of few tokens
    unsigned q_blocks;          // CTAs of the query heads; the others take the key heads
    int row_pairs, pairs;
    float eps, inv_d;
    unsigned long long turn[kQkMaxD / 2];   // a position step's angle in 2^-64 turns
};

// Cosine and sine of position * turn: the product's low 64 bits are the angle
// modulo a turn, exactly; its top 32 bits go on as a signed float.
__device__ __forceinline__ void turned(int p, unsigned long long turn, float &c, float &s)
{
    const unsigned long long f = static_cast<unsigned long long>(static_cast<long long>(p)) * turn;
    sincospif(static_cast<float>(static_cast<int>(f >> 32)) * 0x1p-31f, &s, &c);
}

__device__ __forceinline__ long long token_off(unsigned n, unsigned px, const View &v, unsigned W, int joined, int bytes)
{
    return n * v.bstride + pixel_off(px, W, joined != 0, v.pitch, bytes);
}

// VE: elements of a vector, NV: vectors a lane holds of each half.  INTER: pairs
// are neighbours.  A lane's pairs are (lo[i], hi[i]), or, of neighbours, those
// inside lo and then those inside hi (VE 1: lo and hi are neighbours).
template <int VE, bool INTER>
__device__ __forceinline__ void to_pairs(const float (&lo)[VE], const float (&hi)[VE], float (&a)[VE], float (&b)[VE])
{
#pragma unroll
    for (int i = 0; i < VE; i++) {
        if (INTER && VE > 1) {
            a[i] = i < VE / 2 ? lo[(2 * i) % VE] : hi[(2 * i) % VE];
            b[i] = i < VE / 2 ? lo[(2 * i) % VE + 1] : hi[(2 * i) % VE + 1];
        } else {
            a[i] = lo[i];
            b[i] = hi[i];
        }
    }
}
template <int VE, bool INTER>
__device__ __forceinline__ void from_pairs(const float (&a)[VE], const float (&b)[VE], float (&lo)[VE], float (&hi)[VE])
{
#pragma unroll
    for (int i = 0; i < VE; i++) {
        if (INTER && VE > 1) {
            lo[i] = (i & 1) ? b[i / 2] : a[i / 2];
            hi[i] = (i & 1) ? b[VE / 2 + i / 2] : a[VE / 2 + i / 2];
        } else {
            lo[i] = a[i];
            hi[i] = b[i];
        }
    }
}

// What a lane holds of every head: the channels of its vectors, their gammas and
// its pairs' numbers.
template <class T, int VE, int NV, bool INTER>
struct QkLane {
    int lo[NV], hi[NV], pair[NV];   // first channel of either vector; the first pair (of hi's half where INTER: + half / 2)
    bool on[NV];
    float ga[NV][VE], gb[NV][VE];
    float cs[NV][VE], sn[NV][VE];

    __device__ __forceinline__ void place(int sub, int lanes, int half)
    {
#pragma unroll
        for (int v = 0; v < NV; v++) {
            const int idx = sub + v * lanes;
            on[v] = idx * VE < half;
            lo[v] = INTER && VE == 1 ? 2 * idx : idx * VE;
            hi[v] = INTER && VE == 1 ? 2 * idx + 1 : half + idx * VE;
            pair[v] = INTER && VE > 1 ? idx * VE / 2 : idx * VE;
        }
    }
    __device__ __forceinline__ void gammas(const float *g)
    {
#pragma unroll
        for (int v = 0; v < NV; v++) {
            float l[VE], h[VE];
#pragma unroll
            for (int i = 0; i < VE; i++) {
                l[i] = g && on[v] ? g[lo[v] + i] : 1.0f;
                h[i] = g && on[v] ? g[hi[v] + i] : 1.0f;
            }
            to_pairs<VE, INTER>(l, h, ga[v], gb[v]);
        }
    }
    __device__ __forceinline__ void angles(const unsigned long long *turn, int row, int col, int row_pairs, int half)
    {
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int i = 0; i < VE; i++) {
                int j = pair[v] + i;
                if (INTER && VE > 1 && i >= VE / 2) j += (half - VE) / 2;
                if (!on[v]) j = 0;
                turned(j < row_pairs ? row : col, turn[j], cs[v][i], sn[v][i]);
            }
    }
};

__device__ __forceinline__ float group_sum(float v, int lanes)
{
    for (int o = lanes >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One warp takes a token's heads (or a run of them) at a time, U groups' vectors
// read before the first is used.
template <class T, int VE, int NV, bool INTER, bool GRAD, int U>
__global__ void __launch_bounds__(kQkThreads) k_qk_norm(const __grid_constant__ QkArgs a)
{
    using V = Raw<T, VE>;
    __shared__ unsigned long long turn[kQkMaxD / 2];
    __shared__ float sums[GRAD ? kQkWarps : 1][GRAD ? kQkMaxD : 1];
    grid_launch_dependents();
    const int half = a.D / 2;
    for (int i = threadIdx.x; i < half; i += kQkThreads) turn[i] = a.turn[i];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool keys = blockIdx.x >= a.q_blocks;
    const unsigned block = keys ? blockIdx.x - a.q_blocks : blockIdx.x;
    const unsigned blocks = keys ? gridDim.x - a.q_blocks : a.q_blocks;
    const int heads = keys ? a.k_heads : a.q_heads, first = keys ? a.q_heads : 0;
    const int lanes = a.lanes, at_once = 32 / lanes, group = lane / lanes;
    QkLane<T, VE, NV, INTER> k;
    k.place(lane & (lanes - 1), lanes, half);
    __syncthreads();
    grid_dependency_wait();
    k.gammas(keys ? a.gk : a.gq);
    float da[NV][VE], db[NV][VE];
    if (GRAD) {
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int i = 0; i < VE; i++) da[v][i] = db[v][i] = 0.0f;
    }
    const int chunk = (heads + a.chunks - 1) / a.chunks;
    const unsigned long long items = static_cast<unsigned long long>(a.tokens) * a.chunks;
    for (unsigned long long item = static_cast<unsigned long long>(block) * kQkWarps + warp; item < items;
         item += static_cast<unsigned long long>(blocks) * kQkWarps) {
        const unsigned t = static_cast<unsigned>(a.chunks == 1 ? item : item / a.chunks);
        const int h0 = static_cast<int>(item - static_cast<unsigned long long>(t) * a.chunks) * chunk;
        const int h1 = min(heads, h0 + chunk);
        const unsigned n = t / a.HW, px = t - n * a.HW;
        const uint8_t *xt = a.x.p + token_off(n, px, a.x, a.W, a.x_joined, a.x_px);
        const uint8_t *dt = GRAD ? a.dy.p + token_off(n, px, a.dy, a.W, a.dy_joined, a.dy_px) : nullptr;
        uint8_t *yt = a.y.p + token_off(n, px, a.y, a.W, a.y_joined, a.y_px);
        bool ready = false;
        for (int h = h0; h < h1; h += U * at_once) {
            V x[U][NV][2], d[GRAD ? U : 1][NV][2];
#pragma unroll
            for (int u = 0; u < U; u++)
#pragma unroll
                for (int v = 0; v < NV; v++) {
                    const int hd = h + u * at_once + group;
                    const long long off = static_cast<long long>(first + hd) * a.D;
                    if (hd < h1 && k.on[v]) {
                        x[u][v][0] = __ldcs(reinterpret_cast<const V *>(xt + (off + k.lo[v]) * sizeof(T)));
                        x[u][v][1] = __ldcs(reinterpret_cast<const V *>(xt + (off + k.hi[v]) * sizeof(T)));
                        if (GRAD) {
                            d[u][v][0] = __ldcs(reinterpret_cast<const V *>(dt + (off + k.lo[v]) * sizeof(T)));
                            d[u][v][1] = __ldcs(reinterpret_cast<const V *>(dt + (off + k.hi[v]) * sizeof(T)));
                        }
                    } else {
                        x[u][v][0] = x[u][v][1] = V{};
                        if (GRAD) d[u][v][0] = d[u][v][1] = V{};
                    }
                }
            if (!ready) {
                // under the first vectors' flight
                const unsigned prow = px / a.W;
                int row = static_cast<int>(prow), col = static_cast<int>(px - prow * a.W);
                if (a.pos) {
                    const int2 p = reinterpret_cast<const int2 *>(a.pos)[t];
                    row = p.x;
                    col = p.y;
                }
                k.angles(turn, row, col, a.row_pairs, half);
                ready = true;
            }
#pragma unroll
            for (int u = 0; u < U; u++) {
                if (h + u * at_once >= h1) break;   // the same for the whole warp
                const int hd = h + u * at_once + group;
                const long long off = static_cast<long long>(first + hd) * a.D;
                float xa[NV][VE], xb[NV][VE], wa[NV][VE], wb[NV][VE];
                float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
                for (int v = 0; v < NV; v++) {
                    float lo[VE], hi[VE];
                    unpack<T, VE>(x[u][v][0], lo);
                    unpack<T, VE>(x[u][v][1], hi);
                    to_pairs<VE, INTER>(lo, hi, xa[v], xb[v]);
#pragma unroll
                    for (int i = 0; i < VE; i++) s1 = fmaf(xa[v][i], xa[v][i], fmaf(xb[v][i], xb[v][i], s1));
                    if (GRAD) {
                        float ya[VE], yb[VE];
                        unpack<T, VE>(d[u][v][0], lo);
                        unpack<T, VE>(d[u][v][1], hi);
                        to_pairs<VE, INTER>(lo, hi, ya, yb);
#pragma unroll
                        for (int i = 0; i < VE; i++) {
                            // turned back; dg's term lacks r, w has gamma
                            wa[v][i] = fmaf(ya[i], k.cs[v][i], yb[i] * k.sn[v][i]);
                            wb[v][i] = fmaf(yb[i], k.cs[v][i], -ya[i] * k.sn[v][i]);
                            s2 = fmaf(wa[v][i] * k.ga[v][i], xa[v][i], fmaf(wb[v][i] * k.gb[v][i], xb[v][i], s2));
                        }
                    }
                }
                s1 = group_sum(s1, lanes);
                if (GRAD) s2 = group_sum(s2, lanes);
                const float r = rsqrtf(fmaf(s1, a.inv_d, a.eps));
                const float m = GRAD ? r * r * r * (s2 * a.inv_d) : 0.0f;
#pragma unroll
                for (int v = 0; v < NV; v++) {
                    float oa[VE], ob[VE], lo[VE], hi[VE];
#pragma unroll
                    for (int i = 0; i < VE; i++) {
                        if (GRAD) {
                            if (hd < h1) {      // r of a lane without a head is not finite for eps 0
                                da[v][i] = fmaf(wa[v][i] * xa[v][i], r, da[v][i]);
                                db[v][i] = fmaf(wb[v][i] * xb[v][i], r, db[v][i]);
                            }
                            oa[i] = fmaf(wa[v][i] * k.ga[v][i], r, -xa[v][i] * m);
                            ob[i] = fmaf(wb[v][i] * k.gb[v][i], r, -xb[v][i] * m);
                        } else {
                            const float ua = xa[v][i] * r * k.ga[v][i], ub = xb[v][i] * r * k.gb[v][i];
                            oa[i] = fmaf(ua, k.cs[v][i], -ub * k.sn[v][i]);
                            ob[i] = fmaf(ua, k.sn[v][i], ub * k.cs[v][i]);
                        }
                    }
                    if (hd < h1 && k.on[v]) {
                        from_pairs<VE, INTER>(oa, ob, lo, hi);
                        *reinterpret_cast<V *>(yt + (off + k.lo[v]) * sizeof(T)) = pack<T, VE>(lo);
                        *reinterpret_cast<V *>(yt + (off + k.hi[v]) * sizeof(T)) = pack<T, VE>(hi);
                    }
                }
            }
        }
    }
    if constexpr (GRAD) {
        if (!a.part) return;
        // the groups of a warp, then the warps in order
#pragma unroll
        for (int v = 0; v < NV; v++) {
            float lo[VE], hi[VE];
#pragma unroll
            for (int i = 0; i < VE; i++)
                for (int o = lanes; o < 32; o <<= 1) {
                    da[v][i] += __shfl_xor_sync(0xffffffffu, da[v][i], o);
                    db[v][i] += __shfl_xor_sync(0xffffffffu, db[v][i], o);
                }
            from_pairs<VE, INTER>(da[v], db[v], lo, hi);
            if (group == 0 && k.on[v])
#pragma unroll
                for (int i = 0; i < VE; i++) {
                    sums[warp][k.lo[v] + i] = lo[i];
                    sums[warp][k.hi[v] + i] = hi[i];
                }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.D; c += kQkThreads) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kQkWarps; w++) s += sums[w][c];
            a.part[static_cast<long long>(blockIdx.x) * a.D + c] = s;
        }
    }
}

// dgamma of the queries (blockIdx.y 0) and keys: the CTAs' sums, 32 channels a
// block, each of its warps a row in eight, joined in order.
__global__ void __launch_bounds__(256) k_qk_params(const float *part, unsigned q_blocks, unsigned blocks, int D, float *dq,
                                                   float *dk)
{
    __shared__ float sh[8][32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    const unsigned from = blockIdx.y ? q_blocks : 0, to = blockIdx.y ? blocks : q_blocks;
    float s = 0.0f;
    if (c < D) {
#pragma unroll 8
        for (unsigned r = from + w; r < to; r += 8) s += part[static_cast<long long>(r) * D + c];
    }
    sh[w][lane] = s;
    __syncthreads();
    float *out = blockIdx.y ? dk : dq;
    if (w || c >= D || !out) return;
#pragma unroll
    for (int i = 1; i < 8; i++) s += sh[i][lane];
    out[c] = s;
}

// ------------------------------------------------------------------ host side

struct QkPlan {
    Shape x, y;
    size_t workspace;
};

int qk_check(const rz_qk *d, QkPlan *p)
{
    if (!d) return RZ_ERR_ARG;
    const size_t es = dtype_size(d->dtype);
    p->x = {d->N, d->H, d->W, d->C, es};
    p->y = {d->N, d->H, d->W, d->out_C, es};
    p->workspace = sizeof(float) * static_cast<size_t>(kQkBlocks) * kQkMaxD;
    if (!es || !shape_ok(p->x) || !shape_ok(p->y)) return RZ_ERR_ARG;
    if (d->q_heads < 0 || d->k_heads < 0 || d->q_heads > RZ_MAX_DIM || d->k_heads > RZ_MAX_DIM) return RZ_ERR_ARG;
    if (d->q_heads + d->k_heads < 1 || d->D < 2 || d->D > kQkMaxD || d->D % 2) return RZ_ERR_ARG;
    const long long c = static_cast<long long>(d->q_heads + d->k_heads) * d->D;
    if (c > d->C || c > d->out_C) return RZ_ERR_ARG;
    if (d->row_pairs < 0 || d->col_pairs < 0 || d->row_pairs > d->D / 2 || d->col_pairs > d->D / 2 - d->row_pairs)
        return RZ_ERR_ARG;
    if (!(d->eps >= 0.0f) || !(d->eps <= 3.0e38f) || !(d->base > 0.0) || !std::isfinite(d->base) || !std::isfinite(d->scale))
        return RZ_ERR_ARG;
    // tokens are numbered in 32 bits
    if (!p->x.empty() && static_cast<long long>(d->N) > 0x7fffffffLL / (p->x.H * p->x.W)) return RZ_ERR_UNSUPPORTED;
    return RZ_OK;
}

// Turns of a position step in 2^-64, whole turns left out.
unsigned long long turn_of(double base, double scale, int j, int pairs)
{
    const double f = scale * std::pow(base, -static_cast<double>(j) / pairs) * 0.15915494309189533577;
    if (!std::isfinite(f)) return 0;
    const double frac = f - std::floor(f);
    return frac < 1.0 ? static_cast<unsigned long long>(std::ldexp(frac, 64)) : 0ull;
}

template <class T, int VE, int NV, bool GRAD>
cudaError_t qk_launch(const QkArgs &a, bool inter, unsigned blocks, void *stream)
{
    constexpr int U = NV > 1 ? 1 : GRAD ? 2 : 4;
    const auto fn = inter ? k_qk_norm<T, VE, NV, true, GRAD, U> : k_qk_norm<T, VE, NV, false, GRAD, U>;
    return launch(fn, dim3(blocks), kQkThreads, 0, stream, a);
}

template <class T, bool GRAD>
cudaError_t qk_dispatch(QkArgs &a, const rz_qk *d, int ve, unsigned *total, void *stream)
{
    constexpr int W = 16 / sizeof(T);
    const int half = d->D / 2, vecs = half / ve;
    int lanes = 1;
    while (lanes < vecs && lanes < 32) lanes *= 2;
    a.lanes = lanes;
    const int u = ve == 1 ? 1 : GRAD ? 2 : 4, heads = a.q_heads + a.k_heads;
    // about two CTAs' worth of warps an SM before a token's heads stay in one warp
    a.chunks = 1;
    const int most = (std::max(a.q_heads, a.k_heads) * lanes + 32 * u - 1) / (32 * u);
    while (a.chunks < most && static_cast<long long>(a.tokens) * a.chunks < 2 * kQkSms * kQkWarps) a.chunks++;
    const unsigned long long need =
        (static_cast<unsigned long long>(a.tokens) * a.chunks + kQkWarps - 1) / kQkWarps;
    // CTAs are shared out by heads
    const auto share = [&](int h) {
        if (!h) return 0u;
        const unsigned long long s = std::max(1ull, static_cast<unsigned long long>(kQkBlocks - 1) * h / heads);
        return static_cast<unsigned>(std::min(need, s));
    };
    a.q_blocks = share(a.q_heads);
    const unsigned blocks = *total = a.q_blocks + share(a.k_heads);
    if (ve == W) return qk_launch<T, W, 1, GRAD>(a, d->interleaved != 0, blocks, stream);
    if (sizeof(T) == 2 && ve == 4) return qk_launch<T, 4, 1, GRAD>(a, d->interleaved != 0, blocks, stream);
    return qk_launch<T, 1, 4, GRAD>(a, d->interleaved != 0, blocks, stream);
}

template <bool GRAD>
int qk_run(const rz_qk *d, const QkPlan &p, const rz_map *x, const rz_map *dy, const rz_map *y, const float *gamma_q,
           const float *gamma_k, const int *positions, float *part, unsigned *q_blocks, unsigned *blocks, void *stream)
{
    QkArgs a{};
    a.x = view(x);
    a.y = view(y);
    const Shape &sy = GRAD ? p.x : p.y;
    const auto px = [](const Shape &s) { return static_cast<int>(s.C * s.es); };
    a.x_px = px(p.x);
    a.y_px = px(sy);
    a.x_joined = rows_joined(*x, p.x);
    a.y_joined = rows_joined(*y, sy);
    if (GRAD) {
        a.dy = view(dy);
        a.dy_px = px(p.y);
        a.dy_joined = rows_joined(*dy, p.y);
    }
    a.gq = gamma_q;
    a.gk = gamma_k;
    a.pos = positions;
    a.part = part;
    a.HW = static_cast<unsigned>(p.x.H * p.x.W);
    a.W = static_cast<unsigned>(p.x.W);
    a.tokens = static_cast<unsigned>(d->N) * a.HW;
    a.q_heads = d->q_heads;
    a.k_heads = d->k_heads;
    a.D = d->D;
    a.row_pairs = d->row_pairs;
    a.pairs = d->row_pairs + d->col_pairs;
    a.eps = d->eps;
    a.inv_d = 1.0f / static_cast<float>(d->D);
    for (int j = 0; j < a.pairs; j++)
        a.turn[j] = j < d->row_pairs ? turn_of(d->base, d->scale, j, d->row_pairs)
                                     : turn_of(d->base, d->scale, j - d->row_pairs, d->col_pairs);
    const auto fits = [&](int ve) {
        const size_t b = ve * p.x.es;
        return d->D / 2 % ve == 0 && a.x_px % b == 0 && a.y_px % b == 0 && map_aligned(*x, p.x, b) && map_aligned(*y, sy, b) &&
               (!GRAD || (a.dy_px % b == 0 && map_aligned(*dy, p.y, b)));
    };
    const int wide = 16 / static_cast<int>(p.x.es);
    const int ve = fits(wide) ? wide : p.x.es == 2 && fits(4) ? 4 : 1;
    cudaError_t e;
    if (d->dtype == RZ_F32)
        e = qk_dispatch<float, GRAD>(a, d, ve, blocks, stream);
    else if (d->dtype == RZ_BF16)
        e = qk_dispatch<__nv_bfloat16, GRAD>(a, d, ve, blocks, stream);
    else
        e = qk_dispatch<__half, GRAD>(a, d, ve, blocks, stream);
    *q_blocks = a.q_blocks;
    if (e != cudaSuccess) {
        record_cuda_error(static_cast<int>(e));
        return RZ_ERR_CUDA;
    }
    return RZ_OK;
}

bool floats_ok(const float *p) { return reinterpret_cast<uintptr_t>(p) % sizeof(float) == 0; }

}  // namespace
}  // namespace rz

using namespace rz;

extern "C" {

int map_qk_norm(const rz_qk *d, const rz_map *x, const rz_map *y, const float *gamma_q, const float *gamma_k,
                const int *positions, void *stream)
{
    QkPlan p;
    if (const int rc = qk_check(d, &p)) return rc;
    if (p.x.empty()) return RZ_OK;
    if (!maps::map_ok(x, p.x) || !maps::map_ok(y, p.y)) return RZ_ERR_ARG;
    if (!floats_ok(gamma_q) || !floats_ok(gamma_k) || reinterpret_cast<uintptr_t>(positions) % 8) return RZ_ERR_ARG;
    const bool same = d->C == d->out_C && maps::map_same(*x, *y, p.x);
    if (!same && maps::map_overlap(*x, p.x, *y, p.y)) return RZ_ERR_ARG;
    unsigned qb, b;
    return qk_run<false>(d, p, x, nullptr, y, gamma_q, gamma_k, positions, nullptr, &qb, &b, stream);
}

int map_qk_norm_grad_workspace(const rz_qk *d, size_t *bytes)
{
    QkPlan p;
    const int rc = bytes ? qk_check(d, &p) : RZ_ERR_ARG;
    if (rc) return rc;
    *bytes = p.x.empty() ? 0 : p.workspace;
    return RZ_OK;
}

int map_qk_norm_grad(const rz_qk *d, const rz_map *dy, const rz_map *x, const rz_map *dx, const float *gamma_q,
                     const float *gamma_k, const int *positions, float *dgamma_q, float *dgamma_k, void *workspace,
                     size_t workspace_bytes, void *stream)
{
    QkPlan p;
    if (const int rc = qk_check(d, &p)) return rc;
    if (!floats_ok(gamma_q) || !floats_ok(gamma_k) || !floats_ok(dgamma_q) || !floats_ok(dgamma_k)) return RZ_ERR_ARG;
    const bool sums = dgamma_q || dgamma_k;
    unsigned qb = 0, blocks = 0;
    if (!p.x.empty()) {
        if (!maps::map_ok(x, p.x) || !maps::map_ok(dy, p.y) || !maps::map_ok(dx, p.x)) return RZ_ERR_ARG;
        if (reinterpret_cast<uintptr_t>(positions) % 8) return RZ_ERR_ARG;
        const bool same = d->C == d->out_C && maps::map_same(*dy, *dx, p.x);
        if ((!same && maps::map_overlap(*dx, p.x, *dy, p.y)) || maps::map_overlap(*dx, p.x, *x, p.x)) return RZ_ERR_ARG;
        if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 || workspace_bytes < p.workspace) return RZ_ERR_ARG;
        const int rc = qk_run<true>(d, p, x, dy, dx, gamma_q, gamma_k, positions,
                                    sums ? static_cast<float *>(workspace) : nullptr, &qb, &blocks, stream);
        if (rc) return rc;
    }
    if (!sums) return RZ_OK;
    const dim3 grid((d->D + 31) / 32, 2);
    const cudaError_t e = maps::launch(k_qk_params, grid, 256, 0, stream, static_cast<const float *>(workspace), qb, blocks,
                                       d->D, dgamma_q, dgamma_k);
    if (e == cudaSuccess) return RZ_OK;
    record_cuda_error(static_cast<int>(e));
    return RZ_ERR_CUDA;
}

}  // extern "C"
