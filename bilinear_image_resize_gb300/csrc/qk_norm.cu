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
#include "token_rules.h"

namespace rz {
namespace {

using namespace maps;
using dev::grid_dependency_wait;
using dev::grid_launch_dependents;

constexpr int kQkSms = rules::kSms;
constexpr int kQkThreads = 256;
constexpr int kQkWarps = kQkThreads / 32;
constexpr int kQkMaxD = 256;
constexpr int kQkBlocks = 4 * kQkSms;   // most CTAs of a call, each of a gradient's with a row of partial sums

struct QkArgs {
    View x, y, dy;              // forward: x -> y; gradient: x, dy -> y
    const float *g[2];          // of queries and keys
    const int *pos;             // null: the pixel's place
    float *part;                // gradient: [blocks][2][D] partial sums, or null
    unsigned tokens, H, W;
    int x_px, y_px, dy_px;      // bytes of a pixel
    int q_heads, heads, D;
    int lanes;                  // lanes of a head's group
    int chunks, chunk;          // runs of heads a token is cut into, for calls of few tokens, and the heads of a run
    int row_pairs;
    float eps, inv_d;
    unsigned long long turn[kQkMaxD / 2];   // a position step's angle in 2^-64 turns
};

// Cosine and sine of position * turn: the product's low 64 bits are the angle
// modulo a turn, off by what the step is (2^-63 of a turn) for each position; its top
// 32 bits go on as a signed float.  16-bit results take the GPU's approximate
// functions, off by 2^-21.2 in [-pi, pi] (with the angle's rounding 7e-7).
template <class T>
__device__ __forceinline__ void turned(int p, unsigned long long turn, float &c, float &s)
{
    const unsigned long long f = static_cast<unsigned long long>(static_cast<long long>(p)) * turn;
    const float half_turns = static_cast<float>(static_cast<int>(f >> 32)) * 0x1p-31f;
    if constexpr (sizeof(T) == 4)
        sincospif(half_turns, &s, &c);
    else
        __sincosf(half_turns * 3.14159265f, &s, &c);
}

// A head's vectors as pairs' members, two pairs at a time.  VE: elements of a
// vector; INTER: pairs are neighbours.  Pair i of a lane is (lo[i], hi[i]), or, of
// neighbours, those inside lo and then those inside hi (VE 1: lo and hi are
// neighbours).
template <int VE, bool INTER>
__device__ __forceinline__ void to_pairs(const float (&lo)[VE], const float (&hi)[VE], float2 (&a)[kPairs<VE>], float2 (&b)[kPairs<VE>])
{
#pragma unroll
    for (int i = 0; i < kPairs<VE>; i++) {
        if constexpr (VE == 1) {
            a[i] = make_float2(lo[0], 0.0f);
            b[i] = make_float2(hi[0], 0.0f);
        } else if constexpr (INTER) {
            const float(&v)[VE] = i < VE / 4 ? lo : hi;
            const int k = 4 * i % VE;
            a[i] = make_float2(v[k], v[k + 2]);
            b[i] = make_float2(v[k + 1], v[k + 3]);
        } else {
            a[i] = make_float2(lo[2 * i], lo[2 * i + 1]);
            b[i] = make_float2(hi[2 * i], hi[2 * i + 1]);
        }
    }
}
template <int VE, bool INTER>
__device__ __forceinline__ void from_pairs(const float2 (&a)[kPairs<VE>], const float2 (&b)[kPairs<VE>], float (&lo)[VE], float (&hi)[VE])
{
#pragma unroll
    for (int i = 0; i < kPairs<VE>; i++) {
        if constexpr (VE == 1) {
            lo[0] = a[i].x;
            hi[0] = b[i].x;
        } else if constexpr (INTER) {
            float(&v)[VE] = i < VE / 4 ? lo : hi;
            const int k = 4 * i % VE;
            v[k] = a[i].x;
            v[k + 1] = b[i].x;
            v[k + 2] = a[i].y;
            v[k + 3] = b[i].y;
        } else {
            lo[2 * i] = a[i].x;
            lo[2 * i + 1] = a[i].y;
            hi[2 * i] = b[i].x;
            hi[2 * i + 1] = b[i].y;
        }
    }
}

template <class T, int VE, bool INTER>
__device__ __forceinline__ void pairs_of(const Raw<T, VE> &first, const Raw<T, VE> &second, float2 (&a)[kPairs<VE>],
                                         float2 (&b)[kPairs<VE>])
{
    float lo[VE], hi[VE];
    unpack<T, VE>(first, lo);
    unpack<T, VE>(second, hi);
    to_pairs<VE, INTER>(lo, hi, a, b);
}
template <class T, int VE, bool INTER>
__device__ __forceinline__ void write_pairs(uint8_t *first, uint8_t *second, const float2 (&a)[kPairs<VE>], const float2 (&b)[kPairs<VE>])
{
    float lo[VE], hi[VE];
    from_pairs<VE, INTER>(a, b, lo, hi);
    *reinterpret_cast<Raw<T, VE> *>(first) = pack<T, VE>(lo);
    *reinterpret_cast<Raw<T, VE> *>(second) = pack<T, VE>(hi);
}

// What a lane has of every head: vector v of its first half begins at channel
// lo(v), the matching one of the second half at hi(v).
template <int VE, bool INTER>
struct QkLane {
    int sub, lanes, half;
    __device__ __forceinline__ int idx(int v) const { return sub + v * lanes; }
    __device__ __forceinline__ bool on(int v) const { return idx(v) * VE < half; }
    __device__ __forceinline__ int lo(int v) const { return INTER && VE == 1 ? 2 * idx(v) : idx(v) * VE; }
    __device__ __forceinline__ int hi(int v) const { return INTER && VE == 1 ? 2 * idx(v) + 1 : half + idx(v) * VE; }
    // The lane's entries of a table with one for each pair: those of VE pairs in a
    // row, or, of neighbours, of half as many inside each vector.
    __device__ __forceinline__ void pairs(const float *t, int v, float2 (&out)[kPairs<VE>]) const
    {
        if constexpr (VE == 1) {
            out[0] = make_float2(t[idx(v)], 0.0f);
        } else {
#pragma unroll
            for (int i = 0; i < VE / 2; i += 2) {
                const int at = !INTER ? idx(v) * VE + 2 * i : i < VE / 4 ? idx(v) * VE / 2 + 2 * i : (half + idx(v) * VE) / 2 + 2 * i - VE / 2;
                if constexpr (VE == 4 && INTER) {
                    const int second = (half + idx(v) * VE) / 2;
                    out[0] = *reinterpret_cast<const float2 *>(t + idx(v) * VE / 2);
                    out[1] = *reinterpret_cast<const float2 *>(t + second);
                } else {
                    const float4 q = *reinterpret_cast<const float4 *>(t + at);
                    out[i] = make_float2(q.x, q.y);
                    out[i + 1] = make_float2(q.z, q.w);
                }
            }
        }
    }
};

__device__ __forceinline__ float group_sum(float v, int lanes)
{
    for (int o = lanes >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Tables of a token, an entry for each pair.  Forward, for queries and keys each,
// gamma and the turn as one: cos ga, -sin gb, sin ga, cos gb.  Gradient: cos, sin,
// -sin.  Gamma by pairs' members, [part][member], follows the tables.
constexpr int kQkTables = 8, kQkGradTables = 3;
__host__ __device__ constexpr int qk_row(int half) { return (half + 3) / 4 * 4; }

template <bool INTER>
__device__ __forceinline__ void gammas_by_member(const QkArgs &a, float *to, int half, int row)
{
    for (int i = threadIdx.x; i < 4 * half; i += kQkThreads) {
        const int j = i % half, member = i / half % 2;
        const float *g = a.g[i / (2 * half)];
        to[(i / half) * row + j] = g ? g[INTER ? 2 * j + member : j + member * half] : 1.0f;
    }
}

// A walk over a warp's items: tokens, or runs of the heads of few tokens.
struct QkWalk {
    unsigned long long item, items;
    unsigned step, n, h, w, dn, dh, dw;
    int h0, h1;

    __device__ __forceinline__ void begin(const QkArgs &a)
    {
        items = static_cast<unsigned long long>(a.tokens) * a.chunks;
        step = gridDim.x * kQkWarps;
        place(a, step);
        dn = n, dh = h, dw = w;
        item = static_cast<unsigned long long>(blockIdx.x) * kQkWarps + (threadIdx.x >> 5);
        h0 = 0;
        h1 = a.heads;
        if (live()) find(a);
    }
    __device__ __forceinline__ bool live() const { return item < items; }
    __device__ __forceinline__ void place(const QkArgs &a, unsigned t)
    {
        const unsigned r = t / a.W;
        w = t - r * a.W;
        n = r / a.H;
        h = r - n * a.H;
    }
    __device__ __forceinline__ unsigned token(const QkArgs &a) const { return static_cast<unsigned>(a.chunks == 1 ? item : item / a.chunks); }
    __device__ __forceinline__ void find(const QkArgs &a)
    {
        const unsigned t = token(a);
        place(a, t);
        if (a.chunks > 1) {
            h0 = static_cast<int>(item - static_cast<unsigned long long>(t) * a.chunks) * a.chunk;
            h1 = min(a.heads, h0 + a.chunk);
        }
    }
    __device__ __forceinline__ void next(const QkArgs &a)
    {
        item += step;
        if (a.chunks > 1) {
            if (live()) find(a);
            return;
        }
        w += dw;
        h += dh + (w >= a.W ? 1 : 0);
        if (w >= a.W) w -= a.W;
        n += dn + (h >= a.H ? 1 : 0);
        if (h >= a.H) h -= a.H;
    }
    __device__ __forceinline__ uint8_t *at(const View &m, int px) const
    {
        return m.p + n * m.bstride + h * m.pitch + static_cast<long long>(w) * px;
    }
    __device__ __forceinline__ int2 position(const QkArgs &a) const
    {
        if (a.pos) return __ldg(reinterpret_cast<const int2 *>(a.pos) + token(a));
        return make_int2(static_cast<int>(h), static_cast<int>(w));
    }
};

// A warp takes a token (or a run of the heads of few tokens) at a time: while its
// first vectors are on their way it works out the token's turns, once for all of
// its heads, into shared memory of its own.  U: groups' vectors read before the
// first is used.  12 x 64 x 64 tokens of 40 heads of 64, bf16: 86 us, 5.9 TB/s (109
// with the turns worked out by every group of lanes for itself).
template <class T, int VE, int NV, bool INTER, int U>
__global__ void __launch_bounds__(kQkThreads, NV == 1 ? 4 : 1) k_qk_norm(const __grid_constant__ QkArgs a)
{
    using V = Raw<T, VE>;
    constexpr int P = kPairs<VE>;
    extern __shared__ float4 shared[];
    __shared__ unsigned long long turn[kQkMaxD / 2];
    grid_launch_dependents();
    const int half = a.D / 2, row = qk_row(half);
    for (int i = threadIdx.x; i < half; i += kQkThreads) turn[i] = a.turn[i];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lanes = a.lanes, at_once = 32 / lanes, group = lane / lanes;
    const QkLane<VE, INTER> k{lane & (lanes - 1), lanes, half};
    float *tables = reinterpret_cast<float *>(shared) + warp * kQkTables * row;
    float *gammas = reinterpret_cast<float *>(shared) + kQkWarps * kQkTables * row;
    grid_dependency_wait();
    gammas_by_member<INTER>(a, gammas, half, row);
    __syncthreads();
    QkWalk it;
    for (it.begin(a); it.live(); it.next(a)) {
        const int h0 = it.h0, h1 = it.h1;
        const uint8_t *xt = it.at(a.x, a.x_px);
        uint8_t *yt = it.at(a.y, a.y_px);
        V x[U][NV][2];
        const auto read = [&](int from) {
#pragma unroll
            for (int u = 0; u < U; u++)
#pragma unroll
                for (int v = 0; v < NV; v++) {
                    const int hd = from + u * at_once + group;
                    if (hd < h1 && k.on(v)) {
                        x[u][v][0] = __ldcs(reinterpret_cast<const V *>(xt + (hd * a.D + k.lo(v)) * static_cast<int>(sizeof(T))));
                        x[u][v][1] = __ldcs(reinterpret_cast<const V *>(xt + (hd * a.D + k.hi(v)) * static_cast<int>(sizeof(T))));
                    } else {
                        x[u][v][0] = x[u][v][1] = V{};
                    }
                }
        };
        read(h0);
        // the turns, under the vectors' flight
        const int2 p = it.position(a);
        __syncwarp();
        for (int j = lane; j < half; j += 32) {
            float c, s;
            turned<T>(j < a.row_pairs ? p.x : p.y, turn[j], c, s);
#pragma unroll
            for (int part = 0; part < 2; part++) {
                const float ga = gammas[2 * part * row + j], gb = gammas[(2 * part + 1) * row + j];
                float *to = tables + part * 4 * row + j;
                to[0] = c * ga;
                to[row] = -s * gb;
                to[2 * row] = s * ga;
                to[3 * row] = c * gb;
            }
        }
        __syncwarp();
        for (int from = h0; from < h1; from += U * at_once) {
            if (from != h0) read(from);
#pragma unroll
            for (int u = 0; u < U; u++) {
                if (from + u * at_once >= h1) break;    // the same for the whole warp
                const int hd = from + u * at_once + group;
                float2 xa[NV][P], xb[NV][P], s = both(0.0f);
#pragma unroll
                for (int v = 0; v < NV; v++) {
                    pairs_of<T, VE, INTER>(x[u][v][0], x[u][v][1], xa[v], xb[v]);
#pragma unroll
                    for (int i = 0; i < P; i++) s = __ffma2_rn(xa[v][i], xa[v][i], __ffma2_rn(xb[v][i], xb[v][i], s));
                }
                const float r = rsqrtf(fmaf(group_sum(s.x + s.y, lanes), a.inv_d, a.eps));
                const float *tab = tables + (hd < a.q_heads ? 0 : 4 * row);
#pragma unroll
                for (int v = 0; v < NV; v++) {
                    if (hd >= h1 || !k.on(v)) continue;
                    float2 t[P], oa[P], ob[P];
                    k.pairs(tab, v, t);
#pragma unroll
                    for (int i = 0; i < P; i++) oa[i] = __fmul2_rn(xa[v][i], t[i]);
                    k.pairs(tab + row, v, t);
#pragma unroll
                    for (int i = 0; i < P; i++) oa[i] = __fmul2_rn(__ffma2_rn(xb[v][i], t[i], oa[i]), both(r));
                    k.pairs(tab + 2 * row, v, t);
#pragma unroll
                    for (int i = 0; i < P; i++) ob[i] = __fmul2_rn(xa[v][i], t[i]);
                    k.pairs(tab + 3 * row, v, t);
#pragma unroll
                    for (int i = 0; i < P; i++) ob[i] = __fmul2_rn(__ffma2_rn(xb[v][i], t[i], ob[i]), both(r));
                    write_pairs<T, VE, INTER>(yt + (hd * a.D + k.lo(v)) * static_cast<int>(sizeof(T)),
                                              yt + (hd * a.D + k.hi(v)) * static_cast<int>(sizeof(T)), oa, ob);
                }
            }
        }
    }
}

// The gradient: the same walk, a step of a warp being one group of heads of one
// kind.  (Every item has a step: two walks count the places, one as it fills them
// and one as it uses them.)  A step's vectors are copied into places in shared memory that only their
// lane reads, kQkAhead steps before they are used, across tokens: in registers the
// four vectors of two steps left 16 warps an SM waiting a memory's latency for
// each (16 x 37 x 50 tokens of 20 heads of 128, f16: 106 us; so 85 us, 5.3 TB/s).
constexpr int kQkAhead = 3;

template <class T, int VE, int NV, bool INTER>
__global__ void __launch_bounds__(kQkThreads, NV == 1 ? 2 : 1) k_qk_grad(const __grid_constant__ QkArgs a)
{
    using V = Raw<T, VE>;
    constexpr int P = kPairs<VE>, kPlaces = kQkAhead + 1;
    extern __shared__ float4 shared[];
    __shared__ unsigned long long turn[kQkMaxD / 2];
    grid_launch_dependents();
    const int half = a.D / 2, row = qk_row(half);
    for (int i = threadIdx.x; i < half; i += kQkThreads) turn[i] = a.turn[i];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lanes = a.lanes, at_once = 32 / lanes, group = lane / lanes;
    const QkLane<VE, INTER> k{lane & (lanes - 1), lanes, half};
    float *tables = reinterpret_cast<float *>(shared) + warp * kQkGradTables * row;
    float *gammas = reinterpret_cast<float *>(shared) + kQkWarps * kQkGradTables * row;
    // [warp][place][vector of x lo, x hi, dy lo, dy hi][lane]
    V *places = reinterpret_cast<V *>(gammas + 4 * row) + warp * kPlaces * NV * 4 * 32 + lane;
    grid_dependency_wait();
    gammas_by_member<INTER>(a, gammas, half, row);
    __syncthreads();
    float2 da[2][NV][P], db[2][NV][P];
#pragma unroll
    for (int part = 0; part < 2; part++)
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int i = 0; i < P; i++) da[part][v][i] = db[part][v][i] = both(0.0f);

    // the steps to copy run ahead of those to use
    QkWalk it, ahead;
    it.begin(a);
    ahead.begin(a);
    int next_from = ahead.h0, place = 0, filled = 0;
    const auto end_of = [&](const QkWalk &w, int from) { return from < a.q_heads ? min(w.h1, a.q_heads) : w.h1; };
    const auto copy = [&] {
        if (ahead.live()) {
            const int to = end_of(ahead, next_from), hd = next_from + group;
            const uint8_t *xt = ahead.at(a.x, a.x_px), *dt = ahead.at(a.dy, a.dy_px);
#pragma unroll
            for (int v = 0; v < NV; v++)
                if (hd < to && k.on(v)) {
                    V *p = places + (filled * NV + v) * 4 * 32;
                    const int lo = (hd * a.D + k.lo(v)) * static_cast<int>(sizeof(T)), hi = (hd * a.D + k.hi(v)) * static_cast<int>(sizeof(T));
                    copy_async(p, reinterpret_cast<const V *>(xt + lo));
                    copy_async(p + 32, reinterpret_cast<const V *>(xt + hi));
                    copy_async(p + 64, reinterpret_cast<const V *>(dt + lo));
                    copy_async(p + 96, reinterpret_cast<const V *>(dt + hi));
                }
            next_from = min(next_from + at_once, to);
            if (next_from >= ahead.h1) {
                ahead.next(a);
                next_from = ahead.h0;
            }
        }
        copies_commit();
        filled = filled + 1 == kPlaces ? 0 : filled + 1;
    };
    for (int i = 0; i < kQkAhead; i++) copy();
    for (; it.live(); it.next(a)) {
        uint8_t *yt = it.at(a.y, a.y_px);
        const int2 p = it.position(a);
        __syncwarp();
        for (int j = lane; j < half; j += 32) {
            float c, s;
            turned<T>(j < a.row_pairs ? p.x : p.y, turn[j], c, s);
            tables[j] = c;
            tables[row + j] = s;
            tables[2 * row + j] = -s;
        }
        __syncwarp();
#pragma unroll
        for (int part = 0; part < 2; part++) {
            const int p0 = part ? max(it.h0, a.q_heads) : it.h0, p1 = part ? it.h1 : min(it.h1, a.q_heads);
            for (int from = p0; from < p1; from += at_once) {
                copy();
                copies_left<kQkAhead>();
                const int hd = from + group;
                float2 xa[NV][P], xb[NV][P], wa[NV][P], wb[NV][P], s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
                for (int v = 0; v < NV; v++) {
#pragma unroll
                    for (int i = 0; i < P; i++) xa[v][i] = xb[v][i] = wa[v][i] = wb[v][i] = both(0.0f);
                    if (hd >= p1 || !k.on(v)) continue;
                    const V *at = places + (place * NV + v) * 4 * 32;
                    float2 ya[P], yb[P], t[P];
                    pairs_of<T, VE, INTER>(at[0], at[32], xa[v], xb[v]);
                    pairs_of<T, VE, INTER>(at[64], at[96], ya, yb);
#pragma unroll
                    for (int i = 0; i < P; i++) s1 = __ffma2_rn(xa[v][i], xa[v][i], __ffma2_rn(xb[v][i], xb[v][i], s1));
                    // turned back
                    k.pairs(tables, v, t);
#pragma unroll
                    for (int i = 0; i < P; i++) {
                        wa[v][i] = __fmul2_rn(ya[i], t[i]);
                        wb[v][i] = __fmul2_rn(yb[i], t[i]);
                    }
                    k.pairs(tables + row, v, t);
#pragma unroll
                    for (int i = 0; i < P; i++) wa[v][i] = __ffma2_rn(yb[i], t[i], wa[v][i]);
                    k.pairs(tables + 2 * row, v, t);
#pragma unroll
                    for (int i = 0; i < P; i++) wb[v][i] = __ffma2_rn(ya[i], t[i], wb[v][i]);
                    // dgamma's terms lack r: wa xa, wb xb, which times gamma are those of the other sum
                    k.pairs(gammas + 2 * part * row, v, t);
#pragma unroll
                    for (int i = 0; i < P; i++) s2 = __ffma2_rn(__fmul2_rn(wa[v][i], xa[v][i]), t[i], s2);
                    k.pairs(gammas + (2 * part + 1) * row, v, t);
#pragma unroll
                    for (int i = 0; i < P; i++) s2 = __ffma2_rn(__fmul2_rn(wb[v][i], xb[v][i]), t[i], s2);
                }
                place = place + 1 == kPlaces ? 0 : place + 1;
                const float sum1 = group_sum(s1.x + s1.y, lanes), sum2 = group_sum(s2.x + s2.y, lanes);
                const float r = rsqrtf(fmaf(sum1, a.inv_d, a.eps)), m = sum2 * a.inv_d * r * r * r;    // r^3 alone may pass the range
#pragma unroll
                for (int v = 0; v < NV; v++) {
                    // r of a group without a head is not finite for eps 0
                    if (hd >= p1 || !k.on(v)) continue;
                    float2 t[P];
                    k.pairs(gammas + 2 * part * row, v, t);
#pragma unroll
                    for (int i = 0; i < P; i++) {
                        const float2 wr = __fmul2_rn(wa[v][i], both(r));
                        da[part][v][i] = __ffma2_rn(wr, xa[v][i], da[part][v][i]);
                        wa[v][i] = __ffma2_rn(wr, t[i], __fmul2_rn(xa[v][i], both(-m)));
                    }
                    k.pairs(gammas + (2 * part + 1) * row, v, t);
#pragma unroll
                    for (int i = 0; i < P; i++) {
                        const float2 wr = __fmul2_rn(wb[v][i], both(r));
                        db[part][v][i] = __ffma2_rn(wr, xb[v][i], db[part][v][i]);
                        wb[v][i] = __ffma2_rn(wr, t[i], __fmul2_rn(xb[v][i], both(-m)));
                    }
                    write_pairs<T, VE, INTER>(yt + (hd * a.D + k.lo(v)) * static_cast<int>(sizeof(T)),
                                              yt + (hd * a.D + k.hi(v)) * static_cast<int>(sizeof(T)), wa[v], wb[v]);
                }
            }
        }
    }
    copies_left<0>();
    if (!a.part) return;
    // the groups of a warp, then the warps in order
    __syncthreads();
    float *sums = reinterpret_cast<float *>(shared);    // [warp][D]
#pragma unroll
    for (int part = 0; part < 2; part++) {
#pragma unroll
        for (int v = 0; v < NV; v++) {
            float lo[VE], hi[VE];
#pragma unroll
            for (int i = 0; i < P; i++)
                for (int o = lanes; o < 32; o <<= 1) {
                    float2 &pa = da[part][v][i], &pb = db[part][v][i];
                    pa = __fadd2_rn(pa, make_float2(__shfl_xor_sync(0xffffffffu, pa.x, o), __shfl_xor_sync(0xffffffffu, pa.y, o)));
                    pb = __fadd2_rn(pb, make_float2(__shfl_xor_sync(0xffffffffu, pb.x, o), __shfl_xor_sync(0xffffffffu, pb.y, o)));
                }
            from_pairs<VE, INTER>(da[part][v], db[part][v], lo, hi);
            if (group == 0 && k.on(v))
#pragma unroll
                for (int i = 0; i < VE; i++) {
                    sums[warp * a.D + k.lo(v) + i] = lo[i];
                    sums[warp * a.D + k.hi(v) + i] = hi[i];
                }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.D; c += kQkThreads) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < kQkWarps; i++) s += sums[i * a.D + c];
            a.part[(static_cast<long long>(blockIdx.x) * 2 + part) * a.D + c] = s;
        }
        __syncthreads();
    }
}

// dgamma of the queries (blockIdx.y 0) and keys: the CTAs' sums, 32 channels a
// block, each of its warps a row in eight, joined in order.
__global__ void __launch_bounds__(256) k_qk_params(const float *part, unsigned blocks, int D, float *dq, float *dk)
{
    __shared__ float sh[8][32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < D) {
        const float *from = part + static_cast<long long>(blockIdx.y) * D + c;
#pragma unroll 16
        for (unsigned r = w; r < blocks; r += 8) s += from[static_cast<long long>(r) * 2 * D];
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
    if (!es || !shape_ok(p->x) || !shape_ok(p->y)) return RZ_ERR_ARG;
    if (d->q_heads < 0 || d->k_heads < 0 || d->q_heads > RZ_MAX_DIM || d->k_heads > RZ_MAX_DIM) return RZ_ERR_ARG;
    if (d->q_heads + d->k_heads < 1 || d->D < 2 || d->D > kQkMaxD || d->D % 2) return RZ_ERR_ARG;
    const long long c = static_cast<long long>(d->q_heads + d->k_heads) * d->D;
    if (c > d->C || c > d->out_C) return RZ_ERR_ARG;
    if (d->row_pairs < 0 || d->col_pairs < 0 || d->row_pairs > d->D / 2 || d->col_pairs > d->D / 2 - d->row_pairs)
        return RZ_ERR_ARG;
    if (!(d->eps >= 0.0f) || !(d->eps <= 3.0e38f) || !(d->base > 0.0) || !std::isfinite(d->base) || !std::isfinite(d->scale))
        return RZ_ERR_ARG;
    p->workspace = sizeof(float) * 2 * static_cast<size_t>(kQkBlocks) * d->D;
    // tokens are numbered in 32 bits
    if (!p->x.empty() && static_cast<long long>(d->N) > 0x7fffffffLL / (p->x.H * p->x.W)) return RZ_ERR_UNSUPPORTED;
    return RZ_OK;
}

template <class T, int VE, int NV, bool GRAD>
cudaError_t qk_launch(const QkArgs &a, bool inter, unsigned blocks, void *stream)
{
    const size_t row = sizeof(float) * qk_row(a.D / 2);
    if constexpr (GRAD) {
        const auto fn = inter ? k_qk_grad<T, VE, NV, true> : k_qk_grad<T, VE, NV, false>;
        const size_t smem = row * (kQkWarps * kQkGradTables + 4) + kQkWarps * (kQkAhead + 1) * NV * 4 * 32 * sizeof(Raw<T, VE>);
        if (const cudaError_t e = shared_opt_in(reinterpret_cast<const void *>(fn))) return e;
        return launch(fn, dim3(blocks), kQkThreads, std::max(smem, sizeof(float) * kQkWarps * a.D), stream, a);
    } else {
        constexpr int U = NV > 1 ? 1 : 2;
        const auto fn = inter ? k_qk_norm<T, VE, NV, true, U> : k_qk_norm<T, VE, NV, false, U>;
        return launch(fn, dim3(blocks), kQkThreads, row * (kQkWarps * kQkTables + 4), stream, a);
    }
}

template <class T, bool GRAD>
cudaError_t qk_dispatch(QkArgs &a, const rz_qk *d, int ve, unsigned *blocks, void *stream)
{
    constexpr int W = 16 / sizeof(T);
    const int vecs = (d->D / 2 + ve - 1) / ve;
    int lanes = 1;
    while (lanes < vecs && lanes < 32) lanes *= 2;
    a.lanes = lanes;
    const rules::Runs runs = rules::head_runs(a.heads, lanes, a.tokens, kQkWarps);
    a.chunks = runs.chunks;
    a.chunk = runs.chunk;
    const unsigned long long need = (static_cast<unsigned long long>(a.tokens) * a.chunks + kQkWarps - 1) / kQkWarps;
    *blocks = static_cast<unsigned>(std::min<unsigned long long>(need, GRAD ? 2 * kQkSms : kQkBlocks));
    const bool inter = d->interleaved != 0;
    if (ve == W) return qk_launch<T, W, 1, GRAD>(a, inter, *blocks, stream);
    if (sizeof(T) == 2 && ve == 4) return qk_launch<T, 4, 1, GRAD>(a, inter, *blocks, stream);
    return qk_launch<T, 1, 4, GRAD>(a, inter, *blocks, stream);
}

template <bool GRAD>
int qk_run(const rz_qk *d, const QkPlan &p, const rz_map *x, const rz_map *dy, const rz_map *y, const float *gamma_q,
           const float *gamma_k, const int *positions, float *part, unsigned *blocks, void *stream)
{
    QkArgs a{};
    a.x = view(x);
    a.y = view(y);
    const Shape &sy = GRAD ? p.x : p.y;
    const auto px = [](const Shape &s) { return static_cast<int>(s.C * s.es); };
    a.x_px = px(p.x);
    a.y_px = px(sy);
    if (GRAD) {
        a.dy = view(dy);
        a.dy_px = px(p.y);
    }
    a.g[0] = gamma_q;
    a.g[1] = gamma_k;
    a.pos = positions;
    a.part = part;
    a.H = static_cast<unsigned>(p.x.H);
    a.W = static_cast<unsigned>(p.x.W);
    a.tokens = static_cast<unsigned>(d->N) * a.H * a.W;
    a.q_heads = d->q_heads;
    a.heads = d->q_heads + d->k_heads;
    a.D = d->D;
    a.row_pairs = d->row_pairs;
    a.eps = d->eps;
    a.inv_d = 1.0f / static_cast<float>(d->D);
    rules::turns_of(d->base, d->scale, d->row_pairs, a.turn);
    rules::turns_of(d->base, d->scale, d->col_pairs, a.turn + d->row_pairs);
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
    unsigned blocks;
    return qk_run<false>(d, p, x, nullptr, y, gamma_q, gamma_k, positions, nullptr, &blocks, stream);
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
    unsigned blocks = 0;
    if (!p.x.empty()) {
        if (!maps::map_ok(x, p.x) || !maps::map_ok(dy, p.y) || !maps::map_ok(dx, p.x)) return RZ_ERR_ARG;
        if (reinterpret_cast<uintptr_t>(positions) % 8) return RZ_ERR_ARG;
        const bool same = d->C == d->out_C && maps::map_same(*dy, *dx, p.x);
        if ((!same && maps::map_overlap(*dx, p.x, *dy, p.y)) || maps::map_overlap(*dx, p.x, *x, p.x)) return RZ_ERR_ARG;
        if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 || workspace_bytes < p.workspace) return RZ_ERR_ARG;
        const int rc = qk_run<true>(d, p, x, dy, dx, gamma_q, gamma_k, positions,
                                    sums ? static_cast<float *>(workspace) : nullptr, &blocks, stream);
        if (rc) return rc;
    }
    if (!sums) return RZ_OK;
    const dim3 grid((d->D + 31) / 32, 2);
    const cudaError_t e = maps::launch(k_qk_params, grid, 256, 0, stream, static_cast<const float *>(workspace), blocks, d->D,
                                       dgamma_q, dgamma_k);
    if (e == cudaSuccess) return RZ_OK;
    record_cuda_error(static_cast<int>(e));
    return RZ_ERR_CUDA;
}

}  // extern "C"
