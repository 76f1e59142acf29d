// Group norm with an activation and dropout on channels-last maps, and its
// gradient.  For image n and group g of Cg = C / G channels, M = H W Cg values:
//   mean = sum x / M,  var = sum (x - mean)^2 / M,  rstd = (var + eps)^-1/2
//   xh = (x - mean) rstd,  z = xh gamma_c + beta_c,  y = drop(act(z))
// and, with da = drop(dy) under the same mask and dz = da act'(z),
//   dbeta_c = sum dz,  dgamma_c = sum dz xh  (over images and pixels)
//   A = sum gamma dz / M,  B = sum gamma dz xh / M  (over the group)
//   dx = rstd (gamma dz - A - xh B).
//
// Memory bounds both.  A thread keeps one vector of channels and walks
// pixels, so that sums are taken per channel whatever the group's width, and
// groups are put together from channels afterwards.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "map_ops.h"
#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {

using namespace maps;
using dev::grid_dependency_wait;
using dev::grid_launch_dependents;

constexpr int kGnThreads = 256;
constexpr int kGnRows = 8;      // pixels a thread loads before it uses the first

struct GnArgs {
    View x, dy, y;              // y: the output (dx for the gradient)
    const float *gamma, *beta;  // may be null (1 and 0)
    float *mean, *rstd;         // [N][G]
    float *dgamma, *dbeta;      // [C], may be null
    int N, C, G, Cg;
    unsigned HW, W;             // pixels an image and a row
    int joined;                 // rows follow one another in every map
    int act;
    float eps, inv_m;
    Drop drop;
    float2 *part;               // [N][chunks][C]: a chunk's {mean, sum (x - mean)^2}, or {sum dz, sum dz xh}
    float2 *chan;               // [N][C]: {sum dz, sum dz xh}
    float2 *grp;                // [N][G]: {A, B}
    unsigned chunk_px;
    int chunks;
};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the block, for every thread; `scratch` holds 32 floats.
__device__ __forceinline__ float block_sum(float v, float *scratch)
{
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (unsigned i = 0; i < blockDim.x / 32; i++) s += scratch[i];
    return s;
}

// The thread's place: `c` the first channel of its vector, number `vec` of the
// block's `width`; `lane` its pixel lane of `lanes`.
struct Place {
    int c, lane, lanes, vec, width;
    bool on;
};

template <int VE>
__device__ __forceinline__ Place place(const GnArgs &a)
{
    const int all = a.C / VE, first = blockIdx.y * kGnThreads;
    const int width = min(all - first, kGnThreads);
    const int lanes = kGnThreads / width, lane = threadIdx.x / width, vec = threadIdx.x - lane * width;
    return {(first + vec) * VE, lane, lanes, vec, width, lane < lanes};
}

template <class T, int VE>
__device__ __forceinline__ const Raw<T, VE> *at(const View &v, const GnArgs &a, unsigned px, int n, int c)
{
    return reinterpret_cast<const Raw<T, VE> *>(
        v.p + n * v.bstride + pixel_off(px, a.W, a.joined, v.pitch, a.C * static_cast<int>(sizeof(T))) +
        c * static_cast<int>(sizeof(T)));
}

// One chunk's mean and sum of squared distances for every channel.  A thread
// takes kGnRows pixels at a time: their mean, their squared distances from
// it, and the two joined to what it holds (the pairwise update of Chan, Golub
// and LeVeque, "Updating formulae and a pairwise algorithm for computing
// sample variances"), so that nothing cancels where the mean is far above the
// deviation.
template <class T, int VE>
__global__ void __launch_bounds__(kGnThreads) k_gn_stats(const GnArgs a)
{
    __shared__ float2 sh[kGnThreads * VE];
    __shared__ int count[kGnThreads];
    grid_launch_dependents();
    grid_dependency_wait();
    const Place t = place<VE>(a);
    const int n = blockIdx.z;
    const unsigned p0 = blockIdx.x * a.chunk_px, p1 = min(a.HW, p0 + a.chunk_px);
    float mean[VE], m2[VE];
#pragma unroll
    for (int i = 0; i < VE; i++) mean[i] = m2[i] = 0.0f;
    int have = 0;
    if (t.on) {
        for (unsigned p = p0 + t.lane; p < p1; p += t.lanes * kGnRows) {
            const int rows = min(kGnRows, static_cast<int>((p1 - p + t.lanes - 1) / t.lanes));
            Raw<T, VE> r[kGnRows];
#pragma unroll
            for (int j = 0; j < kGnRows; j++)
                if (j < rows) r[j] = *at<T, VE>(a.x, a, p + j * t.lanes, n, t.c);
            float m[VE], q[VE];
#pragma unroll
            for (int i = 0; i < VE; i++) m[i] = q[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < kGnRows; j++)
                if (j < rows) {
                    float f[VE];
                    unpack<T, VE>(r[j], f);
#pragma unroll
                    for (int i = 0; i < VE; i++) m[i] += f[i];
                }
            const float inv = 1.0f / rows;
#pragma unroll
            for (int i = 0; i < VE; i++) m[i] *= inv;
#pragma unroll
            for (int j = 0; j < kGnRows; j++)
                if (j < rows) {
                    float f[VE];
                    unpack<T, VE>(r[j], f);
#pragma unroll
                    for (int i = 0; i < VE; i++) q[i] = fmaf(f[i] - m[i], f[i] - m[i], q[i]);
                }
            have += rows;
            const float share = static_cast<float>(rows) / have, weight = share * (have - rows);
#pragma unroll
            for (int i = 0; i < VE; i++) {
                const float d = m[i] - mean[i];
                mean[i] = fmaf(d, share, mean[i]);
                m2[i] += fmaf(d * d, weight, q[i]);
            }
        }
    }
    // join the pixel lanes, a thread to a channel
    if (t.on) {
#pragma unroll
        for (int i = 0; i < VE; i++) sh[(t.lane * t.width + t.vec) * VE + i] = make_float2(mean[i], m2[i]);
        if (t.vec == 0) count[t.lane] = have;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < t.width * VE; c += kGnThreads) {
        float s = 0.0f;
        for (int l = 0; l < t.lanes; l++) s = fmaf(sh[l * t.width * VE + c].x, static_cast<float>(count[l]), s);
        const float m = s / (p1 - p0);
        float q = 0.0f;
        for (int l = 0; l < t.lanes; l++) {
            const float2 v = sh[l * t.width * VE + c];
            q += fmaf((v.x - m) * (v.x - m), static_cast<float>(count[l]), v.y);
        }
        a.part[(static_cast<long long>(n) * a.chunks + blockIdx.x) * a.C + blockIdx.y * kGnThreads * VE + c] =
            make_float2(m, q);
    }
}

// A group's mean and 1 / deviation from its chunks' and channels' values.
__global__ void __launch_bounds__(128) k_gn_finish(const GnArgs a)
{
    __shared__ float scratch[32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int g = blockIdx.x, n = blockIdx.y;
    const float2 *part = a.part + static_cast<long long>(n) * a.chunks * a.C + g * a.Cg;
    const int items = a.chunks * a.Cg;
    float s = 0.0f;
    for (int i = threadIdx.x; i < items; i += 128) {
        const int k = i / a.Cg;
        s = fmaf(part[static_cast<long long>(k) * a.C + (i - k * a.Cg)].x,
                 static_cast<float>(min(a.chunk_px, a.HW - k * a.chunk_px)), s);
    }
    const float mean = block_sum(s, scratch) * a.inv_m;
    float q = 0.0f;
    for (int i = threadIdx.x; i < items; i += 128) {
        const int k = i / a.Cg;
        const float2 v = part[static_cast<long long>(k) * a.C + (i - k * a.Cg)];
        q += fmaf((v.x - mean) * (v.x - mean), static_cast<float>(min(a.chunk_px, a.HW - k * a.chunk_px)), v.y);
    }
    q = block_sum(q, scratch);
    if (threadIdx.x == 0) {
        a.mean[n * a.G + g] = mean;
        a.rstd[n * a.G + g] = 1.0f / sqrtf(fmaf(q, a.inv_m, a.eps));
    }
}

// What a vector's channels are normalised with.
template <int VE>
struct Channel {
    float mean[VE], rstd[VE], gamma[VE], beta[VE];
    __device__ __forceinline__ void load(const GnArgs &a, int n, int c)
    {
#pragma unroll
        for (int i = 0; i < VE; i++) {
            const int g = (c + i) / a.Cg;
            mean[i] = a.mean[n * a.G + g];
            rstd[i] = a.rstd[n * a.G + g];
            gamma[i] = a.gamma ? a.gamma[c + i] : 1.0f;
            beta[i] = a.beta ? a.beta[c + i] : 0.0f;
        }
    }
};

template <class T, int VE, bool DROP, int ACT>
__device__ __forceinline__ void gn_apply(const GnArgs &a)
{
    const Place t = place<VE>(a);
    if (!t.on) return;
    const int n = blockIdx.z;
    const unsigned p0 = blockIdx.x * a.chunk_px, p1 = min(a.HW, p0 + a.chunk_px);
    Channel<VE> k;
    k.load(a, n, t.c);
#pragma unroll
    for (int i = 0; i < VE; i++) k.gamma[i] *= k.rstd[i];
    constexpr int U = 4;
    for (unsigned p = p0 + t.lane; p < p1; p += t.lanes * U) {
        Raw<T, VE> r[U];
#pragma unroll
        for (int j = 0; j < U; j++)
            if (p + j * t.lanes < p1) r[j] = __ldcs(at<T, VE>(a.x, a, p + j * t.lanes, n, t.c));
#pragma unroll
        for (int j = 0; j < U; j++) {
            const unsigned px = p + j * t.lanes;
            if (px >= p1) break;
            float f[VE];
            unpack<T, VE>(r[j], f);
#pragma unroll
            for (int i = 0; i < VE; i++) f[i] = act_value<ACT>(fmaf(f[i] - k.mean[i], k.gamma[i], k.beta[i]));
            if (DROP)
                drop_elements<VE>(f, (static_cast<unsigned long long>(n) * a.HW + px) * a.C + t.c, a.drop);
            __stcs(const_cast<Raw<T, VE> *>(at<T, VE>(a.y, a, px, n, t.c)), pack<T, VE>(f));
        }
    }
}

template <class T, int VE, bool DROP>
__global__ void __launch_bounds__(kGnThreads) k_gn_apply(const GnArgs a)
{
    grid_launch_dependents();
    grid_dependency_wait();
    switch (a.act) {
    case RZ_ACT_SILU: gn_apply<T, VE, DROP, RZ_ACT_SILU>(a); break;
    case RZ_ACT_GELU: gn_apply<T, VE, DROP, RZ_ACT_GELU>(a); break;
    default: gn_apply<T, VE, DROP, RZ_ACT_NONE>(a); break;
    }
}

// dz of one vector: x and dy in, xh and dz out.
template <int VE, bool DROP, int ACT>
__device__ __forceinline__ void gn_dz(const GnArgs &a, const Channel<VE> &k, unsigned long long e, float (&x)[VE],
                                      float (&d)[VE])
{
    if (DROP) drop_elements<VE>(d, e, a.drop);
#pragma unroll
    for (int i = 0; i < VE; i++) {
        x[i] = (x[i] - k.mean[i]) * k.rstd[i];
        if (ACT != RZ_ACT_NONE) d[i] *= act_slope<ACT>(fmaf(x[i], k.gamma[i], k.beta[i]));
    }
}

// One chunk's sums of dz and dz xh for every channel.
template <class T, int VE, bool DROP, int ACT>
__device__ __forceinline__ void gn_sums(const GnArgs &a, float2 *sh)
{
    const Place t = place<VE>(a);
    const int n = blockIdx.z;
    const unsigned p0 = blockIdx.x * a.chunk_px, p1 = min(a.HW, p0 + a.chunk_px);
    if (t.on) {
        Channel<VE> k;
        k.load(a, n, t.c);
        float s1[VE], s2[VE];
#pragma unroll
        for (int i = 0; i < VE; i++) s1[i] = s2[i] = 0.0f;
        constexpr int U = 4;
        for (unsigned p = p0 + t.lane; p < p1; p += t.lanes * U) {
            Raw<T, VE> rx[U], rd[U];
#pragma unroll
            for (int j = 0; j < U; j++)
                if (p + j * t.lanes < p1) {
                    rx[j] = *at<T, VE>(a.x, a, p + j * t.lanes, n, t.c);
                    rd[j] = *at<T, VE>(a.dy, a, p + j * t.lanes, n, t.c);
                }
#pragma unroll
            for (int j = 0; j < U; j++) {
                const unsigned px = p + j * t.lanes;
                if (px >= p1) break;
                float x[VE], d[VE];
                unpack<T, VE>(rx[j], x);
                unpack<T, VE>(rd[j], d);
                gn_dz<VE, DROP, ACT>(a, k, (static_cast<unsigned long long>(n) * a.HW + px) * a.C + t.c, x, d);
#pragma unroll
                for (int i = 0; i < VE; i++) {
                    s1[i] += d[i];
                    s2[i] = fmaf(d[i], x[i], s2[i]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < VE; i++) sh[(t.lane * t.width + t.vec) * VE + i] = make_float2(s1[i], s2[i]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < t.width * VE; c += kGnThreads) {
        float2 s = make_float2(0.0f, 0.0f);
        for (int l = 0; l < t.lanes; l++) {
            const float2 v = sh[l * t.width * VE + c];
            s.x += v.x;
            s.y += v.y;
        }
        a.part[(static_cast<long long>(n) * a.chunks + blockIdx.x) * a.C + blockIdx.y * kGnThreads * VE + c] = s;
    }
}

template <class T, int VE, bool DROP>
__global__ void __launch_bounds__(kGnThreads) k_gn_sums(const GnArgs a)
{
    __shared__ float2 sh[kGnThreads * VE];
    grid_launch_dependents();
    grid_dependency_wait();
    switch (a.act) {
    case RZ_ACT_SILU: gn_sums<T, VE, DROP, RZ_ACT_SILU>(a, sh); break;
    case RZ_ACT_GELU: gn_sums<T, VE, DROP, RZ_ACT_GELU>(a, sh); break;
    default: gn_sums<T, VE, DROP, RZ_ACT_NONE>(a, sh); break;
    }
}

// The sums of an image's channels and groups from its chunks'.
__global__ void __launch_bounds__(128) k_gn_finish_sums(const GnArgs a)
{
    __shared__ float scratch[32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int g = blockIdx.x, n = blockIdx.y;
    float ga = 0.0f, gb = 0.0f;
    for (int c = g * a.Cg + threadIdx.x; c < (g + 1) * a.Cg; c += 128) {
        float2 s = make_float2(0.0f, 0.0f);
        for (int k = 0; k < a.chunks; k++) {
            const float2 v = a.part[(static_cast<long long>(n) * a.chunks + k) * a.C + c];
            s.x += v.x;
            s.y += v.y;
        }
        a.chan[static_cast<long long>(n) * a.C + c] = s;
        const float gamma = a.gamma ? a.gamma[c] : 1.0f;
        ga = fmaf(gamma, s.x, ga);
        gb = fmaf(gamma, s.y, gb);
    }
    ga = block_sum(ga, scratch);
    gb = block_sum(gb, scratch);
    if (threadIdx.x == 0) a.grp[n * a.G + g] = make_float2(ga * a.inv_m, gb * a.inv_m);
}

// dgamma and dbeta: the images' sums in order.
__global__ void __launch_bounds__(128) k_gn_params(const GnArgs a)
{
    grid_launch_dependents();
    grid_dependency_wait();
    const int c = blockIdx.x * 128 + threadIdx.x;
    if (c >= a.C) return;
    float2 s = make_float2(0.0f, 0.0f);
    for (int n = 0; n < a.N; n++) {
        const float2 v = a.chan[static_cast<long long>(n) * a.C + c];
        s.x += v.x;
        s.y += v.y;
    }
    if (a.dbeta) a.dbeta[c] = s.x;
    if (a.dgamma) a.dgamma[c] = s.y;
}

template <class T, int VE, bool DROP, int ACT>
__device__ __forceinline__ void gn_dx(const GnArgs &a)
{
    const Place t = place<VE>(a);
    if (!t.on) return;
    const int n = blockIdx.z;
    const unsigned p0 = blockIdx.x * a.chunk_px, p1 = min(a.HW, p0 + a.chunk_px);
    Channel<VE> k;
    k.load(a, n, t.c);
    float2 ab[VE];
#pragma unroll
    for (int i = 0; i < VE; i++) ab[i] = a.grp[n * a.G + (t.c + i) / a.Cg];
    constexpr int U = 4;
    for (unsigned p = p0 + t.lane; p < p1; p += t.lanes * U) {
        Raw<T, VE> rx[U], rd[U];
#pragma unroll
        for (int j = 0; j < U; j++)
            if (p + j * t.lanes < p1) {
                rx[j] = __ldcs(at<T, VE>(a.x, a, p + j * t.lanes, n, t.c));
                rd[j] = __ldcs(at<T, VE>(a.dy, a, p + j * t.lanes, n, t.c));
            }
#pragma unroll
        for (int j = 0; j < U; j++) {
            const unsigned px = p + j * t.lanes;
            if (px >= p1) break;
            float x[VE], d[VE];
            unpack<T, VE>(rx[j], x);
            unpack<T, VE>(rd[j], d);
            gn_dz<VE, DROP, ACT>(a, k, (static_cast<unsigned long long>(n) * a.HW + px) * a.C + t.c, x, d);
#pragma unroll
            for (int i = 0; i < VE; i++)
                d[i] = k.rstd[i] * (fmaf(k.gamma[i], d[i], -ab[i].x) - x[i] * ab[i].y);
            __stcs(const_cast<Raw<T, VE> *>(at<T, VE>(a.y, a, px, n, t.c)), pack<T, VE>(d));
        }
    }
}

template <class T, int VE, bool DROP>
__global__ void __launch_bounds__(kGnThreads) k_gn_dx(const GnArgs a)
{
    grid_launch_dependents();
    grid_dependency_wait();
    switch (a.act) {
    case RZ_ACT_SILU: gn_dx<T, VE, DROP, RZ_ACT_SILU>(a); break;
    case RZ_ACT_GELU: gn_dx<T, VE, DROP, RZ_ACT_GELU>(a); break;
    default: gn_dx<T, VE, DROP, RZ_ACT_NONE>(a); break;
    }
}

// ------------------------------------------------------------------ host side

constexpr int kGnMaxChunks = 1024;   // chunks an image: at most this many partial sums a channel

// Chunks of an image and their pixels: about eight CTAs an SM over the call,
// at least 2 kGnRows pixels a thread.
void gn_chunks(GnArgs &a, int ve)
{
    const int vecs = a.C / ve, width = std::min(vecs, kGnThreads), lanes = kGnThreads / width;
    const long long slabs = (vecs + kGnThreads - 1) / kGnThreads;
    const long long want = std::max(1LL, 8LL * 152 / (slabs * a.N));
    const long long least = 2LL * kGnRows * lanes;
    const long long chunks = std::clamp((a.HW + least - 1) / least, 1LL, std::min<long long>(want, kGnMaxChunks));
    a.chunk_px = static_cast<unsigned>((a.HW + chunks - 1) / chunks);
    a.chunks = static_cast<int>((a.HW + a.chunk_px - 1) / a.chunk_px);
}

struct GnWorkspace {
    size_t part, chan, grp, stat, total;
};

GnWorkspace gn_workspace(const GnArgs &a)
{
    auto up = [](size_t v) { return (v + 255) & ~size_t{255}; };
    GnWorkspace w;
    w.part = 0;
    w.chan = up(sizeof(float2) * a.N * a.chunks * static_cast<size_t>(a.C));
    w.grp = w.chan + up(sizeof(float2) * a.N * static_cast<size_t>(a.C));
    w.stat = w.grp + up(sizeof(float2) * a.N * static_cast<size_t>(a.G));
    w.total = w.stat + up(2 * sizeof(float) * a.N * static_cast<size_t>(a.G));
    return w;
}

int gn_check(const rz_norm *d, Shape *s)
{
    if (!d) return RZ_ERR_ARG;
    *s = {d->N, d->H, d->W, d->C, dtype_size(d->dtype)};
    if (!s->es || !shape_ok(*s) || d->groups < 1 || d->C % d->groups != 0) return RZ_ERR_ARG;
    if (d->act != RZ_ACT_NONE && d->act != RZ_ACT_SILU && d->act != RZ_ACT_GELU) return RZ_ERR_ARG;
    if (!(d->eps > 0.0f) || !(d->eps <= 3.0e38f)) return RZ_ERR_ARG;
    return d->N > 65535 ? RZ_ERR_UNSUPPORTED : RZ_OK;
}

void gn_fill(const rz_norm *d, const Shape &s, GnArgs &a)
{
    a = GnArgs{};
    a.N = d->N;
    a.C = d->C;
    a.G = d->groups;
    a.Cg = d->C / d->groups;
    a.HW = static_cast<unsigned>(s.H * s.W);
    a.W = static_cast<unsigned>(s.W);
    a.act = d->act;
    a.eps = d->eps;
    a.inv_m = s.empty() ? 0.0f : static_cast<float>(1.0 / (static_cast<double>(a.HW) * a.Cg));
}

template <class T, int VE>
cudaError_t gn_forward(const GnArgs &a, bool drop, void *stream)
{
    const dim3 grid(a.chunks, (a.C / VE + kGnThreads - 1) / kGnThreads, a.N);
    cudaError_t e = launch(k_gn_stats<T, VE>, grid, kGnThreads, 0, stream, a);
    if (e == cudaSuccess) e = launch(k_gn_finish, dim3(a.G, a.N), 128, 0, stream, a);
    if (e == cudaSuccess)
        e = launch(drop ? k_gn_apply<T, VE, true> : k_gn_apply<T, VE, false>, grid, kGnThreads, 0, stream, a);
    return e;
}

template <class T, int VE>
cudaError_t gn_backward(const GnArgs &a, bool drop, void *stream)
{
    const dim3 grid(a.chunks, (a.C / VE + kGnThreads - 1) / kGnThreads, a.N);
    cudaError_t e =
        launch(drop ? k_gn_sums<T, VE, true> : k_gn_sums<T, VE, false>, grid, kGnThreads, 0, stream, a);
    if (e == cudaSuccess) e = launch(k_gn_finish_sums, dim3(a.G, a.N), 128, 0, stream, a);
    if (e == cudaSuccess)
        e = launch(drop ? k_gn_dx<T, VE, true> : k_gn_dx<T, VE, false>, grid, kGnThreads, 0, stream, a);
    if (e == cudaSuccess && (a.dgamma || a.dbeta))
        e = launch(k_gn_params, dim3((a.C + 127) / 128), 128, 0, stream, a);
    return e;
}

// Elements an access moves: 16 bytes, half of it for 16-bit types whose
// pixels are a multiple of 8 bytes, else one element.
int gn_vector(const Shape &s, const rz_map *x, const rz_map *y, const rz_map *z)
{
    for (int ve = 16 / static_cast<int>(s.es); ve >= 4; ve /= 2)
        if (s.C % ve == 0 && map_aligned(*x, s, ve * s.es) && map_aligned(*y, s, ve * s.es) &&
            (!z || map_aligned(*z, s, ve * s.es)))
            return ve;
    return 1;
}

template <class Fn>
cudaError_t gn_dispatch(int dtype, int ve, Fn fn)
{
    if (dtype == RZ_F32) return ve == 4 ? fn(float{}, std::integral_constant<int, 4>{}) : fn(float{}, std::integral_constant<int, 1>{});
    auto half = [&](auto t) {
        if (ve == 8) return fn(t, std::integral_constant<int, 8>{});
        return ve == 4 ? fn(t, std::integral_constant<int, 4>{}) : fn(t, std::integral_constant<int, 1>{});
    };
    return dtype == RZ_BF16 ? half(__nv_bfloat16{}) : half(__half{});
}

bool gn_floats_ok(std::initializer_list<const float *> ps)
{
    for (const float *p : ps)
        if (reinterpret_cast<uintptr_t>(p) % sizeof(float)) return false;
    return true;
}

int gn_status(cudaError_t e)
{
    if (e == cudaSuccess) return RZ_OK;
    record_cuda_error(static_cast<int>(e));
    return RZ_ERR_CUDA;
}

}  // namespace
}  // namespace rz

using namespace rz;

extern "C" {

int map_group_norm_workspace(const rz_norm *d, size_t *bytes)
{
    maps::Shape s;
    const int rc = gn_check(d, &s);
    if (rc != RZ_OK) return rc;
    if (!bytes) return RZ_ERR_ARG;
    *bytes = 0;
    if (s.empty()) return RZ_OK;
    GnArgs a;
    gn_fill(d, s, a);
    // enough for every vector width, the one thing that the maps' alignment decides
    for (int ve : {8, 4, 1})
        if (a.C % ve == 0) {
            gn_chunks(a, ve);
            *bytes = std::max(*bytes, gn_workspace(a).total);
        }
    return RZ_OK;
}

int map_group_norm(const rz_norm *d, const rz_drop *drop, const rz_map *x, const rz_map *y, const float *gamma, const float *beta,
                   float *mean, float *rstd, void *workspace, size_t workspace_bytes, void *stream)
{
    maps::Shape s;
    const int rc = gn_check(d, &s);
    if (rc != RZ_OK) return rc;
    if (!maps::drop_ok(drop)) return RZ_ERR_ARG;
    if (!gn_floats_ok({gamma, beta, mean, rstd})) return RZ_ERR_ARG;
    if (s.empty()) return RZ_OK;
    if (!maps::map_ok(x, s) || !maps::map_ok(y, s) || maps::map_overlap(*x, s, *y, s)) return RZ_ERR_ARG;
    GnArgs a;
    gn_fill(d, s, a);
    a.x = maps::view(x);
    a.y = maps::view(y);
    a.joined = maps::rows_joined(*x, s) && maps::rows_joined(*y, s);
    const int ve = gn_vector(s, x, y, nullptr);
    gn_chunks(a, ve);
    const GnWorkspace w = gn_workspace(a);
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 || workspace_bytes < w.total) return RZ_ERR_ARG;
    uint8_t *base = static_cast<uint8_t *>(workspace);
    a.part = reinterpret_cast<float2 *>(base + w.part);
    float *stat = reinterpret_cast<float *>(base + w.stat);
    a.gamma = gamma;
    a.beta = beta;
    a.mean = mean ? mean : stat;
    a.rstd = rstd ? rstd : stat + static_cast<size_t>(a.N) * a.G;
    a.drop = maps::make_drop(drop);
    const bool dropping = maps::drop_threshold(drop) != 0;
    return gn_status(gn_dispatch(d->dtype, ve, [&](auto t, auto v) {
        return gn_forward<decltype(t), decltype(v)::value>(a, dropping, stream);
    }));
}

int map_group_norm_grad(const rz_norm *d, const rz_drop *drop, const rz_map *dy, const rz_map *x, const rz_map *dx, const float *gamma,
                        const float *beta, const float *mean, const float *rstd, float *dgamma, float *dbeta,
                        void *workspace, size_t workspace_bytes, void *stream)
{
    maps::Shape s;
    const int rc = gn_check(d, &s);
    if (rc != RZ_OK) return rc;
    if (!maps::drop_ok(drop)) return RZ_ERR_ARG;
    if (!gn_floats_ok({gamma, beta, mean, rstd, dgamma, dbeta})) return RZ_ERR_ARG;
    if (s.empty()) {
        for (float *g : {dgamma, dbeta})
            if (g) {
                const cudaError_t e =
                    cudaMemsetAsync(g, 0, sizeof(float) * d->C, static_cast<cudaStream_t>(stream));
                if (e != cudaSuccess) return gn_status(e);
            }
        return RZ_OK;
    }
    if (!maps::map_ok(x, s) || !maps::map_ok(dy, s) || !maps::map_ok(dx, s) || maps::map_overlap(*x, s, *dx, s) ||
        maps::map_overlap(*dy, s, *dx, s) || !mean || !rstd)
        return RZ_ERR_ARG;
    GnArgs a;
    gn_fill(d, s, a);
    a.x = maps::view(x);
    a.dy = maps::view(dy);
    a.y = maps::view(dx);
    a.joined = maps::rows_joined(*x, s) && maps::rows_joined(*dy, s) && maps::rows_joined(*dx, s);
    const int ve = gn_vector(s, x, dx, dy);
    gn_chunks(a, ve);
    const GnWorkspace w = gn_workspace(a);
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 || workspace_bytes < w.total) return RZ_ERR_ARG;
    uint8_t *base = static_cast<uint8_t *>(workspace);
    a.part = reinterpret_cast<float2 *>(base + w.part);
    a.chan = reinterpret_cast<float2 *>(base + w.chan);
    a.grp = reinterpret_cast<float2 *>(base + w.grp);
    a.gamma = gamma;
    a.beta = beta;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    a.drop = maps::make_drop(drop);
    const bool dropping = maps::drop_threshold(drop) != 0;
    return gn_status(gn_dispatch(d->dtype, ve, [&](auto t, auto v) {
        return gn_backward<decltype(t), decltype(v)::value>(a, dropping, stream);
    }));
}

}  // extern "C"
