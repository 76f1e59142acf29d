// Group norm and its gradient for images of any size and layout, in passes: a
// launch that sums each channel by chunks of an image, a small one that joins
// the chunks, and one that applies the result, from the map's end backwards.
// group_norm.cu states the formulas.  Of a map up to L2's size the second
// reading costs no DRAM; cutting larger calls into batches that fit L2 measured
// slower than reading them twice (batches of 64 MB: the gradient of 4 x 512 x
// 512 x 128 bf16 278 us against 231 us as it then was).
//
// The forward is bound by DRAM: 4 x 512 x 512 x 128 bf16 138 us, three
// transfers of the map at 5.8 TB/s (141 us with SiLU; 180 with dropout, bound by
// the generator's arithmetic).  The gradient is bound by the instructions that
// its warps issue: 8 x 128 x 128 x 512 bf16 124 us (five transfers, 5.4 TB/s),
// as much with SiLU, 142 with dropout, which both passes make again (146 where
// each call is made by itself and not from a graph).
//
// A thread keeps one vector of channels and walks pixels, so sums are taken by
// channel whatever the group's width; groups are put together from channels at
// the head of the applying launch.  All sums go through memory in a fixed
// order.
#pragma once

#include "gn_device.h"
#include "map_ops.h"
#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {

using namespace maps;

constexpr int kGpThreads = 256, kGpWarps = kGpThreads / 32;
// Pixels a thread loads before it uses the first, and the CTAs an SM that its
// registers are held to: 4 x 512 x 512 x 128 bf16 with SiLU forward 152 us so
// (later steps took it to 141), 164 at two CTAs an SM, 155 with the loads through
// shared memory.
constexpr int kGpStats = 4, kGpStatsCtas = 4, kGpApply = 4, kGpApplyCtas = 4;
// The gradient, whose constants and sums fill the registers, has its loads on
// their way in shared memory, kGpAhead pixels of x and dy a thread, and so a
// third CTA an SM: 8 x 128 x 128 x 512 bf16 with SiLU and dropout 155 us, 171
// with four pixels in registers and two CTAs; four CTAs spill, 183.  Pointers
// that step from pixel to pixel, in place of each one's offset, took it to 142.
constexpr int kGpAhead = 3, kGpGradCtas = 3;
template <class V> constexpr int kGpRing = 2 * kGpAhead * kGpThreads * static_cast<int>(sizeof(V));

// The thread's place: vector `vec` of the block's `width`, pixel lane `lane`
// of `lanes`; `c` its first channel, `first` the block's.
struct GpPlace {
    int n, first, c, width, vec, lanes, lane;
    unsigned p0, p1;
    bool on;
};

// BACK: from the last image's last chunk on, so that the pass which applies
// begins with what the summing one has left in L2.
template <int VE, bool BACK>
__device__ __forceinline__ GpPlace gp_place(const GnArgs &a)
{
    GpPlace t;
    const int start = blockIdx.y * kGpThreads;
    t.width = min(a.C / VE - start, kGpThreads);
    t.lanes = kGpThreads / t.width;
    t.lane = threadIdx.x / t.width;
    t.vec = threadIdx.x - t.lane * t.width;
    t.n = BACK ? gridDim.z - 1 - blockIdx.z : blockIdx.z;
    t.first = start * VE;
    t.c = t.first + t.vec * VE;
    t.p0 = (BACK ? gridDim.x - 1 - blockIdx.x : blockIdx.x) * a.chunk_px;
    t.p1 = min(a.HW, t.p0 + a.chunk_px);
    t.on = t.lane < t.lanes;
    return t;
}

template <class T, int VE>
__device__ __forceinline__ const Raw<T, VE> *gp_at(const View &v, const GnArgs &a, const GpPlace &t, unsigned px)
{
    return reinterpret_cast<const Raw<T, VE> *>(
        v.p + t.n * v.bstride + pixel_off(px, a.W, a.joined, v.pitch, a.C * static_cast<int>(sizeof(T))) +
        t.c * static_cast<int>(sizeof(T)));
}

// Elements before the thread's vector of pixel px.
__device__ __forceinline__ unsigned long long gp_element(const GnArgs &a, const GpPlace &t, unsigned px)
{
    return (static_cast<unsigned long long>(t.n) * a.HW + px) * a.C + t.c;
}

// A pixel's vectors as they were read.
template <class T, int VE>
struct One {
    Raw<T, VE> x;
};

// Walks the thread's pixels, U at a time while there are U, then one by one:
// load(pixel) and use(values, count, pixel).
template <int U, class Load, class Use>
__device__ __forceinline__ void gp_walk(const GpPlace &t, Load load, Use use)
{
    using R = decltype(load(0u));
    unsigned p = t.p0 + t.lane;
    const unsigned step = U * t.lanes, reach = (U - 1) * t.lanes;
    if (p + reach < t.p1) {
        R some[U];
#pragma unroll
        for (int j = 0; j < U; j++) some[j] = load(p + j * t.lanes);
        while (true) {
            use(some, Int<U>{}, p);
            p += step;
            if (p + reach >= t.p1) break;
            // asked for at the loop's end, where they overlap the arithmetic before
#pragma unroll
            for (int j = 0; j < U; j++) some[j] = load(p + j * t.lanes);
        }
    }
    for (; p < t.p1; p += t.lanes) {
        const R last[1] = {load(p)};
        use(last, Int<1>{}, p);
    }
}

// The thread's vector in a map, pixel after pixel; `step` bytes apart where the
// rows follow one another.
template <class T, int VE>
struct GpWalker {
    const uint8_t *at;
    __device__ __forceinline__ GpWalker(const View &v, const GnArgs &a, const GpPlace &t, unsigned px)
        : at(reinterpret_cast<const uint8_t *>(gp_at<T, VE>(v, a, t, px)))
    {
    }
    __device__ __forceinline__ void go(const View &v, const GnArgs &a, const GpPlace &t, unsigned px, unsigned step)
    {
        if (a.joined)
            at += step;
        else
            at = reinterpret_cast<const uint8_t *>(gp_at<T, VE>(v, a, t, px));
    }
    __device__ __forceinline__ Raw<T, VE> *get() const
    {
        return const_cast<Raw<T, VE> *>(reinterpret_cast<const Raw<T, VE> *>(at));
    }
};

// Bytes from one of the thread's pixels to the next: at most 256 threads' vectors
// and a pixel's channels, far below 4 GB.
template <class T>
__device__ __forceinline__ unsigned gp_step(const GnArgs &a, const GpPlace &t)
{
    return t.lanes * a.C * static_cast<unsigned>(sizeof(T));
}

// Walks the thread's pixels with kGpAhead of them, x and dy, on their way into
// the thread's places in `ring`: use(x, dy, element, pixel).
template <class T, int VE, class Use>
__device__ __forceinline__ void gp_stream(const GnArgs &a, const GpPlace &t, Raw<T, VE> *ring, Use use)
{
    using V = Raw<T, VE>;
    const unsigned step = gp_step<T>(a, t);
    unsigned next = t.p0 + t.lane;
    unsigned long long e = gp_element(a, t, next);
    GpWalker<T, VE> x(a.x, a, t, next), dy(a.dy, a, t, next);
    const auto copy = [&](V *to) {
        if (next < t.p1) {
            copy_async(to, x.get());
            copy_async(to + kGpThreads, dy.get());
        }
        copies_commit();
        next += t.lanes;
        x.go(a.x, a, t, next, step);
        dy.go(a.dy, a, t, next, step);
    };
    V *const end = ring + 2 * kGpAhead * kGpThreads;
    for (V *to = ring; to != end; to += 2 * kGpThreads) copy(to);
    V *at = ring;
    for (unsigned p = t.p0 + t.lane; p < t.p1; p += t.lanes, e += t.lanes * static_cast<unsigned>(a.C)) {
        copies_left<kGpAhead - 1>();
        const V vx = at[0], vd = at[kGpThreads];
        copy(at);
        at = at + 2 * kGpThreads == end ? ring : at + 2 * kGpThreads;
        use(vx, vd, e, p);
    }
}

__device__ __forceinline__ float2 *gp_part(const GnArgs &a, int n, int chunk)
{
    return a.part + (static_cast<long long>(n) * a.chunks + chunk) * a.C;
}

// One chunk's mean and sum of squared distances for every channel.  A thread
// takes kGpStats pixels at a time: their mean, their squared distances from it,
// and the two joined to what it holds (the pairwise update of Chan, Golub and
// LeVeque, "Updating formulae and a pairwise algorithm for computing sample
// variances"), so that nothing cancels where the mean is far above the
// deviation.
template <class T, int VE>
__global__ void __launch_bounds__(kGpThreads, kGpStatsCtas) k_gp_stats(const GnArgs a)
{
    __shared__ __align__(16) float sh[kGpThreads * VE];
    __shared__ int count[kGpThreads];
    dev::grid_launch_dependents();
    dev::grid_dependency_wait();
    const GpPlace t = gp_place<VE, false>(a);
    float2 mean[kPairs<VE>], m2[kPairs<VE>];
#pragma unroll
    for (int i = 0; i < kPairs<VE>; i++) mean[i] = m2[i] = both(0.0f);
    int have = 0;
    const auto take = [&](const auto &r, auto count, unsigned) {
        constexpr int U = decltype(count)::value;
        float2 m[kPairs<VE>], q[kPairs<VE>], f[kPairs<VE>];
#pragma unroll
        for (int i = 0; i < kPairs<VE>; i++) m[i] = q[i] = both(0.0f);
#pragma unroll
        for (int j = 0; j < U; j++) {
            unpack2<T, VE>(r[j].x, f);
#pragma unroll
            for (int i = 0; i < kPairs<VE>; i++) m[i] = __fadd2_rn(m[i], f[i]);
        }
#pragma unroll
        for (int i = 0; i < kPairs<VE>; i++) m[i] = __fmul2_rn(m[i], both(-1.0f / U));   // minus the mean
#pragma unroll
        for (int j = 0; j < U; j++) {
            unpack2<T, VE>(r[j].x, f);
#pragma unroll
            for (int i = 0; i < kPairs<VE>; i++) {
                const float2 d = __fadd2_rn(f[i], m[i]);
                q[i] = __ffma2_rn(d, d, q[i]);
            }
        }
        have += U;
        const float share = __fdividef(static_cast<float>(U), static_cast<float>(have)), weight = share * (have - U);
#pragma unroll
        for (int i = 0; i < kPairs<VE>; i++) {
            const float2 d = __fadd2_rn(m[i], mean[i]);     // what was held minus what is new
            mean[i] = __ffma2_rn(d, both(-share), mean[i]);
            m2[i] = __fadd2_rn(m2[i], __ffma2_rn(__fmul2_rn(d, d), both(weight), q[i]));
        }
    };
    if (t.on)
        gp_walk<kGpStats>(t, [&](unsigned px) { return One<T, VE>{*gp_at<T, VE>(a.x, a, t, px)}; }, take);
    // join the pixel lanes, a thread to a channel: the chunk's mean, then the distances about it
    float *mine = sh + (t.lane * t.width + t.vec) * VE;
    if (t.on) {
        gn_save<VE>(mine, mean);
        if (t.vec == 0) count[t.lane] = have;
    }
    __syncthreads();
    constexpr int kOwn = VE;    // channels a thread joins at most
    float m[kOwn], q[kOwn];
#pragma unroll
    for (int k = 0; k < kOwn; k++) {
        const int c = threadIdx.x + k * kGpThreads;
        m[k] = q[k] = 0.0f;
        if (c < t.width * VE) {
            float s = 0.0f;
            for (int l = 0; l < t.lanes; l++) s = fmaf(sh[l * t.width * VE + c], static_cast<float>(count[l]), s);
            m[k] = s / (t.p1 - t.p0);
            for (int l = 0; l < t.lanes; l++) {
                const float d = sh[l * t.width * VE + c] - m[k];
                q[k] = fmaf(d * d, static_cast<float>(count[l]), q[k]);
            }
        }
    }
    __syncthreads();
    if (t.on) gn_save<VE>(mine, m2);
    __syncthreads();
    float2 *out = gp_part(a, blockIdx.z, blockIdx.x) + blockIdx.y * kGpThreads * VE;
#pragma unroll
    for (int k = 0; k < kOwn; k++) {
        const int c = threadIdx.x + k * kGpThreads;
        if (c < t.width * VE) {
            for (int l = 0; l < t.lanes; l++) q[k] += sh[l * t.width * VE + c];
            out[c] = make_float2(m[k], q[k]);
        }
    }
}

// The constants of the block's channels, from the groups' statistics: -mean,
// a, beta.
__device__ __forceinline__ void gp_constants(const GnArgs &a, const GpPlace &t, int channels, float *cst, int c, float mean,
                                             float rstd)
{
    cst[c] = -mean;
    cst[channels + c] = a.gamma ? rstd * a.gamma[t.first + c] : rstd;
    cst[2 * channels + c] = a.beta ? a.beta[t.first + c] : 0.0f;
}

template <int VE>
__device__ __forceinline__ void gp_channel(const GpPlace &t, const float *cst, Channel<VE> &k)
{
    gn_load<VE>(k.shift, cst + t.vec * VE);
    gn_load<VE>(k.a, cst + t.width * VE + t.vec * VE);
    gn_load<VE>(k.beta, cst + 2 * t.width * VE + t.vec * VE);
}

// For each group that the block's channels belong to, fn(g, {sum, sum}) by
// every lane of a warp, with the sums over all its channels of get(c).
template <class Get, class Fn>
__device__ __forceinline__ void gp_groups(const GnArgs &a, const GpPlace &t, int channels, Get get, Fn fn)
{
    const int lane = threadIdx.x & 31, g1 = (t.first + channels - 1) / a.Cg;
    for (int g = t.first / a.Cg + (threadIdx.x >> 5); g <= g1; g += kGpWarps) {
        float2 s = make_float2(0.0f, 0.0f);
        for (int c = g * a.Cg + lane; c < (g + 1) * a.Cg; c += 32) s = __fadd2_rn(s, get(c));
        fn(g, make_float2(warp_sum(s.x), warp_sum(s.y)));
    }
}

template <class T, int VE, bool DROP, int ACT>
__global__ void __launch_bounds__(kGpThreads, kGpApplyCtas) k_gp_apply(const GnArgs a)
{
    extern __shared__ __align__(16) float gp_smem[];    // three constants a channel, then two statistics a group
    dev::grid_launch_dependents();
    const GpPlace t = gp_place<VE, true>(a);
    const int channels = t.width * VE, g0 = t.first / a.Cg;
    float2 *group = reinterpret_cast<float2 *>(gp_smem + align_up(3 * channels, 2));
    dev::grid_dependency_wait();
    const float2 *chan = a.chan + static_cast<long long>(t.n) * a.C;
    const float pixels = static_cast<float>(a.HW);
    gp_groups(
        a, t, channels, [&](int c) { return make_float2(chan[c].x * pixels, 0.0f); },
        [&](int g, float2 s) {
            if ((threadIdx.x & 31) == 0) group[g - g0].x = s.x * a.inv_m;
        });
    __syncthreads();
    gp_groups(
        a, t, channels,
        [&](int c) {
            const float2 v = chan[c];
            const float d = v.x - group[c / a.Cg - g0].x;
            return make_float2(fmaf(d * d, pixels, v.y), 0.0f);
        },
        [&](int g, float2 s) {
            if ((threadIdx.x & 31)) return;
            const float rstd = rsqrtf(fmaf(s.x, a.inv_m, a.eps));
            group[g - g0].y = rstd;
            if (blockIdx.x == 0 && g * a.Cg >= t.first) {
                a.mean[t.n * a.G + g] = group[g - g0].x;
                a.rstd[t.n * a.G + g] = rstd;
            }
        });
    __syncthreads();
    for (int c = threadIdx.x; c < channels; c += kGpThreads) {
        const float2 v = group[(t.first + c) / a.Cg - g0];
        gp_constants(a, t, channels, gp_smem, c, v.x, v.y);
    }
    __syncthreads();
    if (!t.on) return;
    Channel<VE> k;
    gp_channel<VE>(t, gp_smem, k);
    gp_walk<kGpApply>(
        t, [&](unsigned px) { return One<T, VE>{__ldcs(gp_at<T, VE>(a.x, a, t, px))}; },
        [&](const auto &r, auto count, unsigned p) {
#pragma unroll
            for (int j = 0; j < decltype(count)::value; j++) {
                const unsigned px = p + j * t.lanes;
                const unsigned long long e = gp_element(a, t, px);
                __stcs(const_cast<Raw<T, VE> *>(gp_at<T, VE>(a.y, a, t, px)),
                       gn_value<T, VE, DROP, ACT>(r[j].x, k, a.drop, e >> 3, e & 7));
            }
        });
}

// One chunk's sums of dz and dz xh for every channel.
template <class T, int VE, bool DROP, int ACT>
__global__ void __launch_bounds__(kGpThreads, kGpGradCtas) k_gp_sums(const GnArgs a)
{
    // vectors on their way; three constants a channel, then the threads' sums
    extern __shared__ __align__(16) uint8_t gp_bytes[];
    using V = Raw<T, VE>;
    V *ring = reinterpret_cast<V *>(gp_bytes) + threadIdx.x;
    float *gp_smem = reinterpret_cast<float *>(gp_bytes + kGpRing<V>);
    dev::grid_launch_dependents();
    const GpPlace t = gp_place<VE, false>(a);
    const int channels = t.width * VE;
    dev::grid_dependency_wait();
    for (int c = threadIdx.x; c < channels; c += kGpThreads) {
        const int g = t.n * a.G + (t.first + c) / a.Cg;
        gp_constants(a, t, channels, gp_smem, c, a.mean[g], a.rstd[g]);
    }
    __syncthreads();
    float2 s1[kPairs<VE>], s2[kPairs<VE>];
#pragma unroll
    for (int i = 0; i < kPairs<VE>; i++) s1[i] = s2[i] = both(0.0f);
    if (t.on) {
        Channel<VE> k;
        gp_channel<VE>(t, gp_smem, k);
        gp_stream<T, VE>(a, t, ring, [&](const V &x, const V &dy, unsigned long long e, unsigned) {
            float2 d[kPairs<VE>], dz[kPairs<VE>];
            gn_dz<T, VE, DROP, ACT>(x, dy, k, a.drop, e >> 3, e & 7, d, dz);
#pragma unroll
            for (int i = 0; i < kPairs<VE>; i++) {
                s1[i] = __fadd2_rn(s1[i], dz[i]);
                s2[i] = __ffma2_rn(dz[i], d[i], s2[i]);
            }
        });
    }
    float2 *out = gp_part(a, blockIdx.z, blockIdx.x) + blockIdx.y * kGpThreads * VE;
    float u[VE];    // this thread's channels' sums of dz
#pragma unroll
    for (int z = 0; z < 2; z++) {
        __syncthreads();
        if (t.on) gn_save<VE>(gp_smem + (t.lane * t.width + t.vec) * VE, z ? s2 : s1);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < VE; k++) {
            const int c = threadIdx.x + k * kGpThreads;
            if (c < channels) {
                float s = 0.0f;
                for (int l = 0; l < t.lanes; l++) s += gp_smem[l * channels + c];
                if (z)
                    out[c] = make_float2(u[k] * a.drop.scale, s * a.drop.scale * a.rstd[t.n * a.G + (t.first + c) / a.Cg]);
                else
                    u[k] = s;
            }
        }
    }
}

// dx = a dz - rstd A - rstd^2 B d; the dropout's scale, which dz lacks, goes
// with a.
template <class T, int VE, bool DROP, int ACT>
__global__ void __launch_bounds__(kGpThreads, kGpGradCtas) k_gp_dx(const GnArgs a)
{
    // vectors on their way; five constants a channel, then two sums a group
    extern __shared__ __align__(16) uint8_t gp_bytes[];
    using V = Raw<T, VE>;
    V *ring = reinterpret_cast<V *>(gp_bytes) + threadIdx.x;
    float *gp_smem = reinterpret_cast<float *>(gp_bytes + kGpRing<V>);
    dev::grid_launch_dependents();
    const GpPlace t = gp_place<VE, true>(a);
    const int channels = t.width * VE, g0 = t.first / a.Cg;
    float2 *group = reinterpret_cast<float2 *>(gp_smem + align_up(5 * channels, 2));
    dev::grid_dependency_wait();
    const float2 *chan = a.chan + static_cast<long long>(t.n) * a.C;
    gp_groups(
        a, t, channels,
        [&](int c) {
            const float gamma = a.gamma ? a.gamma[c] : 1.0f;
            return make_float2(gamma * chan[c].x, gamma * chan[c].y);
        },
        [&](int g, float2 s) {
            const float r = a.rstd[t.n * a.G + g];
            if ((threadIdx.x & 31) == 0) group[g - g0] = make_float2(-r * (s.x * a.inv_m), -r * r * (s.y * a.inv_m));
        });
    __syncthreads();
    for (int c = threadIdx.x; c < channels; c += kGpThreads) {
        const int g = (t.first + c) / a.Cg;
        gp_constants(a, t, channels, gp_smem, c, a.mean[t.n * a.G + g], a.rstd[t.n * a.G + g]);
        gp_smem[3 * channels + c] = group[g - g0].x;
        gp_smem[4 * channels + c] = group[g - g0].y;
    }
    __syncthreads();
    if (!t.on) return;
    Channel<VE> k;
    float2 k0[kPairs<VE>], k1[kPairs<VE>];
    gp_channel<VE>(t, gp_smem, k);
    gn_load<VE>(k0, gp_smem + 3 * channels + t.vec * VE);
    gn_load<VE>(k1, gp_smem + 4 * channels + t.vec * VE);
    const unsigned step = gp_step<T>(a, t);
    GpWalker<T, VE> out(a.y, a, t, t.p0 + t.lane);
    gp_stream<T, VE>(a, t, ring, [&](const V &x, const V &dy, unsigned long long e, unsigned px) {
        float2 d[kPairs<VE>], dz[kPairs<VE>];
        gn_dz<T, VE, DROP, ACT>(x, dy, k, a.drop, e >> 3, e & 7, d, dz);
#pragma unroll
        for (int i = 0; i < kPairs<VE>; i++) {
            if (DROP) dz[i] = __fmul2_rn(dz[i], both(a.drop.scale));
            dz[i] = __ffma2_rn(d[i], k1[i], __ffma2_rn(dz[i], k.a[i], k0[i]));
        }
        __stcs(out.get(), pack2<T, VE>(dz));
        out.go(a.y, a, t, px + t.lanes, step);
    });
}

// The chunks' shares joined, kJoinWide channels a block, the chunks over its
// threads, each of which asks for all of its own at once: forward, sets of
// unlike counts and means; gradient, sums.  A thread takes about four chunks
// where the largest block allows it (blocks of 64 rows whatever the chunks: 16
// x 64 x 64 x 320 forward 35 us against 30).
constexpr int kJoinThreads = 1024, kJoinWide = 16, kJoinFew = 4;
constexpr int kJoinEach = (kGnMaxChunks * kJoinWide + kJoinThreads - 1) / kJoinThreads;

template <bool GRAD>
__global__ void __launch_bounds__(kJoinThreads) k_gp_join(const GnArgs a)
{
    __shared__ float2 sh[2][kJoinThreads / 32][kJoinWide];
    dev::grid_launch_dependents();
    const int lane = threadIdx.x % kJoinWide, row = threadIdx.x / kJoinWide, rows = blockDim.x / kJoinWide;
    const int c = blockIdx.x * kJoinWide + lane;
    const float2 *part = gp_part(a, blockIdx.y, 0) + c;
    // over the warp's two rows, then over the warps, every other one a row
    const auto total = [&](float2 s, int z) {
        s.x += __shfl_xor_sync(0xffffffffu, s.x, kJoinWide);
        s.y += __shfl_xor_sync(0xffffffffu, s.y, kJoinWide);
        if ((row & 1) == 0) sh[z][row / 2][lane] = s;
        __syncthreads();
        s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kJoinThreads / 64; k++) {
            const int w = 2 * k + (row & 1);
            if (w < rows / 2) s = __fadd2_rn(s, sh[z][w][lane]);
        }
        s.x += __shfl_xor_sync(0xffffffffu, s.x, kJoinWide);
        s.y += __shfl_xor_sync(0xffffffffu, s.y, kJoinWide);
        return s;
    };
    dev::grid_dependency_wait();
    float2 v[kJoinEach];
#pragma unroll
    for (int k = 0; k < kJoinEach; k++) {
        const int chunk = row + k * rows;
        v[k] = c < a.C && chunk < a.chunks ? part[static_cast<long long>(chunk) * a.C] : make_float2(0.0f, 0.0f);
    }
    float2 s = make_float2(0.0f, 0.0f);
    if (GRAD) {
#pragma unroll
        for (int k = 0; k < kJoinEach; k++) s = __fadd2_rn(s, v[k]);
        s = total(s, 0);
    } else {
        float px[kJoinEach];    // the chunks' pixels; 0 past the last
#pragma unroll
        for (int k = 0; k < kJoinEach; k++) {
            const int chunk = row + k * rows;
            px[k] = chunk < a.chunks ? static_cast<float>(min(a.chunk_px, a.HW - chunk * a.chunk_px)) : 0.0f;
            s.x = fmaf(v[k].x, px[k], s.x);
        }
        const float mean = total(s, 0).x / a.HW;
        s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kJoinEach; k++) s.y += fmaf((v[k].x - mean) * (v[k].x - mean), px[k], v[k].y);
        s = make_float2(mean, total(s, 1).y);
    }
    if (row == 0 && c < a.C) a.chan[static_cast<long long>(blockIdx.y) * a.C + c] = s;
}

// ------------------------------------------------------------------ host side

template <class T, class Fn>
cudaError_t gp_vectors(int ve, Fn fn)
{
    if constexpr (sizeof(T) == 2)
        if (ve == 8) return fn(Int<8>{});
    return ve == 4 ? fn(Int<4>{}) : fn(Int<1>{});
}

inline dim3 gp_grid(const GnArgs &a, int ve)
{
    return dim3(a.chunks, (a.C / ve + kGpThreads - 1) / kGpThreads, a.N);
}

template <bool GRAD>
cudaError_t gp_join(const GnArgs &a, void *stream)
{
    static_assert(kJoinEach >= kJoinFew, "");
    const int warps = std::min((a.chunks + 2 * kJoinFew - 1) / (2 * kJoinFew), kJoinThreads / 32);
    return launch(k_gp_join<GRAD>, dim3((a.C + kJoinWide - 1) / kJoinWide, a.N), 32 * warps, 0, stream, a);
}

// Floats of shared memory: `each` a channel and two a group, or one for each
// thread's elements where that is more.
inline size_t gp_shared(const GnArgs &a, int ve, int each)
{
    const int channels = std::min(a.C, kGpThreads * ve), groups = channels / a.Cg + 2;
    return sizeof(float) * std::max(align_up(each * channels, 2) + 2 * groups, kGpThreads * ve);
}

inline cudaError_t gp_launch(void (*fn)(GnArgs), dim3 grid, size_t smem, void *stream, const GnArgs &a)
{
    const cudaError_t e = shared_opt_in(reinterpret_cast<const void *>(fn));
    return e != cudaSuccess ? e : launch(fn, grid, kGpThreads, smem, stream, a);
}

}  // namespace

template <class T>
cudaError_t gn_passes_forward(const GnArgs &a, int ve, bool drop, void *stream)
{
    return gp_vectors<T>(ve, [&](auto v) {
        constexpr int VE = decltype(v)::value;
        const dim3 grid = gp_grid(a, VE);
        cudaError_t e = launch(k_gp_stats<T, VE>, grid, kGpThreads, 0, stream, a);
        if (e == cudaSuccess)
            e = gp_join<false>(a, stream);
        if (e != cudaSuccess) return e;
        return gn_kinds(a.act, drop, [&](auto dr, auto act) {
            return gp_launch(k_gp_apply<T, VE, decltype(dr)::value, decltype(act)::value>, grid, gp_shared(a, VE, 3),
                             stream, a);
        });
    });
}

template <class T>
cudaError_t gn_passes_backward(const GnArgs &a, int ve, bool drop, void *stream)
{
    return gp_vectors<T>(ve, [&](auto v) {
        constexpr int VE = decltype(v)::value;
        const dim3 grid = gp_grid(a, VE);
        return gn_kinds(a.act, drop, [&](auto dr, auto act) {
            constexpr bool D = decltype(dr)::value;
            constexpr int A = decltype(act)::value;
            constexpr size_t ring = kGpRing<Raw<T, VE>>;
            cudaError_t e = gp_launch(k_gp_sums<T, VE, D, A>, grid, ring + gp_shared(a, VE, 3), stream, a);
            if (e == cudaSuccess)
                e = gp_join<true>(a, stream);
            return e != cudaSuccess ? e : gp_launch(k_gp_dx<T, VE, D, A>, grid, ring + gp_shared(a, VE, 5), stream, a);
        });
    });
}

}  // namespace rz
