// Group norm and its gradient where a slab of an image (some neighbouring
// groups, all pixels) fits the shared memory of one cluster of CTAs: the map is
// read once, the statistics meet through distributed shared memory, and what
// was kept is put through and written.  group_norm.cu states the formulas.
//
// A warp's lanes are `lv` vectors of a pixel by 32 / lv pixels; a thread keeps
// `keep` vectors of its own, copied in asynchronously to places that only it
// reads, so that the loops over them stay short whatever their number.  A
// cluster takes unit after unit (a slab of an image): as a thread is done with
// a place, the next unit's vector is asked for into it, so that DRAM reads go
// on while results are put through and written.
// Channels are joined into groups only after the sums over pixels, so groups
// may end anywhere inside a vector.
//
// Each map crosses DRAM once, and what bounds the kernels is the arithmetic of
// a round's phases, at 16 warps an SM and about half of the issue slots: 64 x 32
// x 32 x 256 bf16 forward 18 us (3.7 TB/s), 26 with SiLU and dropout, gradient
// 32 and 42; 16 x 64 x 64 x 320 with both 36 us, where its 128 units make two
// rounds of 76 clusters; 2 x 14 x 14 x 256 4 us, one launch's latency.  More
// warps measured slower: ten a CTA spill (40 us at 16 x 64 x 64 x 320), and
// three CTAs an SM keep fewer vectors each, in larger clusters.
#include <algorithm>
#include <mutex>

#include "gn_device.h"
#include "map_ops.h"
#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {

using namespace maps;

constexpr int kGcWarps = 8, kGcThreads = 32 * kGcWarps;
constexpr int kGcCtas = 2;          // resident CTAs an SM
constexpr int kGcMaxVecs = 32;      // vectors a slab: one warp wide

__device__ __forceinline__ void cluster_arrive()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait()
{
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// *p in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ float2 remote(const float2 *p, int rank)
{
    unsigned at = dev::smem_addr(p);
    float2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(at) : "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}

// Shared memory of a CTA, byte offsets.
struct GcLayout {
    int warp, cst, cta, total;
};
// slot: bytes a kept vector takes.
__host__ __device__ inline GcLayout gc_layout(int keep, int slot, int ve, int lv, int channels, int groups)
{
    GcLayout l;
    l.warp = keep * slot * kGcThreads;                          // [warps][channels], float2
    l.cst = l.warp + 8 * kGcWarps * lv * ve;                    // [channels] x 5 floats
    l.cta = l.cst + align_up(5 * 4 * channels, 16);             // [groups], float2
    l.total = l.cta + 8 * groups;
    return l;
}

// The thread's place in its slab: vector v of a pixel, pixel lp of its warp's
// `pixels`; c its first channel, c0 the slab's; `have` vectors from pixel
// `first` on, a `step` apart.
struct GcPlace {
    int rank, n, lane, warp, v, lp, pixels, c, c0, channels, groups, have;
    unsigned first, step;
    bool on;
};

// Units are counted slab by slab, image by image.
template <int VE>
__device__ __forceinline__ GcPlace gc_place(const GnArgs &a, unsigned unit)
{
    GcPlace t;
    t.n = unit / a.slabs;
    const int slab = unit - t.n * a.slabs;
    t.rank = blockIdx.x % a.cl;
    t.lane = threadIdx.x & 31;
    t.warp = threadIdx.x >> 5;
    t.pixels = 32 / a.lv;
    t.lp = t.lane / a.lv;
    t.v = t.lane - t.lp * a.lv;
    t.groups = min(a.gs, a.G - slab * a.gs);
    t.channels = t.groups * a.Cg;
    t.c0 = slab * a.gs * a.Cg;
    t.c = t.c0 + t.v * VE;
    t.step = kGcWarps * t.pixels;
    t.first = t.rank * a.keep * t.step + t.warp * t.pixels + t.lp;
    t.on = t.lp < t.pixels && t.v * VE < t.channels;
    t.have = t.on && t.first < a.HW ? min(a.keep, static_cast<int>((a.HW - t.first + t.step - 1) / t.step)) : 0;
    return t;
}

// Pixels of [0, HW) that CTA `rank` holds.
__device__ __forceinline__ int gc_count(const GnArgs &a, unsigned per_cta, int rank)
{
    const unsigned first = rank * per_cta;
    return first >= a.HW ? 0 : static_cast<int>(min(per_cta, a.HW - first));
}

__device__ __forceinline__ void copy16(void *to, const void *from)
{
    copy_async(static_cast<uint4 *>(to), static_cast<const uint4 *>(from));
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Two values of each of a vector's channels to the warp's row.
template <int VE>
__device__ __forceinline__ void gc_save(const GcPlace &t, float2 *row, const float2 (&p)[kPairs<VE>],
                                        const float2 (&q)[kPairs<VE>])
{
    if (!t.on || t.lp) return;
    float4 *at = reinterpret_cast<float4 *>(row + t.warp * t.channels + t.v * VE);
#pragma unroll
    for (int i = 0; i < kPairs<VE>; i++) at[i] = make_float4(p[i].x, q[i].x, p[i].y, q[i].y);
}

// The other CTAs' values of a group: all asked for before the first is used.
__device__ __forceinline__ void gc_others(const float2 *p, int cl, float2 (&v)[kGnMaxCluster])
{
#pragma unroll
    for (int r = 0; r < kGnMaxCluster; r++)
        if (r < cl) v[r] = cl > 1 ? remote(p, r) : *p;
}

// The statistics by the pairwise update of Chan, Golub and LeVeque ("Updating
// formulae and a pairwise algorithm for computing sample variances"): a thread's
// own mean and squared distances first, joined over lanes, warps and CTAs.
template <class T, int VE, bool DROP, int ACT>
__global__ void __launch_bounds__(kGcThreads, kGcCtas) k_gc_forward(const GnArgs a)
{
    extern __shared__ __align__(16) uint8_t gc_smem[];
    __shared__ float counts[kGcWarps];
    using V = Raw<T, VE>;
    dev::grid_launch_dependents();
    const unsigned units = a.N * a.slabs, clusters = gridDim.x / a.cl;
    unsigned unit = blockIdx.x / a.cl;
    GcPlace t = gc_place<VE>(a, unit);
    V *data = reinterpret_cast<V *>(gc_smem) + threadIdx.x;      // every kGcThreads-th
    // from one of a thread's vectors to the next: bytes, and the generator's blocks of eight elements (a step is a
    // multiple of eight pixels); all of an image's slab in a cluster is far below 4 GB
    const long long px_bytes = a.C * static_cast<long long>(sizeof(T));
    const unsigned hop = t.step * static_cast<unsigned>(px_bytes), blocks = t.step / 8 * a.C;
    const auto offset = [&](const View &v, const GcPlace &o) {
        return v.p + o.n * v.bstride + o.first * px_bytes + o.c * static_cast<int>(sizeof(T));
    };
    dev::grid_dependency_wait();
    {
        const uint8_t *in = offset(a.x, t);
#pragma unroll 4
        for (int j = 0; j < t.have; j++) copy16(data + j * kGcThreads, in + j * hop);
    }
    const int own = threadIdx.x / a.Cg;     // the group of channel threadIdx.x
    const unsigned per_cta = a.keep * t.step;
    const int mine = gc_count(a, per_cta, t.rank);
    const float mine_inv = mine ? 1.0f / (static_cast<float>(mine) * a.Cg) : 0.0f;
    while (true) {
    const GcLayout l = gc_layout(a.keep, 16, VE, a.lv, t.channels, t.groups);
    float2 *row = reinterpret_cast<float2 *>(gc_smem + l.warp), *cta = reinterpret_cast<float2 *>(gc_smem + l.cta);
    float *cst = reinterpret_cast<float *>(gc_smem + l.cst);    // -mean, a, beta of the channels
    float gamma = 1.0f, beta = 0.0f;
    if (threadIdx.x < t.channels) {
        if (a.gamma) gamma = a.gamma[t.c0 + threadIdx.x];
        if (a.beta) beta = a.beta[t.c0 + threadIdx.x];
    }
    copies_done();

    // the thread's mean, and its squared distances from it
    float2 f[kPairs<VE>], m[kPairs<VE>], q[kPairs<VE>];
#pragma unroll
    for (int i = 0; i < kPairs<VE>; i++) m[i] = q[i] = both(0.0f);
#pragma unroll 4
    for (int j = 0; j < t.have; j++) {
        unpack2<T, VE>(data[j * kGcThreads], f);
#pragma unroll
        for (int i = 0; i < kPairs<VE>; i++) m[i] = __fadd2_rn(m[i], f[i]);
    }
    const float inv = t.have ? -1.0f / t.have : 0.0f;
#pragma unroll
    for (int i = 0; i < kPairs<VE>; i++) m[i] = __fmul2_rn(m[i], both(inv));    // minus the mean
#pragma unroll 4
    for (int j = 0; j < t.have; j++) {
        unpack2<T, VE>(data[j * kGcThreads], f);
#pragma unroll
        for (int i = 0; i < kPairs<VE>; i++) {
            const float2 d = __fadd2_rn(f[i], m[i]);
            q[i] = __ffma2_rn(d, d, q[i]);
        }
    }
    // over the warp's pixels, two sets at a time (Chan, Golub and LeVeque)
    int count = t.have;
    for (int half = t.pixels; half > 1;) {
        const int h = (half + 1) / 2, by = h * a.lv;
        const bool take = t.lp + h < half;
        const int below = __shfl_down_sync(0xffffffffu, count, by), other = take ? below : 0;
        const float share = count + other ? __fdividef(static_cast<float>(other), static_cast<float>(count + other)) : 0.0f;
        const float weight = share * count;
#pragma unroll
        for (int i = 0; i < kPairs<VE>; i++) {
            float2 om, oq;
            om.x = __shfl_down_sync(0xffffffffu, m[i].x, by);
            om.y = __shfl_down_sync(0xffffffffu, m[i].y, by);
            oq.x = __shfl_down_sync(0xffffffffu, q[i].x, by);
            oq.y = __shfl_down_sync(0xffffffffu, q[i].y, by);
            if (take) {
                const float2 d = __ffma2_rn(m[i], both(-1.0f), om);
                m[i] = __ffma2_rn(d, both(share), m[i]);
                q[i] = __fadd2_rn(q[i], __ffma2_rn(__fmul2_rn(d, d), both(weight), oq));
            }
        }
        count += other;
        half = h;
    }
    gc_save<VE>(t, row, m, q);
    if (t.lane == 0) counts[t.warp] = static_cast<float>(count);
    __syncthreads();
    // over the warps and a group's channels, a warp to a group, a lane to a channel: the CTA's mean, then the
    // distances about it
    for (int g = t.warp; g < t.groups; g += kGcWarps) {
        const float2 *at = row + g * a.Cg;
        float2 e[kGcWarps];
        float n[kGcWarps], s = 0.0f, v = 0.0f;
#pragma unroll
        for (int w = 0; w < kGcWarps; w++) n[w] = counts[w];
        for (int c = t.lane; c < a.Cg; c += 32) {
#pragma unroll
            for (int w = 0; w < kGcWarps; w++) e[w] = at[w * t.channels + c];
#pragma unroll
            for (int w = 0; w < kGcWarps; w++) s = fmaf(e[w].x, n[w], s);
        }
        s = warp_sum(s) * mine_inv;     // minus the mean
        for (int c = t.lane; c < a.Cg; c += 32) {
            if (a.Cg > 32) {
#pragma unroll
                for (int w = 0; w < kGcWarps; w++) e[w] = at[w * t.channels + c];
            }
#pragma unroll
            for (int w = 0; w < kGcWarps; w++)
                if (n[w] > 0.0f) v += fmaf((e[w].x - s) * (e[w].x - s), n[w], e[w].y);
        }
        v = warp_sum(v);
        if (t.lane == 0) cta[g] = make_float2(-s, v);
    }
    if (a.cl > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    // over the cluster, a thread to a channel
    if (threadIdx.x < t.channels) {
        float2 v[kGnMaxCluster];
        gc_others(cta + own, a.cl, v);
        float2 e = v[0];
        float n = static_cast<float>(gc_count(a, per_cta, 0)) * a.Cg;
#pragma unroll
        for (int r = 1; r < kGnMaxCluster; r++)
            if (r < a.cl) {
                const float on = static_cast<float>(gc_count(a, per_cta, r)) * a.Cg, share = __fdividef(on, n + on);
                const float d = v[r].x - e.x;
                e = make_float2(fmaf(d, share, e.x), e.y + fmaf(d * d, share * n, v[r].y));
                n += on;
            }
        const float rstd = rsqrtf(fmaf(e.y, a.inv_m, a.eps));
        if (t.rank == 0 && threadIdx.x == own * a.Cg) {
            const int g = t.n * a.G + t.c0 / a.Cg + own;
            a.mean[g] = e.x;
            a.rstd[g] = rstd;
        }
        cst[threadIdx.x] = -e.x;
        cst[t.channels + threadIdx.x] = rstd * gamma;
        cst[2 * t.channels + threadIdx.x] = beta;
    }
    if (a.cl > 1) cluster_arrive();   // this CTA has read the others' memory
    __syncthreads();
    // put through and written; the next unit's vectors come into the places
    const bool more = unit + clusters < units;
    const GcPlace o = more ? gc_place<VE>(a, unit + clusters) : t;
    const uint8_t *in = offset(a.x, o);
    const int coming = more ? o.have : 0;
    if (t.have) {
        Channel<VE> k;
        gn_load<VE>(k.shift, cst + t.v * VE);
        gn_load<VE>(k.a, cst + t.channels + t.v * VE);
        gn_load<VE>(k.beta, cst + 2 * t.channels + t.v * VE);
        uint8_t *out = const_cast<uint8_t *>(offset(a.y, t));
        const unsigned long long e = (static_cast<unsigned long long>(t.n) * a.HW + t.first) * a.C + t.c;
        constexpr int kUnroll = DROP || ACT == RZ_ACT_GELU ? 2 : 4;
#pragma unroll kUnroll
        for (int j = 0; j < t.have; j++) {
            const V r = data[j * kGcThreads];
            if (j < coming) copy16(data + j * kGcThreads, in + j * hop);
            __stcs(reinterpret_cast<V *>(out + j * hop), gn_value<T, VE, DROP, ACT>(r, k, a.drop, (e >> 3) + j * blocks, e & 7));
        }
    }
    for (int j = t.have; j < coming; j++) copy16(data + j * kGcThreads, in + j * hop);
    if (a.cl > 1) cluster_wait();
    if (!more) return;
    t = o;
    unit += clusters;
    }
}

// The gradient.  x stays as it was read; dz, of which the second pass needs
// every bit and which costs most of the arithmetic, takes dy's place as float32.
template <class T, int VE, bool DROP, int ACT>
__global__ void __launch_bounds__(kGcThreads, kGcCtas) k_gc_backward(const GnArgs a)
{
    extern __shared__ __align__(16) uint8_t gc_smem[];
    using V = Raw<T, VE>;
    dev::grid_launch_dependents();
    const unsigned units = a.N * a.slabs, clusters = gridDim.x / a.cl;
    unsigned unit = blockIdx.x / a.cl;
    GcPlace t = gc_place<VE>(a, unit);
    V *x = reinterpret_cast<V *>(gc_smem) + threadIdx.x;         // every kGcThreads-th
    float4 *z = reinterpret_cast<float4 *>(gc_smem + a.keep * 16 * kGcThreads) + threadIdx.x;
    // from one of a thread's vectors to the next: bytes, and the generator's blocks of eight elements (a step is a
    // multiple of eight pixels); all of an image's slab in a cluster is far below 4 GB
    const long long px_bytes = a.C * static_cast<long long>(sizeof(T));
    const unsigned hop = t.step * static_cast<unsigned>(px_bytes), blocks = t.step / 8 * a.C;
    const auto offset = [&](const View &v, const GcPlace &o) {
        return v.p + o.n * v.bstride + o.first * px_bytes + o.c * static_cast<int>(sizeof(T));
    };
    // what a channel is normalised with, a thread to a channel: read a unit ahead
    float mean = 0.0f, rstd = 0.0f, gamma = 1.0f, beta = 0.0f;
    const auto channel = [&](const GcPlace &o) {
        if (threadIdx.x >= o.channels) return;
        const int c = o.c0 + threadIdx.x, g = o.n * a.G + c / a.Cg;
        mean = a.mean[g];
        rstd = a.rstd[g];
        if (a.gamma) gamma = a.gamma[c];
        if (a.beta) beta = a.beta[c];
    };
    dev::grid_dependency_wait();
    {
        const uint8_t *in = offset(a.x, t), *din = offset(a.dy, t);
#pragma unroll 4
        for (int j = 0; j < t.have; j++) {
            copy16(x + j * kGcThreads, in + j * hop);
            copy16(z + j * (VE / 4) * kGcThreads, din + j * hop);
        }
    }
    channel(t);
    const int own = threadIdx.x / a.Cg;     // the group of channel threadIdx.x
    while (true) {
    const GcLayout l = gc_layout(a.keep, 16 + 4 * VE, VE, a.lv, t.channels, t.groups);
    float2 *row = reinterpret_cast<float2 *>(gc_smem + l.warp), *cta = reinterpret_cast<float2 *>(gc_smem + l.cta);
    float *cst = reinterpret_cast<float *>(gc_smem + l.cst);     // -mean, a, beta, then what dx takes from the group's sums
    if (threadIdx.x < t.channels) {
        cst[threadIdx.x] = -mean;
        cst[t.channels + threadIdx.x] = rstd * gamma;
        cst[2 * t.channels + threadIdx.x] = beta;
    }
    copies_done();
    __syncthreads();
    Channel<VE> k;
    if (t.on) {
        gn_load<VE>(k.shift, cst + t.v * VE);
        gn_load<VE>(k.a, cst + t.channels + t.v * VE);
        gn_load<VE>(k.beta, cst + 2 * t.channels + t.v * VE);
    }
    float2 s1[kPairs<VE>], s2[kPairs<VE>];
#pragma unroll
    for (int i = 0; i < kPairs<VE>; i++) s1[i] = s2[i] = both(0.0f);
    const unsigned long long e = (static_cast<unsigned long long>(t.n) * a.HW + t.first) * a.C + t.c;
#pragma unroll 2
    for (int j = 0; j < t.have; j++) {
        float2 d[kPairs<VE>], dz[kPairs<VE>];
        float4 *zj = z + j * (VE / 4) * kGcThreads;
        gn_dz<T, VE, DROP, ACT>(x[j * kGcThreads], *reinterpret_cast<const V *>(zj), k, a.drop, (e >> 3) + j * blocks, e & 7, d, dz);
#pragma unroll
        for (int i = 0; i < kPairs<VE>; i++) {
            s1[i] = __fadd2_rn(s1[i], dz[i]);
            s2[i] = __ffma2_rn(dz[i], d[i], s2[i]);
        }
#pragma unroll
        for (int i = 0; i < VE / 4; i++)
            zj[i * kGcThreads] = make_float4(dz[2 * i].x, dz[2 * i].y, dz[2 * i + 1].x, dz[2 * i + 1].y);
    }
    for (int half = t.pixels; half > 1;) {
        const int h = (half + 1) / 2, by = h * a.lv;
        const bool take = t.lp + h < half;
#pragma unroll
        for (int i = 0; i < kPairs<VE>; i++) {
            float2 o1, o2;
            o1.x = __shfl_down_sync(0xffffffffu, s1[i].x, by);
            o1.y = __shfl_down_sync(0xffffffffu, s1[i].y, by);
            o2.x = __shfl_down_sync(0xffffffffu, s2[i].x, by);
            o2.y = __shfl_down_sync(0xffffffffu, s2[i].y, by);
            if (take) {
                s1[i] = __fadd2_rn(s1[i], o1);
                s2[i] = __fadd2_rn(s2[i], o2);
            }
        }
        half = h;
    }
    gc_save<VE>(t, row, s1, s2);
    __syncthreads();
    // the groups' sums of a dz and a dz d, a = rstd gamma, a warp to a group, a lane to a channel
    for (int g = t.warp; g < t.groups; g += kGcWarps) {
        const float2 *at = row + g * a.Cg;
        float2 v = make_float2(0.0f, 0.0f);
        for (int c = t.lane; c < a.Cg; c += 32) {
            float2 u = at[c];
#pragma unroll
            for (int w = 1; w < kGcWarps; w++) u = __fadd2_rn(u, at[w * t.channels + c]);
            v = __ffma2_rn(u, both(cst[t.channels + g * a.Cg + c]), v);
        }
        v = make_float2(warp_sum(v.x), warp_sum(v.y));
        if (t.lane == 0) cta[g] = v;
    }
    if (a.cl > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    // over the cluster, a thread to a channel
    if (threadIdx.x < t.channels) {
        float2 o[kGnMaxCluster];
        gc_others(cta + own, a.cl, o);
        float2 v = o[0];
#pragma unroll
        for (int r = 1; r < kGnMaxCluster; r++)
            if (r < a.cl) v = __fadd2_rn(v, o[r]);
        const float share = -a.inv_m * a.drop.scale;
        cst[3 * t.channels + threadIdx.x] = share * v.x;
        cst[4 * t.channels + threadIdx.x] = share * rstd * rstd * v.y;
    }
    if (a.cl > 1) cluster_arrive();     // this CTA has read the others' memory
    __syncthreads();
    // put through and written; the next unit's vectors come into the places
    const bool more = unit + clusters < units;
    const GcPlace o = more ? gc_place<VE>(a, unit + clusters) : t;
    const uint8_t *in = offset(a.x, o), *din = offset(a.dy, o);
    const int coming = more ? o.have : 0;
    const float row_scale = a.drop.scale * rstd;
    if (more) channel(o);
    if (t.have) {
        float2 k0[kPairs<VE>], k1[kPairs<VE>];
        gn_load<VE>(k0, cst + 3 * t.channels + t.v * VE);
        gn_load<VE>(k1, cst + 4 * t.channels + t.v * VE);
#pragma unroll
        for (int i = 0; i < kPairs<VE>; i++) k.a[i] = __fmul2_rn(k.a[i], both(a.drop.scale));
        uint8_t *out = const_cast<uint8_t *>(offset(a.y, t));
#pragma unroll 4
        for (int j = 0; j < t.have; j++) {
            float2 d[kPairs<VE>];
            unpack2<T, VE>(x[j * kGcThreads], d);
            float4 *zj = z + j * (VE / 4) * kGcThreads;
#pragma unroll
            for (int i = 0; i < VE / 4; i++) {
                const float4 q = zj[i * kGcThreads];
                d[2 * i] = __ffma2_rn(__fadd2_rn(d[2 * i], k.shift[2 * i]), k1[2 * i],
                                      __ffma2_rn(make_float2(q.x, q.y), k.a[2 * i], k0[2 * i]));
                d[2 * i + 1] = __ffma2_rn(__fadd2_rn(d[2 * i + 1], k.shift[2 * i + 1]), k1[2 * i + 1],
                                          __ffma2_rn(make_float2(q.z, q.w), k.a[2 * i + 1], k0[2 * i + 1]));
            }
            if (j < coming) {
                copy16(x + j * kGcThreads, in + j * hop);
                copy16(zj, din + j * hop);
            }
            __stcs(reinterpret_cast<V *>(out + j * hop), pack2<T, VE>(d));
        }
    }
    for (int j = t.have; j < coming; j++) {
        copy16(x + j * kGcThreads, in + j * hop);
        copy16(z + j * (VE / 4) * kGcThreads, din + j * hop);
    }
    // this CTA's {sum dz, sum dz xh} of its channels: a row of its own for dgamma and dbeta
    if (threadIdx.x < t.channels) {
        float2 v = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kGcWarps; w++) v = __fadd2_rn(v, row[w * t.channels + threadIdx.x]);
        a.chan[(static_cast<long long>(t.n) * a.cl + t.rank) * a.C + t.c0 + threadIdx.x] =
            make_float2(v.x * a.drop.scale, v.y * row_scale);
    }
    if (a.cl > 1) cluster_wait();
    if (!more) return;
    t = o;
    unit += clusters;
    __syncthreads();    // the constants and rows have been read
    }
}

// ------------------------------------------------------------------ host side

cudaError_t gc_launch(void (*fn)(GnArgs), const GnArgs &a, int smem, void *stream)
{
    const cudaError_t e = shared_opt_in(reinterpret_cast<const void *>(fn));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.cl) * a.clusters, 1, 1);
    cfg.blockDim = dim3(kGcThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(a.cl), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fn, a);
}

template <class Fn>
cudaError_t gc_types(int dtype, Fn fn)
{
    if (dtype == RZ_F32) return fn(float{});
    return dtype == RZ_BF16 ? fn(__nv_bfloat16{}) : fn(__half{});
}

int gc_bytes(const GnArgs &a, size_t es, bool grad, int keep)
{
    const int ve = 16 / static_cast<int>(es);
    return gc_layout(keep, grad ? 16 + 4 * ve : 16, ve, a.lv, a.gs * a.Cg, a.gs).total;
}


// Clusters of each size that are resident at once (a cluster lies within one
// of the GPU's parts of some SMs), asked once a device for the largest CTAs.
cudaError_t gc_resident(int *clusters)
{
    static std::mutex mu;
    static int known[64][kGnMaxCluster + 1] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    int (&row)[kGnMaxCluster + 1] = known[dev & 63];
    if (!row[1]) {
        const auto fn = k_gc_forward<__nv_bfloat16, 8, true, RZ_ACT_SILU>;
        e = shared_opt_in(reinterpret_cast<const void *>(fn));
        for (int cl = kGnMaxCluster; cl >= 1 && e == cudaSuccess; cl--) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(cl, 1, 1);
            cfg.blockDim = dim3(kGcThreads, 1, 1);
            cfg.dynamicSmemBytes = kMapShared;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim = {static_cast<unsigned>(cl), 1, 1};
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            e = cudaOccupancyMaxActiveClusters(&n, fn, &cfg);
            row[cl] = std::max(1, n);
        }
        if (e != cudaSuccess) {
            row[1] = 0;
            return e;
        }
    }
    std::copy(row, row + kGnMaxCluster + 1, clusters);
    return cudaSuccess;
}

}  // namespace

// Of the slabs from 128 bytes of a pixel down to 32 (a DRAM sector) and the
// clusters of up to eight CTAs that hold an image's slab, the pair with the
// least estimated time: the rounds of units that the resident clusters need,
// each of a fixed part, one for each vector that a thread keeps and one for the
// cluster's barriers, in microseconds as measured on 512 x 16 x 16 x 512 to
// 64 x 64 x 64 x 256 bf16 maps at slabs of 2 to 8 vectors and clusters of 1 to
// 8 (a round with 8 vectors a thread: forward 5.6 us alone, 6.3 in clusters of
// four; gradient 7.3 and 9.1).
cudaError_t gn_cluster_plan(GnArgs &args, size_t es, bool grad, bool *fits)
{
    *fits = false;
    GnArgs a = args;
    const int ve = 16 / static_cast<int>(es);
    int base = 1;   // groups whose channels fill whole vectors
    while (static_cast<long long>(base) * a.Cg % ve) base++;
    const long long base_vecs = static_cast<long long>(base) * a.Cg / ve;
    if (base_vecs > kGcMaxVecs) return cudaSuccess;
    int resident[kGnMaxCluster + 1];
    const cudaError_t e = gc_resident(resident);
    if (e != cudaSuccess) return e;
    double best = 0.0;
    for (int m = std::max(1, 8 / static_cast<int>(base_vecs)); m >= 1; m--) {
        a.lv = static_cast<int>(base_vecs) * m;
        a.gs = base * m;
        if (a.lv < 2 && a.gs < a.G) break;
        const int row = kGcWarps * (32 / a.lv), rows = static_cast<int>((a.HW + row - 1) / row);
        const int fixed = gc_bytes(a, es, grad, 0), most = (kMapShared - fixed) / (gc_bytes(a, es, grad, 1) - fixed);
        a.slabs = (a.G + a.gs - 1) / a.gs;
        const long long units = static_cast<long long>(a.N) * a.slabs;
        if (units > 0x7fffffffLL) continue;
        for (int cl = 1; cl <= kGnMaxCluster; cl++) {
            a.keep = (rows + cl - 1) / cl;
            if (a.keep > most || (rows + a.keep - 1) / a.keep != cl) continue;
            const long long rounds = (units + resident[cl] - 1) / resident[cl];
            const double barrier = cl == 1 ? 0.0 : grad ? 0.3 * cl : 0.6 + 0.1 * cl;
            const double cost = rounds * ((grad ? 2.3 + 0.62 * a.keep : 2.8 + 0.35 * a.keep) + barrier);
            if (*fits && cost >= best) continue;
            best = cost;
            *fits = true;
            a.cl = cl;
            a.clusters = static_cast<int>((units + rounds - 1) / rounds);   // no fewer rounds with more
            a.rows = a.N * cl;
            args = a;
        }
    }
    return cudaSuccess;
}

cudaError_t gn_cluster_forward(const GnArgs &a, int dtype, bool drop, void *stream)
{
    return gc_types(dtype, [&](auto t) {
        using T = decltype(t);
        return gn_kinds(a.act, drop, [&](auto dr, auto act) {
            return gc_launch(k_gc_forward<T, 16 / sizeof(T), decltype(dr)::value, decltype(act)::value>, a,
                             gc_bytes(a, sizeof(T), false, a.keep), stream);
        });
    });
}

cudaError_t gn_cluster_backward(const GnArgs &a, int dtype, bool drop, void *stream)
{
    return gc_types(dtype, [&](auto t) {
        using T = decltype(t);
        return gn_kinds(a.act, drop, [&](auto dr, auto act) {
            return gc_launch(k_gc_backward<T, 16 / sizeof(T), decltype(dr)::value, decltype(act)::value>, a,
                             gc_bytes(a, sizeof(T), true, a.keep), stream);
        });
    });
}

}  // namespace rz
