// Group norm and its gradient where a slab of an image (some neighbouring
// groups, all pixels) fits the shared memory of one cluster of CTAs: the map is
// read once, the statistics meet through distributed shared memory, and what
// was kept is put through and written.  group_norm.cu states the formulas.
//
// A warp's lanes are `lv` vectors of a pixel by 32 / lv pixels; a thread keeps
// `keep` vectors of its own, copied in asynchronously to places that only it
// reads, so that the loops over them stay short whatever their number.
// Channels are joined into groups only after the sums over pixels, so groups
// may end anywhere inside a vector.
#include <algorithm>

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
    int red, part, cst, cta, total;
};
// slot: bytes a kept vector takes; values: floats a channel is reduced to.
__host__ __device__ inline GcLayout gc_layout(int keep, int slot, int ve, int lv, int values, int channels, int groups)
{
    GcLayout l;
    l.red = keep * slot * kGcThreads;                                               // [rows][channels] x values
    l.part = l.red + 4 * values * kGcWarps * ((32 / lv + 1) / 2) * lv * ve;         // [segments][groups] x values
    l.cst = l.part + align_up(8 * (groups > kGcWarps ? groups : kGcWarps), 16);     // [channels] x 5 floats
    l.cta = l.cst + align_up(5 * 4 * channels, 16);                                 // [groups], float2
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

// CTAs are counted slab by slab, image by image.
template <int VE>
__device__ __forceinline__ GcPlace gc_place(const GnArgs &a)
{
    GcPlace t;
    const unsigned row = a.cl * a.slabs;
    t.n = blockIdx.x / row;
    const int at = blockIdx.x - t.n * row, slab = at / a.cl;
    t.rank = at - slab * a.cl;
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
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dev::smem_addr(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Writes each channel's value a thread (V floats) to red[rows][channels], the
// warp's pixels joined by halves first; the rows of a CTA.
template <int VE, int V>
__device__ __forceinline__ int gc_rows(const GcPlace &t, int lv, float2 (&f)[V][kPairs<VE>], float *red)
{
    const int half = (t.pixels + 1) / 2;
#pragma unroll
    for (int z = 0; z < V; z++)
#pragma unroll
        for (int i = 0; i < kPairs<VE>; i++) {
            const float x = __shfl_down_sync(0xffffffffu, f[z][i].x, half * lv);
            const float y = __shfl_down_sync(0xffffffffu, f[z][i].y, half * lv);
            if (t.lp + half < t.pixels) f[z][i] = __fadd2_rn(f[z][i], make_float2(x, y));
        }
    if (t.on && t.lp < half) {
        float *at = red + ((t.warp * half + t.lp) * t.channels + t.v * VE) * V;
        if constexpr (V == 1) {
            gn_save<VE>(at, f[0]);
        } else {
#pragma unroll
            for (int i = 0; i < kPairs<VE>; i++)
                reinterpret_cast<float4 *>(at)[i] = make_float4(f[0][i].x, f[1][i].x, f[0][i].y, f[1][i].y);
        }
    }
    return kGcWarps * half;
}

// Sums over the CTA's rows and each group's channels: get(row, channel) by all
// warps, several to a group where there are few, into part[segment][group];
// the number of segments.
template <class Get>
__device__ __forceinline__ int gc_groups(const GcPlace &t, int cg, int rows, float2 *part, Get get)
{
    const int segments = max(1, kGcWarps / t.groups), wide = min(cg, 32), at_once = 32 / wide;
    const int l0 = t.lane / wide, c0 = t.lane - l0 * wide;
    for (int i = t.warp; i < segments * t.groups; i += kGcWarps) {
        const int seg = i / t.groups, g = i - seg * t.groups;
        float2 s = make_float2(0.0f, 0.0f);
        if (l0 < at_once)
            for (int r = seg * at_once + l0; r < rows; r += segments * at_once)
                for (int c = c0; c < cg; c += wide) s = __fadd2_rn(s, get(r, g * cg + c));
        s = make_float2(warp_sum(s.x), warp_sum(s.y));
        if (t.lane == 0) part[i] = s;
    }
    return segments;
}

template <class T, int VE, bool DROP, int ACT>
__global__ void __launch_bounds__(kGcThreads, kGcCtas) k_gc_forward(const GnArgs a)
{
    extern __shared__ __align__(16) uint8_t gc_smem[];
    using V = Raw<T, VE>;
    dev::grid_launch_dependents();
    const GcPlace t = gc_place<VE>(a);
    const GcLayout l = gc_layout(a.keep, 16, VE, a.lv, 1, t.channels, t.groups);
    V *data = reinterpret_cast<V *>(gc_smem) + threadIdx.x;      // every kGcThreads-th
    float *red = reinterpret_cast<float *>(gc_smem + l.red);
    float2 *part = reinterpret_cast<float2 *>(gc_smem + l.part), *cta = reinterpret_cast<float2 *>(gc_smem + l.cta);
    float *cst = reinterpret_cast<float *>(gc_smem + l.cst);    // -mean, a, beta of the channels
    const long long px_bytes = a.C * static_cast<long long>(sizeof(T)), hop = t.step * px_bytes;
    const uint8_t *in = a.x.p + t.n * a.x.bstride + t.first * px_bytes + t.c * static_cast<int>(sizeof(T));
    dev::grid_dependency_wait();
#pragma unroll 4
    for (int j = 0; j < t.have; j++) copy16(data + j * kGcThreads, in + j * hop);
    float gamma = 1.0f, beta = 0.0f;
    if (threadIdx.x < t.channels) {
        if (a.gamma) gamma = a.gamma[t.c0 + threadIdx.x];
        if (a.beta) beta = a.beta[t.c0 + threadIdx.x];
    }
    copies_done();

    // the CTA's group means, then the squared distances from them
    float2 f[kPairs<VE>], s[1][kPairs<VE>], m[kPairs<VE>];
#pragma unroll
    for (int i = 0; i < kPairs<VE>; i++) s[0][i] = both(0.0f);
#pragma unroll 4
    for (int j = 0; j < t.have; j++) {
        unpack2<T, VE>(data[j * kGcThreads], f);
#pragma unroll
        for (int i = 0; i < kPairs<VE>; i++) s[0][i] = __fadd2_rn(s[0][i], f[i]);
    }
    const auto get = [&](int r, int c) { return make_float2(red[r * t.channels + c], 0.0f); };
    const int rows = gc_rows<VE, 1>(t, a.lv, s, red);
    __syncthreads();
    int segments = gc_groups(t, a.Cg, rows, part, get);
    __syncthreads();
    const unsigned per_cta = a.keep * t.step;
    const int mine = gc_count(a, per_cta, t.rank);
    const int own = threadIdx.x / a.Cg;                          // the group of channel threadIdx.x
    if (threadIdx.x < t.channels) {
        float v = 0.0f;
        for (int k = 0; k < segments; k++) v += part[k * t.groups + own].x;
        cst[threadIdx.x] = mine ? -v / (static_cast<float>(mine) * a.Cg) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPairs<VE>; i++) s[0][i] = both(0.0f);
    if (t.on) gn_load<VE>(m, cst + t.v * VE);
#pragma unroll 4
    for (int j = 0; j < t.have; j++) {
        unpack2<T, VE>(data[j * kGcThreads], f);
#pragma unroll
        for (int i = 0; i < kPairs<VE>; i++) {
            const float2 d = __fadd2_rn(f[i], m[i]);
            s[0][i] = __ffma2_rn(d, d, s[0][i]);
        }
    }
    gc_rows<VE, 1>(t, a.lv, s, red);
    __syncthreads();
    segments = gc_groups(t, a.Cg, rows, part, get);
    __syncthreads();
    if (threadIdx.x < t.channels && threadIdx.x == own * a.Cg) {
        float v = 0.0f;
        for (int k = 0; k < segments; k++) v += part[k * t.groups + own].x;
        cta[own] = make_float2(-cst[threadIdx.x], v);
    }
    if (a.cl > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    // over the cluster, a thread to a channel: sets of unlike counts and means (Chan, Golub and LeVeque)
    if (threadIdx.x < t.channels) {
        float2 e = a.cl > 1 ? remote(cta + own, 0) : cta[own];
        float n = static_cast<float>(gc_count(a, per_cta, 0)) * a.Cg;
        for (int r = 1; r < a.cl; r++) {
            const float2 o = remote(cta + own, r);
            const float on = static_cast<float>(gc_count(a, per_cta, r)) * a.Cg, share = __fdividef(on, n + on);
            const float d = o.x - e.x;
            e = make_float2(fmaf(d, share, e.x), e.y + fmaf(d * d, share * n, o.y));
            n += on;
        }
        const float rstd = 1.0f / sqrtf(fmaf(e.y, a.inv_m, a.eps));
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
    if (t.have) {
        Channel<VE> k;
        gn_load<VE>(k.shift, cst + t.v * VE);
        gn_load<VE>(k.a, cst + t.channels + t.v * VE);
        gn_load<VE>(k.beta, cst + 2 * t.channels + t.v * VE);
        uint8_t *out = a.y.p + t.n * a.y.bstride + t.first * px_bytes + t.c * static_cast<int>(sizeof(T));
        unsigned long long e = (static_cast<unsigned long long>(t.n) * a.HW + t.first) * a.C + t.c;
        const unsigned long long e_hop = static_cast<unsigned long long>(t.step) * a.C;
#pragma unroll 4
        for (int j = 0; j < t.have; j++) {
            __stcs(reinterpret_cast<V *>(out + j * hop),
                   gn_value<T, VE, DROP, ACT>(data[j * kGcThreads], k, a.drop, e + j * e_hop));
        }
    }
    if (a.cl > 1) cluster_wait();
}

// The gradient.  x stays as it was read; dz, of which the second pass needs
// every bit and which costs most of the arithmetic, takes dy's place as float32.
template <class T, int VE, bool DROP, int ACT>
__global__ void __launch_bounds__(kGcThreads, kGcCtas) k_gc_backward(const GnArgs a)
{
    extern __shared__ __align__(16) uint8_t gc_smem[];
    using V = Raw<T, VE>;
    dev::grid_launch_dependents();
    const GcPlace t = gc_place<VE>(a);
    const GcLayout l = gc_layout(a.keep, 16 + 4 * VE, VE, a.lv, 2, t.channels, t.groups);
    V *x = reinterpret_cast<V *>(gc_smem) + threadIdx.x;         // every kGcThreads-th
    float4 *z = reinterpret_cast<float4 *>(gc_smem + a.keep * 16 * kGcThreads) + threadIdx.x;
    float2 *red = reinterpret_cast<float2 *>(gc_smem + l.red);
    float2 *part = reinterpret_cast<float2 *>(gc_smem + l.part), *cta = reinterpret_cast<float2 *>(gc_smem + l.cta);
    float *cst = reinterpret_cast<float *>(gc_smem + l.cst);     // -mean, a, beta, then what dx takes from the group's sums
    const long long px_bytes = a.C * static_cast<long long>(sizeof(T)), hop = t.step * px_bytes;
    const long long at = t.first * px_bytes + t.c * static_cast<int>(sizeof(T));
    const uint8_t *in = a.x.p + t.n * a.x.bstride + at, *din = a.dy.p + t.n * a.dy.bstride + at;
    dev::grid_dependency_wait();
#pragma unroll 4
    for (int j = 0; j < t.have; j++) {
        copy16(x + j * kGcThreads, in + j * hop);
        copy16(z + j * (VE / 4) * kGcThreads, din + j * hop);
    }
    float rstd = 0.0f;
    if (threadIdx.x < t.channels) {
        const int c = threadIdx.x, g = t.n * a.G + (t.c0 + c) / a.Cg;
        rstd = a.rstd[g];
        cst[c] = -a.mean[g];
        cst[t.channels + c] = a.gamma ? rstd * a.gamma[t.c0 + c] : rstd;
        cst[2 * t.channels + c] = a.beta ? a.beta[t.c0 + c] : 0.0f;
    }
    copies_done();
    __syncthreads();
    Channel<VE> k;
    if (t.on) {
        gn_load<VE>(k.shift, cst + t.v * VE);
        gn_load<VE>(k.a, cst + t.channels + t.v * VE);
        gn_load<VE>(k.beta, cst + 2 * t.channels + t.v * VE);
    }
    float2 s[2][kPairs<VE>];
#pragma unroll
    for (int i = 0; i < kPairs<VE>; i++) s[0][i] = s[1][i] = both(0.0f);
    const unsigned long long e = (static_cast<unsigned long long>(t.n) * a.HW + t.first) * a.C + t.c;
    const unsigned long long e_hop = static_cast<unsigned long long>(t.step) * a.C;
#pragma unroll 2
    for (int j = 0; j < t.have; j++) {
        float2 d[kPairs<VE>], dz[kPairs<VE>];
        float4 *zj = z + j * (VE / 4) * kGcThreads;
        gn_dz<T, VE, DROP, ACT>(x[j * kGcThreads], *reinterpret_cast<const V *>(zj), k, a.drop, e + j * e_hop, d, dz);
#pragma unroll
        for (int i = 0; i < kPairs<VE>; i++) {
            s[0][i] = __fadd2_rn(s[0][i], dz[i]);
            s[1][i] = __ffma2_rn(dz[i], d[i], s[1][i]);
        }
#pragma unroll
        for (int i = 0; i < VE / 4; i++)
            zj[i * kGcThreads] = make_float4(dz[2 * i].x, dz[2 * i].y, dz[2 * i + 1].x, dz[2 * i + 1].y);
    }
    const int rows = gc_rows<VE, 2>(t, a.lv, s, reinterpret_cast<float *>(red));
    __syncthreads();
    // the groups' sums of a dz and a dz d, a = rstd gamma
    const int segments = gc_groups(t, a.Cg, rows, part, [&](int r, int c) {
        return __fmul2_rn(red[r * t.channels + c], both(cst[t.channels + c]));
    });
    __syncthreads();
    const int own = threadIdx.x / a.Cg;                          // the group of channel threadIdx.x
    if (threadIdx.x < t.channels && threadIdx.x == own * a.Cg) {
        float2 v = make_float2(0.0f, 0.0f);
        for (int q = 0; q < segments; q++) v = __fadd2_rn(v, part[q * t.groups + own]);
        cta[own] = v;
    }
    if (a.cl > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    // over the cluster, a thread to a channel
    if (threadIdx.x < t.channels) {
        float2 v = a.cl > 1 ? remote(cta + own, 0) : cta[own];
        for (int r = 1; r < a.cl; r++) v = __fadd2_rn(v, remote(cta + own, r));
        const float share = -a.inv_m * a.drop.scale;
        cst[3 * t.channels + threadIdx.x] = share * v.x;
        cst[4 * t.channels + threadIdx.x] = share * rstd * rstd * v.y;
    }
    if (a.cl > 1) cluster_arrive();     // this CTA has read the others' memory
    __syncthreads();
    if (t.have) {
        float2 k0[kPairs<VE>], k1[kPairs<VE>];
        gn_load<VE>(k0, cst + 3 * t.channels + t.v * VE);
        gn_load<VE>(k1, cst + 4 * t.channels + t.v * VE);
#pragma unroll
        for (int i = 0; i < kPairs<VE>; i++) k.a[i] = __fmul2_rn(k.a[i], both(a.drop.scale));
        uint8_t *out = a.y.p + t.n * a.y.bstride + at;
#pragma unroll 4
        for (int j = 0; j < t.have; j++) {
            float2 d[kPairs<VE>];
            unpack2<T, VE>(x[j * kGcThreads], d);
#pragma unroll
            for (int i = 0; i < VE / 4; i++) {
                const float4 q = z[(j * (VE / 4) + i) * kGcThreads];
                d[2 * i] = __ffma2_rn(__fadd2_rn(d[2 * i], k.shift[2 * i]), k1[2 * i],
                                      __ffma2_rn(make_float2(q.x, q.y), k.a[2 * i], k0[2 * i]));
                d[2 * i + 1] = __ffma2_rn(__fadd2_rn(d[2 * i + 1], k.shift[2 * i + 1]), k1[2 * i + 1],
                                          __ffma2_rn(make_float2(q.z, q.w), k.a[2 * i + 1], k0[2 * i + 1]));
            }
            __stcs(reinterpret_cast<V *>(out + j * hop), pack2<T, VE>(d));
        }
    }
    // this CTA's {sum dz, sum dz xh} of its channels: a row of its own for dgamma and dbeta
    if (threadIdx.x < t.channels) {
        float2 v = make_float2(0.0f, 0.0f);
        for (int r = 0; r < rows; r++) v = __fadd2_rn(v, red[r * t.channels + threadIdx.x]);
        a.chan[(static_cast<long long>(t.n) * a.cl + t.rank) * a.C + t.c0 + threadIdx.x] =
            make_float2(v.x * a.drop.scale, v.y * a.drop.scale * rstd);
    }
    if (a.cl > 1) cluster_wait();
}

// ------------------------------------------------------------------ host side

cudaError_t gc_launch(void (*fn)(GnArgs), const GnArgs &a, int smem, void *stream)
{
    const cudaError_t e = gn_shared(reinterpret_cast<const void *>(fn));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.cl) * a.slabs * a.N, 1, 1);
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
    return gc_layout(keep, grad ? 16 + 4 * ve : 16, ve, a.lv, grad ? 2 : 1, a.gs * a.Cg, a.gs).total;
}

}  // namespace

// The widest slab from 128 bytes of a pixel down to 32 (a DRAM sector) whose
// image eight CTAs hold; then more CTAs a cluster, of fewer vectors each, where
// SMs would otherwise stay without their two.  Eight is the portable limit, and
// sixteen measured slower: their CTAs start together, so SMs wait (the gradient
// of 8 x 128 x 128 x 512 bf16 in 216 us, 147 us by passes).
bool gn_cluster_plan(GnArgs &args, size_t es, bool grad)
{
    GnArgs a = args;
#ifdef X_NOCLUSTER
    return false;
#endif
    const int ve = 16 / static_cast<int>(es);
    int base = 1;   // groups whose channels fill whole vectors
    while (static_cast<long long>(base) * a.Cg % ve) base++;
    const long long base_vecs = static_cast<long long>(base) * a.Cg / ve;
    if (base_vecs > kGcMaxVecs) return false;
    for (int m = std::max(1, 8 / static_cast<int>(base_vecs)); m >= 1; m--) {
        a.lv = static_cast<int>(base_vecs) * m;
        a.gs = base * m;
        if (a.lv < 2 && a.gs < a.G) break;
        const int row = kGcWarps * (32 / a.lv), rows = static_cast<int>((a.HW + row - 1) / row);
        int keep = 1;
        while (gc_bytes(a, es, grad, keep + 1) <= kGnShared) keep++;
        int cl = (rows + keep - 1) / keep;
        if (cl > kGnMaxCluster) continue;
        a.slabs = (a.G + a.gs - 1) / a.gs;
        const long long units = static_cast<long long>(a.N) * a.slabs;
        if (units > 0x7fffffffLL / kGnMaxCluster) return false;
        cl = std::max(cl, static_cast<int>(std::min<long long>(kGnMaxCluster, (kGcCtas * kGnSms + units - 1) / units)));
        a.keep = (rows + cl - 1) / cl;
        a.cl = (rows + a.keep - 1) / a.keep;
        a.rows = a.N * a.cl;
        args = a;
        return true;
    }
    return false;
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
