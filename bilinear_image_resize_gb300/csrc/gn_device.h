// Group norm: what its kernels share.  group_norm.cu has the entry points and
// the kernels for images of any size, gn_cluster.cu those that keep an image's
// channels on chip between the statistics and their use.
#pragma once

#include <type_traits>

#include "map_ops.h"

namespace rz {

using maps::both;
using maps::kPairs;
using maps::pack2;
using maps::unpack2;

constexpr float kLog2e = 1.44269504f;
constexpr int kGnSms = 152;
constexpr int kGnMaxChunks = 4 * kGnSms;  // chunks of an image, pass kernels
constexpr int kGnMaxCluster = 8;    // CTAs a cluster (the portable limit)

struct GnArgs {
    maps::View x, dy, y;        // y: the output (dx for the gradient)
    const float *gamma, *beta;  // may be null (1 and 0)
    float *mean, *rstd;         // [N][G]
    float *dgamma, *dbeta;      // [C], may be null
    int N, C, G, Cg;
    unsigned HW, W;             // pixels an image and a row
    int joined;                 // rows follow one another in every map
    int act;
    float eps, inv_m;
    maps::Drop drop;
    float2 *chan;               // [N][C]: {mean, squared distances}; [rows][C]: {sum dz, sum dz xh}
    int rows;
    // cluster kernels: groups and vectors a slab, slabs an image, CTAs a cluster, vectors a thread keeps, clusters
    int gs, lv, slabs, cl, keep, clusters;
    // pass kernels: chunks of an image and their pixels
    float2 *part;               // [N][chunks][C]: a chunk's share of chan
    int chunks;
    unsigned chunk_px;
};

// Cluster kernels (gn_cluster.cu): whether an image's slab fits a cluster; sets
// gs, lv, slabs, cl, keep, clusters and rows.
cudaError_t gn_cluster_plan(GnArgs &a, size_t es, bool grad, bool *fits);
cudaError_t gn_cluster_forward(const GnArgs &a, int dtype, bool drop, void *stream);
cudaError_t gn_cluster_backward(const GnArgs &a, int dtype, bool drop, void *stream);

// Pass kernels (gn_passes.h), one translation unit a type.
template <class T> cudaError_t gn_passes_forward(const GnArgs &a, int ve, bool drop, void *stream);
template <class T> cudaError_t gn_passes_backward(const GnArgs &a, int ve, bool drop, void *stream);

template <int V> using Int = std::integral_constant<int, V>;

// Calls fn(DROP, ACT) for a call's dropout and activation.
template <class Fn>
cudaError_t gn_kinds(int act, bool drop, Fn fn)
{
    auto on = [&](auto d) {
        if (act == RZ_ACT_SILU) return fn(d, Int<RZ_ACT_SILU>{});
        return act == RZ_ACT_GELU ? fn(d, Int<RZ_ACT_GELU>{}) : fn(d, Int<RZ_ACT_NONE>{});
    };
    return drop ? on(std::true_type{}) : on(std::false_type{});
}

// 1 / (1 + 2^(-z log2 e)) by the GPU's exp2 and reciprocal.  Rounding the
// exponent costs up to |z| units of 2^-24 of the value where z is below 0 (4 at
// -4, 31 at -40; 2 above 0), and below -87.3 the reciprocal's subnormal becomes
// 0, for 1.1e-36 at most.  expf and a division are within 3 units everywhere,
// but the float32 maps that could show it took 18% longer (64 x 32 x 32 x 256
// forward 36.8 us against 31.1, gradient 61.4 against 52.5) and 16-bit ones,
// which cannot, 40 to 57% (16 x 64 x 64 x 320 with dropout 53.8 against 36.4).
__device__ __forceinline__ float2 sigmoid2(float2 z)
{
    const float2 t = __fmul2_rn(z, both(-kLog2e));
    const float2 q = __fadd2_rn(make_float2(maps::exp2_approx(t.x), maps::exp2_approx(t.y)), both(1.0f));
    return make_float2(maps::rcp_approx(q.x), maps::rcp_approx(q.y));
}

template <int ACT>
__device__ __forceinline__ float2 act_value2(float2 z)
{
    if constexpr (ACT == RZ_ACT_SILU) return __fmul2_rn(z, sigmoid2(z));
    if constexpr (ACT == RZ_ACT_GELU) return make_float2(maps::gelu(z.x), maps::gelu(z.y));
    return z;
}

// silu'(z) = s + s z (1 - s)
template <int ACT>
__device__ __forceinline__ float2 act_slope2(float2 z)
{
    if constexpr (ACT == RZ_ACT_SILU) {
        const float2 s = sigmoid2(z);
        return __ffma2_rn(s, __fmul2_rn(z, __ffma2_rn(s, both(-1.0f), both(1.0f))), s);
    }
    if constexpr (ACT == RZ_ACT_GELU) return make_float2(maps::gelu_slope(z.x), maps::gelu_slope(z.y));
    return both(1.0f);
}

// Zeroes the dropped ones of the VE elements from lane `lane` of a block; the
// scale of the kept ones is left to the caller.
template <int VE>
__device__ __forceinline__ void drop2(float2 (&f)[kPairs<VE>], unsigned long long block, unsigned lane, const maps::Drop &d)
{
    bool keep[VE];
    maps::kept<VE>(keep, block, lane, d);
#pragma unroll
    for (int i = 0; i < VE; i++) {
        float &v = (i & 1) ? f[i / 2].y : f[i / 2].x;
        v = keep[i] ? v : 0.0f;
    }
}

// The thread's vector of channels: d = x + shift, z = d a + beta, with
// shift = -mean and a = rstd gamma.
template <int VE>
struct Channel {
    float2 shift[kPairs<VE>], a[kPairs<VE>], beta[kPairs<VE>];
};

// VE channels' values from an array of them.
template <int VE>
__device__ __forceinline__ void gn_load(float2 (&f)[kPairs<VE>], const float *from)
{
    if constexpr (VE == 1) {
        f[0] = make_float2(*from, 0.0f);
    } else {
#pragma unroll
        for (int i = 0; i < VE / 4; i++) {
            const float4 v = reinterpret_cast<const float4 *>(from)[i];
            f[2 * i] = make_float2(v.x, v.y);
            f[2 * i + 1] = make_float2(v.z, v.w);
        }
    }
}
template <int VE>
__device__ __forceinline__ void gn_save(float *to, const float2 (&f)[kPairs<VE>])
{
    if constexpr (VE == 1) {
        *to = f[0].x;
    } else {
#pragma unroll
        for (int i = 0; i < VE / 4; i++)
            reinterpret_cast<float4 *>(to)[i] = make_float4(f[2 * i].x, f[2 * i].y, f[2 * i + 1].x, f[2 * i + 1].y);
    }
}

// One vector forward: x in, y out.
template <class T, int VE, bool DROP, int ACT>
__device__ __forceinline__ maps::Raw<T, VE> gn_value(const maps::Raw<T, VE> &x, const Channel<VE> &k,
                                                     const maps::Drop &drop, unsigned long long block,
                                                     unsigned lane)
{
    float2 f[kPairs<VE>];
    unpack2<T, VE>(x, f);
#pragma unroll
    for (int i = 0; i < kPairs<VE>; i++) {
        f[i] = act_value2<ACT>(__ffma2_rn(__fadd2_rn(f[i], k.shift[i]), k.a[i], k.beta[i]));
        if (DROP) f[i] = __fmul2_rn(f[i], both(drop.scale));
    }
    if (DROP) drop2<VE>(f, block, lane, drop);
    return pack2<T, VE>(f);
}

// One vector backward: x and dy in; d = x - mean and dz out, dz short of the
// dropout's scale.
template <class T, int VE, bool DROP, int ACT>
__device__ __forceinline__ void gn_dz(const maps::Raw<T, VE> &x, const maps::Raw<T, VE> &dy, const Channel<VE> &k,
                                      const maps::Drop &drop, unsigned long long block, unsigned lane,
                                      float2 (&d)[kPairs<VE>], float2 (&dz)[kPairs<VE>])
{
    unpack2<T, VE>(x, d);
    unpack2<T, VE>(dy, dz);
    if (DROP) drop2<VE>(dz, block, lane, drop);
#pragma unroll
    for (int i = 0; i < kPairs<VE>; i++) {
        d[i] = __fadd2_rn(d[i], k.shift[i]);
        if (ACT != RZ_ACT_NONE) dz[i] = __fmul2_rn(dz[i], act_slope2<ACT>(__ffma2_rn(d[i], k.a[i], k.beta[i])));
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace rz
