// Bilinear resize of channels-last maps with any number of channels, and its
// gradient, under the clamp rule and with the float weights of the library's
// resizes (axis_linear in api.cu): output index d samples x = num / den,
// num = (2d + 1) n_in - n_out, den = 2 n_out; near tap i = floor(x), far tap
// i + 1, both clamped, far weight u = (num - i den) / den.
//
// Forward: dst[n] = base[n] + resize(src[n]); one source image may serve every
// n (a position table).  Gradient: source index s is read by the outputs d
// with floor(x_d) in {s - 1, s}, a range whose ends are exact integer
// divisions, so each source value gathers its own terms in order and nothing
// is added atomically.
#include <algorithm>

#include "map_ops.h"
#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {

using namespace maps;

constexpr int kMapThreads = 256;

struct ResampleArgs {
    View src, base, dst;        // gradient: dst is ddst, src is dsrc; base.p null: none
    int N, src_n, H, W, OH, OW, C;
    float *sum;                 // gradient of a table: [OH][OW][C], ddst summed over the images
};

// Taps of output index d: near, far and the far tap's weight.
struct Tap {
    int a, b;
    float u;
};

__device__ __forceinline__ Tap tap(int d, int n_in, int n_out)
{
    const long long num = (2LL * d + 1) * n_in - n_out;
    const int den = 2 * n_out, i = dev::floor_div_exact(num, den);
    const int r = static_cast<int>(num - static_cast<long long>(i) * den);
    return {max(i, 0), min(i + 1, n_in - 1), __fdiv_rn(static_cast<float>(r), static_cast<float>(den))};
}

// Outputs [lo, hi) that read source index s, and the weight with which d does.
__device__ __forceinline__ long long ceil_div(long long a, long long b) { return a >= 0 ? (a + b - 1) / b : -(-a / b); }
__device__ __forceinline__ int2 readers(int s, int n_in, int n_out)
{
    const long long lo = s == 0 ? 0 : ceil_div((2LL * s - 1) * n_out - n_in, 2LL * n_in);
    const long long hi = s == n_in - 1 ? n_out : ceil_div((2LL * s + 3) * n_out - n_in, 2LL * n_in);
    return make_int2(static_cast<int>(max(lo, 0LL)), static_cast<int>(min(hi, static_cast<long long>(n_out))));
}
__device__ __forceinline__ float tap_weight(int d, int s, int n_in, int n_out)
{
    const Tap t = tap(d, n_in, n_out);
    return (t.a == s ? 1.0f - t.u : 0.0f) + (t.b == s ? t.u : 0.0f);
}

template <class T, int VE>
__device__ __forceinline__ const Raw<T, VE> *map_at(const View &v, long long n, int y, int x, int C, int c)
{
    return reinterpret_cast<const Raw<T, VE> *>(v.p + n * v.bstride + y * v.pitch +
                                                (static_cast<long long>(x) * C + c) * static_cast<int>(sizeof(T)));
}

// A thread forms one vector of channels of one output pixel: once for every
// image where the source is one table, else for image blockIdx.z.
template <class S, class T, int VE>
__global__ void __launch_bounds__(kMapThreads) k_resize_map(const ResampleArgs a)
{
    dev::grid_launch_dependents();
    dev::grid_dependency_wait();
    const int vecs = a.C / VE;
    const long long i = blockIdx.x * static_cast<long long>(kMapThreads) + threadIdx.x;
    if (i >= static_cast<long long>(a.OW) * vecs) return;
    const int ox = static_cast<int>(i / vecs), c = static_cast<int>(i - static_cast<long long>(ox) * vecs) * VE;
    const Tap tx = tap(ox, a.W, a.OW);
    for (int oy = blockIdx.y; oy < a.OH; oy += gridDim.y) {
        const Tap ty = tap(oy, a.H, a.OH);
        for (int s = blockIdx.z; s < a.src_n; s += gridDim.z) {
            float p[VE], q[VE], out[VE];
            unpack<S, VE>(*map_at<S, VE>(a.src, s, ty.a, tx.a, a.C, c), p);
            unpack<S, VE>(*map_at<S, VE>(a.src, s, ty.a, tx.b, a.C, c), q);
#pragma unroll
            for (int k = 0; k < VE; k++) out[k] = fmaf(tx.u, q[k] - p[k], p[k]);
            unpack<S, VE>(*map_at<S, VE>(a.src, s, ty.b, tx.a, a.C, c), p);
            unpack<S, VE>(*map_at<S, VE>(a.src, s, ty.b, tx.b, a.C, c), q);
#pragma unroll
            for (int k = 0; k < VE; k++) out[k] = fmaf(ty.u, fmaf(tx.u, q[k] - p[k], p[k]) - out[k], out[k]);
            const int n0 = a.src_n == 1 ? 0 : s, n1 = a.src_n == 1 ? a.N : s + 1;
            for (int n = n0; n < n1; n++) {
                float f[VE];
#pragma unroll
                for (int k = 0; k < VE; k++) f[k] = out[k];
                if (a.base.p) {
                    unpack<T, VE>(__ldcs(map_at<T, VE>(a.base, n, oy, ox, a.C, c)), p);
#pragma unroll
                    for (int k = 0; k < VE; k++) f[k] += p[k];
                }
                __stcs(const_cast<Raw<T, VE> *>(map_at<T, VE>(a.dst, n, oy, ox, a.C, c)), pack<T, VE>(f));
            }
        }
    }
}

// sum[y][x][c] = the images' ddst added up in order.
template <class T, int VE>
__global__ void __launch_bounds__(kMapThreads) k_sum_images(const ResampleArgs a)
{
    dev::grid_launch_dependents();
    dev::grid_dependency_wait();
    const int vecs = a.C / VE;
    const long long i = blockIdx.x * static_cast<long long>(kMapThreads) + threadIdx.x;
    if (i >= static_cast<long long>(a.OW) * vecs) return;
    const int ox = static_cast<int>(i / vecs), c = static_cast<int>(i - static_cast<long long>(ox) * vecs) * VE;
    for (int oy = blockIdx.y; oy < a.OH; oy += gridDim.y) {
        float s[VE];
#pragma unroll
        for (int k = 0; k < VE; k++) s[k] = 0.0f;
        for (int n = 0; n < a.N; n++) {
            float f[VE];
            unpack<T, VE>(__ldcs(map_at<T, VE>(a.dst, n, oy, ox, a.C, c)), f);
#pragma unroll
            for (int k = 0; k < VE; k++) s[k] += f[k];
        }
        float *out = a.sum + (static_cast<long long>(oy) * a.OW + ox) * a.C + c;
#pragma unroll
        for (int k = 0; k < VE; k++) out[k] = s[k];
    }
}

// A thread gathers one vector of channels of one source pixel.
template <class S, class T, int VE>
__global__ void __launch_bounds__(kMapThreads) k_resize_map_grad(const ResampleArgs a)
{
    dev::grid_launch_dependents();
    dev::grid_dependency_wait();
    const int vecs = a.C / VE;
    const long long i = blockIdx.x * static_cast<long long>(kMapThreads) + threadIdx.x;
    if (i >= static_cast<long long>(a.W) * vecs) return;
    const int x = static_cast<int>(i / vecs), c = static_cast<int>(i - static_cast<long long>(x) * vecs) * VE;
    const int2 rx = readers(x, a.W, a.OW);
    for (int y = blockIdx.y; y < a.H; y += gridDim.y) {
        const int2 ry = readers(y, a.H, a.OH);
        for (int n = blockIdx.z; n < a.src_n; n += gridDim.z) {
            float s[VE];
#pragma unroll
            for (int k = 0; k < VE; k++) s[k] = 0.0f;
            for (int oy = ry.x; oy < ry.y; oy++) {
                float h[VE];
#pragma unroll
                for (int k = 0; k < VE; k++) h[k] = 0.0f;
                for (int ox = rx.x; ox < rx.y; ox++) {
                    const float w = tap_weight(ox, x, a.W, a.OW);
                    float f[VE];
                    unpack<T, VE>(*map_at<T, VE>(a.dst, n, oy, ox, a.C, c), f);
#pragma unroll
                    for (int k = 0; k < VE; k++) h[k] = fmaf(w, f[k], h[k]);
                }
                const float w = tap_weight(oy, y, a.H, a.OH);
#pragma unroll
                for (int k = 0; k < VE; k++) s[k] = fmaf(w, h[k], s[k]);
            }
            *const_cast<Raw<S, VE> *>(map_at<S, VE>(a.src, n, y, x, a.C, c)) = pack<S, VE>(s);
        }
    }
}

// ------------------------------------------------------------------ host side

struct Checked {
    Shape src, dst;
};

int resample_check(const rz_resample *d, Checked *s)
{
    if (!d) return RZ_ERR_ARG;
    s->src = {d->src_n, d->H, d->W, d->C, dtype_size(d->src_dtype)};
    s->dst = {d->N, d->out_h, d->out_w, d->C, dtype_size(d->dtype)};
    if (!s->src.es || !s->dst.es || !shape_ok(s->src) || !shape_ok(s->dst)) return RZ_ERR_ARG;
    if (d->src_dtype != d->dtype && d->src_dtype != RZ_F32) return RZ_ERR_ARG;
    if (d->H < 1 || d->W < 1 || d->H > RZ_MAX_DIM || d->W > RZ_MAX_DIM || d->out_h > RZ_MAX_DIM ||
        d->out_w > RZ_MAX_DIM)
        return RZ_ERR_ARG;
    return d->src_n == 1 || d->src_n == d->N ? RZ_OK : RZ_ERR_ARG;
}

void resample_fill(const rz_resample *d, ResampleArgs &a)
{
    a = ResampleArgs{};
    a.N = d->N;
    a.src_n = d->src_n;
    a.H = d->H;
    a.W = d->W;
    a.OH = d->out_h;
    a.OW = d->out_w;
    a.C = d->C;
}

dim3 map_grid(int W, int vecs, int rows, int images)
{
    return dim3(static_cast<unsigned>((static_cast<long long>(W) * vecs + kMapThreads - 1) / kMapThreads),
                static_cast<unsigned>(std::min(rows, 65535)), static_cast<unsigned>(std::min(images, 65535)));
}

// Calls fn(S{}, T{}, VE) for the map types; VE is the elements of 16 bytes of
// the wider type where `wide`.
template <class Fn>
cudaError_t resample_dispatch(const rz_resample *d, bool wide, Fn fn)
{
    auto width = [&](auto s, auto t) {
        constexpr int V = 16 / static_cast<int>(sizeof(s));
        return wide ? fn(s, t, std::integral_constant<int, V>{}) : fn(s, t, std::integral_constant<int, 1>{});
    };
    if (d->dtype == RZ_F32) return width(float{}, float{});
    if (d->dtype == RZ_BF16)
        return d->src_dtype == RZ_F32 ? width(float{}, __nv_bfloat16{}) : width(__nv_bfloat16{}, __nv_bfloat16{});
    return d->src_dtype == RZ_F32 ? width(float{}, __half{}) : width(__half{}, __half{});
}

int resample_status(cudaError_t e)
{
    if (e == cudaSuccess) return RZ_OK;
    record_cuda_error(static_cast<int>(e));
    return RZ_ERR_CUDA;
}

size_t sum_bytes(const rz_resample *d)
{
    return d->src_n == 1 && d->N > 1 ? sizeof(float) * d->out_h * static_cast<size_t>(d->out_w) * d->C : 0;
}

}  // namespace
}  // namespace rz

using namespace rz;

extern "C" {

int resize_map(const rz_resample *d, const rz_map *src, const rz_map *base, const rz_map *dst, void *stream)
{
    Checked s;
    const int rc = resample_check(d, &s);
    if (rc != RZ_OK) return rc;
    if (s.dst.empty()) return RZ_OK;
    if (!maps::map_ok(src, s.src) || !maps::map_ok(dst, s.dst) || (base && !maps::map_ok(base, s.dst)))
        return RZ_ERR_ARG;
    if (maps::map_overlap(*src, s.src, *dst, s.dst)) return RZ_ERR_ARG;
    if (base && maps::map_overlap(*base, s.dst, *dst, s.dst) && !maps::map_same(*base, *dst, s.dst)) return RZ_ERR_ARG;
    ResampleArgs a;
    resample_fill(d, a);
    a.src = maps::view(src);
    a.dst = maps::view(dst);
    if (base) a.base = maps::view(base);
    const size_t ve = 16 / s.src.es;
    const bool wide = d->C % ve == 0 && maps::map_aligned(*src, s.src, 16) &&
                      maps::map_aligned(*dst, s.dst, ve * s.dst.es) &&
                      (!base || maps::map_aligned(*base, s.dst, ve * s.dst.es));
    return resample_status(resample_dispatch(d, wide, [&](auto ts, auto td, auto v) {
        constexpr int V = decltype(v)::value;
        return maps::launch(k_resize_map<decltype(ts), decltype(td), V>, map_grid(a.OW, a.C / V, a.OH, a.src_n),
                            kMapThreads, 0, stream, a);
    }));
}

int resize_map_grad_workspace(const rz_resample *d, size_t *bytes)
{
    Checked s;
    const int rc = resample_check(d, &s);
    if (rc != RZ_OK) return rc;
    if (!bytes) return RZ_ERR_ARG;
    *bytes = sum_bytes(d);
    return RZ_OK;
}

int resize_map_grad(const rz_resample *d, const rz_map *ddst, const rz_map *dsrc, void *workspace,
                    size_t workspace_bytes, void *stream)
{
    Checked s;
    const int rc = resample_check(d, &s);
    if (rc != RZ_OK) return rc;
    if (s.src.empty()) return RZ_OK;
    if (!maps::map_ok(dsrc, s.src)) return RZ_ERR_ARG;
    ResampleArgs a;
    resample_fill(d, a);
    a.src = maps::view(dsrc);
    size_t ve = 16 / s.src.es;
    bool wide = d->C % ve == 0 && maps::map_aligned(*dsrc, s.src, 16);
    if (s.dst.empty()) {
        a.OH = a.OW = 0;   // no reader: zeros
    } else {
        if (!maps::map_ok(ddst, s.dst) || maps::map_overlap(*ddst, s.dst, *dsrc, s.src)) return RZ_ERR_ARG;
        a.dst = maps::view(ddst);
        wide = wide && maps::map_aligned(*ddst, s.dst, ve * s.dst.es);
        const size_t need = sum_bytes(d);
        if (need) {
            if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 || workspace_bytes < need) return RZ_ERR_ARG;
            a.sum = static_cast<float *>(workspace);
        }
    }
    return resample_status(resample_dispatch(d, wide, [&](auto ts, auto td, auto v) {
        using S = decltype(ts);
        using T = decltype(td);
        constexpr int V = decltype(v)::value;
        ResampleArgs g = a;
        if (a.sum) {
            const cudaError_t e = maps::launch(k_sum_images<T, V>, map_grid(a.OW, a.C / V, a.OH, 1), kMapThreads, 0,
                                               stream, a);
            if (e != cudaSuccess) return e;
            g.dst = {reinterpret_cast<uint8_t *>(a.sum), static_cast<long long>(sizeof(float)) * a.OW * a.C, 0};
            return maps::launch(k_resize_map_grad<S, float, V>, map_grid(a.W, a.C / V, a.H, 1), kMapThreads, 0,
                                stream, g);
        }
        return maps::launch(k_resize_map_grad<S, T, V>, map_grid(a.W, a.C / V, a.H, a.src_n), kMapThreads, 0, stream,
                            g);
    }));
}

}  // extern "C"
