// Group norm with an activation and dropout on channels-last maps, and its
// gradient.  For image n and group g of Cg = C / G channels, M = H W Cg values:
//   mean = sum x / M,  var = sum (x - mean)^2 / M,  rstd = (var + eps)^-1/2
//   xh = (x - mean) rstd,  z = xh gamma_c + beta_c,  y = drop(act(z))
// and, with da = drop(dy) under the same mask and dz = da act'(z),
//   dbeta_c = sum dz,  dgamma_c = sum dz xh  (over images and pixels)
//   A = sum gamma dz / M,  B = sum gamma dz xh / M  (over the group)
//   dx = rstd (gamma dz - A - xh B).
//
// A call's floor is each map read or written once; the arithmetic (the generator,
// the sigmoid) comes near it or above.  Small images are kept on chip between the two passes
// (gn_cluster.cu), others are read twice, the second time out of L2 as far as
// it holds them (gn_passes.h).
#include <algorithm>
#include <initializer_list>
#include <mutex>

#include "gn_device.h"
#include "map_ops.h"
#include "rz_device.h"
#include "rz_internal.h"
#include "token_rules.h"

namespace rz {
namespace {

using namespace maps;
using dev::grid_dependency_wait;
using dev::grid_launch_dependents;

// dgamma and dbeta: the rows' sums, 32 channels a block, each of its warps a
// row in eight, joined in order.
__global__ void __launch_bounds__(256) k_gn_params(const GnArgs a)
{
    __shared__ float2 sh[8][32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float2 s = make_float2(0.0f, 0.0f);
    if (c < a.C) {
#pragma unroll 4
        for (int r = w; r < a.rows; r += 8) s = __fadd2_rn(s, a.chan[static_cast<long long>(r) * a.C + c]);
    }
    sh[w][lane] = s;
    __syncthreads();
    if (w || c >= a.C) return;
#pragma unroll
    for (int i = 1; i < 8; i++) s = __fadd2_rn(s, sh[i][lane]);
    if (a.dbeta) a.dbeta[c] = s.x;
    if (a.dgamma) a.dgamma[c] = s.y;
}

// ------------------------------------------------------------------ host side

constexpr int kGnBlock = 256;   // threads of a pass kernel's CTA

// Chunks of an image for the pass kernels: as many CTAs over the call as are
// resident at once (four an SM forward, three in the gradient; two waves of the
// gradient's measured 47.0 against 42.0 us on 16 x 64 x 64 x 320 bf16, 24.8
// against 21.4 on 1 x 256 x 256 x 128), and at least eight pixels a thread.
void gn_passes_plan(GnArgs &a, int ve, bool grad)
{
    const long long vecs = a.C / ve, blocks = (vecs + kGnBlock - 1) / kGnBlock;
    const long long lanes = kGnBlock / std::min<long long>(vecs, kGnBlock);
    const long long want = std::max(1LL, (grad ? 3 : 4) * kGnSms / (blocks * a.N));
    const long long chunks = std::clamp(a.HW / (8 * lanes), 1LL, std::min<long long>(want, kGnMaxChunks));
    a.chunk_px = static_cast<unsigned>((a.HW + chunks - 1) / chunks);
    a.chunks = static_cast<int>((a.HW + a.chunk_px - 1) / a.chunk_px);
}

struct GnWorkspace {
    size_t part, chan, stat, total;
};

GnWorkspace gn_workspace(const GnArgs &a)
{
    auto up = [](size_t v) { return (v + 255) & ~size_t{255}; };
    GnWorkspace w;
    w.part = 0;
    w.chan = up(sizeof(float2) * a.N * static_cast<size_t>(a.chunks) * a.C);
    w.stat = w.chan + up(sizeof(float2) * kGnMaxCluster * a.N * static_cast<size_t>(a.C));
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
    // the grid's depth, and statistics that the kernels number in 32 bits
    if (d->N > 65535 || static_cast<long long>(d->N) * d->groups > 0x7fffffffLL) return RZ_ERR_UNSUPPORTED;
    return RZ_OK;
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

cudaError_t gn_passes(const GnArgs &a, int dtype, int ve, bool drop, bool grad, void *stream)
{
    const auto run = [&](auto forward, auto backward) { return (grad ? backward : forward)(a, ve, drop, stream); };
    if (dtype == RZ_F32) return run(gn_passes_forward<float>, gn_passes_backward<float>);
    if (dtype == RZ_BF16) return run(gn_passes_forward<__nv_bfloat16>, gn_passes_backward<__nv_bfloat16>);
    return run(gn_passes_forward<__half>, gn_passes_backward<__half>);
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

namespace rz {

cudaError_t maps::shared_opt_in(const void *fn, int bytes)
{
    static std::mutex mu;
    static rules::Granted granted;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    return static_cast<cudaError_t>(granted.have(dev, fn, bytes, [fn](int n) {
        return static_cast<int>(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, n));
    }));
}

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
    // enough for every vector width, which the maps' alignment decides
    for (int ve : {8, 4, 1})
        for (bool grad : {false, true})
            if (a.C % ve == 0) {
                gn_passes_plan(a, ve, grad);
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
    gn_passes_plan(a, ve, false);
    const GnWorkspace w = gn_workspace(a);
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 || workspace_bytes < w.total) return RZ_ERR_ARG;
    uint8_t *base = static_cast<uint8_t *>(workspace);
    a.part = reinterpret_cast<float2 *>(base + w.part);
    a.chan = reinterpret_cast<float2 *>(base + w.chan);
    float *stat = reinterpret_cast<float *>(base + w.stat);
    a.gamma = gamma;
    a.beta = beta;
    a.mean = mean ? mean : stat;
    a.rstd = rstd ? rstd : stat + static_cast<size_t>(a.N) * a.G;
    a.drop = maps::make_drop(drop);
    const bool dropping = maps::drop_threshold(drop) != 0;
    bool cluster = false;
    if (a.joined && ve * s.es == 16) {
        const cudaError_t e = gn_cluster_plan(a, s.es, false, &cluster);
        if (e != cudaSuccess) return gn_status(e);
    }
    return gn_status(cluster ? gn_cluster_forward(a, d->dtype, dropping, stream)
                             : gn_passes(a, d->dtype, ve, dropping, false, stream));
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
    gn_passes_plan(a, ve, true);
    a.rows = a.N;
    const GnWorkspace w = gn_workspace(a);
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 || workspace_bytes < w.total) return RZ_ERR_ARG;
    uint8_t *base = static_cast<uint8_t *>(workspace);
    a.part = reinterpret_cast<float2 *>(base + w.part);
    a.chan = reinterpret_cast<float2 *>(base + w.chan);
    a.gamma = gamma;
    a.beta = beta;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    a.drop = maps::make_drop(drop);
    const bool dropping = maps::drop_threshold(drop) != 0;
    bool cluster = false;
    cudaError_t e = cudaSuccess;
    if (a.joined && ve * s.es == 16) e = gn_cluster_plan(a, s.es, true, &cluster);
    if (e == cudaSuccess)
        e = cluster ? gn_cluster_backward(a, d->dtype, dropping, stream)
                    : gn_passes(a, d->dtype, ve, dropping, true, stream);
    if (e == cudaSuccess && (a.dgamma || a.dbeta))
        e = maps::launch(k_gn_params, dim3((a.C + 31) / 32), 256, 0, stream, a);
    return gn_status(e);
}

}  // extern "C"
