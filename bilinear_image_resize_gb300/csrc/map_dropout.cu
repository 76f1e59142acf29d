// Dropout of a channels-last map, and the add of a residual that follows it in
// a block: y = drop(x) + residual, the mask made from a counter as the map
// passes through (map_ops.h), never stored.  One read of each input and one
// write: memory bounds it where the generator's arithmetic (about 70 integer
// instructions for eight elements) stays below it.
#include <algorithm>

#include "map_ops.h"
#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {

using namespace maps;

constexpr int kDropThreads = 256;

struct DropArgs {
    View x, r, y;               // r.p null: no residual
    unsigned long long rows;    // N H rows, or one for the whole map
    unsigned long long row;     // elements of a row
    unsigned H;                 // rows an image
    Drop drop;
    int dropping;
};

// Thread i takes vectors i, i + stride, ... of the map's elements.
template <class T, int VE>
__global__ void __launch_bounds__(kDropThreads) k_dropout(const DropArgs a)
{
    dev::grid_launch_dependents();
    dev::grid_dependency_wait();
    const unsigned long long per_row = a.row / VE, total = a.rows * per_row;
    for (unsigned long long v = blockIdx.x * static_cast<unsigned long long>(kDropThreads) + threadIdx.x; v < total;
         v += static_cast<unsigned long long>(gridDim.x) * kDropThreads) {
        const unsigned long long row = a.rows == 1 ? 0 : v / per_row;
        const unsigned long long n = a.rows == 1 ? 0 : row / a.H, h = row - n * a.H;
        const long long j = static_cast<long long>(v - row * per_row) * VE * static_cast<long long>(sizeof(T));
        const auto in = [&](const View &m) {
            return reinterpret_cast<const Raw<T, VE> *>(m.p + n * m.bstride + h * m.pitch + j);
        };
        float f[VE];
        unpack<T, VE>(__ldcs(in(a.x)), f);
        if (a.dropping) drop_elements<VE>(f, v * VE, a.drop);
        if (a.r.p) {
            float r[VE];
            unpack<T, VE>(__ldcs(in(a.r)), r);
#pragma unroll
            for (int i = 0; i < VE; i++) f[i] += r[i];
        }
        __stcs(const_cast<Raw<T, VE> *>(in(a.y)), pack<T, VE>(f));
    }
}

template <class T, int VE>
cudaError_t drop_launch(const DropArgs &a, void *stream)
{
    const unsigned long long blocks = (a.rows * (a.row / VE) + kDropThreads - 1) / kDropThreads;
    return launch(k_dropout<T, VE>, dim3(static_cast<unsigned>(std::min(blocks, 152ull * 64))), kDropThreads, 0,
                  stream, a);
}

}  // namespace
}  // namespace rz

using namespace rz;

extern "C" {

int map_dropout(const rz_map *x, const rz_map *residual, const rz_map *y, int N, int H, int W, int C, int dtype,
                const rz_drop *drop, void *stream)
{
    const maps::Shape s{N, H, W, C, maps::dtype_size(dtype)};
    if (!s.es || !maps::shape_ok(s) || !drop || !maps::drop_ok(drop)) return RZ_ERR_ARG;
    if (s.empty()) return RZ_OK;
    if (!maps::map_ok(x, s) || !maps::map_ok(y, s) || (residual && !maps::map_ok(residual, s))) return RZ_ERR_ARG;
    if (!maps::map_same(*x, *y, s) && maps::map_overlap(*x, s, *y, s)) return RZ_ERR_ARG;
    if (residual && !maps::map_same(*residual, *y, s) && maps::map_overlap(*residual, s, *y, s)) return RZ_ERR_ARG;
    const auto whole = [&](const rz_map *m) {
        return !m || (maps::rows_joined(*m, s) && (s.N == 1 || m->batch_stride == s.H * s.row()));
    };
    DropArgs a{};
    a.x = maps::view(x);
    a.y = maps::view(y);
    if (residual) a.r = maps::view(residual);
    const bool one = whole(x) && whole(y) && whole(residual);
    a.rows = one ? 1 : static_cast<unsigned long long>(s.N) * s.H;
    a.row = static_cast<unsigned long long>(s.W) * s.C * (one ? s.N * s.H : 1);
    a.H = one ? 1 : static_cast<unsigned>(s.H);
    a.drop = maps::make_drop(drop);
    a.dropping = maps::drop_threshold(drop) != 0;
    const int ve = 16 / static_cast<int>(s.es);
    const bool wide = a.row % ve == 0 && maps::map_aligned(*x, s, 16) && maps::map_aligned(*y, s, 16) &&
                      (!residual || maps::map_aligned(*residual, s, 16));
    cudaError_t e;
    if (dtype == RZ_F32)
        e = wide ? drop_launch<float, 4>(a, stream) : drop_launch<float, 1>(a, stream);
    else if (dtype == RZ_BF16)
        e = wide ? drop_launch<__nv_bfloat16, 8>(a, stream) : drop_launch<__nv_bfloat16, 1>(a, stream);
    else
        e = wide ? drop_launch<__half, 8>(a, stream) : drop_launch<__half, 1>(a, stream);
    if (e == cudaSuccess) return RZ_OK;
    record_cuda_error(static_cast<int>(e));
    return RZ_ERR_CUDA;
}

}  // extern "C"
