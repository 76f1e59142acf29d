// Dropout of a channels-last map, and the add of a residual that follows it in
// a block: y = drop(x) + residual, the mask made from a counter as the map
// passes through (map_ops.h), never stored.  One read of each input and one
// write: DRAM bounds it, for the generator's arithmetic (about 70 integer
// instructions for eight elements) fits below.  32 x 64 x 64 x 1024 bf16 with a
// residual 115 us, 7.0 TB/s; 7 x 61 x 83 x 200 f16 7.6 us, 5.6 TB/s (8.5 where
// none of its maps is left in L2); a small call 1.7 us, the launch.
#include <algorithm>
#include <initializer_list>

#include "map_ops.h"
#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {

using namespace maps;

constexpr int kDropThreads = 256;
constexpr int kDropVecs = 4;    // vectors a thread reads before it uses the first (115 us as above, 133 with one)

struct DropArgs {
    View x, r, y;               // r.p null: no residual
    unsigned long long total;   // vectors
    unsigned long long row;     // vectors of a row
    unsigned H;                 // rows an image
    unsigned tail;              // elements after the last vector of maps whose elements follow one another
    Drop drop;
    int dropping;
};

// One element of maps whose elements follow one another.
template <class T, bool RESIDUAL>
__device__ __forceinline__ void drop_one(const DropArgs &a, unsigned long long e)
{
    float f[1], r[1];
    unpack<T, 1>(reinterpret_cast<const Raw<T, 1> *>(a.x.p)[e], f);
    if (a.dropping) drop_elements<1>(f, e, a.drop);
    if (RESIDUAL) {
        unpack<T, 1>(reinterpret_cast<const Raw<T, 1> *>(a.r.p)[e], r);
        f[0] += r[0];
    }
    reinterpret_cast<Raw<T, 1> *>(a.y.p)[e] = pack<T, 1>(f);
}

// A CTA takes kDropVecs x kDropThreads consecutive vectors.  WHOLE: the maps'
// elements follow one another; else vectors are found by row and image.
template <class T, int VE, bool WHOLE, bool RESIDUAL>
__global__ void __launch_bounds__(kDropThreads) k_dropout(const DropArgs a)
{
    using V = Raw<T, VE>;
    dev::grid_launch_dependents();
    const unsigned long long first = blockIdx.x * static_cast<unsigned long long>(kDropVecs * kDropThreads) + threadIdx.x;
    const auto at = [&](const View &m, int u) {
        const unsigned long long v = first + u * kDropThreads;
        if (WHOLE) return reinterpret_cast<V *>(m.p) + v;
        const unsigned long long row = v / a.row, n = row / a.H;
        return reinterpret_cast<V *>(m.p + n * m.bstride + (row - n * a.H) * m.pitch) + (v - row * a.row);
    };
    dev::grid_dependency_wait();
    if (WHOLE && VE > 1 && first < a.tail) drop_one<T, RESIDUAL>(a, a.total * VE + first);
    V x[kDropVecs], r[kDropVecs];
#pragma unroll
    for (int u = 0; u < kDropVecs; u++)
        if (first + u * kDropThreads < a.total) {
            x[u] = __ldcs(at(a.x, u));
            if (RESIDUAL) r[u] = __ldcs(at(a.r, u));
        }
#pragma unroll
    for (int u = 0; u < kDropVecs; u++)
        if (first + u * kDropThreads < a.total) {
            float f[VE];
            unpack<T, VE>(x[u], f);
            if (a.dropping) drop_elements<VE>(f, (first + u * kDropThreads) * VE, a.drop);
            if (RESIDUAL) {
                float g[VE];
                unpack<T, VE>(r[u], g);
#pragma unroll
                for (int i = 0; i < VE; i++) f[i] += g[i];
            }
            __stcs(at(a.y, u), pack<T, VE>(f));
        }
}

template <class T, int VE>
cudaError_t drop_launch(const DropArgs &a, bool whole, void *stream)
{
    const unsigned long long blocks = std::max(1ull, (a.total + kDropVecs * kDropThreads - 1) / (kDropVecs * kDropThreads));
    if (blocks > 0x7fffffffull) return cudaErrorInvalidConfiguration;
    const auto fn = whole ? (a.r.p ? k_dropout<T, VE, true, true> : k_dropout<T, VE, true, false>)
                          : (a.r.p ? k_dropout<T, VE, false, true> : k_dropout<T, VE, false, false>);
    return launch(fn, dim3(static_cast<unsigned>(blocks)), kDropThreads, 0, stream, a);
}

// Launches over `all` elements of maps in rows of `row`; ONE: the maps' elements
// follow one another, and a vector may cross rows.
int drop_run(DropArgs &a, int dtype, bool one, bool aligned, unsigned long long row, unsigned long long all,
             const rz_drop *drop, void *stream)
{
    const unsigned ve = 16 / static_cast<unsigned>(dtype_size(dtype));
    const bool wide = (one || row % ve == 0) && aligned;
    a.drop = make_drop(drop);
    a.dropping = drop_threshold(drop) != 0;
    a.row = wide ? row / ve : row;
    a.total = wide ? all / ve : all;
    a.tail = wide ? static_cast<unsigned>(all % ve) : 0;
    // one element at a time a map of 2^41 elements would pass the grid's width
    if (a.total / (kDropVecs * kDropThreads) >= 0x7fffffffull) return RZ_ERR_UNSUPPORTED;
    cudaError_t e;
    if (dtype == RZ_F32)
        e = wide ? drop_launch<float, 4>(a, one, stream) : drop_launch<float, 1>(a, one, stream);
    else if (dtype == RZ_BF16)
        e = wide ? drop_launch<__nv_bfloat16, 8>(a, one, stream) : drop_launch<__nv_bfloat16, 1>(a, one, stream);
    else
        e = wide ? drop_launch<__half, 8>(a, one, stream) : drop_launch<__half, 1>(a, one, stream);
    if (e == cudaSuccess) return RZ_OK;
    record_cuda_error(static_cast<int>(e));
    return RZ_ERR_CUDA;
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
    a.H = static_cast<unsigned>(s.H);
    const bool one = whole(x) && whole(y) && whole(residual);
    const auto aligned = [&](const rz_map *m) {
        return !m || (one ? reinterpret_cast<uintptr_t>(m->data) % 16 == 0 : maps::map_aligned(*m, s, 16));
    };
    const unsigned long long row = static_cast<unsigned long long>(s.W) * s.C;
    return drop_run(a, dtype, one, aligned(x) && aligned(y) && aligned(residual), row, row * s.N * s.H, drop, stream);
}

int map_dropout_packed(const void *x, const void *residual, void *y, size_t n, int dtype, const rz_drop *drop, void *stream)
{
    const size_t es = maps::dtype_size(dtype);
    if (!es || n > (size_t{1} << 46) || !drop || !maps::drop_ok(drop)) return RZ_ERR_ARG;
    if (n == 0) return RZ_OK;
    const auto at = [](const void *p) { return reinterpret_cast<uintptr_t>(p); };
    if (!x || !y || at(x) % es || at(y) % es || at(residual) % es) return RZ_ERR_ARG;
    for (const void *p : {x, residual})
        if (p && p != y && at(p) < at(y) + n * es && at(y) < at(p) + n * es) return RZ_ERR_ARG;
    DropArgs a{};
    a.x.p = static_cast<uint8_t *>(const_cast<void *>(x));
    a.y.p = static_cast<uint8_t *>(y);
    a.r.p = static_cast<uint8_t *>(const_cast<void *>(residual));
    return drop_run(a, dtype, true, (at(x) | at(y) | at(residual)) % 16 == 0, n, n, drop, stream);
}

}  // extern "C"
