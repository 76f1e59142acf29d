// Linear layer of a map with its epilogue, and its gradient:
//   z = x W^T + b,  y = act(z) + residual;
//   dz = dy act'(z),  dx = dz W,  dW = dz^T x,  db = sum dz.
#include <algorithm>
#include <cmath>

#include "map_ops.h"
#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {

using namespace maps;
using dev::grid_dependency_wait;
using dev::grid_launch_dependents;

// A matrix inside a map or a weight: row r at row_off(r), its columns packed.
struct Rows {
    View v;
    unsigned HW, W;     // pixels of an image and of its rows (HW 0: rows `pitch` apart)
    int joined, bytes;  // a row's bytes where the map's rows are joined
};

__device__ __forceinline__ long long row_off(const Rows &m, unsigned r)
{
    if (!m.HW) return r * m.v.pitch;
    const unsigned n = r / m.HW;
    return n * m.v.bstride + pixel_off(r - n * m.HW, m.W, m.joined != 0, m.v.pitch, m.bytes);
}
template <class T>
__device__ __forceinline__ float element(const Rows &m, unsigned r, unsigned c)
{
    return static_cast<float>(reinterpret_cast<const T *>(m.v.p + row_off(m, r))[c]);
}
template <class T>
__device__ __forceinline__ void put(const Rows &m, unsigned r, unsigned c, float v)
{
    reinterpret_cast<T *>(m.v.p + row_off(m, r))[c] = static_cast<T>(v);
}

__device__ __forceinline__ float activated(float z, int act)
{
    if (act == RZ_ACT_SILU) return z < -87.3f ? 0.0f : z * rcp_approx(1.0f + exp2_approx(-1.44269504f * z));
    return act == RZ_ACT_GELU ? gelu(z) : z;
}
__device__ __forceinline__ float act_slope(float z, int act)
{
    if (act == RZ_ACT_SILU) {
        const float s = z < -87.3f ? 0.0f : rcp_approx(1.0f + exp2_approx(-1.44269504f * z));
        return s * fmaf(z, 1.0f - s, 1.0f);
    }
    return act == RZ_ACT_GELU ? gelu_slope(z) : 1.0f;
}

// D[m][n] = sum_k A(m, k) B(n, k), an element read by its row and column: of a
// transposed operand k is the row.  64 x 64 a CTA, 16 terms at a time.
struct SimpleArgs {
    Rows a, b, out, pre, residual, slope;   // slope: pre of A, which A is multiplied by act' of
    const float *bias;
    unsigned M, N, K;
    int a_turned, b_turned, act, has_pre, has_residual, has_slope;
};

template <class T, class O>
__global__ void __launch_bounds__(256) k_linear_simple(const __grid_constant__ SimpleArgs p)
{
    __shared__ float sa[16][65], sb[16][65];
    grid_launch_dependents();
    grid_dependency_wait();
    const unsigned tiles_n = (p.N + 63) / 64, m0 = blockIdx.x / tiles_n * 64, n0 = blockIdx.x % tiles_n * 64;
    const unsigned tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (unsigned k0 = 0; k0 < p.K; k0 += 16) {
        for (unsigned i = threadIdx.x; i < 1024; i += 256) {
            const unsigned k = i % 16, r = i / 16;
            float a = 0.0f, b = 0.0f;
            if (k0 + k < p.K && m0 + r < p.M) {
                const unsigned row = p.a_turned ? k0 + k : m0 + r, col = p.a_turned ? m0 + r : k0 + k;
                a = element<T>(p.a, row, col);
                if (p.has_slope) a *= act_slope(element<T>(p.slope, row, col), p.act);
            }
            if (k0 + k < p.K && n0 + r < p.N)
                b = p.b_turned ? element<T>(p.b, k0 + k, n0 + r) : element<T>(p.b, n0 + r, k0 + k);
            sa[k][r] = a;
            sb[k][r] = b;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; k++)
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) acc[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; i++)
        for (int j = 0; j < 4; j++) {
            const unsigned m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (m >= p.M || n >= p.N) continue;
            float z = acc[i][j];
            if (!p.has_slope) {
                if (p.bias) z += p.bias[n];
                if (p.has_pre) put<T>(p.pre, m, n, z);
                z = activated(z, p.act);
                if (p.has_residual) z += element<T>(p.residual, m, n);
            }
            put<O>(p.out, m, n, z);
        }
}

// Column sums of dz, a column a warp.
template <class T>
__global__ void __launch_bounds__(256) k_linear_sums(const __grid_constant__ SimpleArgs p, float *dbias)
{
    grid_launch_dependents();
    grid_dependency_wait();
    const unsigned c = blockIdx.x * 8 + threadIdx.x / 32;
    if (c >= p.N) return;
    float s = 0.0f;
    for (unsigned r = threadIdx.x % 32; r < p.M; r += 32) {
        float v = element<T>(p.a, r, c);
        if (p.has_slope) v *= act_slope(element<T>(p.slope, r, c), p.act);
        s += v;
    }
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (threadIdx.x % 32 == 0) dbias[c] = s;
}

// ------------------------------------------------------------------ host side

struct LinPlan {
    Shape x, y;
    unsigned P;
};

int lin_check(const rz_linear *d, LinPlan *p)
{
    if (!d) return RZ_ERR_ARG;
    const size_t es = dtype_size(d->dtype);
    p->x = {d->N, d->H, d->W, d->C, es};
    p->y = {d->N, d->H, d->W, d->K, es};
    if (!es || !shape_ok(p->x) || !shape_ok(p->y)) return RZ_ERR_ARG;
    if (d->act != RZ_ACT_NONE && d->act != RZ_ACT_SILU && d->act != RZ_ACT_GELU) return RZ_ERR_ARG;
    if (!p->x.empty() && d->N > 0x7fffffffLL / (p->x.H * p->x.W)) return RZ_ERR_UNSUPPORTED;
    p->P = p->x.empty() ? 0 : static_cast<unsigned>(p->x.N * p->x.H * p->x.W);
    return RZ_OK;
}

Rows rows_of(const rz_map *m, const Shape &s)
{
    Rows r{};
    r.v = view(m);
    r.bytes = static_cast<int>(s.C * s.es);
    r.joined = rows_joined(*m, s);
    r.HW = static_cast<unsigned>(s.H * s.W);
    r.W = static_cast<unsigned>(s.W);
    return r;
}
Rows rows_of(const void *p, size_t pitch)
{
    Rows r{};
    r.v = {static_cast<uint8_t *>(const_cast<void *>(p)), static_cast<long long>(pitch), 0};
    return r;
}

bool matrix_ok(const void *p, size_t pitch, long long rows, long long cols, size_t es)
{
    const size_t row = static_cast<size_t>(cols) * es;
    return p && reinterpret_cast<uintptr_t>(p) % es == 0 && pitch % es == 0 && (rows == 1 || pitch >= row) &&
           pitch <= (size_t{1} << 40);
}
// The bytes of a matrix and of a map, for overlaps.
struct Range {
    uintptr_t from, to;
};
Range range_of(const void *p, size_t pitch, long long rows, long long cols, size_t es)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + static_cast<size_t>(rows - 1) * pitch + static_cast<size_t>(cols) * es};
}
Range range_of(const rz_map &m, const Shape &s)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(m.data);
    return {a, a + s.extent(m)};
}
bool meet(const Range &a, const Range &b) { return a.from < b.to && b.from < a.to; }

int lin_status(cudaError_t e)
{
    if (e == cudaSuccess) return RZ_OK;
    record_cuda_error(static_cast<int>(e));
    return RZ_ERR_CUDA;
}

template <class T, class O = T>
cudaError_t simple(const SimpleArgs &p, void *stream)
{
    const long long tiles = static_cast<long long>((p.M + 63) / 64) * ((p.N + 63) / 64);
    if (tiles > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch(k_linear_simple<T, O>, dim3(static_cast<unsigned>(tiles)), 256, 0, stream, p);
}
template <class T>
cudaError_t simple_to(const SimpleArgs &p, int out, void *stream)
{
    return out == RZ_F32 ? simple<T, float>(p, stream) : simple<T>(p, stream);
}
cudaError_t simple_of(const SimpleArgs &p, int dtype, int out, void *stream)
{
    if (dtype == RZ_F32) return simple<float>(p, stream);
    return dtype == RZ_BF16 ? simple_to<__nv_bfloat16>(p, out, stream) : simple_to<__half>(p, out, stream);
}

}  // namespace
}  // namespace rz

using namespace rz;

extern "C" {

int map_linear_workspace(const rz_linear *d, const rz_map *x, const void *weight, size_t weight_pitch, size_t *bytes)
{
    LinPlan p;
    const int rc = bytes ? lin_check(d, &p) : RZ_ERR_ARG;
    if (rc) return rc;
    *bytes = 0;
    if (p.x.empty()) return RZ_OK;
    if (!maps::map_ok(x, p.x) || !matrix_ok(weight, weight_pitch, d->K, d->C, p.x.es)) return RZ_ERR_ARG;
    return RZ_OK;
}

int map_linear(const rz_linear *d, const rz_map *x, const void *weight, size_t weight_pitch, const float *bias,
               const rz_map *residual, const rz_map *pre, const rz_map *y, void *workspace, size_t workspace_bytes, int *status,
               void *stream)
{
    LinPlan p;
    if (const int rc = lin_check(d, &p)) return rc;
    if (p.x.empty()) return RZ_OK;
    const auto map = [](const rz_map *m, const maps::Shape &s) { return !m || maps::map_ok(m, s); };
    if (!x || !y || !map(x, p.x) || !map(y, p.y) || !map(residual, p.y) || !map(pre, p.y)) return RZ_ERR_ARG;
    if (!matrix_ok(weight, weight_pitch, d->K, d->C, p.x.es)) return RZ_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(bias) % 4 || reinterpret_cast<uintptr_t>(status) % 4) return RZ_ERR_ARG;
    const Range ry = range_of(*y, p.y), rx = range_of(*x, p.x), rw = range_of(weight, weight_pitch, d->K, d->C, p.x.es);
    const Range rb{reinterpret_cast<uintptr_t>(bias), reinterpret_cast<uintptr_t>(bias) + (bias ? 4 * size_t(d->K) : 0)};
    if (meet(ry, rx) || meet(ry, rw) || (bias && meet(ry, rb))) return RZ_ERR_ARG;
    if (residual && !maps::map_same(*residual, *y, p.y) && meet(ry, range_of(*residual, p.y))) return RZ_ERR_ARG;
    if (pre) {
        const Range rp = range_of(*pre, p.y);
        if (meet(rp, rx) || meet(rp, rw) || meet(rp, ry) || (bias && meet(rp, rb)) ||
            (residual && meet(rp, range_of(*residual, p.y))))
            return RZ_ERR_ARG;
    }
    SimpleArgs s{};
    s.a = rows_of(x, p.x);
    s.b = rows_of(weight, weight_pitch);
    s.out = rows_of(y, p.y);
    s.M = p.P;
    s.N = static_cast<unsigned>(d->K);
    s.K = static_cast<unsigned>(d->C);
    s.bias = bias;
    s.act = d->act;
    if (pre) s.pre = rows_of(pre, p.y);
    if (residual) s.residual = rows_of(residual, p.y);
    s.has_pre = pre != nullptr;
    s.has_residual = residual != nullptr;
    return lin_status(simple_of(s, d->dtype, d->dtype, stream));
}

int map_linear_grad_workspace(const rz_linear *d, const rz_map *dy, const rz_map *x, const void *weight, size_t weight_pitch,
                              size_t *bytes)
{
    LinPlan p;
    const int rc = bytes ? lin_check(d, &p) : RZ_ERR_ARG;
    if (rc) return rc;
    *bytes = 0;
    if (p.x.empty()) return RZ_OK;
    if (!maps::map_ok(x, p.x) || !maps::map_ok(dy, p.y) || !matrix_ok(weight, weight_pitch, d->K, d->C, p.x.es))
        return RZ_ERR_ARG;
    return RZ_OK;
}

int map_linear_grad(const rz_linear *d, const rz_map *dy, const rz_map *x, const void *weight, size_t weight_pitch,
                    const rz_map *pre, const rz_map *dx, void *dweight, size_t dweight_pitch, int dweight_dtype, float *dbias,
                    void *workspace, size_t workspace_bytes, int *status, void *stream)
{
    LinPlan p;
    if (const int rc = lin_check(d, &p)) return rc;
    const size_t dw_es = maps::dtype_size(dweight_dtype);
    if (dweight && ((dweight_dtype != d->dtype && dweight_dtype != RZ_F32) ||
                    !matrix_ok(dweight, dweight_pitch, d->K, d->C, dw_es)))
        return RZ_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(dbias) % 4 || reinterpret_cast<uintptr_t>(status) % 4) return RZ_ERR_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p.x.empty()) {
        cudaError_t e = dweight ? cudaMemset2DAsync(dweight, std::max<size_t>(dweight_pitch, d->C * dw_es), 0, d->C * dw_es, d->K, st)
                                : cudaSuccess;
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, 4 * static_cast<size_t>(d->K), st);
        return lin_status(e);
    }
    if (!maps::map_ok(x, p.x) || !maps::map_ok(dy, p.y) || (dx && !maps::map_ok(dx, p.x))) return RZ_ERR_ARG;
    if (d->act != RZ_ACT_NONE ? !maps::map_ok(pre, p.y) : pre && !maps::map_ok(pre, p.y)) return RZ_ERR_ARG;
    if (!matrix_ok(weight, weight_pitch, d->K, d->C, p.x.es)) return RZ_ERR_ARG;
    // no output meets an input or another output
    Range in[4] = {range_of(*x, p.x), range_of(*dy, p.y), range_of(weight, weight_pitch, d->K, d->C, p.x.es), {}}, out[3];
    int nin = 3, nout = 0;
    if (pre) in[nin++] = range_of(*pre, p.y);
    if (dx) out[nout++] = range_of(*dx, p.x);
    if (dweight) out[nout++] = range_of(dweight, dweight_pitch, d->K, d->C, dw_es);
    if (dbias) out[nout++] = {reinterpret_cast<uintptr_t>(dbias), reinterpret_cast<uintptr_t>(dbias) + 4 * size_t(d->K)};
    for (int i = 0; i < nout; i++) {
        for (int j = 0; j < nin; j++)
            if (meet(out[i], in[j])) return RZ_ERR_ARG;
        for (int j = 0; j < i; j++)
            if (meet(out[i], out[j])) return RZ_ERR_ARG;
    }
    SimpleArgs s{};
    s.a = rows_of(dy, p.y);
    s.act = d->act;
    s.has_slope = d->act != RZ_ACT_NONE;
    if (s.has_slope) s.slope = rows_of(pre, p.y);
    cudaError_t e = cudaSuccess;
    if (dx) {
        SimpleArgs q = s;
        q.b = rows_of(weight, weight_pitch);
        q.b_turned = 1;
        q.out = rows_of(dx, p.x);
        q.M = p.P;
        q.N = static_cast<unsigned>(d->C);
        q.K = static_cast<unsigned>(d->K);
        e = simple_of(q, d->dtype, d->dtype, stream);
    }
    if (dweight && e == cudaSuccess) {
        SimpleArgs q = s;
        q.a_turned = q.b_turned = 1;
        q.b = rows_of(x, p.x);
        q.out = rows_of(dweight, dweight_pitch);
        q.M = static_cast<unsigned>(d->K);
        q.N = static_cast<unsigned>(d->C);
        q.K = p.P;
        e = simple_of(q, d->dtype, dweight_dtype, stream);
    }
    if (dbias && e == cudaSuccess) {
        s.M = p.P;
        s.N = static_cast<unsigned>(d->K);
        const dim3 grid((s.N + 7) / 8);
        if (d->dtype == RZ_F32)
            e = maps::launch(k_linear_sums<float>, grid, 256, 0, stream, s, dbias);
        else if (d->dtype == RZ_BF16)
            e = maps::launch(k_linear_sums<__nv_bfloat16>, grid, 256, 0, stream, s, dbias);
        else
            e = maps::launch(k_linear_sums<__half>, grid, 256, 0, stream, s, dbias);
    }
    return lin_status(e);
}

}  // extern "C"
