// Linear layer of a map with its epilogue, and its gradient:
//   z = x W^T + b,  y = act(z) + residual;
//   dz = dy act'(z),  dx = dz W,  dW = dz^T x,  db = sum dz.
// The products run on the tensor cores (linear_tc.cu), which take 16-bit
// operands whose rows TMA can address (16-byte pitch and start).  What is not of
// that kind is laid out first: float32 as three bfloat16 planes, rows of odd
// widths or with gaps as packed ones; so is dz, in one pass that also adds up its
// columns.  Sums too long for few tiles are cut into parts that a last kernel joins
// in order.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "linear.h"
#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {

using namespace lin;
using dev::grid_dependency_wait;
using dev::grid_launch_dependents;

constexpr int kLinSms = 152;
constexpr int kPackThreads = 256;
constexpr int kPackWarps = kPackThreads / 32;

// Rows of a map or weight, times act'(slope) if there is one, laid out for the
// tensor cores: 16-bit rows of `pitch` bytes, float32 as three planes of bfloat16
// (each the leading 8 bits of what is left: together all 24).  And their column
// sums, by chunks of rows.
//
// dz = dy act'(pre) of 16-bit maps is rounded to their type here, which a result of that
// type (dx, dweight) shows no more than its own rounding (2.3e-3 of a bf16 result's
// size in the 2-norm, 1.7e-3 without it): a second plane would double their products, 90 of the 130 us
// of 32768 x 1024 -> 1024.  A float32 dweight does take it: what the rounding left,
// rounded in turn, is a second plane.  A float16 dz past 65504 is infinite.
struct PackArgs {
    Rows in, slope;
    uint8_t *to;            // null: sums only
    long long pitch, plane;
    float *sums;            // [chunks][C], or null
    unsigned M, C;
    unsigned chunk;         // rows of a CTA
    int lanes;              // lanes side by side in a row, eight columns each
    int has_slope, act, wide;
    int second;             // 16-bit: a second plane holds what the first one's rounding left
    unsigned blocks, across;    // CTAs, and of them along a row
};
// The matrices of a call in one launch, their CTAs one after another.
struct PackJobs {
    PackArgs job[3];
    int count;
};

// Eight elements: as they come, or with those past the row's end 0.
template <class T, bool WIDE>
__device__ __forceinline__ void load8(const uint8_t *at, int left, Raw<T, 8> &r)
{
    if constexpr (WIDE) {
        if constexpr (sizeof(T) == 4) {
            r.a = __ldcs(reinterpret_cast<const uint4 *>(at));
            r.b = __ldcs(reinterpret_cast<const uint4 *>(at) + 1);
        } else {
            r = __ldcs(reinterpret_cast<const uint4 *>(at));
        }
    } else {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] = i < left ? static_cast<float>(reinterpret_cast<const T *>(at)[i]) : 0.0f;
        r = pack<T, 8>(f);
    }
}

// The leading 8 bits of v, cut, so that what is left has its sign and no value
// becomes infinite; 0 of one that is not finite.  Those go into the last plane whole,
// which meets but the other operand's first: an infinity times a value is then the
// infinity of its sign, where a lower plane of 0 would have made it NaN.
__device__ __forceinline__ float leading(float v)
{
    return fabsf(v) <= 3.402823466e38f ? __uint_as_float(__float_as_uint(v) & 0xffff0000u) : 0.0f;
}

template <class T, bool WIDE, bool SECOND>
__device__ __forceinline__ void pack_block(const PackArgs &a, unsigned bx, unsigned by, float (&sh)[kPackWarps][256])
{
    constexpr int U = sizeof(T) == 2 ? 4 : 2;       // rows read before the first is used
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rows = 32 / a.lanes, sub = lane % a.lanes, down = lane / a.lanes;
    const unsigned c = (bx * a.lanes + sub) * 8;
    const int left = static_cast<int>(a.C) - static_cast<int>(c);
    const unsigned r0 = by * a.chunk, r1 = min(a.M, r0 + a.chunk), step = kPackWarps * rows;
    float s[8] = {};
    if (left > 0) {
        for (unsigned r = r0 + warp * rows + down; r < r1; r += U * step) {
            Raw<T, 8> in[U], slope[U];
#pragma unroll
            for (int u = 0; u < U; u++) {
                // past the last row: that one again, and not used
                const unsigned ru = min(r + u * step, r1 - 1);
                load8<T, WIDE>(a.in.v.p + row_off(a.in, ru) + static_cast<long long>(c) * sizeof(T), left, in[u]);
                if (a.has_slope) load8<T, WIDE>(a.slope.v.p + row_off(a.slope, ru) + static_cast<long long>(c) * sizeof(T), left, slope[u]);
            }
#pragma unroll
            for (int u = 0; u < U; u++) {
                if (r + u * step >= r1) break;
                float f[8];
                unpack<T, 8>(in[u], f);
                if (a.has_slope) {
                    float z[8];
                    unpack<T, 8>(slope[u], z);
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float2 d = act_slope<T>(make_float2(z[i], z[i + 1]), a.act);
                        f[i] *= d.x;
                        f[i + 1] *= d.y;
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; i++)
                    if (WIDE || i < left) s[i] += f[i];
                if (!a.to) continue;
                uint8_t *at = a.to + (r + u * step) * a.pitch + c * 2;
                if constexpr (sizeof(T) == 2) {
                    const uint4 first = pack<T, 8>(f);
                    *reinterpret_cast<uint4 *>(at) = first;
                    if (SECOND && a.second) {
                        float h[8];
                        unpack<T, 8>(first, h);
#pragma unroll
                        for (int i = 0; i < 8; i++) f[i] = fabsf(h[i]) <= 3.4e38f ? f[i] - h[i] : 0.0f;
                        *reinterpret_cast<uint4 *>(at + a.plane) = pack<T, 8>(f);
                    }
                } else {
#pragma unroll
                    for (int p = 0; p < 3; p++) {
                        float h[8];
#pragma unroll
                        for (int i = 0; i < 8; i++) {
                            h[i] = p < 2 ? leading(f[i]) : f[i];    // (8 bits are left for the last)
                            f[i] -= h[i];
                        }
                        *reinterpret_cast<uint4 *>(at + p * a.plane) = pack<__nv_bfloat16, 8>(h);
                    }
                }
            }
        }
    }
    if (!a.sums) return;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        for (int o = a.lanes; o < 32; o <<= 1) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
        if (down == 0) sh[warp][sub * 8 + i] = s[i];
    }
    __syncthreads();
    const unsigned col = bx * a.lanes * 8 + threadIdx.x;
    if (static_cast<int>(threadIdx.x) >= a.lanes * 8 || col >= a.C) return;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kPackWarps; w++) sum += sh[w][threadIdx.x];
    a.sums[static_cast<long long>(by) * a.C + col] = sum;
}

// WIDE: of every job.  ONE: a single one, whose arguments need no index (32768 x 1024
// with a slope: 34.5 us, 40 where they do).  SECOND: one has a second plane (with the
// question asked at run time, those that have none took 41 us for 31).
template <class T, bool WIDE, bool ONE, bool SECOND>
__global__ void __launch_bounds__(kPackThreads) k_linear_pack(const __grid_constant__ PackJobs jobs)
{
    __shared__ float sh[kPackWarps][256];
    grid_launch_dependents();
    grid_dependency_wait();
    unsigned b = blockIdx.x;
    int j = 0;
    if (!ONE)
        while (j + 1 < jobs.count && b >= jobs.job[j].blocks) b -= jobs.job[j++].blocks;
    const PackArgs &a = jobs.job[ONE ? 0 : j];
    const unsigned by = b / a.across, bx = b - by * a.across;
    if (WIDE || a.wide)
        pack_block<T, true, SECOND>(a, bx, by, sh);
    else
        pack_block<T, false, SECOND>(a, bx, by, sh);
}

// dbias: the chunks' sums, 32 columns a block, each of its warps a chunk in
// eight, joined in order.
struct Sums {
    const float *from;
    float *to;              // null: none
    unsigned chunks, C;
};
__device__ __forceinline__ void sum_columns(const Sums &a, unsigned block)
{
    __shared__ float sh[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const unsigned c = block * 32 + lane;
    float s = 0.0f;
    if (c < a.C) {
#pragma unroll 16
        for (unsigned r = w; r < a.chunks; r += 8) s += a.from[static_cast<long long>(r) * a.C + c];
    }
    sh[w][lane] = s;
    __syncthreads();
    if (w || c >= a.C) return;
#pragma unroll
    for (int i = 1; i < 8; i++) s += sh[i][lane];
    a.to[c] = s;
}
__global__ void __launch_bounds__(256) k_linear_sums(const __grid_constant__ Sums a)
{
    grid_launch_dependents();
    grid_dependency_wait();
    sum_columns(a, blockIdx.x);
}

// The parts of a product joined in order, and its epilogue; one alone where its sums
// took several runs, or its result's rows are not TMA's to write.
struct JoinArgs {
    Finish f;
    const float *part;
    unsigned pitch;         // floats, a multiple of VE
    int parts;
    unsigned blocks;        // those after them sum the bias's columns (a launch of 5 us less)
    Sums sums;
};

constexpr int kJoinUnits = 4;   // units a thread has in flight where vectors do not fit

// UNIT: elements taken at once, a vector, a pair or one.
template <class T, int ACT, int UNIT>
__global__ void __launch_bounds__(256) k_linear_join(const __grid_constant__ JoinArgs a)
{
    constexpr bool WIDE = UNIT * sizeof(T) == 16;
    constexpr int U = WIDE ? 1 : kJoinUnits;
    grid_launch_dependents();
    grid_dependency_wait();
    if (blockIdx.x >= a.blocks) {
        sum_columns(a.sums, blockIdx.x - a.blocks);
        return;
    }
    // a block's first unit by 64-bit division, the others from there
    const unsigned units = a.f.N / UNIT;
    const unsigned long long base = static_cast<unsigned long long>(blockIdx.x) * (256 * U);
    const unsigned m0 = static_cast<unsigned>(base / units), n0 = static_cast<unsigned>(base - static_cast<unsigned long long>(m0) * units);
    const long long step = static_cast<long long>(a.f.M) * a.pitch;
    if constexpr (WIDE) {
        const unsigned q0 = n0 + threadIdx.x, m = m0 + q0 / units, n = q0 % units * UNIT;
        if (m >= a.f.M) return;
        const float *from = a.part + static_cast<long long>(m) * a.pitch + n;
        float2 z[UNIT / 2] = {}, b[UNIT / 2];
#pragma unroll 8
        for (int r = 0; r < a.parts; r++, from += step)
#pragma unroll
            for (int q = 0; q < UNIT; q += 4) {
                const float4 v = __ldcs(reinterpret_cast<const float4 *>(from + q));
                z[q / 2] = __fadd2_rn(z[q / 2], make_float2(v.x, v.y));
                z[q / 2 + 1] = __fadd2_rn(z[q / 2 + 1], make_float2(v.z, v.w));
            }
        bias_of<UNIT>(a.f, n, b);
        Raw<T, UNIT> r{};
        if (a.f.has_residual) r = *vec_at<T, UNIT>(a.f.residual, m, n);
        finish<T, UNIT, ACT>(a.f, m, n, z, b, r);
    } else {
        unsigned m[U], n[U];
        const float *from[U];
        float2 z[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const unsigned q = n0 + threadIdx.x + 256 * u;
            m[u] = m0 + q / units;
            n[u] = q % units * UNIT;
            // past the last: that one again, and not stored
            from[u] = a.part + static_cast<long long>(min(m[u], a.f.M - 1)) * a.pitch + n[u];
            z[u] = both(0.0f);
        }
#pragma unroll 2
        for (int r = 0; r < a.parts; r++)
#pragma unroll
            for (int u = 0; u < U; u++) {
                if (UNIT == 2)
                    z[u] = __fadd2_rn(z[u], __ldcs(reinterpret_cast<const float2 *>(from[u])));
                else
                    z[u].x += __ldcs(from[u]);
                from[u] += step;
            }
#pragma unroll
        for (int u = 0; u < U; u++)
            if (m[u] < a.f.M) finish_unit<T, ACT, UNIT>(a.f, m[u], n[u], z[u]);
    }
}

// Few rows of x, one token's for instance: the weight is all there is to read, so
// no tile is staged.  A warp takes two columns of the result, its lanes the terms, a
// vector of each at a time; `share` warps of a CTA share a column pair's terms where
// there are few of them.  Up to ROWS rows of x (blockIdx.y counts them off) meet
// each vector of the weight.  One row, 4096 x 1024 bf16: 2.8 us in a stream of calls
// that leave the weight in L2, 4 from DRAM (2.1 TB/s): a launch and one chain of loads
// and shuffles.
struct RowsArgs {
    Rows x, w;
    Finish f;
    unsigned C;
    int share;
};
constexpr int kRowsColumns = 2;

template <class T, int ACT, int ROWS, bool WIDE>
__global__ void __launch_bounds__(256) k_linear_rows(const __grid_constant__ RowsArgs a)
{
    constexpr int VE = WIDE ? 16 / sizeof(T) : 1, P = kPairs<VE>, N = kRowsColumns;
    using V = Raw<T, VE>;
    __shared__ float sh[8][N * ROWS];
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned pair = (blockIdx.x * 8 + warp) / a.share, n0 = pair * N, m0 = blockIdx.y * ROWS;
    const int part = warp % a.share;
    const uint8_t *w[N], *x[ROWS];
#pragma unroll
    for (int j = 0; j < N; j++) w[j] = a.w.v.p + row_off(a.w, min(n0 + j, a.f.N - 1));
#pragma unroll
    for (int r = 0; r < ROWS; r++) x[r] = a.x.v.p + row_off(a.x, min(m0 + r, a.f.M - 1));
    float2 s[N][ROWS];
#pragma unroll
    for (int j = 0; j < N; j++)
#pragma unroll
        for (int r = 0; r < ROWS; r++) s[j][r] = both(0.0f);
    grid_dependency_wait();
    const unsigned vecs = a.C / VE;
#pragma unroll(ROWS > 2 ? 2 : 4)
    for (unsigned v = part * 32 + lane; v < vecs; v += 32 * a.share) {
        V wr[N], xr[ROWS];
#pragma unroll
        for (int j = 0; j < N; j++) wr[j] = __ldcs(reinterpret_cast<const V *>(w[j]) + v);
#pragma unroll
        for (int r = 0; r < ROWS; r++) xr[r] = reinterpret_cast<const V *>(x[r])[v];
        float2 wf[N][P];
#pragma unroll
        for (int j = 0; j < N; j++) unpack2<T, VE>(wr[j], wf[j]);
#pragma unroll
        for (int r = 0; r < ROWS; r++) {
            float2 xf[P];
            unpack2<T, VE>(xr[r], xf);
#pragma unroll
            for (int j = 0; j < N; j++)
#pragma unroll
                for (int i = 0; i < P; i++) s[j][r] = __ffma2_rn(wf[j][i], xf[i], s[j][r]);
        }
    }
    // a lane keeps the sum of column lane / ROWS, row lane % ROWS
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < N; j++)
#pragma unroll
        for (int r = 0; r < ROWS; r++) {
            float t = s[j][r].x + s[j][r].y;
#pragma unroll
            for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            if (lane == j * ROWS + r) z = t;
        }
    if (a.share > 1) {
        if (lane < N * ROWS) sh[warp][lane] = z;
        __syncthreads();
        if (part) return;
        if (lane < N * ROWS)
            for (int i = 1; i < a.share; i++) z += sh[warp + i][lane];
    }
    const unsigned n = n0 + lane / ROWS, m = m0 + lane % ROWS;
    if (lane >= N * ROWS || n >= a.f.N || m >= a.f.M) return;
    finish_unit<T, ACT, 1>(a.f, m, n, make_float2(z, 0.0f));
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

// A map's rows are pixels; where they are evenly apart, `HW` is 0.
Rows rows_of(const rz_map *m, const Shape &s)
{
    Rows r{};
    r.v = view(m);
    r.bytes = static_cast<int>(s.C * s.es);
    r.joined = rows_joined(*m, s);
    r.HW = static_cast<unsigned>(s.H * s.W);
    r.W = static_cast<unsigned>(s.W);
    if (r.joined && (s.N == 1 || m->batch_stride == s.H * s.row())) {
        r.HW = 0;
        r.v.pitch = r.bytes;
        r.v.bstride = 0;
    }
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
           pitch <= (size_t{1} << 39);
}
// The bytes of a matrix or a map, for overlaps.
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

size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// A matrix as an operand: itself where TMA can address it, else its place in the
// workspace.
struct Laid {
    Rows in;
    unsigned rows, cols;
    int dtype, planes;
    bool direct;
    size_t pitch, plane, bytes;     // of the layout in the workspace; bytes 0: direct
    size_t at = 0;
};
// planes: of 16-bit rows that are changed on their way, 1 or 2.
Laid lay(const Rows &in, unsigned rows, unsigned cols, int dtype, bool changed, int planes = 1)
{
    Laid l{};
    l.in = in;
    l.rows = rows;
    l.cols = cols;
    l.dtype = dtype;
    l.planes = dtype == RZ_F32 ? 3 : planes;
    l.direct = dtype != RZ_F32 && !changed && !in.HW && reinterpret_cast<uintptr_t>(in.v.p) % 16 == 0 &&
               (rows == 1 || in.v.pitch % 16 == 0);
    if (l.direct) {
        l.pitch = rows == 1 ? up(2 * static_cast<size_t>(cols), 16) : static_cast<size_t>(in.v.pitch);
        return l;
    }
    l.pitch = up(cols, 8) * 2;
    l.plane = l.pitch * rows;
    l.bytes = l.plane * l.planes;
    return l;
}
// rows, terms: of the product; turned: the memory's rows are its terms; planes: the first so many.
Operand operand(const Laid &l, const uint8_t *workspace, bool turned, int planes)
{
    Operand o{};
    o.p = l.direct ? l.in.v.p : workspace + l.at;
    o.pitch = l.pitch;
    o.plane = l.plane;
    o.rows = turned ? l.cols : l.rows;
    o.terms = turned ? l.rows : l.cols;
    o.planes = planes;
    o.turned = turned;
    o.bf16 = l.dtype != RZ_F16;
    return o;
}

// Tile width, CTAs of a tile and parts of a product, by an estimate in clocks of
// what was measured (19456 x 1024, 1024 and 4096 terms): a stage of 64 terms takes 590
// on 256 columns of a pair of CTAs and 320 on 128, 650, 390 and 335 on 256, 128 and
// 64 of one CTA; and the join of parts, which pays for long sums of few tiles (50000
// pixels' gradient of a 64 x 64 weight: 211 us in one part, 18 in 32; of 32768 pixels'
// 1024 x 1024 one: 162 and, in 4, 50).
struct Cut {
    int tile_n, pair, parts, part_chunks, run_chunks;
    unsigned pitch;
    size_t bytes;
};
// through: a single run goes through the workspace as well.  A run is as long as its
// accumulator's cut sums allow (linear_tc.cu says by how much), and long enough that its
// products hide its way out: float32 operands 512 terms (off by 1e-6; 768 terms 1.5e-6 at
// the same speed, 256 terms 4e-7 and 7% slower), 16-bit ones 1024 for a float32 result
// (65536 x 1024 x 4096: 498 us; 446 of 2048 terms, 686 of 512), else 8192 of float16 and
// 16384 of bfloat16, where what is cut is a tenth and a hundredth of half a step.
// Parts are several only where they are a few waves of tiles, so that their sums take
// no more than 60 MB; else there is one, the size of the result.
Cut cut(unsigned M, unsigned N, unsigned terms, int dtype, int out_dtype, bool through, int products)
{
    const long long chunks = (terms + 63) / 64;
    const long long longest = dtype == RZ_F32 ? 8 : out_dtype == RZ_F32 ? 16 : dtype == RZ_F16 ? 128 : 256;
    Cut best{};
    double least = 0.0;
    const unsigned pitch = static_cast<unsigned>(up(N, 8));
    const double of_part = 170.0 + 4.0 * M * pitch / 2500.0;
    for (int pair = 0; pair < 2; pair++)
        for (int tile = 256; tile >= (pair ? 128 : 64); tile /= 2) {
            const long long across = (N + tile - 1) / tile;
            if ((tile > 64 && N <= static_cast<unsigned>(tile) / 2) || (pair && M <= 128)) continue;
            const double stage = tile == 64 ? 335 : tile == 128 ? (pair ? 320 : 390) : pair ? 590 : 650;
            const int rows = pair ? 256 : 128, slots = pair ? kLinSms / 2 : kLinSms;
            const long long tiles = static_cast<long long>((M + rows - 1ull) / rows) * across;
            const auto consider = [&](long long want) {
                const long long part = (chunks + want - 1) / want;
                const int parts = static_cast<int>((chunks + part - 1) / part);
                const long long runs = (part + longest - 1) / longest;
                const double waves = static_cast<double>((tiles * parts + slots - 1) / slots);
                double t = waves * (part * products * stage + 300 * runs) + 8.0 * tile + (pair ? 1000 : 0);
                const bool joined = parts > 1 || runs > 1 || through;
                if (joined) t += 4500 + of_part * parts + 4.0 * M * pitch / 2500.0;
                if (!best.tile_n || t < least) {
                    least = t;
                    best = {tile, pair, parts, static_cast<int>(part), static_cast<int>((part + runs - 1) / runs), pitch,
                            joined ? sizeof(float) * parts * static_cast<size_t>(M) * pitch : 0};
                }
            };
            consider(1);
            // of the parts that make one wave, two or three: as many as there can be, or those whose joins cost what they save
            for (int waves = 1; waves <= 3; waves++) {
                const long long most = std::min<long long>({waves * static_cast<long long>(slots) / tiles, chunks, 64});
                if (most <= 1) continue;
                consider(most);
                const long long even = std::lround(std::sqrt(waves * static_cast<double>(chunks) * products * stage / of_part));
                if (even > 1 && even < most) consider(even);
            }
        }
    return best;
}

// One more matrix to lay out.
void add_job(PackJobs &jobs, const Laid &l, const Rows *slope, int act, float *sums, unsigned chunks, uint8_t *workspace)
{
    PackArgs &a = jobs.job[jobs.count++];
    a.in = l.in;
    if (slope) a.slope = *slope;
    a.has_slope = slope != nullptr;
    a.act = act;
    a.to = l.bytes ? workspace + l.at : nullptr;
    a.pitch = static_cast<long long>(l.pitch);
    a.plane = static_cast<long long>(l.plane);
    a.second = l.planes == 2;
    a.sums = sums;
    a.M = l.rows;
    a.C = l.cols;
    const unsigned vecs = (l.cols + 7) / 8;
    a.lanes = 1;
    while (a.lanes < 32 && static_cast<unsigned>(a.lanes) < vecs) a.lanes *= 2;
    a.chunk = (l.rows + chunks - 1) / chunks;
    const auto wide = [](const Rows &r) {
        return reinterpret_cast<uintptr_t>(r.v.p) % 16 == 0 && r.v.pitch % 16 == 0 && r.v.bstride % 16 == 0 &&
               (!r.HW || r.bytes % 16 == 0);
    };
    a.wide = l.cols % 8 == 0 && wide(l.in) && (!slope || wide(*slope));
    a.across = (vecs + a.lanes - 1) / a.lanes;
    a.blocks = a.across * ((l.rows + a.chunk - 1) / a.chunk);
}
cudaError_t pack_launch(const PackJobs &jobs, int dtype, void *stream)
{
    if (!jobs.count) return cudaSuccess;
    unsigned blocks = 0;
    bool wide = true, second = false;
    for (int i = 0; i < jobs.count; i++) {
        blocks += jobs.job[i].blocks;
        wide = wide && jobs.job[i].wide;
        second = second || jobs.job[i].second;
    }
    const auto of = [&](auto t) {
        using T = decltype(t);
        const auto which = [&](auto s) {
            constexpr bool S = decltype(s)::value;
            if (!wide) return k_linear_pack<T, false, false, S>;
            return jobs.count == 1 ? k_linear_pack<T, true, true, S> : k_linear_pack<T, true, false, S>;
        };
        if constexpr (sizeof(T) == 2)
            if (second) return which(std::true_type{});
        return which(std::false_type{});
    };
    const auto fn = dtype == RZ_F32 ? of(float{}) : dtype == RZ_BF16 ? of(__nv_bfloat16{}) : of(__half{});
    return launch(fn, dim3(blocks), kPackThreads, 0, stream, jobs);
}
// Chunks of rows of a pass over a matrix: about four CTAs an SM, at least 16 rows each.
unsigned pack_chunks(unsigned rows, unsigned cols)
{
    const unsigned vecs = (cols + 7) / 8, blocks = (vecs + 31) / 32;
    const unsigned want = std::max(1u, 4 * kLinSms / blocks);
    const unsigned n = std::clamp((rows + 15) / 16, 1u, std::min(want, 65535u));
    const unsigned chunk = (rows + n - 1) / n;
    return (rows + chunk - 1) / chunk;
}

template <class T, int ACT>
cudaError_t join_launch(JoinArgs a, void *stream)
{
    constexpr int VE = 16 / sizeof(T);
    // pairs: rows of them, two elements' alignment everywhere
    bool even = a.f.N % 2 == 0;
    for (const Rows *r : {&a.f.out, a.f.has_pre ? &a.f.pre : nullptr, a.f.has_residual ? &a.f.residual : nullptr})
        if (r && (reinterpret_cast<uintptr_t>(r->v.p) | static_cast<uintptr_t>(r->v.pitch) | static_cast<uintptr_t>(r->v.bstride) |
                  static_cast<uintptr_t>(r->HW ? r->bytes : 0)) % (2 * sizeof(T)))
            even = false;
    const unsigned unit = a.f.wide ? VE : even ? 2 : 1;
    const unsigned long long n = static_cast<unsigned long long>(a.f.M) * (a.f.N / unit), block = 256ull * (a.f.wide ? 1 : kJoinUnits);
    const unsigned long long blocks = (n + block - 1) / block, columns = a.sums.to ? (a.sums.C + 31) / 32 : 0;
    if (blocks + columns > 0x7fffffffull) return cudaErrorInvalidConfiguration;
    a.blocks = static_cast<unsigned>(blocks);
    const auto fn = a.f.wide ? k_linear_join<T, ACT, VE> : even ? k_linear_join<T, ACT, 2> : k_linear_join<T, ACT, 1>;
    return launch(fn, dim3(static_cast<unsigned>(blocks + columns)), 256, 0, stream, a);
}
template <class T>
cudaError_t join_of(const JoinArgs &a, void *stream)
{
    if (a.f.act == RZ_ACT_SILU) return join_launch<T, RZ_ACT_SILU>(a, stream);
    return a.f.act == RZ_ACT_GELU ? join_launch<T, RZ_ACT_GELU>(a, stream) : join_launch<T, RZ_ACT_NONE>(a, stream);
}

cudaError_t product(const Operand &a, const Operand &b, const Finish &f, int out_dtype, const Cut &c, float *part, int *status,
                    void *stream, const Sums &sums = {})
{
    Product p{};
    p.a = a;
    p.b = b;
    p.f = f;
    p.out_dtype = out_dtype;
    p.parts = c.parts;
    p.part_chunks = c.part_chunks;
    p.run_chunks = c.run_chunks;
    p.part = c.bytes ? part : nullptr;
    p.part_pitch = c.pitch;
    p.tile_n = c.tile_n;
    p.pair = c.pair;
    p.status = status;
    cudaError_t e = launch_product(p, stream);
    if (e != cudaSuccess || !c.bytes) return e;
    const JoinArgs j{f, part, c.pitch, c.parts, 0, sums};
    if (out_dtype == RZ_F32) return join_of<float>(j, stream);
    return out_dtype == RZ_BF16 ? join_of<__nv_bfloat16>(j, stream) : join_of<__half>(j, stream);
}

Finish finish_of(const Rows &out, unsigned M, unsigned N, int dtype, const Rows *pre, const Rows *residual)
{
    Finish f{};
    f.out = out;
    f.M = M;
    f.N = N;
    f.has_pre = pre != nullptr;
    f.has_residual = residual != nullptr;
    if (pre) f.pre = *pre;
    if (residual) f.residual = *residual;
    f.wide = N * dtype_size(dtype) % 16 == 0;
    for (const Rows *r : {&out, pre, residual})
        if (r && (reinterpret_cast<uintptr_t>(r->v.p) % 16 || r->v.pitch % 16 || r->v.bstride % 16 || (r->HW && r->bytes % 16)))
            f.wide = 0;
    return f;
}

// Whether a call of M rows is k_linear_rows's, which reads the weight once for eight of
// them.  K x C, rows / tiles in us: 16-bit, 16 rows, 256 x 256 2.2 / 3.2, 1024 x 1024 3.7 / 5.4,
// 4096 x 1024 11.5 / 7.0; 32 rows 2.4 / 3.2, 6.7 / 5.6, 20.6 / 6.5; float32, 16 rows 2.7 /
// 8.2, 6.1 / 11.1, 14.5 / 22.6; 32 rows 2.7 / 8.2, 10.9 / 10.1, 25.3 / 17.3.
bool is_few(unsigned M, unsigned N, unsigned C, int dtype)
{
    const double read = static_cast<double>((M + 7) / 8) * N * C;
    return M <= 8 || (M <= 32 && read <= (dtype == RZ_F32 ? 4.2e6 : 2.1e6));
}

template <class T, int ACT, int ROWS>
cudaError_t rows_launch(const RowsArgs &a, bool wide, void *stream)
{
    const unsigned pairs = (a.f.N + kRowsColumns - 1) / kRowsColumns;
    const dim3 grid((pairs * a.share + 7) / 8, (a.f.M + ROWS - 1) / ROWS);
    return launch(wide ? k_linear_rows<T, ACT, ROWS, true> : k_linear_rows<T, ACT, ROWS, false>, grid, 256, 0, stream, a);
}
template <class T, int ACT>
cudaError_t rows_of_act(const RowsArgs &a, bool wide, void *stream)
{
    if (a.f.M == 1) return rows_launch<T, ACT, 1>(a, wide, stream);
    if (a.f.M == 2) return rows_launch<T, ACT, 2>(a, wide, stream);
    return a.f.M <= 4 ? rows_launch<T, ACT, 4>(a, wide, stream) : rows_launch<T, ACT, 8>(a, wide, stream);
}
template <class T>
cudaError_t rows_of_type(const RowsArgs &a, bool wide, void *stream)
{
    if (a.f.act == RZ_ACT_SILU) return rows_of_act<T, RZ_ACT_SILU>(a, wide, stream);
    return a.f.act == RZ_ACT_GELU ? rows_of_act<T, RZ_ACT_GELU>(a, wide, stream) : rows_of_act<T, RZ_ACT_NONE>(a, wide, stream);
}
cudaError_t few_rows(const Rows &x, const Rows &w, const Finish &f, unsigned C, int dtype, void *stream)
{
    RowsArgs a{};
    a.x = x;
    a.w = w;
    a.f = f;
    a.C = C;
    const size_t es = dtype_size(dtype);
    const auto aligned = [](const Rows &r) {
        return reinterpret_cast<uintptr_t>(r.v.p) % 16 == 0 && r.v.pitch % 16 == 0 && r.v.bstride % 16 == 0 && (!r.HW || r.bytes % 16 == 0);
    };
    const bool wide = C * es % 16 == 0 && aligned(x) && aligned(w);
    // warps until there are sixteen an SM, but at least a vector a lane (one row, 1, 2, 4 and 8 warps: 1024 x 4096 5.8, 3.9, 3.1
    // and 2.8 us; 1024 x 1024 2.4, 2.1, 1.9 and 1.9; 4096 x 1024 3.0, 2.8, 3.8 and 4.7; 256 x 256 1.4, 1.6, 1.6 and 1.6)
    const unsigned vecs = wide ? static_cast<unsigned>(C * es / 16) : C;
    a.share = 1;
    while (a.share < 8 && (f.N + 1) / 2 * a.share < 16 * kLinSms && vecs >= 64u * a.share) a.share *= 2;
    if (dtype == RZ_F32) return rows_of_type<float>(a, wide, stream);
    return dtype == RZ_BF16 ? rows_of_type<__nv_bfloat16>(a, wide, stream) : rows_of_type<__half>(a, wide, stream);
}

// What a forward call lays out, and where in its workspace.
struct Forward {
    bool few;
    Laid x, w;
    Finish out;
    Cut c;
    size_t part, total;
};
Forward plan_forward(const rz_linear *d, const LinPlan &p, const rz_map *x, const void *weight, size_t weight_pitch, const rz_map *y,
                     const rz_map *pre, const rz_map *residual)
{
    const unsigned C = static_cast<unsigned>(d->C), K = static_cast<unsigned>(d->K);
    Forward f{};
    Rows rp, rr;
    if (pre) rp = rows_of(pre, p.y);
    if (residual) rr = rows_of(residual, p.y);
    f.out = finish_of(rows_of(y, p.y), p.P, K, d->dtype, pre ? &rp : nullptr, residual ? &rr : nullptr);
    f.out.act = d->act;
    f.few = is_few(p.P, K, C, d->dtype);
    f.x = lay(rows_of(x, p.x), p.P, C, d->dtype, false);
    f.w = lay(rows_of(weight, weight_pitch), K, C, d->dtype, false);
    if (f.few) return f;
    f.c = cut(p.P, K, C, d->dtype, d->dtype, !direct_out(f.out, d->dtype), products_of(f.x.planes, f.w.planes));
    f.w.at = up(f.x.bytes, 256);
    f.part = f.w.at + up(f.w.bytes, 256);
    f.total = f.part + f.c.bytes;
    return f;
}

// The same of a gradient call.
struct Backward {
    Laid dz, x, w;
    Finish dx, dw;
    Cut cx, cw;
    unsigned chunks;
    size_t sums, part, total;
};
Backward plan_backward(const rz_linear *d, const LinPlan &p, const rz_map *dy, const rz_map *x, const void *weight, size_t weight_pitch,
                       const rz_map *dx, const void *dweight, size_t dweight_pitch, int dweight_dtype)
{
    const unsigned C = static_cast<unsigned>(d->C), K = static_cast<unsigned>(d->K);
    Backward b{};
    const bool rounded = d->act != RZ_ACT_NONE;
    b.dz = lay(rows_of(dy, p.y), p.P, K, d->dtype, rounded, rounded && dweight && dweight_dtype == RZ_F32 ? 2 : 1);
    if (!dx && !dweight) b.dz.bytes = 0;
    b.x = lay(rows_of(x, p.x), p.P, C, d->dtype, false);
    if (!dweight) b.x.bytes = 0;
    b.w = lay(rows_of(weight, weight_pitch), K, C, d->dtype, false);
    if (!dx) b.w.bytes = 0;
    if (dx) {
        b.dx = finish_of(rows_of(dx, p.x), p.P, C, d->dtype, nullptr, nullptr);
        b.cx = cut(p.P, C, K, d->dtype, d->dtype, !direct_out(b.dx, d->dtype), products_of(b.w.planes, b.w.planes));
    }
    if (dweight) {
        b.dw = finish_of(rows_of(dweight, dweight_pitch), K, C, dweight_dtype, nullptr, nullptr);
        b.cw = cut(K, C, p.P, d->dtype, dweight_dtype, !direct_out(b.dw, dweight_dtype),
                   products_of(b.dz.planes, b.x.planes));
    }
    b.chunks = pack_chunks(p.P, K);
    b.x.at = up(b.dz.bytes, 256);
    b.w.at = b.x.at + up(b.x.bytes, 256);
    b.sums = b.w.at + up(b.w.bytes, 256);
    b.part = b.sums + up(sizeof(float) * b.chunks * static_cast<size_t>(K), 256);
    b.total = b.part + std::max(b.cx.bytes, b.cw.bytes);
    return b;
}

bool workspace_ok(const void *p, size_t bytes, size_t need)
{
    return need == 0 || (p && reinterpret_cast<uintptr_t>(p) % 16 == 0 && bytes >= need);
}

}  // namespace
}  // namespace rz

using namespace rz;

namespace rz {
namespace {

int forward_check(const rz_linear *d, LinPlan *p, const rz_map *x, const void *weight, size_t weight_pitch, const rz_map *residual,
                  const rz_map *pre, const rz_map *y)
{
    if (const int rc = lin_check(d, p)) return rc;
    if (p->x.empty()) return RZ_OK;
    const auto map = [](const rz_map *m, const Shape &s) { return !m || map_ok(m, s); };
    if (!x || !y || !map(x, p->x) || !map(y, p->y) || !map(residual, p->y) || !map(pre, p->y)) return RZ_ERR_ARG;
    return matrix_ok(weight, weight_pitch, d->K, d->C, p->x.es) ? RZ_OK : RZ_ERR_ARG;
}

int backward_check(const rz_linear *d, LinPlan *p, const rz_map *dy, const rz_map *x, const void *weight, size_t weight_pitch,
                   const rz_map *pre, const rz_map *dx, const void *dweight, size_t dweight_pitch, int dweight_dtype)
{
    if (const int rc = lin_check(d, p)) return rc;
    if (dweight && ((dweight_dtype != d->dtype && dweight_dtype != RZ_F32) ||
                    !matrix_ok(dweight, dweight_pitch, d->K, d->C, dtype_size(dweight_dtype))))
        return RZ_ERR_ARG;
    if (p->x.empty()) return RZ_OK;
    if (!map_ok(x, p->x) || !map_ok(dy, p->y) || (dx && !map_ok(dx, p->x))) return RZ_ERR_ARG;
    if (d->act != RZ_ACT_NONE ? !map_ok(pre, p->y) : pre && !map_ok(pre, p->y)) return RZ_ERR_ARG;
    return matrix_ok(weight, weight_pitch, d->K, d->C, p->x.es) ? RZ_OK : RZ_ERR_ARG;
}

}  // namespace
}  // namespace rz

extern "C" {

int map_linear_workspace(const rz_linear *d, const rz_map *x, const void *weight, size_t weight_pitch, const rz_map *residual,
                         const rz_map *pre, const rz_map *y, size_t *bytes)
{
    LinPlan p;
    const int rc = bytes ? forward_check(d, &p, x, weight, weight_pitch, residual, pre, y) : RZ_ERR_ARG;
    if (rc) return rc;
    *bytes = p.x.empty() ? 0 : plan_forward(d, p, x, weight, weight_pitch, y, pre, residual).total;
    return RZ_OK;
}

int map_linear(const rz_linear *d, const rz_map *x, const void *weight, size_t weight_pitch, const float *bias,
               const rz_map *residual, const rz_map *pre, const rz_map *y, void *workspace, size_t workspace_bytes, int *status,
               void *stream)
{
    LinPlan p;
    if (const int rc = forward_check(d, &p, x, weight, weight_pitch, residual, pre, y)) return rc;
    if (p.x.empty()) return RZ_OK;
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
    Forward f = plan_forward(d, p, x, weight, weight_pitch, y, pre, residual);
    if (!workspace_ok(workspace, workspace_bytes, f.total)) return RZ_ERR_ARG;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    f.out.bias = bias;
    if (f.few) return lin_status(few_rows(f.x.in, f.w.in, f.out, static_cast<unsigned>(d->C), d->dtype, stream));
    PackJobs jobs{};
    for (const Laid *l : {&f.x, &f.w})
        if (l->bytes) add_job(jobs, *l, nullptr, 0, nullptr, pack_chunks(l->rows, l->cols), ws);
    if (const cudaError_t e = pack_launch(jobs, d->dtype, stream)) return lin_status(e);
    return lin_status(product(operand(f.x, ws, false, f.x.planes), operand(f.w, ws, false, f.w.planes), f.out, d->dtype, f.c,
                              reinterpret_cast<float *>(ws + f.part), status, stream));
}

int map_linear_grad_workspace(const rz_linear *d, const rz_map *dy, const rz_map *x, const void *weight, size_t weight_pitch,
                              const rz_map *pre, const rz_map *dx, const void *dweight, size_t dweight_pitch, int dweight_dtype,
                              size_t *bytes)
{
    LinPlan p;
    const int rc = bytes ? backward_check(d, &p, dy, x, weight, weight_pitch, pre, dx, dweight, dweight_pitch, dweight_dtype) : RZ_ERR_ARG;
    if (rc) return rc;
    *bytes = p.x.empty() ? 0 : plan_backward(d, p, dy, x, weight, weight_pitch, dx, dweight, dweight_pitch, dweight_dtype).total;
    return RZ_OK;
}

int map_linear_grad(const rz_linear *d, const rz_map *dy, const rz_map *x, const void *weight, size_t weight_pitch,
                    const rz_map *pre, const rz_map *dx, void *dweight, size_t dweight_pitch, int dweight_dtype, float *dbias,
                    void *workspace, size_t workspace_bytes, int *status, void *stream)
{
    LinPlan p;
    if (const int rc = backward_check(d, &p, dy, x, weight, weight_pitch, pre, dx, dweight, dweight_pitch, dweight_dtype)) return rc;
    const size_t dw_es = dweight ? maps::dtype_size(dweight_dtype) : 0;
    if (reinterpret_cast<uintptr_t>(dbias) % 4 || reinterpret_cast<uintptr_t>(status) % 4) return RZ_ERR_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p.x.empty()) {
        cudaError_t e = dweight ? cudaMemset2DAsync(dweight, std::max<size_t>(dweight_pitch, d->C * dw_es), 0, d->C * dw_es, d->K, st)
                                : cudaSuccess;
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, 4 * static_cast<size_t>(d->K), st);
        return lin_status(e);
    }
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
    const Backward b = plan_backward(d, p, dy, x, weight, weight_pitch, dx, dweight, dweight_pitch, dweight_dtype);
    if (!workspace_ok(workspace, workspace_bytes, b.total)) return RZ_ERR_ARG;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    float *sums = reinterpret_cast<float *>(ws + b.sums), *part = reinterpret_cast<float *>(ws + b.part);
    PackJobs jobs{};
    if (dbias || b.dz.bytes) {
        Rows slope;
        const bool sloped = d->act != RZ_ACT_NONE;
        if (sloped) slope = rows_of(pre, p.y);
        add_job(jobs, b.dz, sloped ? &slope : nullptr, d->act, dbias ? sums : nullptr, b.chunks, ws);
    }
    for (const Laid *l : {&b.x, &b.w})
        if (l->bytes) add_job(jobs, *l, nullptr, 0, nullptr, pack_chunks(l->rows, l->cols), ws);
    cudaError_t e = pack_launch(jobs, d->dtype, stream);
    // dbias in the last join that there is, else by itself
    const Sums columns{sums, dbias, b.chunks, static_cast<unsigned>(d->K)};
    const bool with_w = dbias && dweight && b.cw.bytes, with_x = dbias && !with_w && dx && b.cx.bytes;
    if (dx && e == cudaSuccess)
        e = product(operand(b.dz, ws, false, b.w.planes), operand(b.w, ws, true, b.w.planes), b.dx, d->dtype, b.cx, part, status, stream,
                    with_x ? columns : Sums{});
    if (dweight && e == cudaSuccess)
        e = product(operand(b.dz, ws, true, b.dz.planes), operand(b.x, ws, true, b.x.planes), b.dw, dweight_dtype, b.cw, part, status, stream,
                    with_w ? columns : Sums{});
    if (dbias && !with_w && !with_x && e == cudaSuccess)
        e = maps::launch(k_linear_sums, dim3((columns.C + 31) / 32), 256, 0, stream, columns);
    return lin_status(e);
}

}  // extern "C"
