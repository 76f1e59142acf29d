// Learned relative position bias by buckets, and its gradient.  Query (qy, qx) of
// a grid and key (ky, kx) of another have the bias
//   B[q][k] = T[r(ky - qy)][c(kx - qx)],
// T a head's table, r and c each axis's bucket of an offset.  For one query
// column qx the values T[r(e)][c(kx - qx)], e an offset of rows, make a small
// panel E[e][kx], and the bias of query (qy, qx) against rows ky0 .. ky1 of keys
// is one contiguous stretch of it, from row e = ky0 - qy on: the rows of a
// matrix are windows that slide over one panel.  So a CTA gathers a panel once,
// into shared memory, and then only streams: each output element costs one
// shared read and its share of a 16-byte store (with scores: of a load too).
// DRAM bounds it, the gathers are a few percent of the elements: 16 heads of 4096 by
// 4096, bf16, 537 MB in 89 us, 0.89 of a copy's rate; 1024 x 8 windows of 49 by 49 in
// 17.5 us, of which the launch and the gather are 4.
//
// The gradient runs the same sums backwards, without atomics: a thread owns
// places (e, kx) of the panel and adds up what every query row sends there, its
// elements lying one row and one key row further each time; panels of the CTA's
// query columns join in shared memory by offset, D[e][kx - qx], and a second
// kernel gathers each bucket's offsets from the CTAs' sums.  Everything runs in
// a fixed order.  4 x 12 heads of 1850 by 1850, bf16: 94 us, 68 of them the sums, which
// wait for memory (rows of 50 keys: loads of four bytes), 18 the totals and buckets.
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <type_traits>
#include <vector>

#include "map_ops.h"
#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {

using namespace maps;
using dev::grid_dependency_wait;
using dev::grid_launch_dependents;

constexpr int kPbSms = 152;
constexpr int kPbThreads = 256;
constexpr int kPbWarps = kPbThreads / 32;
constexpr int kPbFloats = 16384;    // floats of a panel: 64 KB, 72 with the forward's gaps, three CTAs an SM

// One axis as the kernels see it: axis 0 numbers rows of both grids, axis 1 what
// lies inside them (columns), except that two single-row grids are turned, so
// that a sequence has its length in axis 0.
struct PbGrid {
    int q[2], k[2];             // queries and keys
    int buckets[2];
    const int *lut[2];
    long long step[2];          // table elements between an axis's buckets
    int heads, N;
};

struct PbArgs {
    PbGrid g;
    View scores, out;           // gradient: out is dout
    const float *table;
    float *sums;                // gradient: the units' offset sums
    float *dense;               // gradient: their totals, [head][row offset][column offset]
    int tq, tk, tx;             // a tile: query rows, key rows, key columns
    int gx, gn;                 // gradient: query columns and batch entries of a unit
    int nq, nk, nx, ngx, ngn;   // tiles and groups along each
};

// A panel's place of element i: a gap after every eight, so that lanes eight
// elements apart, from any start, read from different banks.
__device__ __forceinline__ int gapped(int i) { return i + (i >> 3); }

__device__ __forceinline__ float bias_at(const PbArgs &a, int head, int i0, int i1)
{
    const int b0 = __ldg(a.g.lut[0] + i0), b1 = __ldg(a.g.lut[1] + i1);
    if (static_cast<unsigned>(b0) >= static_cast<unsigned>(a.g.buckets[0]) ||
        static_cast<unsigned>(b1) >= static_cast<unsigned>(a.g.buckets[1]))
        return 0.0f;
    return __ldg(a.table + b0 * a.g.step[0] + b1 * a.g.step[1] + head);
}

// One warp streams `len` elements: out[i] = (scores[i] +) panel[from + i].
template <class T, bool WIDE, bool SCORES>
__device__ __forceinline__ void stream_row(uint8_t *out, const uint8_t *scores, const float *panel, int from, int len)
{
    constexpr int VE = WIDE ? 16 / sizeof(T) : 1;
    using V = Raw<T, VE>;
    using E = Raw<T, 1>;
    const int lane = threadIdx.x & 31;
    const auto single = [&](int i) {
        float f[1] = {panel[gapped(from + i)]};
        if (SCORES) {
            float s[1];
            unpack<T, 1>(reinterpret_cast<const E *>(scores)[i], s);
            f[0] += s[0];
        }
        reinterpret_cast<E *>(out)[i] = pack<T, 1>(f);
    };
    int head = 0;
    if (WIDE) {
        head = min(len, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(out) & 15)) & 15) / static_cast<int>(sizeof(T)));
        if (lane < head) single(lane);
    }
    const int vecs = (len - head) / VE, at = from + head;
    constexpr int U = SCORES ? 4 : 1;
    for (int v0 = lane; v0 < vecs; v0 += 32 * U) {
        V s[U];
        if (SCORES) {
#pragma unroll
            for (int u = 0; u < U; u++)
                if (v0 + 32 * u < vecs)
                    s[u] = __ldcs(reinterpret_cast<const V *>(scores + (head + (v0 + 32 * u) * VE) * sizeof(T)));
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int v = v0 + 32 * u;
            if (v >= vecs) break;
            float f[VE], c[VE];
#pragma unroll
            for (int i = 0; i < VE; i++) f[i] = panel[VE == 8 ? 9 * v + gapped(at + i) : gapped(at + v * VE + i)];
            if (SCORES) {
                unpack<T, VE>(s[u], c);
#pragma unroll
                for (int i = 0; i < VE; i++) f[i] += c[i];
            }
            __stcs(reinterpret_cast<V *>(out + (head + v * VE) * sizeof(T)), pack<T, VE>(f));
        }
    }
    const int done = head + vecs * VE;
    if (WIDE && lane < len - done) single(done + lane);
}

// A CTA: one head, one query column, tq x tk x tx of the rest, a share of the batch.
template <class T, bool WIDE, bool SCORES>
__global__ void __launch_bounds__(kPbThreads) k_bias(const __grid_constant__ PbArgs a)
{
    extern __shared__ float panel[];
    grid_launch_dependents();
    unsigned b = blockIdx.x;
    const auto part = [&](int n) {
        const unsigned q = b / n, r = b - q * n;
        b = q;
        return static_cast<int>(r);
    };
    const int ik = part(a.nk), ix = part(a.nx), qx = part(a.g.q[1]), iq = part(a.nq), head = part(a.g.heads);
    const int group = static_cast<int>(b);
    const int q0 = iq * a.tq, q1 = min(a.g.q[0], q0 + a.tq), k0 = ik * a.tk, k1 = min(a.g.k[0], k0 + a.tk);
    const int x0 = ix * a.tx, x1 = min(a.g.k[1], x0 + a.tx), width = x1 - x0;
    const int rows = (k1 - k0) + (q1 - q0) - 1;
    grid_dependency_wait();
    // panel row e: the offset of key row k0 and query row q1 - 1, and e more
    for (int i = threadIdx.x; i < rows * width; i += kPbThreads) {
        const int e = i / width, x = i - e * width;
        panel[gapped(i)] = bias_at(a, head, e + k0 - (q1 - 1) + a.g.q[0] - 1, x0 + x - qx + a.g.q[1] - 1);
    }
    __syncthreads();
    const bool whole = width == a.g.k[1];
    const int pieces = whole ? 1 : k1 - k0, len = whole ? (k1 - k0) * width : width;
    const int n0 = group * a.gn, n1 = min(a.g.N, n0 + a.gn), count = (n1 - n0) * (q1 - q0) * pieces;
    for (int r = threadIdx.x >> 5; r < count; r += kPbWarps) {
        const int row = r / pieces, piece = r - row * pieces;
        const int n = row / (q1 - q0), qy = q0 + row - n * (q1 - q0);
        const long long image = static_cast<long long>(n0 + n) * a.g.heads + head, q = static_cast<long long>(qy) * a.g.q[1] + qx;
        const long long k = static_cast<long long>(k0 + piece) * a.g.k[1] + x0;
        stream_row<T, WIDE, SCORES>(a.out.p + image * a.out.bstride + q * a.out.pitch + k * sizeof(T),
                                    SCORES ? a.scores.p + image * a.scores.bstride + q * a.scores.pitch + k * sizeof(T) : nullptr,
                                    panel, (q1 - 1 - qy + piece) * width, len);
    }
}

// Small matrices of a large batch: a CTA holds a head's whole matrix and streams
// its share of the batch, a matrix a warp.
template <class T, bool WIDE, bool SCORES>
__global__ void __launch_bounds__(kPbThreads) k_bias_whole(const __grid_constant__ PbArgs a)
{
    extern __shared__ float panel[];
    grid_launch_dependents();
    const int head = blockIdx.x % a.g.heads, group = blockIdx.x / a.g.heads;
    const int lk = a.g.k[0] * a.g.k[1], lq = a.g.q[0] * a.g.q[1];
    const int n0 = group * a.gn, n1 = min(a.g.N, n0 + a.gn);
    grid_dependency_wait();
    for (int i = threadIdx.x; i < lq * lk; i += kPbThreads) {
        const int q = i / lk, k = i - q * lk, qy = q / a.g.q[1], ky = k / a.g.k[1];
        panel[gapped(i)] = bias_at(a, head, ky - qy + a.g.q[0] - 1,
                                   (k - ky * a.g.k[1]) - (q - qy * a.g.q[1]) + a.g.q[1] - 1);
    }
    __syncthreads();
    for (int n = n0 + (threadIdx.x >> 5); n < n1; n += kPbWarps) {
        const long long image = static_cast<long long>(n) * a.g.heads + head;
        stream_row<T, WIDE, SCORES>(a.out.p + image * a.out.bstride,
                                    SCORES ? a.scores.p + image * a.scores.bstride : nullptr, panel, 0, lq * lk);
    }
}

// s += the vectors at `row`, `count` of them `step` bytes apart, eight read before
// the first is added.  Of the last few that are missing the last one is read again
// and not added: a load under a condition waits for the one before it.
template <class T, int VE>
__device__ __forceinline__ void add_rows(const uint8_t *row, long long step, int count, float (&s)[VE])
{
    using V = Raw<T, VE>;
    constexpr int B = VE <= 2 ? 16 : 8;
    V x[B];
    float f[VE];
    for (; count >= B; count -= B) {
#pragma unroll
        for (int u = 0; u < B; u++, row += step) x[u] = __ldcs(reinterpret_cast<const V *>(row));
#pragma unroll
        for (int u = 0; u < B; u++) {
            unpack<T, VE>(x[u], f);
#pragma unroll
            for (int j = 0; j < VE; j++) s[j] += f[j];
        }
    }
    const auto rest = [&](auto size) {
        constexpr int L = decltype(size)::value;
#pragma unroll
        for (int u = 0; u < L; u++) {
            x[u] = __ldcs(reinterpret_cast<const V *>(row));
            if (u + 1 < count) row += step;
        }
#pragma unroll
        for (int u = 0; u < L; u++) {
            unpack<T, VE>(x[u], f);
#pragma unroll
            for (int j = 0; j < VE; j++)
                if (u < count) s[j] += f[j];
        }
    };
    // half a batch where that is enough: of loads of up to four bytes (of more, four of them wait as long as eight)
    constexpr int R = VE * sizeof(T) <= 4 ? B / 2 : B;
    if (R < B && count > R)
        rest(std::integral_constant<int, B>{});
    else if (count > 0)
        rest(std::integral_constant<int, R>{});
}

// Gradient: a unit is one head, a tile of rows and keys, gx query columns and gn
// batch entries; D[e][kx - qx] of it in shared memory, then in its place of `sums`:
// [head][iq][ik][e][ix][column group][batch group][column], each of full tile size.
//
// Place (m, kx) of a tile of nk key rows takes, for query row i of nq <= nk, key row
// (i + m) mod nk: every place has as many elements to add, those before the wrap
// of offset row m + nq - 1 and those after it of m - nk + nq - 1.
template <class T, int VE>
__global__ void __launch_bounds__(kPbThreads) k_bias_grad(const __grid_constant__ PbArgs a)
{
    extern __shared__ float D[];
    grid_launch_dependents();
    unsigned b = blockIdx.x;
    const auto part = [&](int n) {
        const unsigned q = b / n, r = b - q * n;
        b = q;
        return static_cast<int>(r);
    };
    const int ik = part(a.nk), ix = part(a.nx), ig = part(a.ngx), iq = part(a.nq), in = part(a.ngn), head = static_cast<int>(b);
    const int q0 = iq * a.tq, q1 = min(a.g.q[0], q0 + a.tq), k0 = ik * a.tk, k1 = min(a.g.k[0], k0 + a.tk);
    const int x0 = ix * a.tx, x1 = min(a.g.k[1], x0 + a.tx);
    const int g0 = ig * a.gx, g1 = min(a.g.q[1], g0 + a.gx);
    const int n0 = in * a.gn, n1 = min(a.g.N, n0 + a.gn);
    const int nq = q1 - q0, nk = k1 - k0, vecs = (x1 - x0) / VE;
    const int rows = a.tq + a.tk - 1, cols = a.gx + a.tx - 1;
    for (int i = threadIdx.x; i < rows * cols; i += kPbThreads) D[i] = 0.0f;
    __syncthreads();
    grid_dependency_wait();
    const int places = nk * vecs;
    // few places: several threads each, which share the batch
    const int subs = max(1, min(n1 - n0, kPbThreads / places));
    const int sub = subs > 1 ? threadIdx.x / places : 0, first = subs > 1 ? threadIdx.x - sub * places : threadIdx.x;
    const int stride = subs > 1 ? places : kPbThreads;
    for (int qx = g0; qx < g1; qx++) {
        const long long side = static_cast<long long>(a.g.k[1]) * sizeof(T), step = a.out.pitch * a.g.q[1] + side;
        for (int p0 = 0; p0 < places; p0 += stride) {
            const int p = p0 + first;
            float s[2][VE];
#pragma unroll
            for (int i = 0; i < VE; i++) s[0][i] = s[1][i] = 0.0f;
            const bool mine = p < places && sub < subs;
            const int m = mine ? p / vecs : 0, v = mine ? p - m * vecs : 0;
            if (mine) {
                const int wrap = min(nq, nk - m);
                for (int n = n0 + sub; n < n1; n += subs) {
                    const uint8_t *at = a.out.p + (static_cast<long long>(n) * a.g.heads + head) * a.out.bstride +
                                        (static_cast<long long>(q0) * a.g.q[1] + qx) * a.out.pitch +
                                        (static_cast<long long>(k0 + m) * a.g.k[1] + x0 + v * VE) * sizeof(T);
                    add_rows<T, VE>(at, step, wrap, s[0]);
                    add_rows<T, VE>(at + wrap * step - nk * side, step, nq - wrap, s[1]);
                }
            }
            const int c = v * VE + (g1 - 1 - qx);
            for (int turn = 0; turn < subs; turn++) {
                if (mine && sub == turn) {
#pragma unroll
                    for (int j = 0; j < VE; j++) D[(m + nq - 1) * cols + c + j] += s[0][j];
                    if (m - nk + nq - 1 >= 0)
#pragma unroll
                        for (int j = 0; j < VE; j++) D[(m - nk + nq - 1) * cols + c + j] += s[1][j];
                }
                if (subs > 1) __syncthreads();
            }
        }
        __syncthreads();
    }
    const int groups = a.nx * a.ngx * a.ngn, mine = (ix * a.ngx + ig) * a.ngn + in;
    float *to = a.sums + (static_cast<long long>(head) * a.nq + iq) * a.nk * rows * groups * cols +
                static_cast<long long>(ik) * rows * groups * cols + static_cast<long long>(mine) * cols;
    for (int i = threadIdx.x; i < rows * cols; i += kPbThreads) {
        const int e = i / cols, c = i - e * cols;
        to[static_cast<long long>(e) * groups * cols + c] = D[i];
    }
}

// An offset of a head a thread: its sums over the units that have it, in their order.
__global__ void __launch_bounds__(kPbThreads) k_bias_dense(const __grid_constant__ PbArgs a)
{
    grid_launch_dependents();
    const int down = a.g.q[0] + a.g.k[0] - 1, wide = a.g.q[1] + a.g.k[1] - 1;
    const long long id = static_cast<long long>(blockIdx.x) * kPbThreads + threadIdx.x;
    const int off = static_cast<int>(id % wide);
    const long long up = id / wide;
    const int ry = static_cast<int>(up % down), head = static_cast<int>(up / down);
    if (head >= a.g.heads) return;
    const int rows = a.tq + a.tk - 1, cols = a.gx + a.tx - 1, groups = a.nx * a.ngx * a.ngn;
    grid_dependency_wait();
    float s = 0.0f;
    for (int iq = 0; iq < a.nq; iq++) {
        const int q1 = min(a.g.q[0], iq * a.tq + a.tq), nq = q1 - iq * a.tq;
        // the tiles of keys that a row offset ry meets: e = below - k0 of nq + nk - 1 rows
        const int below = ry - (a.g.q[0] - 1) + (q1 - 1);
        const int first = max(0, (below - (nq + a.tk - 2) + a.tk - 1) / a.tk), last = min(a.nk - 1, below / a.tk);
        if (below < 0) continue;
        for (int ik = first; ik <= last; ik++) {
            const int k0 = ik * a.tk, e = below - k0;
            if (e >= nq + min(a.g.k[0], k0 + a.tk) - k0 - 1) continue;
            const float *row = a.sums + ((static_cast<long long>(head) * a.nq + iq) * a.nk + ik) * rows * groups * cols +
                               static_cast<long long>(e) * groups * cols;
            for (int ix = 0; ix < a.nx; ix++) {
                // column groups with this offset: from the first with a column g < q and g + at >= 0, to the last whose
                // first column has g + at < nx; its place in a group's sums is at + the group's last column
                const int x0 = ix * a.tx, nx = min(a.g.k[1], x0 + a.tx) - x0, at = off - x0 - (a.g.q[1] - 1);
                if (at + a.g.q[1] < 1 || at >= nx) continue;
                const int from = at < 0 ? -at / a.gx : 0, to = min(a.ngx, (nx - at + a.gx - 1) / a.gx);
                const float *group = row + static_cast<long long>(ix) * a.ngx * a.ngn * cols + at - 1;
                for (int i = 0; i < a.ngn; i++, group += cols)
#pragma unroll 8
                    for (int ig = from; ig < to; ig++)
                        s += group[static_cast<long long>(ig) * a.ngn * cols + min(a.g.q[1], ig * a.gx + a.gx)];
            }
        }
    }
    a.dense[id] = s;
}

// A bucket of a head a warp: the sums of its offsets.
__global__ void __launch_bounds__(kPbThreads) k_bias_fold(const __grid_constant__ PbArgs a, float *dtable)
{
    grid_launch_dependents();
    const long long id = static_cast<long long>(blockIdx.x) * kPbWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int head = static_cast<int>(id % a.g.heads);
    const long long bucket = id / a.g.heads;
    const int b1 = static_cast<int>(bucket % a.g.buckets[1]);
    const long long b0 = bucket / a.g.buckets[1];
    if (b0 >= a.g.buckets[0]) return;
    const int down = a.g.q[0] + a.g.k[0] - 1, wide = a.g.q[1] + a.g.k[1] - 1;
    grid_dependency_wait();
    const float *from = a.dense + static_cast<long long>(head) * down * wide;
    float s = 0.0f;
    if (wide <= 8) {            // rows of a few offsets: one a lane
        unsigned mine = 0;
        for (int c = 0; c < wide; c++) mine |= (__ldg(a.g.lut[1] + c) == b1 ? 1u : 0u) << c;
        for (; mine; mine &= mine - 1) {
            const float *column = from + __ffs(mine) - 1;
#pragma unroll 8
            for (int r = lane; r < down; r += 32) {
                // read whether it is the bucket's or not: a load under a condition waits for the one before it
                const float v = column[static_cast<long long>(r) * wide];
                s += __ldg(a.g.lut[0] + r) == b0 ? v : 0.0f;
            }
        }
    } else {
        // the bucket's rows, four of them asked for at once (past the last that one again, and not added)
        for (int c0 = 0; c0 < wide; c0 += 32) {
            const bool mine = c0 + lane < wide && __ldg(a.g.lut[1] + c0 + lane) == b1;
            if (!__any_sync(0xffffffffu, mine)) continue;
            const float *column = from + min(c0 + lane, wide - 1);
            for (int r0 = 0; r0 < down; r0 += 32) {
                unsigned left = __ballot_sync(0xffffffffu, r0 + lane < down && __ldg(a.g.lut[0] + r0 + lane) == b0);
                while (left) {
                    int r[4], n = 0;
                    float v[4];
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        r[u] = left ? r0 + __ffs(left) - 1 : r[u ? u - 1 : 0];
                        n += left != 0;
                        left &= left - 1;
                    }
#pragma unroll
                    for (int u = 0; u < 4; u++) v[u] = column[static_cast<long long>(r[u]) * wide];
#pragma unroll
                    for (int u = 0; u < 4; u++)
                        if (mine && u < n) s += v[u];
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) dtable[b0 * a.g.step[0] + b1 * a.g.step[1] + head] = s;
}

// ------------------------------------------------------------------ host side

int pb_check(const rz_bias *d, Shape *s)
{
    if (!d) return RZ_ERR_ARG;
    const size_t es = dtype_size(d->dtype);
    if (!es || d->N < 0 || d->heads < 1 || d->q_h < 0 || d->q_w < 0 || d->k_h < 0 || d->k_w < 0) return RZ_ERR_ARG;
    const long long lq = static_cast<long long>(d->q_h) * d->q_w, lk = static_cast<long long>(d->k_h) * d->k_w;
    if (lq > RZ_MAX_DIM || lk > RZ_MAX_DIM || std::max({d->q_h, d->q_w, d->k_h, d->k_w}) > RZ_MAX_DIM) return RZ_ERR_ARG;
    if (d->row_buckets < 1 || d->col_buckets < 1 || static_cast<long long>(d->row_buckets) * d->col_buckets > (1 << 22))
        return RZ_ERR_ARG;
    const long long images = static_cast<long long>(d->N) * d->heads;
    if (images > (1 << 24) || d->heads > RZ_MAX_DIM) return RZ_ERR_ARG;
    *s = {images, lq, 1, std::max(lk, 1LL), es};
    if (lk == 0) s->H = 0;
    return s->empty() || shape_ok(*s) ? RZ_OK : RZ_ERR_ARG;
}

void pb_grid(const rz_bias *d, const int *rows, const int *cols, PbGrid &g)
{
    const bool turn = d->q_h == 1 && d->k_h == 1;
    const int r = turn ? 1 : 0, c = 1 - r;
    g.q[r] = d->q_h;
    g.q[c] = d->q_w;
    g.k[r] = d->k_h;
    g.k[c] = d->k_w;
    g.buckets[r] = d->row_buckets;
    g.buckets[c] = d->col_buckets;
    g.lut[r] = rows;
    g.lut[c] = cols;
    g.step[r] = static_cast<long long>(d->col_buckets) * d->heads;
    g.step[c] = d->heads;
    g.heads = d->heads;
    g.N = d->N;
}

int ceil_div(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

// Tiles of the general forward: rows of 64 by 64 where the panel holds them, else
// fewer, and key columns cut last.
void pb_tiles(PbArgs &a, int columns)
{
    const auto panel = [&] { return static_cast<long long>(a.tq + a.tk - 1) * columns; };
    a.tq = std::min(a.g.q[0], 64);
    a.tk = std::min(a.g.k[0], columns == 1 ? 4096 : 64);
    while (panel() > kPbFloats && (a.tq > 8 || a.tk > 8)) (a.tq > a.tk ? a.tq : a.tk) = (std::max(a.tq, a.tk) + 1) / 2;
}

void pb_count(PbArgs &a)
{
    a.nq = ceil_div(a.g.q[0], a.tq);
    a.nk = ceil_div(a.g.k[0], a.tk);
    a.nx = ceil_div(a.g.k[1], a.tx);
}

void pb_plan_forward(PbArgs &a)
{
    pb_tiles(a, a.g.k[1]);
    a.tx = std::min(a.g.k[1], kPbFloats / (a.tq + a.tk - 1));
    if (a.tx < a.g.k[1] && a.tx > 8) a.tx -= a.tx % 8;
    pb_count(a);
    const auto ctas = [&] { return static_cast<long long>(a.nk) * a.nx * a.g.q[1] * a.nq * a.g.heads; };
    while (ctas() < 6 * kPbSms && a.tq > 8) {
        a.tq = (a.tq + 1) / 2;
        pb_count(a);
    }
    const int split = static_cast<int>(std::clamp<long long>(6 * kPbSms / std::max(1LL, ctas()), 1, a.g.N));
    a.gn = ceil_div(a.g.N, split);
    a.ngn = ceil_div(a.g.N, a.gn);
}

void pb_plan_grad(PbArgs &a)
{
    int most = a.g.k[1] == 1 ? 2048 : 64;
    // even tiles of key rows, and no more query rows than the last of them has
    const auto rows = [&] {
        a.tk = ceil_div(a.g.k[0], ceil_div(a.g.k[0], most));
        a.tq = std::min(a.g.q[0], a.g.k[0] - (ceil_div(a.g.k[0], a.tk) - 1) * a.tk);
    };
    rows();
    a.tx = std::min(a.g.k[1], 128);
    a.gx = std::min(a.g.q[1], 128);
    const auto panel = [&] { return static_cast<long long>(a.tq + a.tk - 1) * (a.gx + a.tx - 1); };
    // a unit's columns first, then its rows
    while (panel() > kPbFloats && a.gx > 32) a.gx = (a.gx + 1) / 2;
    while (panel() > kPbFloats && most > 8) {
        most /= 2;
        rows();
    }
    pb_count(a);
    const auto units = [&] { return static_cast<long long>(a.nk) * a.nx * a.nq * a.g.heads; };
    const long long want = 4 * kPbSms;
    const int groups = static_cast<int>(std::clamp<long long>(want / units(), 1, a.g.q[1]));
    a.gx = std::min(a.gx, ceil_div(a.g.q[1], groups));
    a.ngx = ceil_div(a.g.q[1], a.gx);
    const int split = static_cast<int>(std::clamp<long long>(want / (units() * a.ngx), 1, a.g.N));
    a.gn = ceil_div(a.g.N, split);
    a.ngn = ceil_div(a.g.N, a.gn);
    // long sequences of few heads: fewer query rows a unit (2 x 8 heads of 4096 to 4096: 440 us, in units
    // of 2048 rows 4900)
    while (units() * a.ngx * a.ngn < want / 2 && a.tq > 32) {
        a.tq = (a.tq + 1) / 2;
        pb_count(a);
    }
}

long long pb_units(const PbArgs &a) { return static_cast<long long>(a.nk) * a.nx * a.ngx * a.nq * a.ngn * a.g.heads; }
// The workspace: the units' sums, then their totals.
size_t pb_dense_at(const PbArgs &a)
{
    return (sizeof(float) * static_cast<size_t>(pb_units(a)) * static_cast<size_t>(a.tq + a.tk - 1) *
                static_cast<size_t>(a.gx + a.tx - 1) + 255) / 256 * 256;
}
long long pb_offsets(const PbArgs &a)
{
    return static_cast<long long>(a.g.q[0] + a.g.k[0] - 1) * (a.g.q[1] + a.g.k[1] - 1) * a.g.heads;
}
size_t pb_bytes(const PbArgs &a) { return pb_dense_at(a) + sizeof(float) * static_cast<size_t>(pb_offsets(a)); }
bool pb_too_many(const PbArgs &a)
{
    const long long entries = static_cast<long long>(a.g.buckets[0]) * a.g.buckets[1] * a.g.heads;
    return pb_units(a) > 0x7fffffffLL || pb_offsets(a) / kPbThreads >= 0x7fffffffLL || entries / kPbWarps >= 0x7fffffffLL;
}

int pb_status(cudaError_t e)
{
    if (e == cudaSuccess) return RZ_OK;
    if (e == cudaErrorNotSupported) return RZ_ERR_UNSUPPORTED;
    record_cuda_error(static_cast<int>(e));
    return RZ_ERR_CUDA;
}

template <class K>
cudaError_t pb_launch(K fn, long long blocks, size_t smem, void *stream, const PbArgs &a)
{
    if (smem > 48 * 1024)
        if (const cudaError_t e = shared_opt_in(reinterpret_cast<const void *>(fn))) return e;
    return launch(fn, dim3(static_cast<unsigned>(blocks)), kPbThreads, smem, stream, a);
}

template <class T, bool WIDE, bool SCORES>
cudaError_t pb_forward(PbArgs &a, bool whole, void *stream)
{
    const auto bytes = [](long long n) { return sizeof(float) * static_cast<size_t>(n + n / 8 + 1); };
    if (whole) {
        const int split = static_cast<int>(std::clamp<long long>(ceil_div(4 * kPbSms, a.g.heads), 1, ceil_div(a.g.N, kPbWarps)));
        a.gn = ceil_div(a.g.N, split);
        const long long n = static_cast<long long>(a.g.q[0]) * a.g.q[1] * a.g.k[0] * a.g.k[1];
        return pb_launch(k_bias_whole<T, WIDE, SCORES>, static_cast<long long>(a.g.heads) * ceil_div(a.g.N, a.gn), bytes(n),
                         stream, a);
    }
    pb_plan_forward(a);
    const long long blocks = static_cast<long long>(a.nk) * a.nx * a.g.q[1] * a.nq * a.g.heads * a.ngn;
    if (blocks > 0x7fffffffLL) return cudaErrorNotSupported;
    return pb_launch(k_bias<T, WIDE, SCORES>, blocks, bytes(static_cast<long long>(a.tq + a.tk - 1) * a.tx), stream, a);
}

template <class T>
cudaError_t pb_forward_of(PbArgs &a, bool wide, bool scores, bool whole, void *stream)
{
    if (wide) return scores ? pb_forward<T, true, true>(a, whole, stream) : pb_forward<T, true, false>(a, whole, stream);
    return scores ? pb_forward<T, false, true>(a, whole, stream) : pb_forward<T, false, false>(a, whole, stream);
}

template <class T>
cudaError_t pb_grad_of(const PbArgs &a, int ve, void *stream)
{
    constexpr int W = 16 / sizeof(T);
    const size_t smem = sizeof(float) * static_cast<size_t>(a.tq + a.tk - 1) * static_cast<size_t>(a.gx + a.tx - 1);
    const long long n = pb_units(a);
    if (ve == W) return pb_launch(k_bias_grad<T, W>, n, smem, stream, a);
    if (ve == W / 2) return pb_launch(k_bias_grad<T, W / 2>, n, smem, stream, a);
    if (ve == 2) return pb_launch(k_bias_grad<T, 2>, n, smem, stream, a);
    return pb_launch(k_bias_grad<T, 1>, n, smem, stream, a);
}

}  // namespace
}  // namespace rz

using namespace rz;

extern "C" {

int map_position_bias(const rz_bias *d, const float *table, const int *rows, const int *cols, const rz_map *scores,
                      const rz_map *out, void *stream)
{
    maps::Shape s;
    if (const int rc = pb_check(d, &s)) return rc;
    if (s.empty()) return RZ_OK;
    const auto odd = [](const void *p) { return !p || reinterpret_cast<uintptr_t>(p) % 4 != 0; };
    if (odd(table) || odd(rows) || odd(cols)) return RZ_ERR_ARG;
    if (!maps::map_ok(out, s) || (scores && !maps::map_ok(scores, s))) return RZ_ERR_ARG;
    if (scores && !maps::map_same(*scores, *out, s) && maps::map_overlap(*scores, s, *out, s)) return RZ_ERR_ARG;
    PbArgs a{};
    pb_grid(d, rows, cols, a.g);
    a.table = table;
    a.out = maps::view(out);
    if (scores) a.scores = maps::view(scores);
    // rows that begin alike in their 16 bytes let both be read and written in vectors, from wherever they begin
    const auto apart = [&](size_t x, size_t y) { return (x ^ y) % 16 == 0; };
    const bool wide = !scores || (apart(reinterpret_cast<size_t>(scores->data), reinterpret_cast<size_t>(out->data)) &&
                                  (s.H == 1 || apart(scores->pitch, out->pitch)) &&
                                  (s.N == 1 || apart(scores->batch_stride, out->batch_stride)));
    const auto joined = [&](const rz_map *m) { return !m || maps::rows_joined(*m, s); };
    // A matrix held whole costs its gather, panels a CTA for each query column and head.  Whole / panels in us: 8 heads of
    // 49 x 49, batches of 8, 16 and 1024 5.4 / 4.4, 5.6 / 6.5 and 14 / 149; 4 of 64 x 64, 16 and 64 6.4 / 3.8 and 6.1 / 7.7; 8 of
    // 120 x 120, 16 and 64 17 / 8 and 19 / 22.  (A warp takes a matrix of a head: fewer than eight leave some idle.)
    const bool whole = d->N >= 8 && s.N >= 48 + s.H * s.C / 36 && s.H * s.C <= kPbFloats && joined(out) && joined(scores);
    if (d->dtype == RZ_F32) return pb_status(pb_forward_of<float>(a, wide, scores != nullptr, whole, stream));
    if (d->dtype == RZ_BF16) return pb_status(pb_forward_of<__nv_bfloat16>(a, wide, scores != nullptr, whole, stream));
    return pb_status(pb_forward_of<__half>(a, wide, scores != nullptr, whole, stream));
}

int map_position_bias_grad_workspace(const rz_bias *d, size_t *bytes)
{
    maps::Shape s;
    const int rc = bytes ? pb_check(d, &s) : RZ_ERR_ARG;
    if (rc) return rc;
    *bytes = 0;
    if (s.empty()) return RZ_OK;
    PbArgs a{};
    pb_grid(d, nullptr, nullptr, a.g);
    pb_plan_grad(a);
    if (pb_too_many(a)) return RZ_ERR_UNSUPPORTED;
    *bytes = pb_bytes(a);
    return RZ_OK;
}

int map_position_bias_grad(const rz_bias *d, const rz_map *dout, const int *rows, const int *cols, float *dtable,
                           void *workspace, size_t workspace_bytes, void *stream)
{
    maps::Shape s;
    if (const int rc = pb_check(d, &s)) return rc;
    if (!dtable || reinterpret_cast<uintptr_t>(dtable) % 4) return RZ_ERR_ARG;
    const long long buckets = static_cast<long long>(d->row_buckets) * d->col_buckets;
    if (s.empty())
        return pb_status(cudaMemsetAsync(dtable, 0, sizeof(float) * static_cast<size_t>(buckets * d->heads),
                                         static_cast<cudaStream_t>(stream)));
    const auto odd = [](const void *p) { return !p || reinterpret_cast<uintptr_t>(p) % 4 != 0; };
    if (odd(rows) || odd(cols) || !maps::map_ok(dout, s)) return RZ_ERR_ARG;
    PbArgs a{};
    pb_grid(d, rows, cols, a.g);
    pb_plan_grad(a);
    if (pb_too_many(a)) return RZ_ERR_UNSUPPORTED;
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 || workspace_bytes < pb_bytes(a)) return RZ_ERR_ARG;
    a.out = maps::view(dout);
    a.sums = static_cast<float *>(workspace);
    a.dense = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + pb_dense_at(a));
    // the widest vectors that every row, key row and tile of columns is made of
    int ve = 16 / static_cast<int>(s.es);
    while (ve > 1 && (a.g.k[1] % ve || a.tx % ve || !maps::map_aligned(*dout, s, ve * s.es))) ve /= 2;
    cudaError_t e;
    if (d->dtype == RZ_F32)
        e = pb_grad_of<float>(a, ve, stream);
    else if (d->dtype == RZ_BF16)
        e = pb_grad_of<__nv_bfloat16>(a, ve, stream);
    else
        e = pb_grad_of<__half>(a, ve, stream);
    if (e == cudaSuccess)
        e = maps::launch(k_bias_dense, dim3(static_cast<unsigned>((pb_offsets(a) + kPbThreads - 1) / kPbThreads)), kPbThreads, 0,
                         stream, a);
    if (e == cudaSuccess)
        e = maps::launch(k_bias_fold, dim3(static_cast<unsigned>((buckets * d->heads + kPbWarps - 1) / kPbWarps)), kPbThreads, 0,
                         stream, a, dtable);
    return pb_status(e);
}

int map_position_buckets(int queries, int keys, int shift, int exact, int side, int reach, int *out)
{
    if (queries < 1 || keys < 1 || queries > RZ_MAX_DIM || keys > RZ_MAX_DIM || shift < -RZ_MAX_DIM || shift > RZ_MAX_DIM ||
        exact < 1 || side < exact || side > 1024 || reach <= exact || reach > RZ_MAX_DIM || !out)
        return RZ_ERR_ARG;
    const int r = side - exact;
    // d^r exact^j >= exact^r reach^j: by logarithms, and where those are too near to tell in whole numbers
    const auto reached = [&](int d, int j) {
        const double l = r * std::log(static_cast<double>(d) / exact) - j * std::log(static_cast<double>(reach) / exact);
        if (std::fabs(l) > 1e-9) return l > 0;
        std::vector<uint32_t> u, v;
        const auto power = [](std::vector<uint32_t> &x, int b, int n) {
            for (; n > 0; n--) {
                uint64_t carry = 0;
                for (uint32_t &limb : x) {
                    carry += static_cast<uint64_t>(limb) * static_cast<uint32_t>(b);
                    limb = static_cast<uint32_t>(carry);
                    carry >>= 32;
                }
                if (carry) x.push_back(static_cast<uint32_t>(carry));
            }
        };
        u.assign(1, 1u);
        v.assign(1, 1u);
        power(u, d, r);
        power(u, exact, j);
        power(v, exact, r);
        power(v, reach, j);
        if (u.size() != v.size()) return u.size() > v.size();
        for (size_t i = u.size(); i-- > 0;)
            if (u[i] != v[i]) return u[i] > v[i];
        return true;
    };
    std::vector<int> starts;    // the least distance of bucket exact + j
    try {
        for (int j = 1; j < r; j++) {
            int lo = exact, hi = reach;
            while (lo < hi) {
                const int d = lo + (hi - lo) / 2;
                if (reached(d, j))
                    hi = d;
                else
                    lo = d + 1;
            }
            starts.push_back(lo);
        }
    } catch (...) {
        return RZ_ERR_NOMEM;
    }
    for (int i = 0; i < queries + keys - 1; i++) {
        const int d = i - (queries - 1) - shift, m = std::abs(d);
        int b = m;
        if (m >= exact)
            b = std::min(side - 1, exact + static_cast<int>(std::upper_bound(starts.begin(), starts.end(), m) - starts.begin()));
        out[i] = side - 1 + (d < 0 ? -b : b);
    }
    return RZ_OK;
}

}  // extern "C"
