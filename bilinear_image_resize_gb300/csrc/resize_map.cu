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
constexpr int kMapRun = 16;     // rows a thread walks, at most
constexpr int kMapCtas = 5;     // CTAs an SM
constexpr int kMapImages = 4;   // images whose base a thread reads at a time

// Gradient: the CTAs an SM that its registers and shared memory are held to
// (16-bit 2x as above: 64 us with three, 75 with four), the output rows whose
// readers a thread has on their way in shared memory, and the rows that it
// walks at most.
template <class T, int READERS> constexpr int kGradCtas = sizeof(T) == 4 && READERS < 8 ? 4 : 3;
template <class T, int READERS> constexpr int kGradAhead = (kGradCtas<T, READERS> == 4 ? 12 : 16) / READERS;
constexpr int kGradRun = 32;

struct ResampleArgs {
    View src, base, dst;        // gradient: dst is ddst, src is dsrc; base.p null: none
    int N, src_n, H, W, OH, OW, C;
    int run;                    // rows a thread walks
    int ahead;                  // gradient: 1 or kGradAhead output rows on their way
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
__device__ __forceinline__ int2 readers(int s, int n_in, int n_out)
{
    // rounded up: the first d with floor(x_d) >= s - 1, and the first with floor(x_d) > s
    const int den = 2 * n_in;
    const int lo = s == 0 ? 0 : dev::floor_div_exact((2LL * s - 1) * n_out + n_in - 1, den);
    const int hi = s == n_in - 1 ? n_out : dev::floor_div_exact((2LL * s + 3) * n_out + n_in - 1, den);
    return make_int2(max(lo, 0), min(hi, n_out));
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

// A thread forms one column of output pixels, one vector of channels wide,
// over the block's run of rows.  It holds the horizontally interpolated values
// of the two source rows at hand and takes the lower one over as the next
// upper one, so an upscale reads each source row about once per run where a
// pixel on its own would read four taps; the sampling positions of the rows
// are formed once per block.  A table (TABLE) serves every image: it is
// interpolated once and added to each image's base.
// Instructions bound a 16-bit upscale, and writing a float32 one: 2x, 8 x 128 x
// 128 x 256 bf16 67 us, 5.0 TB/s, float32 111 us, 6.0 TB/s (paired float32
// instructions measured slower, 72 us, for the registers that pairs need).  A
// table is bound by its images: 24 x 24 x 1024 added to 16 of 37 x 50 bf16 22
// us, 5.6 TB/s (22.5 us with three CTAs an SM and no spills).
template <class S, class T, int VE, bool TABLE>
__global__ void __launch_bounds__(kMapThreads, TABLE ? 4 : kMapCtas) k_resize_map(const ResampleArgs a)
{
    __shared__ Tap taps[kMapRun];
    dev::grid_launch_dependents();
    const int y0 = blockIdx.y * a.run, rows = min(a.run, a.OH - y0), s = blockIdx.z;
    if (threadIdx.x < rows) taps[threadIdx.x] = tap(y0 + threadIdx.x, a.H, a.OH);
    __syncthreads();
    const unsigned vecs = a.C / VE;
    const unsigned i = blockIdx.x * kMapThreads + threadIdx.x;
    if (i >= a.OW * vecs) return;
    const int ox = static_cast<int>(i / vecs), c = static_cast<int>(i - ox * vecs) * VE;
    const Tap tx = tap(ox, a.W, a.OW);
    const uint8_t *src = reinterpret_cast<const uint8_t *>(map_at<S, VE>(a.src, s, 0, tx.a, a.C, c));
    const long long far = tx.b == tx.a ? 0 : static_cast<long long>(a.C) * sizeof(S);
    uint8_t *dst = reinterpret_cast<uint8_t *>(const_cast<Raw<T, VE> *>(map_at<T, VE>(a.dst, s, y0, ox, a.C, c)));
    const uint8_t *add = a.base.p ? reinterpret_cast<const uint8_t *>(map_at<T, VE>(a.base, s, y0, ox, a.C, c)) : nullptr;
    float up[VE], low[VE], step[VE];     // step = low - up
#pragma unroll
    for (int k = 0; k < VE; k++) low[k] = 0.0f;
    int iu = -1, il = -1;
    const auto across = [&](int y, float (&f)[VE]) {
        const uint8_t *p = src + y * a.src.pitch;
        const Raw<S, VE> r0 = *reinterpret_cast<const Raw<S, VE> *>(p), r1 = *reinterpret_cast<const Raw<S, VE> *>(p + far);
        float q[VE];
        unpack<S, VE>(r0, f);
        unpack<S, VE>(r1, q);
#pragma unroll
        for (int k = 0; k < VE; k++) f[k] = fmaf(tx.u, q[k] - f[k], f[k]);
    };
    dev::grid_dependency_wait();
    for (int j = 0; j < rows; j++) {
        const Tap ty = taps[j];
        if (ty.a != iu || ty.b != il) {
            // the lower row moves up and the next one comes in below: once, but for a run's first row and rows
            // that a reduction skips
            do {
#pragma unroll
                for (int k = 0; k < VE; k++) up[k] = low[k];
                iu = il;
                il = iu == ty.a ? ty.b : ty.a;
                across(il, low);
            } while (iu != ty.a || il != ty.b);
#pragma unroll
            for (int k = 0; k < VE; k++) step[k] = low[k] - up[k];
        }
        float out[VE];
#pragma unroll
        for (int k = 0; k < VE; k++) out[k] = fmaf(ty.u, step[k], up[k]);
        if (TABLE) {
            uint8_t *to = dst;
            const uint8_t *from = add;
            if (add) {
                int n = 0;
                for (; n + kMapImages <= a.N; n += kMapImages) {
                    Raw<T, VE> r[kMapImages];
#pragma unroll
                    for (int m = 0; m < kMapImages; m++)
                        r[m] = __ldcs(reinterpret_cast<const Raw<T, VE> *>(from + m * a.base.bstride));
#pragma unroll
                    for (int m = 0; m < kMapImages; m++) {
                        float f[VE];
                        unpack<T, VE>(r[m], f);
#pragma unroll
                        for (int k = 0; k < VE; k++) f[k] += out[k];
                        __stcs(reinterpret_cast<Raw<T, VE> *>(to + m * a.dst.bstride), pack<T, VE>(f));
                    }
                    from += kMapImages * a.base.bstride;
                    to += kMapImages * a.dst.bstride;
                }
                for (; n < a.N; n++, from += a.base.bstride, to += a.dst.bstride) {
                    float f[VE];
                    unpack<T, VE>(__ldcs(reinterpret_cast<const Raw<T, VE> *>(from)), f);
#pragma unroll
                    for (int k = 0; k < VE; k++) f[k] += out[k];
                    __stcs(reinterpret_cast<Raw<T, VE> *>(to), pack<T, VE>(f));
                }
            } else {
                const Raw<T, VE> r = pack<T, VE>(out);
                for (int n = 0; n < a.N; n++, to += a.dst.bstride) __stcs(reinterpret_cast<Raw<T, VE> *>(to), r);
            }
        } else {
            if (add) {
                float f[VE];
                unpack<T, VE>(__ldcs(reinterpret_cast<const Raw<T, VE> *>(add)), f);
#pragma unroll
                for (int k = 0; k < VE; k++) out[k] += f[k];
            }
            __stcs(reinterpret_cast<Raw<T, VE> *>(dst), pack<T, VE>(out));
        }
        dst += a.dst.pitch;
        if (add) add += a.base.pitch;
    }
}

// sum[y][x][c] = the images' ddst added up in order: one pass, bound by DRAM.
template <class T, int VE>
__global__ void __launch_bounds__(kMapThreads) k_sum_images(const ResampleArgs a)
{
    dev::grid_launch_dependents();
    dev::grid_dependency_wait();
    const unsigned vecs = a.C / VE;
    const unsigned i = blockIdx.x * kMapThreads + threadIdx.x;
    if (i >= a.OW * vecs) return;
    const int ox = static_cast<int>(i / vecs), c = static_cast<int>(i - ox * vecs) * VE;
    const int y0 = blockIdx.y * a.run, y1 = min(y0 + a.run, a.OH);
    for (int oy = y0; oy < y1; oy++) {
        float s[VE];
#pragma unroll
        for (int k = 0; k < VE; k++) s[k] = 0.0f;
#pragma unroll 8
        for (int n = 0; n < a.N; n++) {
            float f[VE];
            unpack<T, VE>(__ldcs(map_at<T, VE>(a.dst, n, oy, ox, a.C, c)), f);
#pragma unroll
            for (int k = 0; k < VE; k++) s[k] += f[k];
        }
        *reinterpret_cast<Raw<float, VE> *>(a.sum + (static_cast<long long>(oy) * a.OW + ox) * a.C + c) =
            pack<float, VE>(s);
    }
}

// A thread gathers one column of source pixels, one vector of channels wide,
// over the block's run of rows.  It walks the output rows that read them: each
// row's readers of its column are summed under the column's weights (READERS
// of them held in registers, formed once; more only beyond a ratio of
// READERS / 2, weighed as they come), and the sum goes to the two source rows
// that the output row lies between, so that each output row is read once per
// run and not once for each source row.  The readers come through shared
// memory, some rows ahead, in places of the thread's own: held in registers
// they left two CTAs an SM, and the launch waited on its loads.
// 2x, 8 x 128 x 128 x 256 f16: 64 us, 5.3 TB/s (89 us from registers); float32
// 104 us, 6.5 TB/s; 16 images' 37 x 50 x 1024 to a table of 24 x 24: 15.4 us
// with the sum before it (16.3 where none of the maps is left in L2).
template <class S, class T, int VE, int READERS>
__global__ void __launch_bounds__(kMapThreads, kGradCtas<T, READERS>) k_resize_map_grad(const ResampleArgs a)
{
    using V = Raw<T, VE>;
    constexpr int kRows = kGradAhead<T, READERS>;
    constexpr int kTaps = 32;
    extern __shared__ __align__(16) uint8_t grad_smem[];
    __shared__ Tap taps[kTaps];
    V *ring = reinterpret_cast<V *>(grad_smem) + threadIdx.x;
    dev::grid_launch_dependents();
    const unsigned vecs = a.C / VE;
    const unsigned i = blockIdx.x * kMapThreads + threadIdx.x;
    const bool on = i < a.W * vecs;
    const int x = on ? static_cast<int>(i / vecs) : 0, c = on ? static_cast<int>(i - x * vecs) * VE : 0;
    const int2 rx = readers(x, a.W, a.OW);
    const int count = on ? rx.y - rx.x : 0;
    const int vec_bytes = a.C * static_cast<int>(sizeof(T));    // from one reader to the next
    float wx[READERS];
#pragma unroll
    for (int k = 0; k < READERS; k++) wx[k] = k < count ? tap_weight(rx.x + k, x, a.W, a.OW) : 0.0f;
    const int y0 = blockIdx.y * a.run, y1 = min(y0 + a.run, a.H), n = blockIdx.z;
    const int lo = readers(y0, a.H, a.OH).x, hi = readers(y1 - 1, a.H, a.OH).y;
    const uint8_t *row = reinterpret_cast<const uint8_t *>(map_at<T, VE>(a.dst, n, lo, rx.x, a.C, c));
    uint8_t *out = reinterpret_cast<uint8_t *>(const_cast<Raw<S, VE> *>(map_at<S, VE>(a.src, n, y0, x, a.C, c)));
    dev::grid_dependency_wait();
    constexpr int P = kPairs<VE>;
    float2 cur[P], next[P];     // source rows y and y + 1
    int y = y0 - 1;
#pragma unroll
    for (int k = 0; k < P; k++) cur[k] = next[k] = both(0.0f);
    const auto flush = [&] {
        if (y >= y0) {
            if (on) *reinterpret_cast<Raw<S, VE> *>(out) = pack2<S, VE>(cur);
            out += a.src.pitch;
        }
        y++;
#pragma unroll
        for (int k = 0; k < P; k++) {
            cur[k] = next[k];
            next[k] = both(0.0f);
        }
    };
    // the next row's readers, copied to the thread's places in ring slot `slot`
    const uint8_t *ahead = row;
    const auto copy = [&](int slot) {
#pragma unroll
        for (int q = 0; q < READERS; q++)
            if (q < count)
                copy_async(ring + (slot * READERS + q) * kMapThreads, reinterpret_cast<const V *>(ahead + q * vec_bytes));
        ahead += a.dst.pitch;
    };
#pragma unroll
    for (int m = 0; m < kRows; m++) {
        if (m < a.ahead && lo + m < hi) copy(m);
        copies_commit();
    }
    int slot = 0;
    for (int base = lo; base < hi; base += kTaps) {
        const int some = min(kTaps, hi - base);
        __syncthreads();
        if (threadIdx.x < some) taps[threadIdx.x] = tap(base + threadIdx.x, a.H, a.OH);
        __syncthreads();
        for (int j = 0; j < some; j++) {
            float2 h[P];
#pragma unroll
            for (int k = 0; k < P; k++) h[k] = both(0.0f);
            const auto read = [&](const V &v, float w) {
                float2 f[P];
                unpack2<T, VE>(v, f);
#pragma unroll
                for (int k = 0; k < P; k++) h[k] = __ffma2_rn(both(w), f[k], h[k]);
            };
            if (a.ahead == 1)
                copies_left<0>();
            else
                copies_left<kRows - 1>();
#pragma unroll
            for (int q = 0; q < READERS; q++) {
                if (q >= count) break;
                read(ring[(slot * READERS + q) * kMapThreads], wx[q]);
            }
            if (base + j + a.ahead < hi) copy(slot);
            copies_commit();
            slot = slot + 1 == a.ahead ? 0 : slot + 1;
            for (int q = READERS; q < count; q++)
                read(*reinterpret_cast<const V *>(row + static_cast<long long>(q) * vec_bytes),
                     tap_weight(rx.x + q, x, a.W, a.OW));
            row += a.dst.pitch;
            const Tap t = taps[j];
            while (t.a > y && y < y1) flush();
            // the near row may lie before the run and the far one after it: both are then left to other blocks
            const float w = t.b == t.a ? 1.0f : 1.0f - t.u;
            if (t.a == y) {
#pragma unroll
                for (int k = 0; k < P; k++) cur[k] = __ffma2_rn(both(w), h[k], cur[k]);
            }
            if (t.b == y + 1) {
#pragma unroll
                for (int k = 0; k < P; k++) next[k] = __ffma2_rn(both(t.u), h[k], next[k]);
            }
        }
    }
    while (y < y1) flush();
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
    if (d->src_n != 1 && d->src_n != d->N) return RZ_ERR_ARG;
    // the grid's depth, and 32-bit column numbers
    if (d->src_n > 65535 || static_cast<long long>(std::max(d->W, d->out_w)) * d->C > 0x7fffffffLL)
        return RZ_ERR_UNSUPPORTED;
    return RZ_OK;
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

// Rows a thread of a table's launches walks, whose time goes with the images of
// each row and not with the rows: as many as leave eight CTAs an SM.
dim3 map_grid(int W, int vecs, int rows, int images, int *run)
{
    const long long columns = (static_cast<long long>(W) * vecs + kMapThreads - 1) / kMapThreads;
    *run = kMapRun;
    while (*run > 1 && columns * images * ((rows + *run - 1) / *run) < 8 * 152) *run /= 2;
    return dim3(static_cast<unsigned>(columns), static_cast<unsigned>((rows + *run - 1) / *run),
                static_cast<unsigned>(images));
}

// Channels a thread takes: 16 bytes of the map's own type (a float32 table is
// then read 32 bytes at a time), or 8 or 4 bytes or one element where the number
// of channels or an alignment allows no more (8 x 64 x 64 x C bf16 doubled: 24 us
// at C = 320, 29 at 324, 41 at 322, where an element at a time took 68).
int resample_vector(const rz_resample *d, const Checked &s, const rz_map *src, const rz_map *a, const rz_map *b)
{
    for (int ve = 16 / static_cast<int>(s.dst.es); ve >= 2; ve /= 2)
        if (d->C % ve == 0 && map_aligned(*src, s.src, std::min<size_t>(16, ve * s.src.es)) &&
            map_aligned(*a, s.dst, ve * s.dst.es) && (!b || map_aligned(*b, s.dst, ve * s.dst.es)))
            return ve;
    return 1;
}

// Rows a thread walks, at most `most`: the fewest row times, of the waves of
// CTAs (`slots` are resident) and what each takes, one row read beyond its run
// and the set-up, which takes about as long as kSetupRows rows (gradient of 2x,
// 8 x 128 x 128 x 256 f16: 64 us with eight rows, 68 with sixteen, whose last
// wave is half empty; 2x of 2 x 32 x 32 x 256 bf16 3.2 us with two, 4.1 with
// one).
constexpr int kSetupRows = 3;
dim3 wave_grid(int W, int vecs, int rows, int images, int slots, int most, int *run)
{
    const long long columns = (static_cast<long long>(W) * vecs + kMapThreads - 1) / kMapThreads;
    long long best = 0;
    for (int r = most; r >= 1; r /= 2) {
        const long long ctas = columns * images * ((rows + r - 1) / r);
        const long long cost = (ctas + slots - 1) / slots * (r + 1 + kSetupRows);
        if (best && cost >= best) continue;
        best = cost;
        *run = r;
    }
    return dim3(static_cast<unsigned>(columns), static_cast<unsigned>((rows + *run - 1) / *run),
                static_cast<unsigned>(images));
}

// Calls fn(S{}, T{}, VE) for the map types.
template <class Fn>
cudaError_t resample_dispatch(const rz_resample *d, int ve, Fn fn)
{
    auto width = [&](auto s, auto t) {
        if constexpr (sizeof(t) == 2)
            if (ve == 8) return fn(s, t, std::integral_constant<int, 8>{});
        if (ve == 4) return fn(s, t, std::integral_constant<int, 4>{});
        if (ve == 2) return fn(s, t, std::integral_constant<int, 2>{});
        return fn(s, t, std::integral_constant<int, 1>{});
    };
    if (d->dtype == RZ_F32) return width(float{}, float{});
    if (d->dtype == RZ_BF16)
        return d->src_dtype == RZ_F32 ? width(float{}, __nv_bfloat16{}) : width(__nv_bfloat16{}, __nv_bfloat16{});
    return d->src_dtype == RZ_F32 ? width(float{}, __half{}) : width(__half{}, __half{});
}

// Readers of a source column: two where the map shrinks, then about two a
// unit of the ratio (ends and roundings add one).  Fewer places make room for
// more CTAs (8 x 64 x 64 x 256 float32 to 150 x 150: 36 us with six, 44 with
// eight).
template <class S, class T, int V, int READERS>
cudaError_t grad_launch(ResampleArgs a, void *stream)
{
    const auto fn = k_resize_map_grad<S, T, V, READERS>;
    const dim3 grid = wave_grid(a.W, a.C / V, a.H, a.src_n, kGradCtas<T, READERS> * 152, kGradRun, &a.run);
    // the few output rows of one source row: one ahead is as good, and the less shared memory a launch takes, the more
    // of it starts under the one before (16 images' 37 x 50 x 1024 to a table of 24 x 24: 15.7 us, 19.3 with two)
    a.ahead = a.run == 1 ? 1 : kGradAhead<T, READERS>;
    const cudaError_t e = shared_opt_in(reinterpret_cast<const void *>(fn));
    if (e != cudaSuccess) return e;
    return launch(fn, grid, kMapThreads, sizeof(Raw<T, V>) * kMapThreads * READERS * a.ahead, stream, a);
}
template <class S, class T, int V>
cudaError_t grad_launch(const ResampleArgs &a, void *stream)
{
    if (a.OW <= 2LL * a.W) return grad_launch<S, T, V, 4>(a, stream);
    return 2LL * a.OW <= 5LL * a.W ? grad_launch<S, T, V, 6>(a, stream) : grad_launch<S, T, V, 8>(a, stream);
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
    const int ve = resample_vector(d, s, src, dst, base);
    return resample_status(resample_dispatch(d, ve, [&](auto ts, auto td, auto v) {
        constexpr int V = decltype(v)::value;
        const dim3 grid = a.N != a.src_n ? map_grid(a.OW, a.C / V, a.OH, 1, &a.run)
                                        : wave_grid(a.OW, a.C / V, a.OH, a.src_n, kMapCtas * 152, kMapRun, &a.run);
        const auto fn = a.N == a.src_n ? k_resize_map<decltype(ts), decltype(td), V, false>
                                       : k_resize_map<decltype(ts), decltype(td), V, true>;
        return maps::launch(fn, grid, kMapThreads, 0, stream, a);
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
    int ve = 1;
    if (s.dst.empty()) {
        a.OH = a.OW = 0;   // no reader: zeros
    } else {
        if (!maps::map_ok(ddst, s.dst) || maps::map_overlap(*ddst, s.dst, *dsrc, s.src)) return RZ_ERR_ARG;
        a.dst = maps::view(ddst);
        ve = resample_vector(d, s, dsrc, ddst, nullptr);
        const size_t need = sum_bytes(d);
        if (need) {
            if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 || workspace_bytes < need) return RZ_ERR_ARG;
            a.sum = static_cast<float *>(workspace);
        }
    }
    return resample_status(resample_dispatch(d, ve, [&](auto ts, auto td, auto v) {
        using S = decltype(ts);
        using T = decltype(td);
        constexpr int V = decltype(v)::value;
        if (a.sum) {
            const dim3 grid = map_grid(a.OW, a.C / V, a.OH, 1, &a.run);
            const cudaError_t e = maps::launch(k_sum_images<T, V>, grid, kMapThreads, 0, stream, a);
            if (e != cudaSuccess) return e;
            a.dst = {reinterpret_cast<uint8_t *>(a.sum), static_cast<long long>(sizeof(float)) * a.OW * a.C, 0};
            return grad_launch<S, float, (V == 8 ? 4 : V)>(a, stream);
        }
        return grad_launch<S, T, V>(a, stream);
    }));
}

}  // extern "C"
