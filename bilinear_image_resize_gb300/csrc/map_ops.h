// Shared by the feature-map operators (group_norm.cu, map_dropout.cu,
// resize_map.cu): element types, channels-last addressing, the activation
// functions and the counter-based generator.  Maps are (N, H, W, C) with the
// pixels of a row packed, a byte pitch between rows and a byte stride between
// images.  All arithmetic is float32; a 16-bit result is rounded once, as it
// is stored.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "gbresize.h"
#include "rz_device.h"

namespace rz {
namespace maps {

// ------------------------------------------------------------------ host side

inline size_t dtype_size(int dtype) { return dtype == RZ_F32 ? 4 : (dtype == RZ_BF16 || dtype == RZ_F16) ? 2 : 0; }

// A map's geometry as the entry points check it.
struct Shape {
    long long N, H, W, C;
    size_t es;
    size_t row() const { return static_cast<size_t>(W) * static_cast<size_t>(C) * es; }
    bool empty() const { return N == 0 || H == 0 || W == 0; }
    // bytes from the first to past the last element of a non-empty map
    size_t extent(const rz_map &m) const
    {
        return static_cast<size_t>(N - 1) * m.batch_stride + static_cast<size_t>(H - 1) * m.pitch + row();
    }
};

inline bool map_overlap(const rz_map &a, const Shape &sa, const rz_map &b, const Shape &sb)
{
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.data), pb = reinterpret_cast<uintptr_t>(b.data);
    return pa < pb + sb.extent(b) && pb < pa + sa.extent(a);
}

// Geometry limits: no negative size, C in [1, RZ_MAX_DIM], at most 2^31 - 1
// pixels an image (the kernels count pixels in 32 bits) and 2^46 elements, so
// that no offset wraps 64 bits.
inline bool shape_ok(const Shape &s)
{
    if (s.N < 0 || s.H < 0 || s.W < 0 || s.C < 1 || s.C > RZ_MAX_DIM) return false;
    const long long px = s.H * s.W;
    return px <= 0x7fffffffLL && (px == 0 || s.N <= (1LL << 46) / (px * s.C));
}

// Pointer, alignment, pitch and stride of one map (of a non-empty shape).  Rows
// and images lie within 2^60 bytes, so that neither they nor extent() wrap.
inline bool map_ok(const rz_map *m, const Shape &s)
{
    constexpr size_t kMost = size_t{1} << 60;
    if (!m || !m->data) return false;
    if (reinterpret_cast<uintptr_t>(m->data) % s.es || m->pitch % s.es || m->batch_stride % s.es) return false;
    if (m->pitch > (size_t{1} << 46) || m->batch_stride > (size_t{1} << 46)) return false;
    const size_t below = static_cast<size_t>(s.H - 1), before = static_cast<size_t>(s.N - 1);
    if (below && (m->pitch < s.row() || m->pitch > kMost / below)) return false;
    return !before || (m->batch_stride >= below * m->pitch + s.row() && m->batch_stride <= kMost / before);
}

inline bool rows_joined(const rz_map &m, const Shape &s) { return s.H == 1 || m.pitch == s.row(); }

// Whether every vector of `bytes` at a multiple of `bytes` from a row's start
// is aligned.
inline bool map_aligned(const rz_map &m, const Shape &s, size_t bytes)
{
    return reinterpret_cast<uintptr_t>(m.data) % bytes == 0 && (s.H == 1 || m.pitch % bytes == 0) &&
           (s.N == 1 || m.batch_stride % bytes == 0);
}

// The same elements at the same places.
inline bool map_same(const rz_map &a, const rz_map &b, const Shape &s)
{
    return a.data == b.data && (s.H == 1 || a.pitch == b.pitch) && (s.N == 1 || a.batch_stride == b.batch_stride);
}

// Launch of one kernel on `stream`; chained launches of one call are
// programmatic dependents of their predecessors.  Returns a cudaError_t.
template <class... P, class... A>
inline cudaError_t launch(void (*fn)(P...), dim3 grid, int threads, size_t smem, void *stream, A &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...);
}

// Opts a kernel into kMapShared bytes of shared memory (two CTAs an SM), once a
// device (group_norm.cu).
constexpr int kMapShared = 112 * 1024;
cudaError_t shared_opt_in(const void *fn);

// ---------------------------------------------------------------- device side

// A map as a kernel reads it; W is the number of pixels in a row, the whole
// image where its rows follow one another without padding.
struct View {
    uint8_t *p;
    long long pitch, bstride;
};

inline View view(const rz_map *m)
{
    return {static_cast<uint8_t *>(m->data), static_cast<long long>(m->pitch), static_cast<long long>(m->batch_stride)};
}

// Byte offset of pixel `px` of an image with W pixels a row, px_bytes each.
__device__ __forceinline__ long long pixel_off(unsigned px, unsigned W, bool joined, long long pitch, int px_bytes)
{
    if (joined) return static_cast<long long>(px) * px_bytes;
    const unsigned row = px / W;
    return row * pitch + static_cast<long long>(px - row * W) * px_bytes;
}

// VE consecutive elements of type T, moved as one access.
template <int BYTES> struct RawOf;
template <> struct RawOf<2> { using type = unsigned short; };
template <> struct RawOf<4> { using type = unsigned; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<16> { using type = uint4; };
template <> struct RawOf<32> { struct alignas(16) type { uint4 a, b; }; };
template <class T, int VE> using Raw = typename RawOf<sizeof(T) * VE>::type;

__device__ __forceinline__ void unpack_pair(unsigned w, float &a, float &b, __nv_bfloat16)
{
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void unpack_pair(unsigned w, float &a, float &b, __half)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    a = f.x;
    b = f.y;
}
__device__ __forceinline__ unsigned pack_pair(float a, float b, __nv_bfloat16)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const unsigned *>(&h);
}
__device__ __forceinline__ unsigned pack_pair(float a, float b, __half)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const unsigned *>(&h);
}

template <class T, int VE>
__device__ __forceinline__ void unpack(const Raw<T, VE> &r, float (&f)[VE])
{
    if constexpr (sizeof(T) == 4) {
        const float *s = reinterpret_cast<const float *>(&r);
#pragma unroll
        for (int i = 0; i < VE; i++) f[i] = s[i];
    } else if constexpr (VE == 1) {
        f[0] = static_cast<float>(*reinterpret_cast<const T *>(&r));
    } else {
        const unsigned *w = reinterpret_cast<const unsigned *>(&r);
#pragma unroll
        for (int i = 0; i < VE / 2; i++) unpack_pair(w[i], f[2 * i], f[2 * i + 1], T{});
    }
}

template <class T, int VE>
__device__ __forceinline__ Raw<T, VE> pack(const float (&f)[VE])
{
    Raw<T, VE> r;
    if constexpr (sizeof(T) == 4) {
        float *s = reinterpret_cast<float *>(&r);
#pragma unroll
        for (int i = 0; i < VE; i++) s[i] = f[i];
    } else if constexpr (VE == 1) {
        const T h = static_cast<T>(f[0]);
        r = *reinterpret_cast<const Raw<T, VE> *>(&h);
    } else {
        unsigned *w = reinterpret_cast<unsigned *>(&r);
#pragma unroll
        for (int i = 0; i < VE / 2; i++) w[i] = pack_pair(f[2 * i], f[2 * i + 1], T{});
    }
    return r;
}

// VE elements as pairs, for the paired float32 instructions (half the issue
// slots of two scalar ones); a single element leaves the second half 0.
template <int VE> constexpr int kPairs = (VE + 1) / 2;

template <class T, int VE>
__device__ __forceinline__ void unpack2(const Raw<T, VE> &r, float2 (&f)[kPairs<VE>])
{
    float s[2 * kPairs<VE>];
    s[2 * kPairs<VE> - 1] = 0.0f;
    unpack<T, VE>(r, reinterpret_cast<float(&)[VE]>(s));
#pragma unroll
    for (int i = 0; i < kPairs<VE>; i++) f[i] = make_float2(s[2 * i], s[2 * i + 1]);
}

template <class T, int VE>
__device__ __forceinline__ Raw<T, VE> pack2(const float2 (&f)[kPairs<VE>])
{
    float s[2 * kPairs<VE>];
#pragma unroll
    for (int i = 0; i < kPairs<VE>; i++) {
        s[2 * i] = f[i].x;
        s[2 * i + 1] = f[i].y;
    }
    return pack<T, VE>(reinterpret_cast<float(&)[VE]>(s));
}

// Copies a vector to a place in shared memory that only this thread reads:
// asynchronously, in the thread's open group of copies, where it is wide enough.
template <class V>
__device__ __forceinline__ void copy_async(V *to, const V *from)
{
    if constexpr (sizeof(V) == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dev::smem_addr(to)), "l"(from) : "memory");
    else if constexpr (sizeof(V) >= 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dev::smem_addr(to)), "l"(from),
                     "n"(sizeof(V))
                     : "memory");
    else
        *to = *from;
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until all but the last N groups have arrived.
template <int N>
__device__ __forceinline__ void copies_left()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Dropout's mask: Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", SC'11), ten rounds on the counter
// (block, offset) under the key `seed`.  Its four words are cut into eight
// 16-bit lanes, lane j the low or high half of word j / 2, so that one block
// serves eight elements: 16 bits set the drop rate to 1 / 65536, which the
// scale takes into account, and halve the generator's work, the larger part of
// the arithmetic.  An element is dropped where its 16 bits are at most
// `top` = round(65536 p) - 1, else multiplied by `scale`.
struct Drop {
    unsigned key[20];       // the rounds' keys: the same for every thread, formed on the host
    unsigned off_lo, off_hi;
    unsigned top;           // in the high half, the low one all ones: what a kept half of a word, shifted up, is above
    float scale;
};

// Drop rate in 65536ths, half-up; 0 drops nothing.
inline unsigned drop_threshold(const rz_drop *d) { return d ? static_cast<unsigned>(d->p * 65536.0 + 0.5) : 0u; }
inline bool drop_ok(const rz_drop *d) { return !d || (d->p >= 0.0 && d->p <= 1.0); }
inline Drop make_drop(const rz_drop *d)
{
    Drop r = {};
    r.scale = 1.0f;
    const unsigned t = drop_threshold(d);
    if (t == 0) return r;
    const uint64_t seed = d->seed, offset = d->offset;
    for (unsigned i = 0; i < 10; i++) {
        r.key[2 * i] = static_cast<unsigned>(seed) + i * 0x9E3779B9u;
        r.key[2 * i + 1] = static_cast<unsigned>(seed >> 32) + i * 0xBB67AE85u;
    }
    r.off_lo = static_cast<unsigned>(offset);
    r.off_hi = static_cast<unsigned>(offset >> 32);
    r.top = (t - 1) << 16 | 0xffffu;
    r.scale = t < 65536 ? static_cast<float>(65536.0 / (65536 - t)) : 0.0f;
    return r;
}

__device__ __forceinline__ uint4 philox(unsigned long long block, const Drop &d)
{
    uint4 c = {static_cast<unsigned>(block), static_cast<unsigned>(block >> 32), d.off_lo, d.off_hi};
#pragma unroll
    for (int r = 0; r < 10; r++) {
        const unsigned long long a = static_cast<unsigned long long>(c.x) * 0xD2511F53u;
        const unsigned long long b = static_cast<unsigned long long>(c.z) * 0xCD9E8D57u;
        c = {static_cast<unsigned>(b >> 32) ^ c.y ^ d.key[2 * r], static_cast<unsigned>(b),
             static_cast<unsigned>(a >> 32) ^ c.w ^ d.key[2 * r + 1], static_cast<unsigned>(a)};
    }
    return c;
}

// Whether the two elements of a word are kept.
__device__ __forceinline__ void kept_pair(unsigned w, const Drop &d, bool &lo, bool &hi)
{
    lo = w << 16 > d.top;
    hi = w > d.top;
}

// Which of the VE elements from lane `lane` of a block (a multiple of VE, which
// divides eight) are kept.
template <int VE>
__device__ __forceinline__ void kept(bool (&keep)[VE], unsigned long long block, unsigned lane, const Drop &d)
{
    const uint4 c = philox(block, d);
    if constexpr (VE == 8) {
        const unsigned w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 4; i++) kept_pair(w[i], d, keep[2 * i], keep[2 * i + 1]);
    } else if constexpr (VE == 4) {
        kept_pair(lane ? c.z : c.x, d, keep[0], keep[1]);
        kept_pair(lane ? c.w : c.y, d, keep[2], keep[3]);
    } else {
        static_assert(VE == 1, "");
        bool lo, hi;
        kept_pair((lane & 4) ? ((lane & 2) ? c.w : c.z) : ((lane & 2) ? c.y : c.x), d, lo, hi);
        keep[0] = (lane & 1) ? hi : lo;
    }
}

// f[i] = kept ? f[i] * scale : 0.  A dropped element is 0 whatever it held.
template <int VE>
__device__ __forceinline__ void drop_elements(float (&f)[VE], unsigned long long e, const Drop &d)
{
    bool keep[VE];
    kept<VE>(keep, e >> 3, static_cast<unsigned>(e & 7), d);
#pragma unroll
    for (int i = 0; i < VE; i++) f[i] = keep[i] ? f[i] * d.scale : 0.0f;
}

__device__ __forceinline__ float exp2_approx(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp_approx(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// z Phi(z) and its derivative Phi(z) + z phi(z), Phi(z) = (1 + erf(z / sqrt 2)) / 2.
// The sum cancels where z is below 0, so the error is absolute there, up to 1.2e-7,
// which is more than the value itself from z = -5.5 on.  The slope's __expf, off by
// 2 + 0.6 z^2 units of a z phi(z) below 0.25, adds no more than that.
__device__ __forceinline__ float gelu(float z) { return 0.5f * z * (1.0f + erff(z * 0.70710678f)); }
__device__ __forceinline__ float gelu_slope(float z)
{
    return fmaf(z * 0.39894228f, __expf(-0.5f * z * z), fmaf(0.5f, erff(z * 0.70710678f), 0.5f));
}

}  // namespace maps
}  // namespace rz
