// Shared by the linear layer's kernels (linear.cu, linear_tc.cu): matrices
// inside maps and weights, and what is done to a product before it is stored.
#pragma once

#include <cuda.h>   // CUtensorMap (a plain struct; no driver library is linked)

#include "map_ops.h"

namespace rz {
namespace lin {

using namespace maps;

// A matrix: row r at row_off(r), its columns packed.
struct Rows {
    View v;
    unsigned HW, W;     // pixels of an image and of its rows (HW 0: rows `pitch` apart)
    int joined, bytes;  // of an image's rows; bytes of a pixel
};

__device__ __forceinline__ long long row_off(const Rows &m, unsigned r)
{
    if (!m.HW) return r * m.v.pitch;
    const unsigned n = r / m.HW;
    return n * m.v.bstride + pixel_off(r - n * m.HW, m.W, m.joined != 0, m.v.pitch, m.bytes);
}

// The activations.  float32 results take the exact forms.  16-bit ones, which are
// rounded to 2^-8 or 2^-11 of their size, take GELU from the lower tail of the normal
// distribution, two elements at a time: with a = |z|,
//   Phi(-a) = 2^(r(a) - a^2 log2(e) / 2),   GELU(z) = max(z, 0) - a Phi(-a),
// r a polynomial of degree 6 for a <= 6, fitted so that Phi(-a) is off by 3e-4 of
// itself at most and by (25 + 3 a) 2^-26 where that is less (of which the fit has 13 + 3 a,
// the float32 steps 4, the power, off by 2^-22, 8); it stays where it is from there on,
// where Phi(-a) < 1e-9.  One function of the special unit and seven
// packed products an element pair; erff takes thirty instructions an element, which
// on a product of 1024 terms cost more than the product (617 against 330 us on 65536 x
// 1024 x 4096).  Infinities: a is cut at 1e4, where Phi(-a) is 0; the rest passes them
// and NaN on.
__device__ __forceinline__ float2 exp2_both(float2 x) { return make_float2(exp2_approx(x.x), exp2_approx(x.y)); }
__device__ __forceinline__ float2 lower_tail(float2 z, float2 &a, float2 &square)
{
    a = make_float2(fminf(fabsf(z.x), 1.0e4f), fminf(fabsf(z.y), 1.0e4f));
    const float2 m = make_float2(fminf(a.x, 6.0f), fminf(a.y, 6.0f));
    float2 r = __ffma2_rn(m, both(3.0424116e-5f), both(-7.3252892e-4f));
    r = __ffma2_rn(m, r, both(7.9208132e-3f));
    r = __ffma2_rn(m, r, both(-5.3121625e-2f));
    r = __ffma2_rn(m, r, both(0.26234567f));
    r = __ffma2_rn(m, r, both(-1.1511284f));
    r = __ffma2_rn(m, r, both(-0.99999971f));
    square = __fmul2_rn(a, a);
    return exp2_both(__ffma2_rn(square, both(-0.72134752f), r));
}
template <class T, int ACT>
__device__ __forceinline__ float2 activated(float2 z)
{
    if constexpr (ACT == RZ_ACT_SILU) {
        const float2 x = __fmul2_rn(z, both(-1.44269504f));
        const float2 d = __fadd2_rn(make_float2(exp2_approx(x.x), exp2_approx(x.y)), both(1.0f));
        const float2 y = __fmul2_rn(z, make_float2(rcp_approx(d.x), rcp_approx(d.y)));
        return make_float2(z.x < -87.3f ? 0.0f : y.x, z.y < -87.3f ? 0.0f : y.y);
    } else if constexpr (ACT == RZ_ACT_GELU) {
        if constexpr (sizeof(T) == 4) return make_float2(gelu(z.x), gelu(z.y));
        float2 a, square;
        const float2 q = lower_tail(z, a, square);
        const float2 m = __ffma2_rn(make_float2(fabsf(z.x), fabsf(z.y)), both(0.5f), __fmul2_rn(z, both(0.5f)));
        return __ffma2_rn(make_float2(-a.x, -a.y), q, m);
    } else {
        return z;
    }
}
// Their derivatives; GELU's is Phi(z) + z phi(z).  From 1e4 on they are 0 or 1, of an
// infinite z (a float16 pre past its type's range) as well; NaN stays.
__device__ __forceinline__ float within(float z) { return z > 1.0e4f ? 1.0e4f : z < -1.0e4f ? -1.0e4f : z; }
template <class T>
__device__ __forceinline__ float2 act_slope(float2 z, int act)
{
    z = make_float2(within(z.x), within(z.y));
    if (act == RZ_ACT_SILU) {
        const float2 x = __fmul2_rn(z, both(-1.44269504f));
        const float2 d = __fadd2_rn(make_float2(exp2_approx(x.x), exp2_approx(x.y)), both(1.0f));
        const float2 s = make_float2(z.x < -87.3f ? 0.0f : rcp_approx(d.x), z.y < -87.3f ? 0.0f : rcp_approx(d.y));
        return __fmul2_rn(s, __ffma2_rn(z, __ffma2_rn(s, both(-1.0f), both(1.0f)), both(1.0f)));
    }
    if (act != RZ_ACT_GELU) return both(1.0f);
    if constexpr (sizeof(T) == 4) return make_float2(gelu_slope(z.x), gelu_slope(z.y));
    float2 a, square;
    const float2 q = lower_tail(z, a, square), e = exp2_both(__fmul2_rn(square, both(-0.72134752f)));
    const float2 up = __ffma2_rn(q, both(-1.0f), both(1.0f));
    const float2 phi = make_float2(z.x > 0.0f ? up.x : q.x, z.y > 0.0f ? up.y : q.y);
    return __ffma2_rn(__fmul2_rn(z, both(0.39894228f)), e, phi);
}

// What becomes of z = a row of a matrix times one of another: out = act(z + bias)
// + residual, and z + bias to pre.
struct Finish {
    Rows out, pre, residual;
    const float *bias;
    unsigned M, N;      // rows and columns of out
    int has_pre, has_residual, act;
    int wide;           // out, pre and residual are made of whole aligned vectors of 16 bytes
};

template <class T, int VE>
__device__ __forceinline__ Raw<T, VE> *vec_at(const Rows &r, unsigned m, unsigned n)
{
    return reinterpret_cast<Raw<T, VE> *>(r.v.p + row_off(r, m) + static_cast<long long>(n) * sizeof(T));
}
// Columns n .. n + VE - 1 of row m, a vector of each matrix; b: their bias, r: the
// residual's vector.
template <class T, int VE, int ACT>
__device__ __forceinline__ void finish(const Finish &f, unsigned m, unsigned n, float2 (&z)[VE / 2], const float2 (&b)[VE / 2],
                                       const Raw<T, VE> &r)
{
#pragma unroll
    for (int i = 0; i < VE / 2; i++) z[i] = __fadd2_rn(z[i], b[i]);
    if (f.has_pre) *vec_at<T, VE>(f.pre, m, n) = pack2<T, VE>(z);
#pragma unroll
    for (int i = 0; i < VE / 2; i++) z[i] = activated<T, ACT>(z[i]);
    if (f.has_residual) {
        float2 add[VE / 2];
        unpack2<T, VE>(r, add);
#pragma unroll
        for (int i = 0; i < VE / 2; i++) z[i] = __fadd2_rn(z[i], add[i]);
    }
    *vec_at<T, VE>(f.out, m, n) = pack2<T, VE>(z);
}
// UNIT elements, one or an aligned pair, where vectors do not fit.
template <class T, int ACT, int UNIT>
__device__ __forceinline__ void finish_unit(const Finish &f, unsigned m, unsigned n, float2 z)
{
    using V = Raw<T, UNIT>;
    const auto at = [&](const Rows &r) { return vec_at<T, UNIT>(r, m, n); };
    const auto packed = [](float2 v) {
        float e[UNIT];
        e[0] = v.x;
        if (UNIT == 2) e[UNIT - 1] = v.y;
        return pack<T, UNIT>(e);
    };
    V r{};
    if (f.has_residual) r = *at(f.residual);
    if (f.bias) z = __fadd2_rn(z, make_float2(__ldg(f.bias + n), UNIT == 2 ? __ldg(f.bias + n + 1) : 0.0f));
    if (f.has_pre) *at(f.pre) = packed(z);
    z = activated<T, ACT>(z);
    if (f.has_residual) {
        float e[UNIT];
        unpack<T, UNIT>(r, e);
        z = __fadd2_rn(z, make_float2(e[0], UNIT == 2 ? e[UNIT - 1] : 0.0f));
    }
    *at(f.out) = packed(z);
}

template <int VE>
__device__ __forceinline__ void bias_of(const Finish &f, unsigned n, float2 (&b)[VE / 2])
{
#pragma unroll
    for (int i = 0; i < VE / 2; i++)
        b[i] = f.bias ? make_float2(__ldg(f.bias + n + 2 * i), __ldg(f.bias + n + 2 * i + 1)) : both(0.0f);
}

// One operand of a product on the tensor cores: its rows (M or N of the product)
// and the terms of the sum, 16-bit, in `planes` matrices one after another.
struct Operand {
    const void *p;
    size_t pitch;       // bytes, a multiple of 16; p too
    size_t plane;       // bytes between planes
    unsigned rows, terms;
    int planes;
    int turned;         // memory rows are terms
    int bf16;
};

// D = A B^T over the terms.  part: the terms are cut into `parts`, whose float32 sums,
// each added up in runs, go to part[i][M][part_pitch] for k_linear_join; else (one run)
// the kernel itself finishes them, where direct_out says that it can.
struct Product {
    Operand a, b;
    Finish f;
    int out_dtype;
    int parts;
    int part_chunks, run_chunks;    // 64-term chunks of a part and of a run
    float *part;
    unsigned part_pitch;    // floats
    int tile_n;             // 64 (without a pair), 128 or 256
    int pair;               // two CTAs work on a tile of 256 rows, else one on 128
    int *status;
};
// Products of planes that an operand of `a` planes and one of `b` take: of three each
// the six largest, of a second plane its own.
inline int products_of(int a, int b) { return a == 3 && b == 3 ? 6 : a * b; }
bool direct_out(const Finish &f, int dtype);
cudaError_t launch_product(const Product &p, void *stream);

}  // namespace lin
}  // namespace rz
