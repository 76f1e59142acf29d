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

// What becomes of z = a row of a matrix times one of another: out = act(z + bias)
// + residual, and z + bias to pre.
struct Finish {
    Rows out, pre, residual;
    const float *bias;
    unsigned M, N;      // rows and columns of out
    int has_pre, has_residual, act;
    int wide;           // whole vectors of 16 bytes are aligned in out, pre and residual
};

// Columns n .. n + VE - 1 of row m, within the matrix (the last of them may not
// be); b: their bias.
template <class T, int VE>
__device__ __forceinline__ void finish(const Finish &f, unsigned m, unsigned n, float (&z)[VE], const float (&b)[VE])
{
    using V = Raw<T, VE>;
    using E = Raw<T, 1>;
    const bool vec = f.wide && n + VE <= f.N;
    const int left = static_cast<int>(min(static_cast<unsigned>(VE), f.N - n));
    const auto store = [&](const Rows &to) {
        uint8_t *at = to.v.p + row_off(to, m) + static_cast<long long>(n) * sizeof(T);
        if (vec) {
            *reinterpret_cast<V *>(at) = pack<T, VE>(z);
            return;
        }
#pragma unroll
        for (int i = 0; i < VE; i++)
            if (i < left) {
                const float one[1] = {z[i]};
                reinterpret_cast<E *>(at)[i] = pack<T, 1>(one);
            }
    };
#pragma unroll
    for (int i = 0; i < VE; i++) z[i] += b[i];
    if (f.has_pre) store(f.pre);
    if (f.act != RZ_ACT_NONE)
#pragma unroll
        for (int i = 0; i < VE; i++) z[i] = activated(z[i], f.act);
    if (f.has_residual) {
        const uint8_t *at = f.residual.v.p + row_off(f.residual, m) + static_cast<long long>(n) * sizeof(T);
        float r[VE] = {};
        if (vec) {
            unpack<T, VE>(*reinterpret_cast<const V *>(at), r);
        } else {
#pragma unroll
            for (int i = 0; i < VE; i++)
                if (i < left) {
                    float one[1];
                    unpack<T, 1>(reinterpret_cast<const E *>(at)[i], one);
                    r[i] = one[0];
                }
        }
#pragma unroll
        for (int i = 0; i < VE; i++) z[i] += r[i];
    }
    store(f.out);
}

template <int VE>
__device__ __forceinline__ void bias_of(const Finish &f, unsigned n, float (&b)[VE])
{
#pragma unroll
    for (int i = 0; i < VE; i++) b[i] = f.bias && n + i < f.N ? __ldg(f.bias + n + i) : 0.0f;
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

// D = A B^T over the terms.  parts > 1: the terms are cut into so many runs, whose
// float32 sums go to part[run][M][pitch_n] for k_linear_join.
struct Product {
    Operand a, b;
    Finish f;
    int out_dtype;
    int splits;
    float *part;
    unsigned part_pitch;    // floats
    int tile_n;             // 64, 128 or 256
    int *status;
};
cudaError_t launch_product(const Product &p, void *stream);

}  // namespace lin
}  // namespace rz
