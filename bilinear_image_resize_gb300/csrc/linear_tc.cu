// The linear layer's products on the fifth-generation tensor cores.
//
// A CTA computes 128 x tile_n of D = A B^T, 64 terms at a time: one thread asks
// for both operands' tiles by TMA, into a ring of stages in the 128-byte swizzle;
// one thread issues four tcgen05.mma (16 terms each) a stage, accumulating in
// tensor memory; sixteen warps take finished tiles out of it.  Tensor memory holds
// two tiles, so that one is stored while the next is computed.  CTAs are
// persistent and take tiles in turn, those of one row of tiles next to each
// other, so that their rows of A come from L2.
//
// An operand may be stored by rows of the product (its terms packed) or by terms
// (its rows packed, as W in dz W and both in dz^T x): the matrix descriptors say
// which.  float32 operands come as three bfloat16 planes x = x0 + x1 + x2, each
// the leading bits of what the ones before it leave; of the nine products of
// planes the six with i + j <= 2 are summed, the smallest first, in the one
// accumulator: the others are below 2^-23 of |a| |b|.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "linear.h"
#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {

using namespace lin;
using dev::grid_dependency_wait;
using dev::grid_launch_dependents;
using dev::smem_addr;

constexpr int kTerms = 64;                      // terms of a stage: 128 bytes, the swizzle's width
constexpr int kTileM = 128;
constexpr int kBytesA = kTileM * kTerms * 2;
constexpr int kEpiWarps = 16;
constexpr int kThreads = 128 + 32 * kEpiWarps;  // producer, issuer, two idle warps; the epilogue's begin at a multiple of four
constexpr int kStagePitch = 20;                 // floats of a row on its way out: 16 columns and a gap, so that rows differ in their banks
constexpr int kStageBytes = kEpiWarps * 32 * kStagePitch * 4;
constexpr int kShare = 64;                      // most columns of a tile that are one epilogue warp's
constexpr int kSmem = 227 * 1024;
constexpr int kStatic = kEpiWarps * kShare * 4 + 512;   // the kernel's own variables
constexpr int kRing = 8;
constexpr int kSms = 152;

struct TcArgs {
    Finish f;
    float *part;
    unsigned part_pitch;
    unsigned tiles_m, tiles_n, tiles;   // tiles: of all runs
    int tile_n, stages;
    int chunks, all_chunks, run;        // 64-term chunks of a plane product, of all of them, and of a run
    int planes;
    int a_turned, b_turned;
    unsigned idesc;
    int *status;
};

// CG: CTAs that work on one tile, 1 or a pair.  A box of this CTA's share, counted
// by the barrier at `bar` (of a pair, its first CTA's: an address in the cluster).
template <int CG>
__device__ __forceinline__ void load_box(const CUtensorMap *map, uint32_t to, uint32_t bar, int x, int y, int plane)
{
    if constexpr (CG == 1)
        asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                     "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(to),
                     "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(plane), "r"(bar)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
                     "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(to),
                     "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(plane), "r"(bar)
                     : "memory");
}
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void arrive_in_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Matrix descriptor of a tile in the 128-byte swizzle.  By terms packed: 8-row
// groups 1024 bytes apart.  By rows packed (turned): boxes of 64 rows by 64 terms,
// 8-term groups 1024 bytes apart, boxes 8192.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, bool turned)
{
    const uint64_t lead = turned ? 8192 >> 4 : 1;
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (lead << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    if constexpr (CG == 1)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
                     : "memory");
}
// One arrival at the barrier (of a pair: at both CTAs') once the products so far are done.
template <int CG>
__device__ __forceinline__ void commit(uint64_t *bar)
{
    if constexpr (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                     : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                         smem_addr(bar)),
                     "h"(static_cast<uint16_t>(3))
                     : "memory");
}

__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&v)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15}, [%16];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
                   "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
                 : "r"(addr)
                 : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// A tile's place and the chunks of its run.
struct Tile {
    unsigned m, n, run;
    int first, last;
};
__device__ __forceinline__ Tile tile_at(const TcArgs &a, unsigned t)
{
    Tile r;
    r.n = t % a.tiles_n;
    const unsigned q = t / a.tiles_n;
    r.m = q % a.tiles_m;
    r.run = q / a.tiles_m;
    r.first = static_cast<int>(r.run) * a.run;
    r.last = min(a.all_chunks, r.first + a.run);
    return r;
}

// The planes of the j-th product of planes, the smallest first.
__device__ __forceinline__ void planes_of(int planes, int j, int &a, int &b)
{
    if (planes == 1) {
        a = b = 0;
        return;
    }
    // (2,0) (1,1) (0,2) (1,0) (0,1) (0,0)
    a = 0x001012 >> (4 * j) & 0xf;
    b = 0x010210 >> (4 * j) & 0xf;
}

template <class T, int ACT, int CG>
__global__ void __launch_bounds__(kThreads, 1)
k_linear_tc(const __grid_constant__ TcArgs a, const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b)
{
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[kRing], empty[kRing], done[2], taken[2];
    __shared__ uint32_t tmem_slot;
    __shared__ alignas(16) float bias[kEpiWarps][kShare];
    const uint32_t pad = (1024 - (smem_addr(raw) & 1023)) & 1023;
    const uint32_t ring = smem_addr(raw) + pad;
    const int rows_b = a.tile_n / CG;     // this CTA's share of B's rows
    const int stage_bytes = kBytesA + rows_b * kTerms * 2;
    uint32_t rank = 0;
    if constexpr (CG == 2) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const unsigned first_tile = blockIdx.x / CG, tile_step = gridDim.x / CG;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; i++) {
            dev::mbar_init(full + i, 1);
            dev::mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; i++) {
            dev::mbar_init(done + i, 1);
            dev::mbar_init(taken + i, kEpiWarps * CG);
        }
        dev::fence_mbar_init();
    }
    if (warp == 2) {
        if constexpr (CG == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                         "r"(512u)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                         "r"(512u)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_slot;
    grid_dependency_wait();

    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t phase = 0;
            bool ok = true;
            unsigned asked = 0;
            for (unsigned t = first_tile; t < a.tiles && ok; t += tile_step) {
                const Tile w = tile_at(a, t);
                for (int c = w.first; c < w.last; c++) {
                    ok = dev::mbar_wait_bounded(empty + s, phase ^ 1, a.status);
                    if (!ok) break;
                    const int j = c / a.chunks, k0 = (c - j * a.chunks) * kTerms;
                    int pa, pb;
                    planes_of(a.planes, j, pa, pb);
                    const uint32_t sa = ring + s * stage_bytes, sb = sa + kBytesA;
                    if (rank == 0) dev::mbar_arrive_expect_tx(full + s, CG * stage_bytes);
                    const uint32_t bar = CG == 1 ? smem_addr(full + s) : in_cta(smem_addr(full + s), 0);
                    const int m0 = (w.m * CG + rank) * kTileM, n0 = w.n * a.tile_n + rank * rows_b;
                    if (a.a_turned) {
                        load_box<CG>(&map_a, sa, bar, m0, k0, pa);
                        load_box<CG>(&map_a, sa + 8192, bar, m0 + 64, k0, pa);
                    } else {
                        load_box<CG>(&map_a, sa, bar, k0, m0, pa);
                    }
                    if (a.b_turned) {
                        for (int i = 0; i < rows_b; i += 64) load_box<CG>(&map_b, sb + i * 128, bar, n0 + i, k0, pb);
                    } else {
                        load_box<CG>(&map_b, sb, bar, k0, n0, pb);
                    }
                    asked++;
                    if (++s == a.stages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            // nothing may arrive in shared memory that is no longer this CTA's (of a pair the first CTA's barriers
            // count both shares, and neither CTA ends before the other)
            if (!ok && rank == 0)
                for (unsigned i = 0; i < min(asked, static_cast<unsigned>(a.stages)); i++) {
                    const unsigned at = asked - 1 - i;
                    dev::mbar_wait_bounded(full + at % a.stages, at / a.stages & 1, a.status);
                }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            int s = 0;
            uint32_t phase = 0;
            bool ok = true;
            unsigned i = 0;
            const uint32_t step_a = (a.a_turned ? 2048 : 32) >> 4, step_b = (a.b_turned ? 2048 : 32) >> 4;
            for (unsigned t = first_tile; t < a.tiles && ok; t += tile_step, i++) {
                const Tile w = tile_at(a, t);
                const uint32_t acc = tmem + (i & 1) * 256;
                ok = dev::mbar_wait_bounded(taken + (i & 1), (i >> 1 & 1) ^ 1, a.status);
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                for (int c = w.first; c < w.last; c++) {
                    ok = dev::mbar_wait_bounded(full + s, phase, a.status);
                    if (!ok) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t sa = ring + s * stage_bytes;
                    const uint64_t da = tile_desc(sa, a.a_turned), db = tile_desc(sa + kBytesA, a.b_turned);
#pragma unroll
                    for (uint32_t k = 0; k < kTerms / 16; k++)
                        mma<CG>(acc, da + k * step_a, db + k * step_b, a.idesc, c > w.first || k > 0);
                    commit<CG>(empty + s);
                    if (++s == a.stages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
                if (ok) commit<CG>(done + (i & 1));
            }
        }
    } else if (warp >= 4) {
        // four warps share 32 rows, a quarter of the columns each, 16 at a time: out of tensor memory a lane has a row
        // of them, on the way to memory (through `stage`) a vector of each of the rows below
        constexpr int VE = 16 / sizeof(T), per_row = 16 / VE, rows = 32 / per_row, steps = 32 / rows;
        using V = Raw<T, VE>;
        const int e = warp - 4, quarter = warp & 3, cols = a.tile_n / 4, down = lane / per_row, sub = lane % per_row * VE;
        float *stage = reinterpret_cast<float *>(raw + pad + a.stages * stage_bytes) + e * 32 * kStagePitch;
        unsigned i = 0;
        bool ok = true;
        for (unsigned t = first_tile; t < a.tiles && ok; t += tile_step, i++) {
            const Tile w = tile_at(a, t);
            const unsigned m0 = (w.m * CG + rank) * kTileM + 32 * quarter, from = (e >> 2) * cols;
            const unsigned n0 = w.n * a.tile_n + from;
            // what does not wait for the product: its columns' bias, the first residuals
            if (!a.part) {
                __syncwarp();
                for (int c = lane; c < cols; c += 32) bias[e][c] = a.f.bias && n0 + c < a.f.N ? __ldg(a.f.bias + n0 + c) : 0.0f;
                __syncwarp();
            }
            V next[steps] = {};
            const bool reads = !a.part && a.f.wide && a.f.has_residual;
            const auto residuals = [&](unsigned n) {
#pragma unroll
                for (int k = 0; k < steps; k++)
                    if (m0 + k * rows + down < a.f.M && n + sub < a.f.N)
                        next[k] = *vec_at<T, VE>(a.f.residual, m0 + k * rows + down, n + sub);
            };
            if (reads) residuals(n0);
            ok = dev::mbar_wait_bounded(done + (i & 1), i >> 1 & 1, a.status);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t acc = tmem + (i & 1) * 256 + (static_cast<uint32_t>(32 * quarter) << 16) + from;
            for (int c0 = 0; c0 < cols; c0 += 16) {
                uint32_t v[16];
                tmem_load(acc + c0, v);
                if (c0 + 16 >= cols) {
                    // this warp's share of the tile is in registers
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    if (lane == 0) {
                        if constexpr (CG == 1)
                            dev::mbar_arrive(taken + (i & 1));
                        else
                            arrive_in_cluster(in_cta(smem_addr(taken + (i & 1)), 0));
                    }
                }
                const unsigned n = n0 + c0;
                if (n >= a.f.N) continue;
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 4; k++)
                    *reinterpret_cast<uint4 *>(stage + lane * kStagePitch + 4 * k) =
                        make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                __syncwarp();
                if (a.part) {
                    // a float32 row of the run's part: 16 columns, 4 lanes a row
                    float *to = a.part + (static_cast<long long>(w.run) * a.f.M + m0) * a.part_pitch + n;
                    const int c = lane % 4 * 4;
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const int r = k * 8 + lane / 4;
                        if (m0 + r < a.f.M && n + c < a.part_pitch)
                            *reinterpret_cast<float4 *>(to + static_cast<long long>(r) * a.part_pitch + c) =
                                *reinterpret_cast<const float4 *>(stage + r * kStagePitch + c);
                    }
                } else if (a.f.wide) {
                    V now[steps];
#pragma unroll
                    for (int k = 0; k < steps; k++) now[k] = next[k];
                    if (reads && c0 + 16 < cols) residuals(n + 16);
                    if (n + sub < a.f.N) {
                        float2 b[VE / 2];
#pragma unroll
                        for (int q = 0; q < VE; q += 4) {
                            const float4 v4 = *reinterpret_cast<const float4 *>(&bias[e][c0 + sub + q]);
                            b[q / 2] = make_float2(v4.x, v4.y);
                            b[q / 2 + 1] = make_float2(v4.z, v4.w);
                        }
#pragma unroll
                        for (int k = 0; k < steps; k++) {
                            const int r = k * rows + down;
                            float2 z[VE / 2];
#pragma unroll
                            for (int q = 0; q < VE; q += 4) {
                                const float4 v4 = *reinterpret_cast<const float4 *>(stage + r * kStagePitch + sub + q);
                                z[q / 2] = make_float2(v4.x, v4.y);
                                z[q / 2 + 1] = make_float2(v4.z, v4.w);
                            }
                            if (m0 + r < a.f.M) finish<T, VE, ACT>(a.f, m0 + r, n + sub, z, b, now[k]);
                        }
                    }
                } else if (n + lane % 16 < a.f.N) {
                    const int c = lane % 16;
#pragma unroll 1
                    for (int r = lane / 16 * 16; r < lane / 16 * 16 + 16 && m0 + r < a.f.M; r += 8) {
                        float z[8];
#pragma unroll
                        for (int u = 0; u < 8; u++) z[u] = stage[(r + u) * kStagePitch + c];
                        finish_column<T, ACT, 8>(a.f, m0 + r, n + c, z, bias[e][c0 + c]);
                    }
                }
            }
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    if (warp == 2) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if constexpr (CG == 1)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

// ------------------------------------------------------------------ host side

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder()
{
    static std::once_flag once;
    static EncodeFn fn = nullptr;
    std::call_once(once, [] {
        void *q = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &q, 12000, cudaEnableDefault, &r) == cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(q);
    });
    return fn;
}

// The operand's tensor map: boxes of 64 packed elements by `box` memory rows;
// what lies outside the matrix reads as 0.
bool encode(const Operand &o, unsigned box, CUtensorMap *map)
{
    std::memset(map, 0, sizeof(*map));
    const cuuint64_t inner = o.turned ? o.rows : o.terms, outer = o.turned ? o.terms : o.rows;
    const cuuint64_t dims[3] = {inner, outer, static_cast<cuuint64_t>(o.planes)};
    const cuuint64_t strides[2] = {o.pitch, o.planes > 1 ? o.plane : o.pitch};
    const cuuint32_t boxes[3] = {kTerms, box, 1}, steps[3] = {1, 1, 1};
    return encoder()(map, o.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(o.p),
                     dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T, int ACT, int CG>
cudaError_t tc_launch(const TcArgs &a, const CUtensorMap &ma, const CUtensorMap &mb, void *stream)
{
    const auto fn = k_linear_tc<T, ACT, CG>;
    if (const cudaError_t e = shared_opt_in(reinterpret_cast<const void *>(fn), kSmem - kStatic)) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CG * std::min<unsigned>(a.tiles, kSms / CG));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = 1024 + a.stages * static_cast<size_t>(kBytesA + a.tile_n / CG * kTerms * 2) + kStageBytes;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 1 ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, fn, a, ma, mb);
}

template <class T, int CG>
cudaError_t tc_launch_act(const TcArgs &a, const CUtensorMap &ma, const CUtensorMap &mb, void *stream)
{
    // runs of a sum are finished where they are joined
    const int act = a.part ? RZ_ACT_NONE : a.f.act;
    if (act == RZ_ACT_SILU) return tc_launch<T, RZ_ACT_SILU, CG>(a, ma, mb, stream);
    return act == RZ_ACT_GELU ? tc_launch<T, RZ_ACT_GELU, CG>(a, ma, mb, stream) : tc_launch<T, RZ_ACT_NONE, CG>(a, ma, mb, stream);
}
template <class T>
cudaError_t tc_launch_of(const TcArgs &a, const CUtensorMap &ma, const CUtensorMap &mb, int pair, void *stream)
{
    return pair ? tc_launch_act<T, 2>(a, ma, mb, stream) : tc_launch_act<T, 1>(a, ma, mb, stream);
}

}  // namespace

cudaError_t lin::launch_product(const Product &p, void *stream)
{
    if (!encoder()) return cudaErrorNotSupported;
    CUtensorMap ma, mb;
    if (!encode(p.a, p.a.turned ? kTerms : kTileM, &ma) || !encode(p.b, p.b.turned ? kTerms : p.tile_n / (p.pair ? 2 : 1), &mb))
        return cudaErrorInvalidValue;
    TcArgs a{};
    a.f = p.f;
    a.part = p.splits > 1 ? p.part : nullptr;
    a.part_pitch = p.part_pitch;
    a.tile_n = p.tile_n;
    const int cg = p.pair ? 2 : 1;
    a.tiles_m = (p.f.M + cg * kTileM - 1) / (cg * kTileM);
    a.tiles_n = (p.f.N + p.tile_n - 1) / p.tile_n;
    a.planes = p.a.planes;
    a.chunks = static_cast<int>((p.a.terms + kTerms - 1) / kTerms);
    a.all_chunks = a.chunks * (a.planes == 1 ? 1 : 6);
    a.run = (a.all_chunks + p.splits - 1) / p.splits;
    const unsigned long long tiles = static_cast<unsigned long long>(a.tiles_m) * a.tiles_n * p.splits;
    if (tiles > 0x7fffffffull) return cudaErrorInvalidConfiguration;
    a.tiles = static_cast<unsigned>(tiles);
    a.stages = std::min(kRing, (kSmem - kStatic - 1024 - kStageBytes) / (kBytesA + p.tile_n / cg * kTerms * 2));
    a.a_turned = p.a.turned;
    a.b_turned = p.b.turned;
    const unsigned type = p.a.bf16 ? 1u : 0u;
    a.idesc = (1u << 4) | (type << 7) | (type << 10) | (static_cast<unsigned>(p.a.turned) << 15) |
              (static_cast<unsigned>(p.b.turned) << 16) | (static_cast<unsigned>(p.tile_n >> 3) << 17) | (static_cast<unsigned>(cg * kTileM >> 4) << 24);
    a.status = p.status;
    if (p.out_dtype == RZ_F32) return tc_launch_of<float>(a, ma, mb, p.pair, stream);
    return p.out_dtype == RZ_BF16 ? tc_launch_of<__nv_bfloat16>(a, ma, mb, p.pair, stream) : tc_launch_of<__half>(a, ma, mb, p.pair, stream);
}

}  // namespace rz
