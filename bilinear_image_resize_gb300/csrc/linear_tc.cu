// The linear layer's products on the fifth-generation tensor cores.
//
// A CTA computes 128 x tile_n of D = A B^T, 64 terms at a time: two threads ask
// for the operands' tiles by TMA, into a ring of stages in the 128-byte swizzle;
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
constexpr int kThreads = 128 + 32 * kEpiWarps;  // loads of A, issuer, tensor memory, loads of B; the epilogue's begin at a multiple of four
constexpr int kStagePitch = 48;                 // bytes of a row on its way out: 32 and a gap, so that rows differ in their banks
constexpr int kStageBytes = kEpiWarps * 32 * kStagePitch;
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
    unsigned group;                     // rows of tiles that are walked together
    int a_turned, b_turned;
    int a_merged, b_merged;             // a turned operand's rows come in one box
    unsigned idesc;
    int *status;
};

// CG: CTAs that work on one tile, 1 or a pair.  A box of this CTA's share, counted
// by the barrier at `bar` (of a pair, its first CTA's: an address in the cluster).
template <int CG>
__device__ __forceinline__ void load_box(const CUtensorMap *map, uint32_t to, uint32_t bar, int x, int y, int z, int plane)
{
    if constexpr (CG == 1)
        asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                     "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(to),
                     "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(plane), "r"(bar)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
                     "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(to),
                     "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(plane), "r"(bar)
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
    // what it orders is reads of tensor memory, which have their own fence: a release in the cluster would wait for the
    // thread's stores to memory
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
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

// Columns addr .. of this warp's 32 lanes of tensor memory, a row a thread.
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
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&v)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(addr)
                 : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// A wait of at most a second that leaves no gap between its attempts.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, int *status)
{
    if (dev::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = dev::global_ns();
    while (!dev::mbar_try_wait(bar, parity))
        if (dev::global_ns() - t0 > kWaitLimitNs) {
            if (status) atomicExch(status, RZ_ERR_TIMEOUT);
            return false;
        }
    return true;
}

// 32 rows of 32 bytes each through a warp's stage, which turns a row a thread into
// consecutive bytes of a row for consecutive threads and back: lane / 2 + 16 k is
// the row of a lane's k-th 16 bytes, lane % 2 their half of it.
__device__ __forceinline__ void stage_row(uint8_t *stage, const uint4 (&v)[2])
{
    const int lane = threadIdx.x & 31;
    __syncwarp();
    reinterpret_cast<uint4 *>(stage + lane * kStagePitch)[0] = v[0];
    reinterpret_cast<uint4 *>(stage + lane * kStagePitch)[1] = v[1];
    __syncwarp();
}
__device__ __forceinline__ uint4 staged(const uint8_t *stage, int k)
{
    const int lane = threadIdx.x & 31;
    return *reinterpret_cast<const uint4 *>(stage + (lane / 2 + 16 * k) * kStagePitch + lane % 2 * 16);
}

// A row a thread of PC = 32 / sizeof(T) columns to a matrix: rows from m, columns
// from n, as far as it reaches; whole vectors or element by element.
template <class T>
__device__ __forceinline__ void emit(const Rows &to, const Finish &f, unsigned m, unsigned n, uint8_t *stage,
                                     const float2 (&z)[16 / sizeof(T)])
{
    constexpr int PC = 32 / sizeof(T), VE = PC / 2;
    using E = Raw<T, 1>;
    const int lane = threadIdx.x & 31;
    uint4 v[2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
        float2 part[VE / 2];
#pragma unroll
        for (int i = 0; i < VE / 2; i++) part[i] = z[h * VE / 2 + i];
        v[h] = pack2<T, VE>(part);
    }
    stage_row(stage, v);
    if (f.wide) {
#pragma unroll
        for (int k = 0; k < 2; k++) {
            const unsigned r = m + lane / 2 + 16 * k, c = n + lane % 2 * VE;
            if (r < f.M && c < f.N) *vec_at<T, VE>(to, r, c) = staged(stage, k);
        }
    } else {
#pragma unroll
        for (int k = 0; k < PC; k++) {
            const int r = k * (32 / PC) + lane / PC, c = lane % PC;
            if (m + r < f.M && n + c < f.N)
                *reinterpret_cast<E *>(to.v.p + row_off(to, m + r) + static_cast<long long>(n + c) * sizeof(T)) =
                    *reinterpret_cast<const E *>(stage + r * kStagePitch + c * sizeof(T));
        }
    }
}

// A tile's place and the chunks of its run.
struct Tile {
    unsigned m, n, run;
    int first, last;
};
__device__ __forceinline__ Tile tile_at(const TcArgs &a, unsigned t)
{
    Tile r;
    const unsigned all = a.tiles_m * a.tiles_n, x = t % all, per = a.group * a.tiles_n;
    const unsigned g = x / per, y = x - g * per, rows = min(a.group, a.tiles_m - g * a.group);
    r.run = t / all;
    r.m = g * a.group + y % rows;
    r.n = y / rows;
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

    if (warp == 0 || warp == 3) {
        // warp 0 asks for A's tiles, warp 3 for B's: one thread for both spends longer on a stage's requests than the
        // products take (its waits for a free stage were a fifth of its time)
        if (lane == 0) {
            const bool of_b = warp == 3;
            const CUtensorMap *map = of_b ? &map_b : &map_a;
            const int turned = of_b ? a.b_turned : a.a_turned, merged = of_b ? a.b_merged : a.a_merged;
            const int rows = of_b ? rows_b : kTileM;
            const uint32_t to = ring + (of_b ? kBytesA : 0);
            const uint32_t bars = CG == 1 ? smem_addr(full) : in_cta(smem_addr(full), 0);
            int s = 0;
            uint32_t phase = 0;
            bool ok = true;
            unsigned asked = 0;
            for (unsigned t = first_tile; t < a.tiles && ok; t += tile_step) {
                const Tile w = tile_at(a, t);
                const int row = of_b ? static_cast<int>(w.n * a.tile_n + rank * rows_b) : static_cast<int>((w.m * CG + rank) * kTileM);
                int j = w.first / a.chunks, k0 = (w.first - j * a.chunks) * kTerms, pa, pb;
                planes_of(a.planes, j, pa, pb);
                for (int c = w.first; c < w.last; c++) {
                    ok = wait_for(empty + s, phase ^ 1, a.status);
                    if (!ok) break;
                    if (!of_b && rank == 0) dev::mbar_arrive_expect_tx(full + s, CG * stage_bytes);
                    const uint32_t at = to + s * stage_bytes, bar = bars + 8 * s;
                    const int plane = of_b ? pb : pa;
                    if (!turned)
                        load_box<CG>(map, at, bar, k0, row, 0, plane);
                    else if (merged)
                        load_box<CG>(map, at, bar, 0, k0, row / 64, plane);
                    else
                        for (int i = 0; i < rows; i += 64) load_box<CG>(map, at + i * 128, bar, row + i, k0, 0, plane);
                    asked++;
                    if (++s == a.stages) {
                        s = 0;
                        phase ^= 1;
                    }
                    k0 += kTerms;
                    if (k0 >= a.chunks * kTerms) {
                        k0 = 0;
                        planes_of(a.planes, ++j, pa, pb);
                    }
                }
            }
            // nothing may arrive in shared memory that is no longer this CTA's (of a pair the first CTA's barriers
            // count both shares, and neither CTA ends before the other)
            if (!ok && rank == 0)
                for (unsigned i = 0; i < min(asked, static_cast<unsigned>(a.stages)); i++) {
                    const unsigned at = asked - 1 - i;
                    wait_for(full + at % a.stages, at / a.stages & 1, a.status);
                }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            int s = 0;
            uint32_t phase = 0;
            bool ok = true;
            unsigned i = 0;
            const uint64_t desc_a = tile_desc(ring, a.a_turned), desc_b = tile_desc(ring + kBytesA, a.b_turned);
            const uint32_t step_a = (a.a_turned ? 2048 : 32) >> 4, step_b = (a.b_turned ? 2048 : 32) >> 4;
            for (unsigned t = first_tile; t < a.tiles && ok; t += tile_step, i++) {
                const Tile w = tile_at(a, t);
                const uint32_t acc = tmem + (i & 1) * 256;
                ok = wait_for(taken + (i & 1), (i >> 1 & 1) ^ 1, a.status);
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                for (int c = w.first; c < w.last; c++) {
                    ok = wait_for(full + s, phase, a.status);
                    if (!ok) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t at = static_cast<uint32_t>(s * stage_bytes) >> 4;   // the ring lies below 2^18: no carry leaves the address
                    const uint64_t da = desc_a + at, db = desc_b + at;
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
        // four warps share 32 rows of the tile, a quarter of its columns each, 32 bytes of the result's rows at a time
        constexpr int PC = 32 / sizeof(T), VE = PC / 2;
        using E = Raw<T, 1>;
        const int e = warp - 4, quarter = warp & 3, cols = a.tile_n / 4;
        uint8_t *stage = raw + pad + a.stages * stage_bytes + e * 32 * kStagePitch;
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
            uint4 next[2] = {};
            const bool adds = !a.part && a.f.has_residual, ahead = adds && a.f.wide;
            const auto residuals = [&](unsigned n) {
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    const unsigned r = m0 + lane / 2 + 16 * k, c = n + lane % 2 * VE;
                    if (r < a.f.M && c < a.f.N) next[k] = *vec_at<T, VE>(a.f.residual, r, c);
                }
            };
            if (ahead) residuals(n0);
            ok = wait_for(done + (i & 1), i >> 1 & 1, a.status);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t acc = tmem + (i & 1) * 256 + (static_cast<uint32_t>(32 * quarter) << 16) + from;
            for (int c0 = 0; c0 < cols; c0 += PC) {
                uint32_t v[PC];
                tmem_load(acc + c0, v);
                if (c0 + PC >= cols) {
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
                if (n >= a.f.N || m0 >= a.f.M) continue;
                if (a.part) {
                    // float32 rows of the run's part
                    float *to = a.part + static_cast<long long>(w.run) * a.f.M * a.part_pitch;
#pragma unroll
                    for (int h = 0; h < PC; h += 8) {
                        const uint4 row[2] = {make_uint4(v[h], v[h + 1], v[h + 2], v[h + 3]),
                                              make_uint4(v[h + 4], v[h + 5], v[h + 6], v[h + 7])};
                        stage_row(stage, row);
#pragma unroll
                        for (int k = 0; k < 2; k++) {
                            const unsigned r = m0 + lane / 2 + 16 * k, c = n + h + lane % 2 * 4;
                            if (r < a.f.M && c < a.part_pitch)
                                *reinterpret_cast<uint4 *>(to + static_cast<long long>(r) * a.part_pitch + c) = staged(stage, k);
                        }
                    }
                    continue;
                }
                float2 add[PC / 2];
                if (adds) {
                    if (ahead) {
                        const uint4 now[2] = {next[0], next[1]};
                        if (c0 + PC < cols) residuals(n + PC);
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < 2; k++)
                            *reinterpret_cast<uint4 *>(stage + (lane / 2 + 16 * k) * kStagePitch + lane % 2 * 16) = now[k];
                    } else {
                        E now[PC];
#pragma unroll
                        for (int k = 0; k < PC; k++) {
                            const unsigned r = m0 + k * (32 / PC) + lane / PC, c = n + lane % PC;
                            now[k] = r < a.f.M && c < a.f.N
                                         ? *reinterpret_cast<const E *>(a.f.residual.v.p + row_off(a.f.residual, r) +
                                                                        static_cast<long long>(c) * sizeof(T))
                                         : E{};
                        }
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < PC; k++)
                            *reinterpret_cast<E *>(stage + (k * (32 / PC) + lane / PC) * kStagePitch + lane % PC * sizeof(T)) = now[k];
                    }
                    __syncwarp();
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        float2 half[VE / 2];
                        unpack2<T, VE>(reinterpret_cast<const Raw<T, VE> *>(stage + lane * kStagePitch)[h], half);
#pragma unroll
                        for (int q = 0; q < VE / 2; q++) add[h * VE / 2 + q] = half[q];
                    }
                }
                float2 z[PC / 2];
#pragma unroll
                for (int q = 0; q < PC; q += 4) {
                    const float4 b = *reinterpret_cast<const float4 *>(&bias[e][c0 + q]);
                    z[q / 2] = __fadd2_rn(make_float2(__uint_as_float(v[q]), __uint_as_float(v[q + 1])), make_float2(b.x, b.y));
                    z[q / 2 + 1] = __fadd2_rn(make_float2(__uint_as_float(v[q + 2]), __uint_as_float(v[q + 3])), make_float2(b.z, b.w));
                }
                if (a.f.has_pre) emit<T>(a.f.pre, a.f, m0, n, stage, z);
#pragma unroll
                for (int q = 0; q < PC / 2; q++) z[q] = activated<T, ACT>(z[q]);
                if (adds)
#pragma unroll
                    for (int q = 0; q < PC / 2; q++) z[q] = __fadd2_rn(z[q], add[q]);
                emit<T>(a.f.out, a.f, m0, n, stage, z);
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

// The operand's tensor map; what lies outside the matrix reads as 0.  By terms: boxes
// of 64 terms by `share` rows.  Turned: boxes of 64 rows by 64 terms, as many side
// by side as the share has where the matrix is made of them (a thread asks for a
// box in about the time of a stage's products, so two take longer than those: 345
// against 331 us on the weight gradient of 65536 x 1024 x 4096).
bool encode(const Operand &o, unsigned share, CUtensorMap *map, int *merged)
{
    std::memset(map, 0, sizeof(*map));
    *merged = o.turned && o.rows % kTerms == 0;
    const cuuint64_t outer = o.turned ? o.terms : o.rows;
    const cuuint64_t dims[4] = {o.turned ? (*merged ? kTerms : o.rows) : o.terms, outer, *merged ? o.rows / kTerms : 1u,
                                static_cast<cuuint64_t>(o.planes)};
    const cuuint64_t strides[3] = {o.pitch, *merged ? 2 * kTerms : o.pitch, o.planes > 1 ? o.plane : o.pitch};
    const cuuint32_t boxes[4] = {kTerms, o.turned ? kTerms : share, *merged ? share / kTerms : 1u, 1}, steps[4] = {1, 1, 1, 1};
    return encoder()(map, o.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void *>(o.p),
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
    const int cg = p.pair ? 2 : 1;
    CUtensorMap ma, mb;
    TcArgs a{};
    if (!encode(p.a, kTileM, &ma, &a.a_merged) || !encode(p.b, p.tile_n / cg, &mb, &a.b_merged)) return cudaErrorInvalidValue;
    a.f = p.f;
    a.part = p.splits > 1 ? p.part : nullptr;
    a.part_pitch = p.part_pitch;
    a.tile_n = p.tile_n;
    a.tiles_m = (p.f.M + cg * kTileM - 1) / (cg * kTileM);
    a.tiles_n = (p.f.N + p.tile_n - 1) / p.tile_n;
    a.planes = p.a.planes;
    // Tiles of a row next to each other read its A at once, and B out of L2 where that holds it (65536 x 1024 x 4096: 341 us,
    // rows of tiles in groups of eight 373).  A larger B is read once for eight rows of tiles (8192 x 8192 x 8192: 611 us, by
    // single rows 650).
    a.group = 2.0 * p.f.N * p.b.terms * p.b.planes > 48e6 ? 8 : 1;
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
