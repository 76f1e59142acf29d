// The linear layer's products on the fifth-generation tensor cores.
//
// A CTA computes 128 x tile_n of D = A B^T, 64 terms at a time: two warps ask
// for the operands' tiles by TMA, into a ring of stages in the 128-byte swizzle;
// one warp issues four tcgen05.mma (16 terms each) a stage, accumulating in
// tensor memory; eight warps take finished tiles out of it.  The first three run
// whole, with one elected lane for the requests, so that addresses and descriptors
// stay in uniform registers: by one thread in a branch of its own the issue took as
// long as the products, and longer under a busy epilogue (65536 x 1024 x 4096 with
// bias and GELU: 400 us, 368 so).  Tensor memory holds
// two tiles, so that one is stored while the next is computed.  A pair of CTAs
// computes 256 x tile_n, each with its half of A's rows and of B's.  CTAs are
// persistent and take tiles in turn, those of one row of tiles next to each
// other, so that their rows of A come from L2.
//
// What bounds it: products of 65536 x 1024 x 4096 (bf16) run at the power limit,
// 1550 to 1690 TFLOP/s (325 us sustained, 294 alone; with bias and GELU 354 and 303), a
// stage in 530 clocks of the 512 that its products take; a short call by its launch,
// first stages and last epilogue, about 5 us.
//
// An operand may be stored by rows of the product (its terms packed) or by terms
// (its rows packed, as W in dz W and both in dz^T x): the matrix descriptors say
// which.  float32 operands come as three bfloat16 planes x = x0 + x1 + x2, each
// the leading bits of what the ones before it leave; of the nine products of
// planes the six with i + j <= 2 are summed, the smallest first, in the one
// accumulator: the others are below 2^-21 of |a| |b| (2^-24 on the whole).
//
// The accumulator cuts what it adds (it does not round): a sum of n terms of one sign
// ends up smaller by about n 2e-9 of its size, of float16 operands, whose products
// have more bits to lose, by n 6e-9 (up to three times that where a few terms are most
// of a sum).  So long sums are cut into runs, one after another in the same CTA, each
// added to the tile's float32 sums as it leaves (TMA's add, rounded): the sums of a
// tile lie in memory once, however long they are.  Only where there are few tiles do
// several CTAs each take a part of a sum, with sums of its own.  k_linear_join adds the
// parts up and finishes them.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "linear.h"
#include "rz_device.h"
#include "rz_internal.h"
#include "token_rules.h"

namespace rz {
namespace {

using namespace lin;
using dev::grid_dependency_wait;
using dev::grid_launch_dependents;
using dev::smem_addr;

constexpr int kTerms = 64;                      // terms of a stage: 128 bytes, the swizzle's width
constexpr int kTileM = 128;
constexpr int kBytesA = kTileM * kTerms * 2;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;  // loads of A, issuer, tensor memory, loads of B; the epilogue's begin at a multiple of four
constexpr int kBlockRow = 64;                   // bytes of a row of a block on its way out, 32 rows a block
constexpr int kBlockBytes = 32 * kBlockRow;
constexpr int kSmem = 227 * 1024;
constexpr int kRing = 8;
constexpr int kSms = 152;

// What lies in shared memory before the ring, which begins at a multiple of 1024: the kernel's own variables, then
// bias of two tiles.
struct alignas(16) Vars {
    uint64_t full[kRing], empty[kRing], done[2], taken[2];
    uint64_t came[kEpiWarps][2];    // a residual's block, each of a warp's two
    uint32_t tmem;
};
constexpr int kBias = 2 * 256 * sizeof(float);
constexpr int kHead = (static_cast<int>(sizeof(Vars)) + kBias + 1023) / 1024 * 1024;

struct TcArgs {
    Finish f;
    unsigned tiles_m, tiles_n, tiles;   // tiles: of all parts
    int tile_n, stages;
    int chunks, part, run;              // 64-term chunks, and of a part and of a run
    int products;                       // of planes, 1, 2 or 6
    unsigned group;                     // rows of tiles that are walked together
    int a_turned, b_turned;
    int a_merged, b_merged;             // a turned operand's rows come in one box
    int places;                         // an epilogue warp's blocks
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

// Sixteen columns from addr of this warp's 32 lanes of tensor memory, a row a
// thread; they are there after tmem_wait, which the registers pass through so that
// no use of them moves before it.
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&v)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15}, [%16];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
                   "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                   "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
}

// True in one lane of a warp, the same one every time.
__device__ __forceinline__ bool elected()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// A wait of at most a second of the kernel's own time that leaves no gap between its attempts.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, int *status)
{
    if (dev::mbar_try_wait(bar, parity)) return true;
    rules::WaitClock clock(dev::global_ns());
    while (!dev::mbar_try_wait(bar, parity))
        if (clock.over(dev::global_ns(), kWaitLimitNs)) {
            if (status) *static_cast<volatile int *>(status) = RZ_ERR_TIMEOUT;     // every writer's value; the word may lie on the host
            return false;
        }
    return true;
}

// A row a thread of 16 columns, the half `sub` of a block's row where they are
// 16-bit, to and from a block in the 64-byte swizzle (16 bytes at `c` of row r are at
// c ^ (r / 2) % 4, so that eight rows differ in their banks).
template <class T>
__device__ __forceinline__ void block_write(uint8_t *block, int sub, const float2 (&z)[8])
{
    constexpr int VE = 16 / sizeof(T);
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < 16 / VE; h++) {
        float2 v[VE / 2];
#pragma unroll
        for (int i = 0; i < VE / 2; i++) v[i] = z[h * VE / 2 + i];
        const int c = sub * (16 / VE) + h;
        *reinterpret_cast<Raw<T, VE> *>(block + lane * kBlockRow + ((c ^ (lane >> 1 & 3)) << 4)) = pack2<T, VE>(v);
    }
}
template <class T>
__device__ __forceinline__ void block_add(const uint8_t *block, int sub, float2 (&z)[8])
{
    constexpr int VE = 16 / sizeof(T);
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < 16 / VE; h++) {
        float2 v[VE / 2];
        const int c = sub * (16 / VE) + h;
        unpack2<T, VE>(*reinterpret_cast<const Raw<T, VE> *>(block + lane * kBlockRow + ((c ^ (lane >> 1 & 3)) << 4)), v);
#pragma unroll
        for (int i = 0; i < VE / 2; i++) z[h * VE / 2 + i] = __fadd2_rn(z[h * VE / 2 + i], v[i]);
    }
}
// A filled block on its way to memory, clipped to the matrix; `add`: to what is there.
template <bool MAY_ADD>
__device__ __forceinline__ void block_store(const CUtensorMap *map, const uint8_t *block, int n, int m, int part, bool add)
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        if (MAY_ADD && add)
            asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                             reinterpret_cast<uint64_t>(map)),
                         "r"(n), "r"(m), "r"(part), "r"(smem_addr(block))
                         : "memory");
        else
            asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                             reinterpret_cast<uint64_t>(map)),
                         "r"(n), "r"(m), "r"(part), "r"(smem_addr(block))
                         : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
}
// Until all but the last LEFT of this thread's blocks have been read.
template <int LEFT>
__device__ __forceinline__ void blocks_read()
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(LEFT) : "memory");
}

// A tile's place and the chunks of its part.
struct Tile {
    unsigned m, n, part;
    int first, last;
};
__device__ __forceinline__ Tile tile_at(const TcArgs &a, unsigned t)
{
    Tile r;
    const unsigned all = a.tiles_m * a.tiles_n, x = t % all, per = a.group * a.tiles_n;
    const unsigned g = x / per, y = x - g * per, rows = min(a.group, a.tiles_m - g * a.group);
    r.part = t / all;
    r.m = g * a.group + y % rows;
    r.n = y / rows;
    r.first = static_cast<int>(r.part) * a.part;
    r.last = min(a.chunks, r.first + a.part);
    return r;
}

// The planes of the j-th product of planes, the smallest first.
__device__ __forceinline__ void planes_of(int products, int j, int &a, int &b)
{
    if (products <= 2) {
        a = products == 2 && j == 0;
        b = 0;
        return;
    }
    // (2,0) (1,1) (0,2) (1,0) (0,1) (0,0); past the last, none
    a = 0x001012 >> (4 * j) & 0xf;
    b = 0x010210 >> (4 * j) & 0xf;
}

template <class T, int ACT, int CG>
__global__ void __launch_bounds__(kThreads, 1)
k_linear_tc(const __grid_constant__ TcArgs a, const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
            const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_pre,
            const __grid_constant__ CUtensorMap map_residual)
{
    // sums that go to the workspace may come in several runs
    constexpr bool RUNS = sizeof(T) == 4 && ACT == RZ_ACT_NONE;
    extern __shared__ __align__(16) uint8_t raw[];
    __shared__ Vars vars;
    uint64_t *const full = vars.full, *const empty = vars.empty, *const done = vars.done, *const taken = vars.taken;
    auto &came = vars.came;
    const uint32_t pad = kBias + ((1024 - ((smem_addr(raw) + kBias) & 1023)) & 1023);
    const uint32_t ring = smem_addr(raw) + pad;
    const int rows_b = a.tile_n / CG;     // this CTA's share of B's rows
    const int stage_bytes = kBytesA + rows_b * kTerms * 2;
    uint32_t rank = 0;
    if constexpr (CG == 2) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const unsigned first_tile = blockIdx.x / CG, tile_step = gridDim.x / CG;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    grid_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; i++) {
            dev::mbar_init(full + i, 1);
            dev::mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; i++) {
            dev::mbar_init(done + i, 1);
            dev::mbar_init(taken + i, kEpiWarps * CG);
            for (int e = 0; e < kEpiWarps; e++) dev::mbar_init(&came[e][i], 1);
        }
        dev::fence_mbar_init();
    }
    if (warp == 2) {
        if constexpr (CG == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&vars.tmem)),
                         "r"(512u)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&vars.tmem)),
                         "r"(512u)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = vars.tmem;
    grid_dependency_wait();

    if (warp == 0 || warp == 3) {
        // warp 0 asks for A's tiles, warp 3 for B's: one for both spends longer on a stage's requests than the products
        // take (its waits for a free stage were a fifth of its time)
        {
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
                for (int r0 = w.first, r1; r0 < w.last && ok; r0 = r1) {
                    r1 = RUNS ? min(w.last, r0 + a.run) : w.last;
                    // a run's chunks, once for every product of planes (counted in chunks: past the last one's terms may
                    // lie 2^31)
                    int j = 0, chunk = r0, pa, pb;
                    planes_of(a.products, j, pa, pb);
                    for (int c = (r1 - r0) * a.products; c > 0; c--) {
                        ok = __all_sync(0xffffffffu, wait_for(empty + s, phase ^ 1, a.status));
                        if (!ok) break;
                        const uint32_t at = to + s * stage_bytes, bar = bars + 8 * s;
                        const int plane = of_b ? pb : pa, k0 = chunk * kTerms;
                        if (elected()) {
                            if (!of_b && rank == 0) dev::mbar_arrive_expect_tx(full + s, CG * stage_bytes);
                            if (!turned)
                                load_box<CG>(map, at, bar, k0, row, 0, plane);
                            else if (merged)
                                load_box<CG>(map, at, bar, 0, k0, row / 64, plane);
                            else
                                for (int i = 0; i < rows; i += 64) load_box<CG>(map, at + i * 128, bar, row + i, k0, 0, plane);
                        }
                        __syncwarp();
                        asked++;
                        if (++s == a.stages) {
                            s = 0;
                            phase ^= 1;
                        }
                        if (++chunk == r1) {
                            chunk = r0;
                            planes_of(a.products, ++j, pa, pb);
                        }
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
        if (rank == 0) {
            int s = 0;
            uint32_t phase = 0;
            bool ok = true;
            unsigned i = 0;
            const uint64_t desc_a = tile_desc(ring, a.a_turned), desc_b = tile_desc(ring + kBytesA, a.b_turned);
            const uint32_t step_a = (a.a_turned ? 2048 : 32) >> 4, step_b = (a.b_turned ? 2048 : 32) >> 4;
            for (unsigned t = first_tile; t < a.tiles && ok; t += tile_step) {
                const Tile w = tile_at(a, t);
                for (int r0 = w.first, r1; r0 < w.last && ok; r0 = r1, i++) {
                    r1 = RUNS ? min(w.last, r0 + a.run) : w.last;
                    const uint32_t acc = tmem + (i & 1) * 256;
                    ok = __all_sync(0xffffffffu, wait_for(taken + (i & 1), (i >> 1 & 1) ^ 1, a.status));
                    if (!ok) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const int stages = (r1 - r0) * a.products;
                    for (int c = 0; c < stages; c++) {
                        ok = __all_sync(0xffffffffu, wait_for(full + s, phase, a.status));
                        if (!ok) break;
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        // the ring lies below 2^18: no carry leaves the address
                        const uint32_t at = static_cast<uint32_t>(s * stage_bytes) >> 4;
                        const uint64_t da = desc_a + at, db = desc_b + at;
                        if (elected()) {
#pragma unroll
                            for (uint32_t k = 0; k < kTerms / 16; k++)
                                mma<CG>(acc, da + k * step_a, db + k * step_b, a.idesc, c > 0 || k > 0);
                            commit<CG>(empty + s);
                        }
                        __syncwarp();
                        if (++s == a.stages) {
                            s = 0;
                            phase ^= 1;
                        }
                    }
                    if (ok && elected()) commit<CG>(done + (i & 1));
                    __syncwarp();
                }
            }
        }
    } else if (warp >= 4) {
        // Two warps share 32 rows of the tile, half of its columns each.  Results leave and residuals come by TMA in blocks of
        // 64 bytes by 32 rows, in two places in turn: a residual's block comes into the place that its result leaves from,
        // the next one's while this one is worked on.  (Loads and stores of a warp's own took the data path of shared
        // memory for 58% of a call's time, and it is what the products are fed through: 325 against 303 us on 65536 x 1024 x
        // 4096.)  With a residual, pre has a third place.
        constexpr int BC = kBlockRow / sizeof(T), SUBS = BC / 16;
        const int e = warp - 4, quarter = warp & 3, cols = a.tile_n / 2, blocks = cols / BC;
        uint8_t *out = raw + pad + a.stages * stage_bytes + e * a.places * kBlockBytes;
        int flip = 0;
        uint32_t phases = 0, coming = 0;        // a bit of each place: its barrier's phase, and whether a residual is on its way
        unsigned i = 0;
        bool ok = true;
        for (unsigned t = first_tile; t < a.tiles && ok; t += tile_step) {
            const Tile w = tile_at(a, t);
            const unsigned m0 = (w.m * CG + rank) * kTileM + 32 * quarter, n0 = w.n * a.tile_n + (e >> 2) * cols;
            const int live = m0 < a.f.M && n0 < a.f.N ? min(blocks, static_cast<int>((a.f.N - n0 + BC - 1) / BC)) : 0;
            const auto fetch = [&](int b, int place) {
                uint64_t *bar = &came[e][place];
                coming |= 1u << place;
                dev::mbar_arrive_expect_tx(bar, kBlockBytes);
                asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                             "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(out + place * kBlockBytes)),
                             "l"(reinterpret_cast<uint64_t>(&map_residual)), "r"(static_cast<int>(n0) + b * BC),
                             "r"(static_cast<int>(m0)), "r"(0), "r"(smem_addr(bar))
                             : "memory");
            };
            for (int r0 = w.first; r0 < w.last && ok; r0 = RUNS ? r0 + a.run : w.last, i++) {
                const bool more = RUNS && r0 > w.first;
                // sums are added in their order: the run before is in memory
                if (more && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
                // what does not wait for the tile: its first residual, and bias, four columns a lane
                if (a.f.has_residual && live && lane == 0) {
                    blocks_read<1>();
                    fetch(0, flip);
                }
                float bias[4] = {};
                if (a.f.bias)
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        if (4 * lane + q < cols && n0 + 4 * lane + q < a.f.N) bias[q] = __ldg(a.f.bias + n0 + 4 * lane + q);
                ok = __all_sync(0xffffffffu, wait_for(done + (i & 1), i >> 1 & 1, a.status));
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                // the four warps of these columns write the same; none still reads what they held two tiles ago, which all had
                // taken before this tile was begun
                float4 *const columns = reinterpret_cast<float4 *>(raw) + (i & 1) * 64 + (e >> 2) * 32;
                if (a.f.bias) {
                    columns[lane] = make_float4(bias[0], bias[1], bias[2], bias[3]);
                    __syncwarp();
                }
                const uint32_t acc = tmem + (i & 1) * 256 + (static_cast<uint32_t>(32 * quarter) << 16) + (e >> 2) * cols;
                // a block's columns are asked for while the one before is worked on
                uint32_t v[SUBS][16];
#pragma unroll
                for (int q = 0; q < SUBS; q++) tmem_load(acc + 16 * q, v[q]);
                for (int b = 0; b < blocks; b++) {
                    float2 z[SUBS][8];
#pragma unroll
                    for (int q = 0; q < SUBS; q++) {
                        tmem_wait(v[q]);
#pragma unroll
                        for (int j = 0; j < 8; j++) z[q][j] = make_float2(__uint_as_float(v[q][2 * j]), __uint_as_float(v[q][2 * j + 1]));
                    }
                    if (b + 1 < blocks)
#pragma unroll
                        for (int q = 0; q < SUBS; q++) tmem_load(acc + (b + 1) * BC + 16 * q, v[q]);
                    // (read by four columns: by shuffles, one a column, they took the data path of shared memory for 18 us of 368)
                    if (a.f.bias && b < live)
#pragma unroll
                        for (int q = 0; q < SUBS; q++)
#pragma unroll
                            for (int j = 0; j < 8; j += 2) {
                                const float4 c = columns[(b * BC + 16 * q) / 4 + j / 2];
                                z[q][j] = __fadd2_rn(z[q][j], make_float2(c.x, c.y));
                                z[q][j + 1] = __fadd2_rn(z[q][j + 1], make_float2(c.z, c.w));
                            }
                    if (b + 1 == blocks) {
                        // this warp's share of the tile is in registers, its bias read
                        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) {
                            if constexpr (CG == 1)
                                dev::mbar_arrive(taken + (i & 1));
                            else
                                arrive_in_cluster(in_cta(smem_addr(taken + (i & 1)), 0));
                        }
                    }
                    if (b >= live) continue;
                    const int n = static_cast<int>(n0) + b * BC;
                    if (a.f.has_residual && b + 1 < live && lane == 0) {
                        blocks_read<0>();
                        fetch(b + 1, flip ^ 1);
                    }
                    if (a.f.has_pre) {
                        uint8_t *block = out + (a.f.has_residual ? 2 : flip) * kBlockBytes;
                        if (lane == 0) blocks_read<1>();
                        __syncwarp();
#pragma unroll
                        for (int q = 0; q < SUBS; q++) block_write<T>(block, q, z[q]);
                        block_store<false>(&map_pre, block, n, static_cast<int>(m0), 0, false);
                        if (!a.f.has_residual) flip ^= 1;
                    }
#pragma unroll
                    for (int q = 0; q < SUBS; q++)
#pragma unroll
                        for (int j = 0; j < 8; j++) z[q][j] = activated<T, ACT>(z[q][j]);
                    uint8_t *block = out + flip * kBlockBytes;
                    if (a.f.has_residual) {
                        ok = __all_sync(0xffffffffu, wait_for(&came[e][flip], phases >> flip & 1, a.status));
                        if (!ok) break;
                        phases ^= 1u << flip;
                        coming &= ~(1u << flip);
#pragma unroll
                        for (int q = 0; q < SUBS; q++) block_add<T>(block, q, z[q]);
                    } else {
                        if (lane == 0) blocks_read<1>();
                        __syncwarp();
                    }
#pragma unroll
                    for (int q = 0; q < SUBS; q++) block_write<T>(block, q, z[q]);
                    block_store<RUNS>(&map_out, block, n, static_cast<int>(m0), static_cast<int>(w.part), more);
                    flip ^= 1;
                }
            }
        }
        if (lane == 0) {
            for (int place = 0; place < 2; place++)
                if (coming >> place & 1) wait_for(&came[e][place], phases >> place & 1, a.status);
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
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

// A result's (or residual's, or pre's) tensor map: blocks of 64 bytes by 32 rows, of
// `parts` matrices one after another.
bool encode_out(const Rows &r, unsigned M, unsigned N, int dtype, int parts, size_t part_bytes, CUtensorMap *map)
{
    std::memset(map, 0, sizeof(*map));
    const size_t es = dtype_size(dtype), pitch = r.v.pitch % 16 ? N * es : static_cast<size_t>(r.v.pitch);    // of one row it is any
    const cuuint64_t dims[3] = {N, M, static_cast<cuuint64_t>(parts)};
    const cuuint64_t strides[2] = {pitch, parts > 1 ? part_bytes : pitch};
    const cuuint32_t boxes[3] = {static_cast<cuuint32_t>(kBlockRow / es), 32, 1}, steps[3] = {1, 1, 1};
    const CUtensorMapDataType type = dtype == RZ_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : dtype == RZ_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return encoder()(map, type, 3, r.v.p, dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
    CUtensorMap a, b, out, pre, residual;
};

template <class T, int ACT, int CG>
cudaError_t tc_launch(const TcArgs &a, const Maps &m, void *stream)
{
    const auto fn = k_linear_tc<T, ACT, CG>;
    if (const cudaError_t e = shared_opt_in(reinterpret_cast<const void *>(fn), kSmem - sizeof(Vars))) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CG * std::min<unsigned>(a.tiles, kSms / CG));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kHead - sizeof(Vars) + a.stages * static_cast<size_t>(kBytesA + a.tile_n / CG * kTerms * 2) +
                           static_cast<size_t>(kEpiWarps) * a.places * kBlockBytes;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 1 ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, fn, a, m.a, m.b, m.out, m.pre, m.residual);
}

template <class T, int CG>
cudaError_t tc_launch_act(const TcArgs &a, const Maps &m, void *stream)
{
    if (a.f.act == RZ_ACT_SILU) return tc_launch<T, RZ_ACT_SILU, CG>(a, m, stream);
    return a.f.act == RZ_ACT_GELU ? tc_launch<T, RZ_ACT_GELU, CG>(a, m, stream) : tc_launch<T, RZ_ACT_NONE, CG>(a, m, stream);
}
template <class T>
cudaError_t tc_launch_of(const TcArgs &a, const Maps &m, int pair, void *stream)
{
    return pair ? tc_launch_act<T, 2>(a, m, stream) : tc_launch_act<T, 1>(a, m, stream);
}

}  // namespace

bool lin::direct_out(const Finish &f, int dtype)
{
    const auto fits = [&](const Rows &r) {
        return !r.HW && reinterpret_cast<uintptr_t>(r.v.p) % 16 == 0 && (f.M == 1 || r.v.pitch % 16 == 0);
    };
    // TMA clips a row to whole 16 bytes
    return f.N * dtype_size(dtype) % 16 == 0 && fits(f.out) && (!f.has_pre || fits(f.pre)) && (!f.has_residual || fits(f.residual));
}

cudaError_t lin::launch_product(const Product &p, void *stream)
{
    if (!encoder()) return cudaErrorNotSupported;
    const int cg = p.pair ? 2 : 1;
    Maps m;
    TcArgs a{};
    if (!encode(p.a, kTileM, &m.a, &a.a_merged) || !encode(p.b, p.tile_n / cg, &m.b, &a.b_merged)) return cudaErrorInvalidValue;
    a.f = p.f;
    int dtype = p.out_dtype;
    if (p.part) {
        // sums in parts or runs, and what TMA cannot write, leave as they are, float32; k_linear_join finishes them
        dtype = RZ_F32;
        a.f = Finish{};
        a.f.M = p.f.M;
        a.f.N = p.f.N;
        a.f.out.v = {reinterpret_cast<uint8_t *>(p.part), static_cast<long long>(p.part_pitch) * 4, 0};
    }
    if (!encode_out(a.f.out, a.f.M, a.f.N, dtype, p.parts, static_cast<size_t>(p.part_pitch) * 4 * a.f.M, &m.out))
        return cudaErrorInvalidValue;
    m.pre = m.residual = m.out;     // where there is none
    if (a.f.has_pre && !encode_out(a.f.pre, a.f.M, a.f.N, dtype, 1, 0, &m.pre)) return cudaErrorInvalidValue;
    if (a.f.has_residual && !encode_out(a.f.residual, a.f.M, a.f.N, dtype, 1, 0, &m.residual)) return cudaErrorInvalidValue;
    a.places = a.f.has_pre && a.f.has_residual ? 3 : 2;
    a.tile_n = p.tile_n;
    a.tiles_m = (p.f.M + cg * kTileM - 1) / (cg * kTileM);
    a.tiles_n = (p.f.N + p.tile_n - 1) / p.tile_n;
    a.products = products_of(p.a.planes, p.b.planes);
    // Tiles of a row next to each other read its A at once, and B out of L2 where that holds it (65536 x 1024 x 4096: 341 us,
    // rows of tiles in groups of eight 373).  A larger B is read once for eight rows of tiles (8192 x 8192 x 8192: 611 us, by
    // single rows 650).
    a.group = 2.0 * p.f.N * p.b.terms * p.b.planes > 48e6 ? 8 : 1;
    a.chunks = static_cast<int>((p.a.terms + kTerms - 1) / kTerms);
    a.part = p.part_chunks;
    a.run = p.run_chunks;
    const unsigned long long tiles = static_cast<unsigned long long>(a.tiles_m) * a.tiles_n * p.parts;
    if (tiles > 0x7fffffffull) return cudaErrorInvalidConfiguration;
    a.tiles = static_cast<unsigned>(tiles);
    a.stages = std::min(kRing, (kSmem - kHead - kEpiWarps * a.places * kBlockBytes) / (kBytesA + p.tile_n / cg * kTerms * 2));
    a.a_turned = p.a.turned;
    a.b_turned = p.b.turned;
    const unsigned type = p.a.bf16 ? 1u : 0u;
    a.idesc = (1u << 4) | (type << 7) | (type << 10) | (static_cast<unsigned>(p.a.turned) << 15) |
              (static_cast<unsigned>(p.b.turned) << 16) | (static_cast<unsigned>(p.tile_n >> 3) << 17) |
              (static_cast<unsigned>(cg * kTileM >> 4) << 24);
    a.status = p.status;
    if (dtype == RZ_F32) return tc_launch_of<float>(a, m, p.pair, stream);
    return dtype == RZ_BF16 ? tc_launch_of<__nv_bfloat16>(a, m, p.pair, stream) : tc_launch_of<__half>(a, m, p.pair, stream);
}

}  // namespace rz
