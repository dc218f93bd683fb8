// Newton-Schulz orthogonalisation of a weight's update.
//
//   X <- G / (|G|_F + eps), transposed where G is tall, so X is r x c, r <= c
//   steps times:  A = X X^T,   Q = a I + b A + c A A,   X <- Q X
//
// The three products are nearly all of the work: r r c multiply-adds for Q X
// and, A and A A being symmetric, half of r r c and of r r r for the others
// (one triangle of tiles is computed, its mirror image stored).  All of them
// run on one tcgen05 kernel (the TMA ring of the BF16 GEMM) with float16
// operands and float32 accumulators.
//
// Precision.  One float16 operand has 11 significant bits, and what rounding
// an iterate loses does not stay small: the iteration multiplies a singular
// direction far below the largest by a = 3.4 per step, the rounding errors
// that fall on it included.  So each matrix is kept as a sum of float16
// planes, x = x0 + x1 (+ x2), each plane the rounding of what the planes
// before it left over, and a product runs over pairs of planes, all into one
// accumulator.  Which pairs are needed differs by matrix:
//
//   X     Every bit lost in X is lost in its small singular directions, so X
//         carries one plane more than the result's type asks for.
//   A, Q  An error in an entry of A or Q acts on X from the left, spread over
//         the row; only the diagonal, large beside the rest in the late
//         steps, needs the extra plane.  It is kept and multiplied for the
//         256 x 256 blocks on the diagonal alone.
//
//   bfloat16 result:  A one pair, A A one, Q X two (one in the last step,
//                     whose roundings no later step multiplies).
//   float32 result:   A three pairs, A A three, Q X four (three in the last).
//
// Measured in float64 arithmetic on spectra from flat to 1e-3 of the largest
// value (256 .. 1000 rows): the bfloat16 result is off by 1.03 to 1.15 times
// the error of rounding the exact result; one pair throughout by up to 16
// times.  On GB300 at 8192 x 8192: 1.03 (decaying spectrum) and 1.05 times
// (flat).  float32 result, 1000 x 3000: 1.7e-7 for equal singular
// values and 3.3e-6 for log-spaced ones down to 1e-3, where the formula in
// float32 arithmetic is off by 7.3e-7 and 4.5e-6.  A fifth pair for Q X, x1 of
// both, takes 5 % more time; without it the error stays below 1.4 times that of
// float32 arithmetic at every size and spectrum tried (tests hold it to 1.5).
//
// A A is never added to b A: the square is completed,
//   Q = c (A + (b / 2c) I)^2 + (a - b b / 4c) I,
// so that the kernel's whole epilogue is a scaling and a diagonal, and reads
// nothing.  (c = 0: Q = a I + b A straight from X X^T.)
//
// What bounds it, on GB300.  Large sides: an SM's shared memory and then the
// power limit (the 256 x 256 tile, choose_cut()).  4096 x 4096 bfloat16 takes
// 1.28 ms, 1.57 PFLOP/s of float16 products done; 8192 x 8192 9.46 ms, 1.70
// PFLOP/s, where a library's bfloat16 product, under the same limit, sustains
// 1.69.  Middle sides: the 95 GB/s or so at which an SM takes operands in, and
// too few tiles (1000 x 3000 float32 345 us, 5000 x 1000 269 us).  Below 500
// or so the chain of fifteen products, each about 7 us of latency: 1.2 until
// the next kernel starts, 0.7 to the first operands, 1 of MMAs, 2 of exchange
// between ranks, 2 of epilogue and stores (256 x 256 114 us); sides of at most
// 128 have a kernel of their own (orthogonalize_small.cu).
//
// Scaling.  G is multiplied by a power of two only, which keeps bfloat16
// entries exact in float16; the rest of 1 / (|G|_F + eps) goes into the
// epilogues in float32, of the first step unless eps dwarfs |G|_F (Factors).
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "orthogonalize_internal.h"
#include "pipelined_train.h"
#include "tma_ring.cuh"

namespace pg {

namespace orth {

constexpr int BK = 64;                          // K block: 128 bytes of float16
constexpr int kUmmaM = 128;
constexpr int kUmmaK = 16;
constexpr uint32_t kAtomBytes = 64 * BK * 2;    // 64 columns of an MN-major operand: 8 KiB
constexpr int kDiagBlock = 256;                 // side of the diagonal blocks that keep the extra plane
constexpr uint32_t kStagingBytes = 32 * 128;    // per epilogue warp: 32 rows of 128 bytes

// One pair of planes to multiply.  Plane -1 is the diagonal-block plane.
// `range`: all of K, or the K of this tile's rows or columns.
enum Range { kAll, kRows, kCols };
struct Pass {
    signed char left, right, range;
};
constexpr int kMaxPasses = 5;

enum Output { kPlanes, kBf16, kF32 };

struct Maps {
    // Loads, one box per operand and K block, 128-byte swizzle: 64 k by the
    // tile's rows, or for Q X's right operand its columns in groups of 64 by
    // 64 k.
    CUtensorMap left, left_diag, right, right_diag;
    CUtensorMap store, mirror, store_diag, mirror_diag;
};

// The tensor cores add to a float32 accumulator by truncation: n additions in
// a row lose about n 2^-25 of a sum of equal signs (A's diagonal), which a
// bfloat16 result does not notice and a float32 one does.  There (Product.fine)
// each K block (four additions) of the one pass over the leading planes has an
// accumulator of its own, and the epilogue adds them with rounding; the other
// passes' terms are 2^-11 as large and share one.  Error of the float32 result
// against float64, 1000 x 3000, flat and decaying spectrum, the products then
// with a fifth pair in Q X: 9.5e-6 and 1.2e-5 with four K blocks to an
// accumulator, 3.1e-6 and 4.2e-6 with one.  With four pairs and one K block to
// an accumulator: 3.1e-6 and 4.3e-6, the formula in float32 arithmetic 3.7e-6
// and 7.0e-6.
enum Fine { kWhole, kPerBlock, kPerStep }; // one for all, one per K block, one per MMA

// Short sums show what the four additions of a K block lose: with a side r of
// up to this every MMA has an accumulator of its own.
constexpr int kStepSide = 128;

// D (rows x cols, a batch of them) = sum over the passes of left plane times
// right plane over k, scaled by alpha, plus diag on the diagonal.

struct Product {
    int rows, cols, k, batch;
    int symmetric; // compute the tiles on and above the diagonal, store both
    int left_planes, right_planes;
    int passes;
    Pass pass[kMaxPasses];
    int ranks; // CTAs that share a tile's K blocks
    int fine; // Fine: accumulators of the last pass; the passes before it have one
    float alpha, diag;
    int alpha_g, alpha_rho, diag_rho; // powers of this step's Factors
    const Factors *f; // of matrix b at f[b * kFactors]
    int output;                  // Output
    int planes;                  // kPlanes: how many to write
    int planes_pitch;            // kPlanes: planes per matrix of the batch
    int diag_plane;              // kPlanes: also one more on the diagonal blocks
    int transposed;              // final output: D^T
    int out_tma;                 // final output through TMA stores
    void *out;
    long long ldo, out_batch;    // elements
    unsigned int *status;
    unsigned long long wait_limit_ns;
    int withhold;
};

// Tile of MH x 128 rows by BN columns, S ring stages.  The 256 x 256 tile
// fills tensor memory with one accumulator and has each of its eight epilogue
// warps take a quarter's 256 columns in turn; the 128-row tiles, of 128 or 192
// columns, have four or two accumulators and each warp takes 64 columns at
// once, so that it can also sum a tile's accumulators in registers
// (Product.fine).
//
// Split: where the 128 x 128 tiles are fewer than half the SMs, a cluster of
// 2, 4 or 8 CTAs shares a tile's K blocks, each multiplying its run of them.
// A tile is eight units of 32 rows by 64 columns, one per epilogue warp; each
// rank owns 8 / ranks of them, receives the other ranks' sums of those into
// its shared memory, adds them in rank order and stores them.
template <int MH, int BN, int S, bool Split>
struct Tile {
    static constexpr int BM = kUmmaM * MH;
    static constexpr uint32_t kLeftBytes = BM * BK * 2;
    static constexpr uint32_t kStageBytes = kLeftBytes + BN * BK * 2;
    static constexpr int kAccBufs = 512 / (MH * BN);
    static constexpr uint32_t kTmemCols = 512;
    static constexpr int kEpiCols = MH == 2 ? BN : 64; // columns per epilogue warp
    static constexpr int kEpiWarps = 4 * MH * BN / kEpiCols;
    static constexpr int kThreads = (2 + kEpiWarps) * 32;
    static constexpr uint32_t kUnitBytes = 32 * 64 * 4;
    static constexpr uint32_t kReceiveBytes = Split ? kEpiWarps * kUnitBytes : 0;
    static constexpr int kSmem = S * kStageBytes + kEpiWarps * kStagingBytes + kReceiveBytes + 1024 /* barriers */ +
                                 1024 /* slack */;
    static_assert(MH * BN <= 512 && kEpiCols % 64 == 0, "accumulators fit tensor memory");
    static_assert(!Split || kEpiCols == 64, "a unit is what one warp holds");
};

// Tile t of the batch: matrix b, tile row i, tile column j.  The upper
// triangle goes column by column; a full matrix in groups of 16 tile rows.
struct TileAt {
    int b, i, j;
};

__host__ __device__ inline int tiles_of(bool symmetric, int tiles_m, int tiles_n)
{
    return symmetric ? tiles_m * (tiles_m + 1) / 2 : tiles_m * tiles_n;
}

__device__ __forceinline__ TileAt tile_at(int t, bool symmetric, int tiles_m, int tiles_n)
{
    const int per = tiles_of(symmetric, tiles_m, tiles_n);
    TileAt at;
    at.b = t / per;
    int r = t - at.b * per;
    if (symmetric) {
        int j = static_cast<int>((sqrtf(8.0f * static_cast<float>(r) + 1.0f) - 1.0f) * 0.5f);
        while (j * (j + 1) / 2 > r)
            --j;
        while ((j + 1) * (j + 2) / 2 <= r)
            ++j;
        at.j = j;
        at.i = r - j * (j + 1) / 2;
    } else {
        constexpr int kGroup = 16;
        const int group = r / (kGroup * tiles_n);
        const int first = group * kGroup;
        const int gm = min(kGroup, tiles_m - first);
        r -= group * kGroup * tiles_n;
        at.i = first + r % gm;
        at.j = r / gm;
    }
    return at;
}

// K blocks of one pass for a tile whose rows start at row0 and columns at col0.
template <int BM, int BN>
__device__ __forceinline__ void pass_range(const Pass &pass, int k, int row0, int col0, int &k0, int &blocks)
{
    k0 = pass.range == kAll ? 0 : pass.range == kRows ? row0 : col0;
    const int k1 = pass.range == kAll ? k : min(k, k0 + (pass.range == kRows ? BM : BN));
    blocks = (k1 - k0 + BK - 1) / BK;
}

// K blocks of one tile: of all its passes but the last, and of all.
struct Blocks {
    int before, all;
    int lo, hi; // this CTA's
    // How many accumulators that takes.
    __device__ __forceinline__ int accumulators(int fine) const
    {
        if (fine == kWhole)
            return lo < hi ? 1 : 0;
        return (lo < min(before, hi) ? 1 : 0) +
               max(0, hi - max(lo, before)) * (fine == kPerStep ? BK / kUmmaK : 1);
    }
};

template <int BM, int BN>
__device__ __forceinline__ Blocks tile_blocks(const Product &p, const TileAt &at, int rank)
{
    Blocks n{0, 0, 0, 0};
    for (int ps = 0; ps < p.passes; ++ps) {
        int k0, blocks;
        pass_range<BM, BN>(p.pass[ps], p.k, at.i * BM, at.j * BN, k0, blocks);
        n.before = n.all;
        n.all += blocks;
    }
    n.lo = rank * n.all / p.ranks;
    n.hi = (rank + 1) * n.all / p.ranks;
    return n;
}

// An epilogue warp's 4 KiB staging buffers, from which TMA stores move boxes.
// The one of its own is written again when the store before has read it.  In
// a CTA's last tile the ring is idle and lends each warp kLentBufs more, so
// that no write waits.
constexpr int kLentBufs = 3;

struct Staging {
    uint32_t own, lent; // first addresses; lent 0: not now
    int lane;
    uint32_t addr = 0;
    int turn = 0;

    __device__ __forceinline__ void begin()
    {
        if (lent == 0) {
            addr = own;
            if (lane == 0)
                bulk_wait_group_read<0>();
        } else {
            addr = lent + static_cast<uint32_t>(turn) * kStagingBytes;
            turn = turn + 1 == kLentBufs ? 0 : turn + 1;
            if (lane == 0)
                bulk_wait_group_read<kLentBufs - 1>();
        }
        __syncwarp();
    }
    __device__ __forceinline__ void end(const CUtensorMap *map, int x, int y, int z) const
    {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_3d(map, addr, x, y, z);
            bulk_commit_group();
        }
    }
    // 32 words of this lane's row, in the 128-byte swizzle.
    __device__ __forceinline__ void row(const uint32_t (&w)[32]) const
    {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(
                             addr + static_cast<uint32_t>(lane * 128 + ((j ^ (lane & 7)) << 4))),
                         "r"(w[4 * j]), "r"(w[4 * j + 1]), "r"(w[4 * j + 2]), "r"(w[4 * j + 3])
                         : "memory");
    }
    // The transpose of what row() has put into this buffer, 64 rows of 32
    // two-byte elements, in 8 x 8 blocks: taken to registers, and (after
    // begin()) put down in the 64-byte swizzle.
    __device__ __forceinline__ void take_transposed(uint32_t (&w)[32]) const
    {
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint32_t r[4];
            load_blocks_transposed(addr + static_cast<uint32_t>(lane * 128 + ((c ^ (lane & 7)) << 4)), r);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[4 * c + e] = r[e];
        }
    }
    __device__ __forceinline__ void transposed(const uint32_t (&w)[32]) const
    {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int j = c * 8 + lane % 8; // row: the block's column
            const uint32_t r[4] = {w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]};
            store_blocks(addr + static_cast<uint32_t>(j * 64 + (((lane / 8) ^ ((j >> 1) & 3)) << 4)), r);
        }
    }
    // 32 rows of 32 four-byte elements, this lane's column.
    __device__ __forceinline__ void column32(const uint32_t (&w)[32]) const
    {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            asm volatile("st.shared.b32 [%0], %1;\n" ::"r"(addr + static_cast<uint32_t>(j * 128 + lane * 4)), "r"(w[j])
                         : "memory");
    }
};

// RightMN: the right operand's rows are k (Q X); otherwise its rows are D's
// columns (X X^T, and the symmetric A A).
template <int MH, int BN, int S, bool RightMN, bool Split, bool Steps = false>
__global__ void __launch_bounds__(Tile<MH, BN, S, Split>::kThreads, 1)
    product_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Product p)
{
    using T = Tile<MH, BN, S, Split>;
    constexpr int BM = T::BM;
    // Instruction descriptor, kind::f16: D float32 (bits 4-5 = 1), A and B
    // float16 (bits 7-12 = 0), A K-major, B K-major or MN-major (bit 16),
    // N >> 3 at bits 17-22, M >> 4 at bits 24-28.
    constexpr uint32_t kIdesc = (1u << 4) | (RightMN ? 1u << 16 : 0u) | (static_cast<uint32_t>(BN >> 3) << 17) |
                                (static_cast<uint32_t>(kUmmaM >> 4) << 24);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = align_smem(raw, 1024);
    const uint32_t staging0 = base + S * T::kStageBytes;
    const uint32_t receive0 = staging0 + T::kEpiWarps * kStagingBytes;
    const uint32_t bars = receive0 + T::kReceiveBytes;
    const TmaRing<S> ring{bars, bars + 8u * S};
    const uint32_t tmem_full0 = bars + 16u * S;                  // [kAccBufs]
    const uint32_t tmem_empty0 = tmem_full0 + 8u * T::kAccBufs; // [kAccBufs]
    const uint32_t epi_done = tmem_empty0 + 8u * T::kAccBufs;
    const uint32_t mma_done = epi_done + 8u;
    const uint32_t tmem_slot = mma_done + 8u;
    volatile uint32_t *tmem_slot_ptr = reinterpret_cast<volatile uint32_t *>(smem_raw + (tmem_slot - raw));

    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    const bool symmetric = p.symmetric != 0;
    const int tiles_m = (p.rows + BM - 1) / BM;
    const int tiles_n = (p.cols + BN - 1) / BN;
    const int num_tiles = tiles_of(symmetric, tiles_m, tiles_n) * p.batch;
    // A split tile has a cluster of its own, so each CTA has one tile.
    const int rank = Split ? static_cast<int>(cluster_cta_rank()) : 0;
    const int first_tile = Split ? static_cast<int>(blockIdx.x) / p.ranks : static_cast<int>(blockIdx.x);
    const int tile_step = Split ? num_tiles : static_cast<int>(gridDim.x);

    if (threadIdx.x == 0) {
        ring.init(1);
        for (int b = 0; b < T::kAccBufs; ++b) {
            mbar_init(tmem_full0 + 8u * b, 1);
            mbar_init(tmem_empty0 + 8u * b, T::kEpiWarps);
        }
        mbar_init(epi_done, T::kEpiWarps);
        mbar_init(mma_done, 1);
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_map(&maps.left);
        tma_prefetch_map(&maps.right);
        tma_prefetch_map(&maps.store);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, T::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    if constexpr (Split)
        cluster_sync(); // every CTA of the cluster has started
    else
        __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot_ptr;
    grid_launch_next();
    // The kernel before, whose results this one reads and whose operands it
    // overwrites, is waited for by the roles that touch global memory, each at
    // its first access: what they work out before that (a tile's place and its
    // K blocks, about 1 us) no longer stands between two products (2048 x 2048
    // bfloat16: 399 -> 379 us, 256 x 256 129 -> 114).

    if (warp == 0) {
        // ------------------------------------------------------- TMA producer
        if (lane == 0) {
            int f = 0;
            bool ok = true, waited = false;
            for (int t = first_tile; t < num_tiles && ok; t += tile_step) {
                const TileAt at = tile_at(t, symmetric, tiles_m, tiles_n);
                const int row0 = at.i * BM, col0 = at.j * BN;
                const Blocks all = tile_blocks<BM, BN>(p, at, rank);
                int before = 0; // K blocks of the passes before this one
                for (int ps = 0; ps < p.passes && ok; ++ps) {
                    const Pass pass = p.pass[ps];
                    int k0, blocks;
                    pass_range<BM, BN>(pass, p.k, row0, col0, k0, blocks);
                    const int kb_lo = max(0, all.lo - before), kb_hi = min(blocks, all.hi - before);
                    before += blocks;
                    const bool ld = pass.left < 0, rd = pass.right < 0;
                    const CUtensorMap *lmap = ld ? &maps.left_diag : &maps.left;
                    const CUtensorMap *rmap = rd ? &maps.right_diag : &maps.right;
                    const int lz = ld ? at.b : at.b * p.left_planes + pass.left;
                    const int rz = rd ? at.b : at.b * p.right_planes + pass.right;
                    for (int kb = kb_lo; kb < kb_hi; ++kb, ++f) {
                        if (f == p.withhold)
                            continue; // test hook: this position is never filled
                        if (!waited) {
                            grid_wait();
                            waited = true;
                        }
                        if (!ring.producer_acquire(f, p.wait_limit_ns)) {
                            record_error(p.status, kErrFamilyOrthogonalize | kErrRoleProducer);
                            ok = false;
                            break;
                        }
                        const int k = k0 + kb * BK;
                        const int lx = ld ? k % kDiagBlock : k, rx = rd ? k % kDiagBlock : k;
                        const uint32_t dst = base + static_cast<uint32_t>(f % S) * T::kStageBytes;
                        const uint32_t full = ring.full_bar(f);
                        ring.producer_commit(f, T::kStageBytes);
                        tma_load_3d(dst, lmap, full, lx, row0, lz);
                        if constexpr (RightMN)
                            tma_load_4d(dst + T::kLeftBytes, rmap, full, 0, k, col0 / 64, rz);
                        else
                            tma_load_3d(dst + T::kLeftBytes, rmap, full, rx, col0, rz);
                    }
                }
            }
            // Only the last S positions issued can still be in flight.
            bool drained = true;
            for (int g = f > S ? f - S : 0; g < f; ++g)
                if (g != p.withhold && !ring.consumer_wait(g, p.wait_limit_ns))
                    drained = false;
            if (!drained)
                record_error(p.status, kErrFamilyOrthogonalize | kErrRoleDrain);
        }
        if constexpr (Split)
            cluster_sync(); // the epilogue's exchange
    } else if (warp == 1) {
        // ------------------------------------------------------- MMA issuer
        // (Steps, the path of Fine::kPerStep, is a kernel of its own: merely
        // present in this loop it made 2048 x 2048 bfloat16 take 460 us
        // instead of 407.)
        // One thread's instructions stand between the MMAs: with descriptors
        // built anew for each MMA the 256 x 256 tile took 0.65 us a K block,
        // in which its MMAs take 0.52 at 1.96 GHz.  So they are built once;
        // stages and K steps add to their address field (16-byte units).
        {
            const uint32_t on = lane == 0 ? 1u : 0u;
            constexpr uint64_t kStageStep = T::kStageBytes >> 4, kRowsStep = (kUmmaM * 128) >> 4;
            // K step: 32 bytes along a K-major row; 16 rows of 128 bytes of an
            // MN-major box.
            constexpr uint64_t kLeftStep = (kUmmaK * 2) >> 4, kRightStep = (RightMN ? kUmmaK * 128 : kUmmaK * 2) >> 4;
            const uint64_t left0 = smem_desc_sw128(base, 16, 1024);
            const uint64_t right0 = smem_desc_sw128(base + T::kLeftBytes, RightMN ? kAtomBytes : 16, 1024);
            uint64_t left = left0, right = right0;
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            int acc = 0; // accumulators begun
            uint32_t d_tmem = tmem_base, full_bar = tmem_full0;
            auto begin = [&]() { // an accumulator
                const int slot = acc % T::kAccBufs;
                const uint32_t use_parity = static_cast<uint32_t>((acc / T::kAccBufs) & 1);
                if (!__all_sync(0xffffffffu,
                                mbar_wait_bounded(tmem_empty0 + 8u * slot, use_parity ^ 1u, p.wait_limit_ns))) {
                    if (on)
                        record_error(p.status, kErrFamilyOrthogonalize | kErrRoleMma);
                    return false;
                }
                tc_fence_after_sync();
                d_tmem = tmem_base + static_cast<uint32_t>(slot * MH * BN);
                full_bar = tmem_full0 + 8u * slot;
                ++acc;
                return true;
            };
            for (int t = first_tile; t < num_tiles && ok; t += tile_step) {
                const TileAt at = tile_at(t, symmetric, tiles_m, tiles_n);
                const Blocks blocks = tile_blocks<BM, BN>(p, at, rank);
                bool fresh = true; // the next MMA begins an accumulator
                for (int kb = blocks.lo; kb < blocks.hi; ++kb) {
                    const bool steps = Steps && kb >= blocks.before;
                    if (fresh && !steps && !begin()) {
                        ok = false;
                        break;
                    }
                    if (!__all_sync(0xffffffffu, mbar_wait_bounded(ring.full0 + 8u * stage, phase, p.wait_limit_ns))) {
                        if (on)
                            record_error(p.status, kErrFamilyOrthogonalize | kErrRoleMma);
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    bool stepped = false;
                    if constexpr (Steps) {
                        stepped = steps;
                        for (int ks = 0; ks < BK / kUmmaK && ok && steps; ++ks) {
                            ok = begin();
                            if (ok) {
                                mma_f16_ss_if(on, d_tmem, left + ks * kLeftStep, right + ks * kRightStep, kIdesc, 0u);
                                mma_commit_if(on, full_bar);
                            }
                        }
                    }
                    if (!stepped) {
#pragma unroll
                        for (int ks = 0; ks < BK / kUmmaK; ++ks)
#pragma unroll
                            for (int h = 0; h < MH; ++h)
                                mma_f16_ss_if(on, d_tmem + static_cast<uint32_t>(h * BN),
                                           left + (ks * kLeftStep + h * kRowsStep), right + ks * kRightStep, kIdesc,
                                           ks == 0 && fresh ? 0u : 1u);
                        fresh = kb == blocks.hi - 1 || (MH == 1 && p.fine != kWhole && kb >= blocks.before - 1);
                        if (fresh)
                            mma_commit_if(on, full_bar); // accumulator complete
                    }
                    if (!ok)
                        break;
                    mma_commit_if(on, ring.empty0 + 8u * stage); // stage free once these MMAs have read it
                    left += kStageStep;
                    right += kStageStep;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                        left = left0;
                        right = right0;
                    }
                }
            }
            // Every MMA this thread issued must finish before tensor memory is freed.
            mma_commit_if(on, mma_done);
            if (!mbar_wait_bounded(mma_done, 0, p.wait_limit_ns) && on)
                record_error(p.status, kErrFamilyOrthogonalize | kErrRoleDrain);
        }
        if constexpr (Split)
            cluster_sync(); // the epilogue's exchange
        __syncwarp();
        if (!mbar_wait_bounded(epi_done, 0, p.wait_limit_ns) && lane == 0)
            record_error(p.status, kErrFamilyOrthogonalize | kErrRoleDrain);
        tc_fence_after_sync();
        __syncwarp();
        tmem_dealloc(tmem_base, T::kTmemCols);
    } else {
        // ------------------------------------------------------- epilogue
        const int quarter = warp & 3; // the tensor-memory lanes this warp may read
        const int epi = warp - 2;
        const int half = MH == 2 ? epi / 4 : 0;                      // of the tile's rows
        const int first_col = MH == 2 ? 0 : (epi / 4) * T::kEpiCols; // of the tile's columns
        Staging staging{staging0 + static_cast<uint32_t>(epi) * kStagingBytes, 0, lane};
        static_assert(T::kEpiWarps * kLentBufs * kStagingBytes <= S * T::kStageBytes, "the ring has room to lend");
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        int acc = 0; // accumulators taken
        grid_wait();
        for (int t = first_tile; t < num_tiles; t += tile_step) {
            const TileAt at = tile_at(t, symmetric, tiles_m, tiles_n);
            const Factors f = p.f[at.b * kFactors];
            float alpha = p.alpha, diag = p.diag;
            for (int e = 0; e < p.alpha_g; ++e)
                alpha *= f.g;
            if (p.alpha_rho)
                alpha *= f.rho;
            if (p.diag_rho)
                diag *= f.rho;
            const int row0 = at.i * BM + half * kUmmaM + quarter * 32;
            const int row = row0 + lane;
            const bool mirrored = symmetric && at.i != at.j;

            // 64 columns of a finished accumulator, in pairs, to v or added to it.
            auto take = [&](int slot, int column, bool add, unsigned long long (&v)[32]) {
                uint32_t r0[32], r1[32];
                const uint32_t taddr = tmem_base + lanes + static_cast<uint32_t>((slot * MH + half) * BN + column);
                tmem_ld_32x32b_x32(taddr, r0);
                tmem_ld_32x32b_x32(taddr + 32u, r1);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const unsigned long long a = pair(__uint_as_float(r0[2 * j]), __uint_as_float(r0[2 * j + 1]));
                    const unsigned long long b = pair(__uint_as_float(r1[2 * j]), __uint_as_float(r1[2 * j + 1]));
                    v[j] = add ? add2(v[j], a) : a;
                    v[16 + j] = add ? add2(v[16 + j], b) : b;
                }
            };
            // Wait for accumulator `acc`; false when the wait ran out.
            auto wait_full = [&]() {
                const bool ok = mbar_wait_bounded(tmem_full0 + 8u * (acc % T::kAccBufs),
                                                  static_cast<uint32_t>((acc / T::kAccBufs) & 1), p.wait_limit_ns);
                if (!__all_sync(0xffffffffu, ok)) {
                    if (lane == 0)
                        record_error(p.status, kErrFamilyOrthogonalize | kErrRoleEpilogue);
                    return false;
                }
                tc_fence_after_sync();
                return true;
            };
            // The accumulator has been read (tcgen05.wait::ld): hand it back.
            auto release = [&]() {
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(tmem_empty0 + 8u * (acc % T::kAccBufs));
                ++acc;
            };
            // Past the last accumulator of the CTA's last tile: every copy has
            // landed and been multiplied.
            auto borrow = [&]() {
                if (t + tile_step >= num_tiles)
                    staging.lent = base + static_cast<uint32_t>(epi * kLentBufs) * kStagingBytes;
            };
            // 64 columns of this warp's 32 rows, scaled and stored.
            auto emit = [&](unsigned long long (&v)[32], int col0) {
                const unsigned long long scale = pair(alpha, alpha);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    v[j] = mul2(v[j], scale);
                if (p.diag != 0.0f && row0 < col0 + 64 && col0 < row0 + 32) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = add2(v[j], pair(col0 + 2 * j == row ? diag : 0.0f,
                                               col0 + 2 * j + 1 == row ? diag : 0.0f));
                }
                uint32_t w[32];
                float lo, hi;
                if (p.output == kPlanes) {
                    const bool on_diag = p.diag_plane != 0 && row0 / kDiagBlock == col0 / kDiagBlock;
                    const int planes = p.planes + (on_diag ? 1 : 0);
#pragma unroll 1
                    for (int q = 0; q < planes; ++q) {
                        const bool extra = q == p.planes;
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            split(v[j], lo, hi);
                            w[j] = pack_f16(lo, hi);
                        }
                        if (q + 1 < planes) { // what this plane leaves over, exactly
                            const unsigned long long minus = pair(-1.0f, -1.0f);
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                const float2 kept = unpack_f16(w[j]);
                                v[j] = fma2(pair(kept.x, kept.y), minus, v[j]);
                            }
                        }
                        staging.begin();
                        staging.row(w);
                        if (extra)
                            staging.end(&maps.store_diag, col0 % kDiagBlock, row0, at.b);
                        else
                            staging.end(&maps.store, col0, row0, at.b * p.planes_pitch + q);
                        if (mirrored) {
                            staging.take_transposed(w);
                            staging.begin();
                            staging.transposed(w);
                            if (extra)
                                staging.end(&maps.mirror_diag, row0 % kDiagBlock, col0, at.b);
                            else
                                staging.end(&maps.mirror, row0, col0, at.b * p.planes_pitch + q);
                        }
                    }
                } else if (p.out_tma && p.output == kBf16) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        split(v[j], lo, hi);
                        w[j] = pack_bf16(lo, hi);
                    }
                    staging.begin();
                    staging.row(w);
                    if (p.transposed) {
                        staging.take_transposed(w);
                        __syncwarp();
                        staging.transposed(w);
                        staging.end(&maps.store, row0, col0, at.b);
                    } else {
                        staging.end(&maps.store, col0, row0, at.b);
                    }
                } else if (p.out_tma) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (col0 + 32 * h >= p.cols)
                            break; // warp-uniform
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            split(v[16 * h + j], lo, hi);
                            w[2 * j] = __float_as_uint(lo);
                            w[2 * j + 1] = __float_as_uint(hi);
                        }
                        staging.begin();
                        if (p.transposed) {
                            staging.column32(w);
                            staging.end(&maps.store, row0, col0 + 32 * h, at.b);
                        } else {
                            staging.row(w);
                            staging.end(&maps.store, col0 + 32 * h, row0, at.b);
                        }
                    }
                } else if (row < p.rows) {
                    // Rows that TMA cannot store (not 16-byte aligned): one
                    // guarded element each.
                    const long long first = at.b * p.out_batch;
#pragma unroll
                    for (int j = 0; j < 64; ++j) {
                        if (col0 + j < p.cols) {
                            const long long o = first + (p.transposed ? (col0 + j) * p.ldo + row
                                                                      : row * p.ldo + col0 + j);
                            split(v[j / 2], lo, hi);
                            store_f32(p.out, p.output == kBf16, o, j & 1 ? hi : lo);
                        }
                    }
                }
            };

            if constexpr (T::kEpiCols == 64) {
                const int parts = tile_blocks<BM, BN>(p, at, rank).accumulators(p.fine);
                unsigned long long v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    v[j] = 0ull;
                bool ok = true;
                for (int part = 0; part < parts && ok; ++part) {
                    ok = wait_full();
                    if (ok) {
                        take(acc % T::kAccBufs, first_col, true, v);
                        release();
                    }
                }
                bool mine = ok;
                if constexpr (Split) {
                    // This warp's unit goes to its owner, or gathers the other
                    // ranks' sums of it: 16 bytes of 32 lanes side by side.
                    const int unit = quarter * 2 + epi / 4, each = T::kEpiWarps / p.ranks;
                    const int owner = unit / each;
                    const uint32_t slots = receive0 + static_cast<uint32_t>(unit % each * p.ranks) * T::kUnitBytes;
                    mine = ok && owner == rank;
                    if (ok && owner != rank) {
                        const uint32_t to = map_to_cta(slots + static_cast<uint32_t>(rank) * T::kUnitBytes,
                                                       static_cast<uint32_t>(owner)) +
                                            static_cast<uint32_t>(lane) * 16u;
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            float a, b, c, d;
                            split(v[j], a, b);
                            split(v[j + 1], c, d);
                            st_cluster_v4(to + static_cast<uint32_t>(j) * 256u, __float_as_uint(a), __float_as_uint(b),
                                          __float_as_uint(c), __float_as_uint(d));
                        }
                    }
                    cluster_sync(); // also in a CTA whose wait ran out
                    for (int src = 0; src < p.ranks && mine; ++src) {
                        if (src == rank)
                            continue;
                        const uint8_t *from = smem_raw + (slots - raw) + src * T::kUnitBytes + lane * 16;
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            const float4 q = *reinterpret_cast<const float4 *>(from + j * 256);
                            v[j] = add2(v[j], pair(q.x, q.y));
                            v[j + 1] = add2(v[j + 1], pair(q.z, q.w));
                        }
                    }
                }
                if (!ok)
                    break;
                borrow();
                const int col0 = at.j * BN + first_col;
                if (mine && row0 < p.rows && col0 < p.cols) // warp-uniform
                    emit(v, col0);
            } else {
                if (!wait_full())
                    break;
                borrow();
#pragma unroll 1
                for (int c = 0; c < T::kEpiCols; c += 64) {
                    const int col0 = at.j * BN + first_col + c;
                    if (col0 >= p.cols || row0 >= p.rows)
                        break; // warp-uniform: nothing of this box lies in the matrix
                    unsigned long long v[32];
                    take(acc % T::kAccBufs, first_col + c, false, v);
                    emit(v, col0);
                }
                release();
            }
        }
        if (lane == 0)
            bulk_wait_group<0>(); // every store of this warp is done
        __syncwarp();
        if (lane == 0)
            mbar_arrive(epi_done);
    }
}

// ------------------------------------------------------------ norm and planes of G
struct Input {
    Matrix g;
    float eps;
    float4 *partial; // [batch][parts]
    int parts;
    Factors *f; // [batch][kFactors]
    int steps;
    Slow slow[kMaxSteps];
    __half *X; // planes of r x pitch, scaled by kScaleX
    int planes, write_planes, pitch;
};

constexpr int kNormThreads = 256;

// The sums of squares, one set of partial sums per CTA.
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const Input p)
{
    __shared__ float4 scratch[kNormThreads / 32];
    const int b = blockIdx.y;
    const unsigned units = static_cast<unsigned>((p.g.n + 7) / 8);
    const unsigned total = units * static_cast<unsigned>(p.g.m);
    Squares sum;
    for (unsigned u = blockIdx.x * kNormThreads + threadIdx.x; u < total; u += gridDim.x * kNormThreads) {
        const unsigned row = u / units;
        float v[8];
        load8(p.g, b * p.g.batch_pitch + row * p.g.ld, static_cast<int>(u - row * units) * 8, v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum.add(v[e]);
    }
    sum.add_up_warp();
    if (threadIdx.x % 32 == 0)
        scratch[threadIdx.x / 32] = sum.sums();
    __syncthreads();
    if (threadIdx.x == 0) {
        Squares all;
        for (int w = 0; w < kNormThreads / 32; ++w)
            all.add(scratch[w]);
        p.partial[static_cast<long long>(b) * p.parts + blockIdx.x] = all.sums();
    }
}

// X's planes from a 64 x 64 piece of G (transposed where G is tall), after
// the norm from the partial sums, and the factors of every step.
template <bool Tall>
__global__ void __launch_bounds__(kNormThreads) planes_kernel(const Input p)
{
    __shared__ float scale[3];
    __shared__ float piece[Tall ? 64 : 1][65];
    const int b = blockIdx.z;
    grid_launch_next();
    grid_wait();
    if (threadIdx.x < 32) {
        Squares sum;
        for (int k = threadIdx.x; k < p.parts; k += 32)
            sum.add(p.partial[static_cast<long long>(b) * p.parts + k]);
        sum.add_up_warp();
        if (threadIdx.x == 0) {
            int e;
            scale[2] = split_scale(sum, p.eps, &e);
            scale[0] = power_of_two(e / 2);
            scale[1] = power_of_two(e - e / 2);
        }
    }
    __syncthreads();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == kNormThreads - 1) {
        float g = scale[2];
        Factors *f = p.f + b * kFactors;
        for (int k = 0; k < p.steps; ++k)
            f[k] = step_factors(g, p.slow[k]);
        f[p.steps] = Factors{g, 1.0f}; // of the result
    }
    const float s0 = scale[0], s1 = scale[1];
    const int r = Tall ? p.g.n : p.g.m, c = Tall ? p.g.m : p.g.n;
    const int i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
    const int ty = threadIdx.x / 8, tx = threadIdx.x % 8 * 8;
    const long long first = b * p.g.batch_pitch;
    if constexpr (Tall) {
#pragma unroll
        for (int h = 0; h < 64; h += 32) {
            float v[8];
            if (j0 + ty + h < c) {
                load8(p.g, first + (j0 + ty + h) * p.g.ld, i0 + tx, v);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                piece[tx + e][ty + h] = v[e];
        }
        __syncthreads();
    }
#pragma unroll
    for (int h = 0; h < 64; h += 32) {
        const int i = i0 + ty + h;
        if (i >= r)
            break;
        float v[8];
        if constexpr (Tall) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = piece[ty + h][tx + e];
        } else {
            load8(p.g, first + i * p.g.ld, j0 + tx, v);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = v[e] * s0 * s1;
        __half *x = p.X + (static_cast<long long>(b) * p.planes * r + i) * p.pitch + j0 + tx;
        for (int q = 0; q < p.write_planes; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[e] = pack_f16(v[2 * e], v[2 * e + 1]);
                const float2 kept = unpack_f16(w[e]);
                v[2 * e] -= kept.x;
                v[2 * e + 1] -= kept.y;
            }
            *reinterpret_cast<uint4 *>(x + static_cast<long long>(q) * r * p.pitch) =
                make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ------------------------------------------------------------ host side
struct Layout {
    int r, c, rp, cp;   // sizes and 128-byte row pitches in elements
    int xp, ap;         // planes of X; full planes of A and of Q
    int parts;
    size_t partial, f, x[2], a, a_diag, q, q_diag, total;
};

Layout make_layout(int batch, int m, int n, int out_dtype, int sms)
{
    Layout l;
    l.r = std::min(m, n);
    l.c = std::max(m, n);
    l.rp = (l.r + 63) / 64 * 64;
    l.cp = (l.c + 63) / 64 * 64;
    l.xp = out_dtype == GEMM_DTYPE_F32 ? 3 : 2;
    l.ap = out_dtype == GEMM_DTYPE_F32 ? 2 : 1;
    // Enough CTAs for the norm to draw on the whole memory system, none with
    // less than a few vectors per thread.
    const long long units = (static_cast<long long>(m) * n + 8 * kNormThreads - 1) / (8 * kNormThreads);
    l.parts = static_cast<int>(std::max(1ll, std::min<long long>(units, std::max(1, 4 * sms / batch))));
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const size_t nb = static_cast<size_t>(batch);
    l.partial = take(nb * l.parts * sizeof(float4));
    l.f = take(nb * kFactors * sizeof(Factors));
    for (size_t &x : l.x)
        x = take(nb * l.xp * l.r * l.cp * 2);
    l.a = take(nb * l.ap * l.r * l.rp * 2);
    l.a_diag = take(nb * l.r * kDiagBlock * 2);
    l.q = take(nb * l.ap * l.r * l.rp * 2);
    l.q_diag = take(nb * l.r * kDiagBlock * 2);
    l.total = at;
    return l;
}

// A matrix of planes in the workspace: r rows, `pitch` elements apart.
struct Planes {
    void *base;
    int rows, cols, pitch, planes; // planes: over the whole batch
};

int encode(CUtensorMap *map, const Planes &m, uint32_t box_cols, uint32_t box_rows, int swizzle)
{
    const uint64_t pitch = static_cast<uint64_t>(m.pitch) * 2u;
    const uint64_t dims[3] = {static_cast<uint64_t>(m.cols), static_cast<uint64_t>(m.rows),
                              static_cast<uint64_t>(m.planes)};
    const uint64_t pitches[2] = {pitch, pitch * static_cast<uint64_t>(m.rows)};
    const uint32_t box[3] = {box_cols, box_rows, 1};
    return encode_tensor_map(map, kElement16, m.base, 3, dims, pitches, box, swizzle);
}

// The columns in groups of 64, `columns` of them and 64 rows a box.  The last
// group may reach past the matrix into its rows' padding; what is computed
// from that lies outside the result.
int encode_column_groups(CUtensorMap *map, const Planes &m, uint32_t columns)
{
    const uint64_t pitch = static_cast<uint64_t>(m.pitch) * 2u;
    const uint64_t dims[4] = {64, static_cast<uint64_t>(m.rows), static_cast<uint64_t>(m.pitch / 64),
                              static_cast<uint64_t>(m.planes)};
    const uint64_t pitches[3] = {pitch, 128, pitch * static_cast<uint64_t>(m.rows)};
    const uint32_t box[4] = {64, BK, columns / 64, 1};
    return encode_tensor_map(map, kElement16, m.base, 4, dims, pitches, box, 128);
}

template <int MH, int BN, int S, bool RightMN, bool Split, bool Steps = false>
int launch_product_t(const Maps &maps, const Product &p, const Device &d, cudaStream_t s)
{
    using T = Tile<MH, BN, S, Split>;
    static std::atomic<unsigned long long> limit_set[kMaxDevices];
    auto *kernel = product_kernel<MH, BN, S, RightMN, Split, Steps>;
    if (ensure_smem_limit(kernel, T::kSmem, d.index, d.ctx, limit_set) != GEMM_OK)
        return GEMM_ERR_CUDA;
    const long long tiles = static_cast<long long>(tiles_of(p.symmetric != 0, (p.rows + T::BM - 1) / T::BM,
                                                            (p.cols + BN - 1) / BN)) * p.batch;
    const unsigned grid = static_cast<unsigned>(Split ? tiles * p.ranks : std::min<long long>(tiles, d.sms));
    return launch(kernel, dim3(grid), T::kThreads, T::kSmem, true, p.ranks, s, maps, p);
}

// How a product is cut: tiles of 256 x 256, 128 x 192 (Q X only) or 128 x
// 128, the last shared by `ranks` CTAs.
struct Cut {
    int rows, cols, ranks;
};

// Clusters of `ranks` CTAs with the split kernel's shared memory that run at
// once: 76, 36 and 15 of 2, 4 and 8 on GB300, whose GPCs do not hold whole
// numbers of the larger ones.
int cluster_room(int ranks, const Device &d)
{
    static std::atomic<int> known[kMaxDevices][4];
    const int at = ranks == 2 ? 1 : ranks == 4 ? 2 : 3;
    const int have = d.index >= 0 && d.index < kMaxDevices ? known[d.index][at].load() : 0;
    if (have > 0)
        return have;
    using T = Tile<1, 128, 4, true>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(d.sms / ranks * ranks));
    cfg.blockDim = dim3(T::kThreads);
    cfg.dynamicSmemBytes = T::kSmem;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(ranks);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    auto *kernel = product_kernel<1, 128, 4, true, true>;
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    if (d.index >= 0 && d.index < kMaxDevices)
        known[d.index][at].store(n);
    return n;
}

// By the time of one round of tiles, in microseconds measured on GB300: a K
// block takes the 256 x 256 tile 0.65, the 128 x 192 tile 0.43 and the 128 x
// 128 tile 0.34 (64, 40 and 32 KiB at the 64 bytes a clock that an SM takes
// in), with an accumulator of its own the latter two 0.55 and 0.45; storing
// a tile takes about 4.5, 2 and 1.5, an exchange between ranks 1.  Ranks only
// where all tiles run at once.
Cut choose_cut(bool symmetric, int rows, int cols, int batch, int k_blocks, int fine, const Device &d)
{
    auto tiles = [&](int bm, int bn) {
        return static_cast<long long>(tiles_of(symmetric, (rows + bm - 1) / bm, (cols + bn - 1) / bn)) * batch;
    };
    auto rounds = [&](long long n) { return static_cast<double>((n + d.sms - 1) / d.sms); };
    const long long small = tiles(128, 128);
    const double block = fine != kWhole ? 0.45 : 0.34;
    Cut best{128, 128, 1};
    double least = rounds(small) * k_blocks * block + 1.5;
    auto offer = [&](const Cut &cut, double t) {
        if (t < least) {
            least = t;
            best = cut;
        }
    };
    for (int ranks = 2; ranks <= 8 && k_blocks >= 2 * ranks && small * ranks <= d.sms; ranks *= 2)
        if (small <= cluster_room(ranks, d))
            offer(Cut{128, 128, ranks}, (k_blocks + ranks - 1) / ranks * block + 2.5);
    if (!symmetric && fine != kPerStep)
        offer(Cut{128, 192, 1}, rounds(tiles(128, 192)) * k_blocks * (fine != kWhole ? 0.55 : 0.43) + 2.0);
    if (fine == kWhole) {
        const double n = rounds(tiles(256, 256));
        offer(Cut{256, 256, 1}, n * (k_blocks * 0.65 + 4.5));
    }
    return best;
}

constexpr int kSmallTileStages = 6;

template <bool RightMN>
int launch_product(const Cut &cut, const Maps &maps, Product p, const Device &d, cudaStream_t s)
{
    p.ranks = cut.ranks;
    if (p.fine == kPerStep) // 128 x 128 tiles (choose_cut)
        return cut.ranks > 1 ? launch_product_t<1, 128, 4, RightMN, true, true>(maps, p, d, s)
                             : launch_product_t<1, 128, kSmallTileStages, RightMN, false, true>(maps, p, d, s);
    if (cut.rows == 256)
        return launch_product_t<2, 256, 3, RightMN, false>(maps, p, d, s);
    if constexpr (RightMN)
        if (cut.cols == 192)
            return launch_product_t<1, 192, 4, RightMN, false>(maps, p, d, s);
    return cut.ranks > 1 ? launch_product_t<1, 128, 4, RightMN, true>(maps, p, d, s)
                         : launch_product_t<1, 128, kSmallTileStages, RightMN, false>(maps, p, d, s);
}

int run(const Call &call, const Layout &l, uint8_t *ws, const Device &d, unsigned int *status, cudaStream_t s)
{
    const bool wide_result = call.out_dtype == GEMM_DTYPE_F32;
    const bool tall = call.m > call.n;
    const int nb = call.batch;
    const Planes x[2] = {{ws + l.x[0], l.r, l.c, l.cp, nb * l.xp}, {ws + l.x[1], l.r, l.c, l.cp, nb * l.xp}};
    const Planes a{ws + l.a, l.r, l.r, l.rp, nb * l.ap}, q{ws + l.q, l.r, l.r, l.rp, nb * l.ap};
    const Planes a_diag{ws + l.a_diag, l.r, kDiagBlock, kDiagBlock, nb};
    const Planes q_diag{ws + l.q_diag, l.r, kDiagBlock, kDiagBlock, nb};
    Factors *f = reinterpret_cast<Factors *>(ws + l.f);

    // The cuts of X X^T, of the square and of Q X, for the K blocks of the
    // passes a middle step makes.
    const int fine = !wide_result ? kWhole : l.r <= kStepSide ? kPerStep : kPerBlock;
    const int kr = (l.r + BK - 1) / BK, kc = (l.c + BK - 1) / BK;
    const Cut cut_a = choose_cut(true, l.r, l.r, nb, (wide_result ? 3 : 1) * kc, fine, d);
    const Cut cut_s = choose_cut(true, l.r, l.r, nb, (wide_result ? 3 : 1) * kr + std::min(kr, 4), fine, d);
    const Cut cut_x = choose_cut(false, l.r, l.c, nb, (wide_result ? 4 : 2) * kr + std::min(kr, 2), fine, d);
    CUtensorMap x_load[2], x_columns[2], a_load, a_diag_load, q_load, q_diag_load;
    CUtensorMap to_x[2], to_a[4], to_q[4], to_out; // a and q: store, mirror, store_diag, mirror_diag
    int st = GEMM_OK;
    auto enc = [&](CUtensorMap *map, const Planes &m, uint32_t cols, uint32_t rows, int swizzle) {
        if (st == GEMM_OK)
            st = encode(map, m, cols, rows, swizzle);
    };
    for (int i = 0; i < 2; ++i) {
        enc(&x_load[i], x[i], BK, cut_a.rows, 128);
        if (st == GEMM_OK)
            st = encode_column_groups(&x_columns[i], x[i], cut_x.cols);
        enc(&to_x[i], x[i], 64, 32, 128);
    }
    enc(&a_load, a, BK, cut_s.rows, 128);
    enc(&a_diag_load, a_diag, BK, cut_s.rows, 128);
    enc(&q_load, q, BK, cut_x.rows, 128);
    enc(&q_diag_load, q_diag, BK, cut_x.rows, 128);
    auto stores = [&](CUtensorMap *to, const Planes &m, const Planes &m_diag) {
        enc(&to[0], m, 64, 32, 128);
        enc(&to[1], m, 32, 64, 64);
        enc(&to[2], m_diag, 64, 32, 128);
        enc(&to[3], m_diag, 32, 64, 64);
    };
    stores(to_a, a, a_diag);
    stores(to_q, q, q_diag);
    if (st != GEMM_OK)
        return st;
    auto set_stores = [](Maps &maps, const CUtensorMap *to) {
        maps.store = to[0];
        maps.mirror = to[1];
        maps.store_diag = to[2];
        maps.mirror_diag = to[3];
    };
    Maps maps;
    std::memset(&maps, 0, sizeof maps);
    const uint64_t es = wide_result ? 4 : 2;
    const bool out_tma = (reinterpret_cast<uintptr_t>(call.out) & 15u) == 0 && (call.ldo * es) % 16 == 0 &&
                         (nb == 1 || (call.o_batch * es) % 16 == 0);
    std::memset(&to_out, 0, sizeof to_out);
    if (out_tma) {
        const uint64_t dims[3] = {static_cast<uint64_t>(call.n), static_cast<uint64_t>(call.m),
                                  static_cast<uint64_t>(nb)};
        const uint64_t pitches[2] = {call.ldo * es,
                                     nb == 1 ? call.ldo * es * static_cast<uint64_t>(call.m) : call.o_batch * es};
        const uint32_t box[3] = {wide_result || tall ? 32u : 64u, tall && !wide_result ? 64u : 32u, 1};
        st = encode_tensor_map(&to_out, wide_result ? kElement32 : kElement16, call.out, 3, dims, pitches, box,
                               !tall ? 128 : wide_result ? 0 : 64);
        if (st != GEMM_OK)
            return st;
    }

    // Norm and the first iterate.  A bfloat16 G is exact in one plane.
    const bool exact_input = call.dtype == GEMM_DTYPE_BF16;
    Input in{call.matrix(), call.eps, reinterpret_cast<float4 *>(ws + l.partial), l.parts, f, call.steps, {},
             static_cast<__half *>(x[0].base), l.xp, exact_input ? 1 : l.xp, l.cp};
    for (int k = 0; k < call.steps; ++k)
        in.slow[k] = slow_step(call.coefficients + 3 * k);
    st = launch(norm_kernel, dim3(l.parts, nb), kNormThreads, 0, false, 1, s, in);
    if (st != GEMM_OK)
        return st;
    const dim3 pieces((l.c + 63) / 64, (l.r + 63) / 64, nb);
    st = tall ? launch(planes_kernel<true>, pieces, kNormThreads, 0, true, 1, s, in)
              : launch(planes_kernel<false>, pieces, kNormThreads, 0, true, 1, s, in);
    if (st != GEMM_OK)
        return st;

    Product base = {};
    base.batch = nb;
    base.status = status;
    base.wait_limit_ns = call_wait_limit_ns();
    base.withhold = call_withhold();
    base.fine = fine;
    for (int step = 0; step < call.steps; ++step) {
        const float ca = call.coefficients[3 * step], cb = call.coefficients[3 * step + 1],
                    cc = call.coefficients[3 * step + 2];
        const bool first = step == 0, last = step == call.steps - 1;
        const bool one_plane = first && exact_input; // X has no more than that
        const int cur = step & 1;
        base.f = f + step;
        auto add = [](Product &p, int left, int right, Range range) {
            p.pass[p.passes++] = Pass{static_cast<signed char>(left), static_cast<signed char>(right),
                                      static_cast<signed char>(range)};
        };

        // X X^T: to A + (b / 2c) I, or with c = 0 to Q itself.
        Product p = base;
        p.rows = p.cols = l.r;
        p.k = l.c;
        p.symmetric = 1;
        p.left_planes = p.right_planes = l.xp;
        if (wide_result && !one_plane) {
            add(p, 0, 1, kAll);
            add(p, 1, 0, kAll);
        }
        add(p, 0, 0, kAll);
        p.output = kPlanes;
        p.planes = p.planes_pitch = l.ap;
        p.diag_plane = 1;
        if (cc != 0.0f) {
            p.alpha = kScaleA / (kScaleX * kScaleX);
            p.diag = kScaleA * (cb / (2.0f * cc));
            p.alpha_g = 2;
        } else {
            p.alpha = kScaleQ * cb / (kScaleX * kScaleX);
            p.diag = kScaleQ * ca;
            p.alpha_g = 2;
            p.alpha_rho = p.diag_rho = 1;
        }
        maps.left = maps.right = x_load[cur];
        set_stores(maps, cc != 0.0f ? to_a : to_q);
        st = launch_product<false>(cut_a, maps, p, d, s);
        if (st != GEMM_OK)
            return st;

        if (cc != 0.0f) {
            // The square, to Q.
            p = base;
            p.rows = p.cols = p.k = l.r;
            p.symmetric = 1;
            p.left_planes = p.right_planes = l.ap;
            add(p, 0, -1, kCols);
            add(p, -1, 0, kRows);
            if (wide_result) {
                add(p, 0, 1, kAll);
                add(p, 1, 0, kAll);
            }
            add(p, 0, 0, kAll);
            p.output = kPlanes;
            p.planes = p.planes_pitch = l.ap;
            p.diag_plane = 1;
            p.alpha = kScaleQ * cc / (kScaleA * kScaleA);
            p.diag = kScaleQ * static_cast<float>(ca - static_cast<double>(cb) * cb / (4.0 * cc));
            p.alpha_rho = p.diag_rho = 1;
            maps.left = maps.right = a_load;
            maps.left_diag = maps.right_diag = a_diag_load;
            set_stores(maps, to_q);
            st = launch_product<false>(cut_s, maps, p, d, s);
            if (st != GEMM_OK)
                return st;
        }

        // Q X: to the next X, or to the result.
        p = base;
        p.rows = p.k = l.r;
        p.cols = l.c;
        p.left_planes = l.ap;
        p.right_planes = l.xp;
        add(p, -1, 0, kRows);
        if (wide_result) {
            if (!one_plane) {
                if (!last)
                    add(p, 0, 2, kAll);
                add(p, 0, 1, kAll);
            }
            add(p, 1, 0, kAll);
        } else if (!one_plane && !last) {
            add(p, 0, 1, kAll);
        }
        add(p, 0, 0, kAll);
        maps.left = q_load;
        maps.left_diag = q_diag_load;
        maps.right = x_columns[cur];
        maps.store = last ? to_out : to_x[1 - cur];
        if (last) {
            p.output = wide_result ? kF32 : kBf16;
            p.alpha = 1.0f / (kScaleQ * kScaleX);
            p.f = f + call.steps;
            p.alpha_g = 1;
            p.transposed = tall;
            p.out_tma = out_tma;
            p.out = call.out;
            p.ldo = call.ldo;
            p.out_batch = call.o_batch;
        } else {
            p.output = kPlanes;
            // The last step reads one plane less.
            p.planes = step == call.steps - 2 ? l.xp - 1 : l.xp;
            p.planes_pitch = l.xp;
            p.alpha = 1.0f / kScaleQ;
        }
        st = launch_product<true>(cut_x, maps, p, d, s);
        if (st != GEMM_OK)
            return st;
    }
    return GEMM_OK;
}

// Whether the iteration stays where the planes can hold it: with singular
// values x in [0, top] before a step, top 1 at first, and q = a + b x x + c x^4,
// Q is at most 15.5 (31 with g below 2), A + (b / 2c) I at most 7.98, and x q,
// what the step leaves, at most 2.8, which a next A holds; all under 65504 at
// their scales, with room for rounding.  The largest values are at the ends
// and where the derivatives vanish.
int check_coefficients(const float *coefficients, int steps)
{
    double top = 1.0;
    for (int k = 0; k < steps; ++k) {
        const double a = coefficients[3 * k], b = coefficients[3 * k + 1], c = coefficients[3 * k + 2];
        if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c))
            return GEMM_ERR_INVALID_ARG;
        if (c != 0.0 && std::fabs(b) > 8.0 * std::fabs(c))
            return GEMM_ERR_UNSUPPORTED; // completing the square would cancel
        const double end = top * top;
        double most = 0.0, next = 0.0; // of |q| and |x q|
        auto at = [&](double y) {
            if (y >= 0.0 && y <= end) {
                const double q = std::fabs(a + b * y + c * y * y);
                most = std::max(most, q);
                next = std::max(next, std::sqrt(y) * q);
            }
        };
        at(0.0);
        at(end);
        if (c != 0.0) {
            at(-b / (2.0 * c)); // q'
            const double d = 9.0 * b * b - 20.0 * a * c; // (x q)' = a + 3 b y + 5 c y y
            if (d >= 0.0) {
                at((-3.0 * b + std::sqrt(d)) / (10.0 * c));
                at((-3.0 * b - std::sqrt(d)) / (10.0 * c));
            }
        } else if (b != 0.0) {
            at(-a / (3.0 * b));
        }
        const double shift = c != 0.0 ? b / (2.0 * c) : 0.0;
        if (most > 15.5 || next > 2.8 || std::max(std::fabs(shift), std::fabs(end + shift)) > 7.98)
            return GEMM_ERR_UNSUPPORTED;
        top = next;
    }
    return GEMM_OK;
}

bool valid_dtype(int d) { return d == GEMM_DTYPE_F32 || d == GEMM_DTYPE_BF16; }

constexpr int kMaxSide = 1 << 20;
constexpr long long kMaxElements = 0x7fffffffll;
constexpr int kMaxBatch = 65535;

int check_sizes(int batch, int m, int n)
{
    if (batch < 0 || m < 0 || n < 0)
        return GEMM_ERR_INVALID_ARG;
    if (batch > kMaxBatch || m > kMaxSide || n > kMaxSide || static_cast<long long>(m) * n > kMaxElements)
        return GEMM_ERR_UNSUPPORTED;
    // Tiles of the whole batch are counted in an int.
    const long long tiles = (static_cast<long long>(m) + 127) / 128 * ((n + 127) / 128) * batch;
    return tiles > 0x3fffffffll ? GEMM_ERR_UNSUPPORTED : GEMM_OK;
}

} // namespace orth

} // namespace pg

using namespace pg;

extern "C" {

int orthogonalize_workspace(int batch, int m, int n, int out_dtype, size_t *bytes)
{
    if (!bytes || !orth::valid_dtype(out_dtype))
        return GEMM_ERR_INVALID_ARG;
    const int st = orth::check_sizes(batch, m, n);
    if (st != GEMM_OK)
        return st;
    const bool none = batch == 0 || m == 0 || n == 0 || orth::fits_small(m, n, out_dtype);
    *bytes = none ? 0 : orth::make_layout(batch, m, n, out_dtype, device_sms()).total;
    return GEMM_OK;
}

int orthogonalize(int batch, int m, int n, const void *G, long long ldg, long long g_batch, int dtype, void *out,
                  long long ldo, long long o_batch, int out_dtype, int steps, const float *coefficients, float eps,
                  void *workspace, size_t workspace_bytes, void *stream)
{
    if (!orth::valid_dtype(dtype) || !orth::valid_dtype(out_dtype) || steps < 1 || steps > orth::kMaxSteps ||
        !coefficients || !(eps >= 0.0f) || !std::isfinite(eps))
        return GEMM_ERR_INVALID_ARG;
    int st = orth::check_sizes(batch, m, n);
    if (st != GEMM_OK)
        return st;
    st = orth::check_coefficients(coefficients, steps);
    if (st != GEMM_OK)
        return st;
    const bool empty = batch == 0 || m == 0 || n == 0;
    if (!empty) {
        if (ldg < n || ldo < n || !G || !out)
            return GEMM_ERR_INVALID_ARG;
        // One matrix of out after the other, or row by row in turn.
        if (batch > 1 && (g_batch < 0 || (o_batch < ldo * (m - 1) + n &&
                                          (o_batch < n || ldo < o_batch * (batch - 1) + n))))
            return GEMM_ERR_INVALID_ARG;
        const uintptr_t ga = dtype == GEMM_DTYPE_F32 ? 3u : 1u, oa = out_dtype == GEMM_DTYPE_F32 ? 3u : 1u;
        if ((reinterpret_cast<uintptr_t>(G) & ga) != 0 || (reinterpret_cast<uintptr_t>(out) & oa) != 0 ||
            (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
            return GEMM_ERR_MISALIGNED;
    }
    int dev;
    st = device_checked(&dev);
    if (st != GEMM_OK)
        return st;
    if (empty)
        return GEMM_OK;
    const orth::Device d{dev, device_sms(), current_context_id()};
    unsigned int *status = device_status_word(dev, d.ctx);
    if (!status)
        return GEMM_ERR_CUDA;
    const orth::Call call{batch, m, n, G, ldg, g_batch, dtype, out, ldo, o_batch, out_dtype, steps, coefficients, eps};
    if (orth::fits_small(m, n, out_dtype))
        return orth::run_small(call, d, status, static_cast<cudaStream_t>(stream));
    const orth::Layout l = orth::make_layout(batch, m, n, out_dtype, d.sms);
    if (!workspace || workspace_bytes < l.total)
        return GEMM_ERR_INVALID_ARG;
    return orth::run(call, l, static_cast<uint8_t *>(workspace), d, status, static_cast<cudaStream_t>(stream));
}

} // extern "C"
