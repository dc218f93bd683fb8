// Products on the tensor cores by pairs of CTAs, the loop that the gated
// projection, its gradient and the 8-bit product share.
//
// A pair (a cluster of two CTAs, on neighbouring SMs) computes 256 x 256 tiles:
// each CTA loads its own 128 rows of A and 128 of B's 256 columns, and rank 0
// issues MMAs of 256 x 256 that read both CTAs' shared memory.  A CTA then
// moves 32 KiB into shared memory per 128-byte K block for 128 x 256 results,
// where a CTA by itself moves 48 KiB (the fill and the tensor core share the
// shared memory's bandwidth), and its accumulator of 128 x 256 takes half of
// tensor memory: the epilogue of one accumulator overlaps the MMAs of the next.
//
//   warps 0, 2   TMA producers of its CTA's A and B: a ring of kStages stages,
//                16 KiB of each.  Both CTAs' copies complete on rank 0's full
//                barrier; the stage is released on both sides by a multicast
//                tcgen05.commit.
//   warp 1       allocates tensor memory; on rank 0 issues the MMAs.
//   warps 4-11   epilogue: warp w reads tensor-memory lanes 32 (w % 4) .. +31
//                (its CTA's rows), columns 0-127 (warps 4-7) or 128-255 (8-11).
//
// Operands lie in shared memory as 128-byte rows, 128-byte swizzled:
//   K-major   one box of 128 rows (m or n) x 128 bytes of k; 8-row groups 1024
//             bytes apart; an MMA's K step (32 bytes) advances 32 bytes.
//   MN-major  boxes of 128 bytes of m or n; rows are k: for 2-byte elements two
//             boxes of 64 k each, 8 KiB apart (one copy brings both where the
//             matrix is whole columns of 64 wide: as a third dimension, in which
//             TMA would not stop at another width); for 1-byte elements one box
//             of 128 k; 8-k groups 1024 bytes apart; a K step advances 16 rows
//             (2048 bytes) or 32 (4096).
// So a matrix serves as it lies in memory, row-major or transposed, on either
// side of the product.  TMA fills what lies outside a matrix with zeros, which
// add nothing; results outside are not stored.
#pragma once

#include <cstdint>

#include "gemm_internal.h"
#include "ptx.cuh"
#include "tma_ring.cuh"
#include "vector_io.cuh"

namespace pg {
namespace pair_product {

constexpr int kRows = 256;       // of a pair's tile
constexpr int kCols = 256;
constexpr int kStages = 6;
constexpr uint32_t kOperandBytes = 128 * 128; // a CTA's part of A or B in a stage
constexpr uint32_t kStageBytes = 2 * kOperandBytes;
constexpr int kEpilogueWarps = 8;
constexpr int kFirstEpilogueWarp = 4;
constexpr int kThreads = (kFirstEpilogueWarp + kEpilogueWarps) * 32;
constexpr uint32_t kTmemCols = 512; // two 128 x 256 accumulators
constexpr int kGroupTiles = 16;     // rows of tiles per raster group
constexpr int kBarrierBytes = 16 * kStages + 64;
constexpr int kMaxMaps = 7;
constexpr int kMaxProducts = 2;

constexpr int smem_bytes(int extra) { return static_cast<int>(kStages * kStageBytes) + kBarrierBytes + extra + 1024; }

struct Maps {
    CUtensorMap map[kMaxMaps];
};

// How an operand is stored: with k contiguous, or with m (n) contiguous, in the
// latter case of 2-byte elements perhaps in whole columns of 64.
enum Layout : int { kAlongK, kAcrossRagged, kAcross };

// One product of a launch.  Its K blocks come in one or two segments (a sum of
// two products); with `dual` one A meets two Bs, the tile's halves of 128
// columns belonging to one of two results each.
struct Product {
    int rows, cols;   // of the result (dual: of each)
    int tiles_m, tiles_n;
    int blocks;       // K blocks of a segment
    int segments;
    int splits;       // pieces that a tile's K blocks are cut into, each a pair's work
    int dual;
    Layout a_layout, b_layout;
    int a_map, b_map; // first of one (a dual B or two segments: two) maps
    uint32_t idesc;
    int tiles() const { return tiles_m * tiles_n; }
    int units() const { return tiles() * splits; }
};

struct Launch {
    Product product[kMaxProducts];
    int first_units, units; // pieces of work of product 0, of all
    int maps;               // in use
    unsigned int family;    // of the status word's codes
    unsigned int *status;
    unsigned long long wait_limit_ns;
    int withhold;
};

// Instruction descriptor: float32 accumulators (bits 4-5 = 1), formats of A
// and B (bits 7-9, 10-12), MN-major A and B (bits 15, 16), N >> 3 at bits
// 17-22, M >> 4 at bits 24-28.
constexpr uint32_t instruction(uint32_t a_format, uint32_t b_format, Layout a, Layout b)
{
    return (1u << 4) | (a_format << 7) | (b_format << 10) | (a != kAlongK ? 1u << 15 : 0u) |
           (b != kAlongK ? 1u << 16 : 0u) | (static_cast<uint32_t>(kCols >> 3) << 17) |
           (static_cast<uint32_t>(kRows >> 4) << 24);
}

struct Tile {
    int mb, nb;
};

// Unit u of a launch: a product's tile, and the K blocks (of all its segments)
// that are summed there.
struct Unit {
    int which, tile, split, first, count;
};

__device__ __forceinline__ Unit unit_at(const Launch &l, int u)
{
    Unit w;
    w.which = u < l.first_units ? 0 : 1;
    const Product &p = l.product[w.which];
    const int at = w.which ? u - l.first_units : u;
    const int blocks = p.blocks * p.segments;
    if (p.splits == 1) {
        w.tile = at;
        w.split = w.first = 0;
        w.count = blocks;
    } else {
        w.tile = at / p.splits;
        w.split = at - w.tile * p.splits;
        w.first = static_cast<int>(static_cast<long long>(blocks) * w.split / p.splits);
        w.count = static_cast<int>(static_cast<long long>(blocks) * (w.split + 1) / p.splits) - w.first;
    }
    return w;
}

// Tile t of a product: groups of kGroupTiles rows of tiles, within one down
// the rows first, so that the tiles at work share rows of A and columns of B
// in L2.
__device__ __forceinline__ Tile tile_at(const Product &p, int t)
{
    const int per_group = kGroupTiles * p.tiles_n;
    const int group = t / per_group;
    const int first = group * kGroupTiles;
    const int height = min(kGroupTiles, p.tiles_m - first);
    const int r = t - group * per_group;
    return Tile{first + r % height, r / height};
}

// Barriers of a CTA, at the same offsets in both.
struct Barriers {
    TmaRing<kStages> ring;
    uint32_t acc_full, acc_empty; // [2] each
    uint32_t mma_done, tmem_slot;

    __device__ __forceinline__ explicit Barriers(uint32_t at)
        : ring{at, at + 8u * kStages}, acc_full(at + 16u * kStages), acc_empty(acc_full + 16u),
          mma_done(acc_empty + 16u), tmem_slot(mma_done + 8u)
    {
    }
};

template <MmaKind Kind>
struct Element {
    static constexpr int kBlockK = Kind == kMmaF16 ? 64 : 128;       // elements of 128 bytes
    static constexpr uint32_t kMnStep = Kind == kMmaF16 ? 2048 : 4096; // bytes of an MN-major K step
};

// A producer warp of a CTA, of A or of B: each operand has one, as a warp takes
// about 90 cycles to issue a copy and 170 for a stage's waits and announcement,
// and a block's MMAs take 512.  All of the warp runs the loop and one lane
// issues: with a branch on the lane around the loop the copies' operands are
// moved to uniform registers one by one, which took longer than a block's MMAs
// (8192 x 4096 by two 4096 x 8192: 741 us, like this 595).
//
// A lane whose wait has run out leaves the loops alone, so nothing in them may need
// all lanes: what counts is the one that issues, and each comes to the loops' end by
// its own waits.
template <MmaKind Kind, bool IsB>
__device__ __forceinline__ void produce(const Launch &l, const Maps &maps, const Barriers &b, uint32_t base, int rank,
                                        uint32_t leader, int first, int stride)
{
    constexpr int BK = Element<Kind>::kBlockK;
    const uint32_t on = threadIdx.x % 32 == 0;
    if (on && !IsB)
        for (int i = 0; i < l.maps; ++i)
            tma_prefetch_map(&maps.map[i]);
    unsigned f = 0;
    bool ok = true;
    for (int t = first; t < l.units && ok; t += stride) {
        const Unit unit = unit_at(l, t);
        const Product &p = l.product[unit.which];
        const Tile tile = tile_at(p, unit.tile);
        // This CTA's 128 rows (columns).
        const int at = !IsB     ? tile.mb * kRows + rank * 128
                       : p.dual ? tile.nb * 128
                                : tile.nb * kCols + rank * 128;
        const Layout layout = IsB ? p.b_layout : p.a_layout;
        int left = unit.count;
        for (int seg = unit.first >= p.blocks ? 1 : 0, begin = unit.first - seg * p.blocks; left > 0 && ok;
             ++seg, begin = 0) {
            const CUtensorMap *map = &maps.map[IsB ? p.b_map + (p.dual ? rank : seg) : p.a_map + seg];
            const int end = min(p.blocks, begin + left);
            left -= end - begin;
            for (int kb = begin; kb < end; ++kb, ++f) {
                if (static_cast<int>(f) == l.withhold)
                    continue; // test hook: this position is never filled
                if (!b.ring.producer_acquire(f, l.wait_limit_ns)) {
                    if (on)
                        record_error(l.status, l.family | kErrRoleProducer);
                    ok = false;
                    break;
                }
                const uint32_t to = base + (f % kStages) * kStageBytes + (IsB ? kOperandBytes : 0u);
                const uint32_t full = map_to_cta(b.ring.full_bar(f), leader);
                mbar_arrive_expect_tx_if(on && rank == 0, b.ring.full_bar(f), 2 * kOperandBytes); // both CTAs' bytes
                const int k = kb * BK;
                if (layout == kAlongK) {
                    tma_load_2d_pair_if(on, to, map, full, k, at);
                } else if (Kind == kMmaF8) {
                    tma_load_2d_pair_if(on, to, map, full, at, k);
                } else if (layout == kAcross) {
                    tma_load_3d_pair_if(on, to, map, full, 0, k, at / 64);
                } else {
                    tma_load_2d_pair_if(on, to, map, full, at, k);
                    tma_load_2d_pair_if(on, to + kOperandBytes / 2, map, full, at + 64, k);
                }
            }
        }
    }
    if (rank == 0) {
        // Only the last kStages positions can still be in flight, this CTA's
        // and the other's; each is waited for, with its own bound.
        bool drained = true;
        for (unsigned g = f > kStages ? f - kStages : 0; g < f; ++g)
            if (static_cast<int>(g) != l.withhold && !b.ring.consumer_wait(g, l.wait_limit_ns))
                drained = false;
        if (!drained && ok && on)
            record_error(l.status, l.family | kErrRoleDrain);
    }
    if (!ok) {
        // Rank 1 cannot wait on rank 0's barriers, and a barrier that one
        // operand's producer gave up on stays open: after an expired wait the
        // last copies get a millisecond to land.
        const uint64_t t0 = global_timer_ns();
        for (uint32_t poll = 0; poll < kMaxPolls && global_timer_ns() - t0 < 1000000u; ++poll)
            ;
    }
}

// The MMA warp of rank 0.  PerBlock: every K block has an accumulator of its
// own, which the epilogue scales and adds up; otherwise every tile has.
//
// Lanes leave the loops as the producers' do.  (A vote between the waits and the MMAs:
// 8192 cubed in 8 bits 389 -> 412 us, a ballot 401, one vote a tile 395.)
template <MmaKind Kind, bool PerBlock>
__device__ __forceinline__ void multiply(const Launch &l, const Barriers &b, uint32_t base, uint32_t tmem,
                                         uint32_t leader, int first, int stride)
{
    const uint32_t on = threadIdx.x % 32 == 0;
    unsigned f = 0, acc = 0;
    bool ok = true;
    for (int t = first; t < l.units && ok; t += stride) {
        const Unit unit = unit_at(l, t);
        const Product &p = l.product[unit.which];
        const int blocks = unit.count;
        const uint32_t idesc = p.idesc;
        const bool a_along = p.a_layout == kAlongK, b_along = p.b_layout == kAlongK;
        const uint32_t a_step = (a_along ? 32u : Element<Kind>::kMnStep) >> 4;
        const uint32_t b_step = (b_along ? 32u : Element<Kind>::kMnStep) >> 4;
        const uint64_t a0 = smem_desc_sw128(base, a_along ? 16 : 8192, 1024);
        const uint64_t b0 = smem_desc_sw128(base + kOperandBytes, b_along ? 16 : 8192, 1024);
        for (int kb = 0; kb < blocks; ++kb, ++f) {
            // The stage first: it is there while the accumulator is waited for.
            if (!b.ring.consumer_wait(f, l.wait_limit_ns) ||
                ((PerBlock || kb == 0) &&
                 !mbar_wait_bounded(b.acc_empty + 8u * (acc & 1u), ((acc >> 1) & 1u) ^ 1u, l.wait_limit_ns))) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            const uint32_t d = tmem + (acc & 1u) * kCols;
            const uint32_t stage = (f % kStages) * (kStageBytes >> 4);
#pragma unroll
            for (uint32_t ks = 0; ks < 4; ++ks)
                mma_pair_if<Kind>(on, d, a0 + stage + ks * a_step, b0 + stage + ks * b_step, idesc,
                                  (!PerBlock && kb != 0) || ks != 0);
            mma_commit_pair_if(on, b.ring.empty_bar(f), leader);
            if (PerBlock || kb == blocks - 1) {
                mma_commit_pair_if(on, b.acc_full + 8u * (acc & 1u), leader);
                ++acc;
            }
        }
    }
    if (!ok && on)
        record_error(l.status, l.family | kErrRoleMma);
    // Every MMA issued must finish before tensor memory is freed.
    mma_commit_pair_if(on, b.mma_done, leader);
    if (!mbar_wait_bounded(b.mma_done, 0, l.wait_limit_ns) && on)
        record_error(l.status, l.family | kErrRoleDrain);
}

// Sets up the CTA, runs the roles (`helper` in warp 3, `epilogue` in warps 4-11,
// given the tensor
// memory's address) and takes everything down.
// OtherRegisters: what the other four warps keep where the epilogue takes more
// registers than the launch gave it (0: it does not).
// Joins: the launch's clusters are of one or more pairs, which share a tile's K
// blocks (product 0's `splits`; each pair has one unit).  The epilogue then calls
// cluster_sync twice: when the ring is free, and when sums have been left there.
template <MmaKind Kind, bool PerBlock, int OtherRegisters, bool Joins, class Epilogue, class Helper>
__device__ __forceinline__ void run(const Launch &l, const Maps &maps, uint32_t base, const Barriers &b,
                                    Epilogue epilogue, Helper helper)
{
    const int warp = threadIdx.x / 32;
    const uint32_t cta = cluster_cta_rank(), leader = Joins ? cta & ~1u : 0u;
    const int rank = static_cast<int>(cta - leader);
    if (threadIdx.x == 0) {
        b.ring.init(1, 2); // full: announced by both producers
        for (int k = 0; k < 2; ++k) {
            mbar_init(b.acc_full + 8u * k, 1);
            mbar_init(b.acc_empty + 8u * k, 2 * kEpilogueWarps);
        }
        mbar_init(b.mma_done, 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(b.tmem_slot, kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    cluster_sync();
    tc_fence_after_sync();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(tmem) : "r"(b.tmem_slot) : "memory");

    grid_wait(); // for the kernel before, where this one may start ahead of its end
    const int first = static_cast<int>(blockIdx.x) / 2, stride = static_cast<int>(gridDim.x) / 2;
    if constexpr (OtherRegisters > 0)
        if (warp < kFirstEpilogueWarp)
            fewer_registers<OtherRegisters>();
    if (warp == 0) {
        produce<Kind, false>(l, maps, b, base, rank, leader, first, stride);
    } else if (warp == 2) {
        produce<Kind, true>(l, maps, b, base, rank, leader, first, stride);
    } else if (warp == 1) {
        if (rank == 0)
            multiply<Kind, PerBlock>(l, b, base, tmem, leader, first, stride);
    } else if (warp == 3) {
        helper(rank, first, stride);
    } else {
        epilogue(tmem, rank, first, stride);
    }
    if (Joins && warp < kFirstEpilogueWarp) {
        cluster_sync();
        cluster_sync();
    }
    // Neither CTA leaves, or frees tensor memory, before the other's copies,
    // MMAs and arrivals are done.
    tc_fence_before_sync();
    cluster_sync();
    tc_fence_after_sync();
    if (warp == 1)
        tmem_dealloc_pair(tmem, kTmemCols);
}

// Epilogue warps: wait for accumulator `acc` (warp-uniform result), and hand it
// back to rank 0's MMA warp.  `others`: whether what goes with it has come, as the
// lane found.  One vote for both, in which a lane whose other wait has run out takes
// part at once (with two votes the 8-bit product of 4096 x 4096 x 8192 by columns
// took 187 us, with both waits by every lane 176, like this 173).
__device__ __forceinline__ bool acquire(const Launch &l, const Barriers &b, unsigned acc, bool others = true)
{
    const bool ok = others && mbar_wait_bounded(b.acc_full + 8u * (acc & 1u), (acc >> 1) & 1u, l.wait_limit_ns);
    if (!__all_sync(0xffffffffu, ok)) {
        if (threadIdx.x % 32 == 0)
            record_error(l.status, l.family | kErrRoleEpilogue);
        return false;
    }
    tc_fence_after_sync();
    return true;
}

__device__ __forceinline__ void release(uint32_t acc_empty_of_rank0, unsigned acc)
{
    tc_fence_before_sync();
    __syncwarp();
    if (threadIdx.x % 32 == 0)
        mbar_arrive_cluster(acc_empty_of_rank0 + 8u * (acc & 1u));
}

// ------------------------------------------------------------------ stores
// How a result's rows may be written: 32, 16 or single elements' bytes at once.
enum Access : int { kByElement = 0, kBy16 = 16, kBy32 = 32 };

__device__ __forceinline__ void store_32_bytes(void *to, const uint32_t *v)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(to), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Lane i's v[j] becomes lane j's v[i].
__device__ __forceinline__ void transpose(float (&v)[32])
{
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const bool upper = (lane & o) != 0;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if ((j & o) == 0) {
                const float got = __shfl_xor_sync(0xffffffffu, upper ? v[j] : v[j + o], o);
                if (upper)
                    v[j] = got;
                else
                    v[j + o] = got;
            }
    }
}

// The `Units` times 8 words of v as unit j takes what (j + by) % Units had.
template <int Units>
__device__ __forceinline__ void rotate_units(uint32_t (&v)[Units * 8], int by)
{
#pragma unroll
    for (int o = 1; o < Units; o *= 2) {
        uint32_t w[Units * 8];
#pragma unroll
        for (int j = 0; j < Units * 8; ++j)
            w[j] = (by & o) ? v[(j + o * 8) % (Units * 8)] : v[j];
#pragma unroll
        for (int j = 0; j < Units * 8; ++j)
            v[j] = w[j];
    }
}

// The first `left` bytes of v, less than all, as parts of a power of two each:
// `to` is as aligned as `access` says.
template <int Words>
__device__ __forceinline__ void store_rest(uint8_t *to, uint32_t (&v)[Words], int left, int access)
{
#pragma unroll
    for (int part = Words / 2; part >= 1; part /= 2) {
        if (!(left & (part * 4)))
            continue;
        if (part >= 8 && access == kBy32) {
#pragma unroll
            for (int k = 0; k < part; k += 8)
                store_32_bytes(to + k * 4, v + k);
        } else if (part >= 4) {
#pragma unroll
            for (int k = 0; k < part; k += 4)
                *reinterpret_cast<uint4 *>(to + k * 4) = make_uint4(v[k], v[k + 1], v[k + 2], v[k + 3]);
        } else if (part == 2) {
            *reinterpret_cast<uint2 *>(to) = make_uint2(v[0], v[1]);
        } else {
            *reinterpret_cast<uint32_t *>(to) = v[0];
        }
        to += part * 4;
#pragma unroll
        for (int k = 0; k < part; ++k)
            v[k] = v[k + part];
    }
    if (left & 2)
        *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(v[0]);
}

// A warp's 32 x 32 elements, lane i having those of row `row0 + i` from column
// `col` on, to a rows x cols matrix.  A lane writes whole 32-byte sectors of its
// row wherever the rows are aligned, which needs no staging through shared
// memory, and of the last columns parts of 64, 32, ... bytes (transposed, as rows
// that are not aligned: 3354 x 128 -> 212 with G and U kept 11.1 us, like this
// 9.1; 200 x 64 x 100 in 8 bits 6.9 and 5.7).
//
// Rows a multiple of 64 or 128 bytes apart have their sectors at the same places of
// their lines, so that a store of all lanes would meet in half or a quarter of the
// memory's banks: lanes start at different sectors (8 bits, 6606 x 143 x 896 to
// float32: 14.8 -> 12.7 us; 4096 x 8192 x 4096: 173 -> 169; bfloat16 8192 cubed:
// 394 -> 390).
//
// Rows that are not aligned are transposed first, so that the warp writes a row at
// a time (by element from each lane, every store would touch 32 sectors: 397 x 256
// x 373 in 8 bits to such rows took 37 us, like this 12).
template <class T>
__device__ __forceinline__ void store_tile(T *to, long long ld, long long row0, int rows, int col, int cols,
                                           float (&v)[32], int access)
{
    const int lane = threadIdx.x % 32;
    if (access != kByElement) {
        if (row0 + lane >= rows)
            return;
        T *const at = to + (row0 + lane) * ld + col;
        constexpr int kWords = 32 * sizeof(T) / 4;
        uint32_t w[kWords];
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int j = 0; j < kWords; ++j) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t *>(&h);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kWords; ++j)
                w[j] = __float_as_uint(v[j]);
        }
        if (cols - col < 32) {
            store_rest(reinterpret_cast<uint8_t *>(at), w, (cols - col) * static_cast<int>(sizeof(T)), access);
        } else if (access == kBy32) {
            constexpr int kUnits = kWords / 8;
            const int step = static_cast<int>(ld * static_cast<int>(sizeof(T)) / 32) & 3;
            const int by = (step & 1) ? 0 : (step == 0 ? lane : lane >> 1 & 1) & (kUnits - 1);
            rotate_units<kUnits>(w, by);
#pragma unroll
            for (int j = 0; j < kUnits; ++j)
                store_32_bytes(reinterpret_cast<uint32_t *>(at) + ((j + by) & (kUnits - 1)) * 8, w + j * 8);
        } else {
#pragma unroll
            for (int j = 0; j < kWords; j += 4)
                *reinterpret_cast<uint4 *>(reinterpret_cast<uint32_t *>(at) + j) =
                    make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
        }
        return;
    }
    __syncwarp();
    transpose(v);
    if (col + lane < cols) {
        T *const at = to + row0 * ld + col + lane;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (row0 + i < rows)
                at[i * ld] = from_f32<T>(v[i]);
    }
}

inline int row_access(const void *p, long long pitch, int rows, size_t size)
{
    const uintptr_t low = reinterpret_cast<uintptr_t>(p) | (rows > 1 ? static_cast<uintptr_t>(pitch) * size : 0);
    return (low & 31u) == 0 ? kBy32 : (low & 15u) == 0 ? kBy16 : kByElement;
}

// ------------------------------------------------------------------- host
// Layout of a matrix of `cols` columns that are not along k.
inline Layout across(MmaKind kind, int cols) { return kind == kMmaF16 && cols % 64 == 0 ? kAcross : kAcrossRagged; }

// Tensor map of an operand: `matrix` rows x cols row-major.
int encode_operand(CUtensorMap *map, MmaKind kind, const void *matrix, int rows, int cols, long long pitch,
                   Layout layout);

} // namespace pair_product
} // namespace pg
