// The product of two matrices of 8-bit floating point numbers with a scale for
// every 128 of them along the contraction.
//
//   C_mn = sum_b sA(m, b) sB(b, n) sum_{k in block b} A_mk B_kn
//
// The tensor cores (pair_product.cuh) multiply one K block of 128 into an
// accumulator of its own; the epilogue warps read it, scale it and add it up in
// registers (128 x 256 float32 of a CTA in 8 warps, 128 of them a thread), while
// the MMAs of the next block fill the other accumulator.  So scales may be any
// float32, and sums between blocks are float32 FMAs.
//
// What bounds it: a K block's MMAs take 512 cycles, but its accumulator comes free
// only after the commit's way to the epilogue, the epilogue's reading (450) and the
// arrival's way back, and there are two: about 790 a block.  A scale for each
// column of B costs a second FMA-pipe instruction for every two sums, and about
// 1200.  8192 cubed with a scale per 128 x 128 of B 441 us call after call for seconds,
// under the power limit (2.49 PFLOP/s), in some tens of calls 390, with one for each
// column 564; 4096 cubed 70, 4096 x 4096 x 8192 by columns 172.  One token by 8192 x
// 4096: 10 us, 3.4 TB/s.
//
// Few tiles and a long contraction: the pairs of a cluster share a tile's K blocks and
// join their sums through shared memory (splits_for).
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "few_rows.cuh"
#include "pair_product.cuh"
#include "pipelined_ffn.h"

namespace pg {
namespace fp8 {

using namespace pair_product;

constexpr int kBlock = 128;

struct Call {
    Launch launch;
    const float *a_scale, *b_scale;
    long long a_scale_m, a_scale_k, b_scale_k, b_scale_n;
    int a_group; // rows that share a scale: 1 or 128
    void *c;
    long long ldc;
    int access;
    int withhold_scales; // test hook: K block of a CTA whose scales are never announced (-1: none)
};

// The scales of K blocks, which warp 3 copies ahead of the epilogue into a ring:
// the CTA's 128 rows' and the tile's 256 columns' of each block.  Loaded by the
// epilogue itself they cost it registers, and a load's latency in every block
// (8192 cubed 674 us).
struct ScaleRing {
    static constexpr int kStages = 8;
    static constexpr uint32_t kStageBytes = (128 + kCols) * 4;
    static constexpr int kBytes = kStages * (static_cast<int>(kStageBytes) + 16);
    uint32_t base;
    __device__ __forceinline__ uint32_t stage(unsigned f) const { return base + f % kStages * kStageBytes; }
    __device__ __forceinline__ uint32_t full(unsigned f) const
    {
        return base + kStages * kStageBytes + f % kStages * 8u;
    }
    __device__ __forceinline__ uint32_t empty(unsigned f) const { return full(f) + kStages * 8u; }
    static __device__ __forceinline__ uint32_t parity(unsigned f) { return f / kStages & 1u; }
};

// The epilogue's 128 sums and two tensor-memory loads of 32 need more registers a
// thread than 384 threads can have (168); the other 128 threads give theirs:
// 128 * 56 + 256 * 224 = 384 * 168.
constexpr int kEpilogueRegisters = 224, kOtherRegisters = 56;

// sum += v * s for both halves, kept between the tensor-memory loads around it:
// moved past them, more loads' results would be held than there are registers.
__device__ __forceinline__ void add_scaled(unsigned long long &sum, unsigned long long v, unsigned long long s)
{
    asm volatile("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(sum) : "l"(v), "l"(s));
}

// Where, in a ring that has served, the warps of pair `from` of the cluster's
// `splits` leave the sums of 32 of the columns that this pair finishes.
__device__ __forceinline__ uint32_t left_sums(int from, int chunk, int splits)
{
    return ((from * (4 / splits) + chunk) * kEpilogueWarps + threadIdx.x / 32 - kFirstEpilogueWarp) * 4096 +
           threadIdx.x % 32 * 16;
}
static_assert(4 * kEpilogueWarps * 4096 <= kStages * kStageBytes, "all pairs' together");

// Vector: sB differs from column to column; otherwise 128 columns have one.
// Joins: several pairs share a tile's K blocks (see splits_for).
template <class T, bool Vector, bool Joins>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp8_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Call p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = align_smem(smem_u32(smem_raw), 1024);
    const ScaleRing scales{base + kStages * kStageBytes};
    const Barriers b(scales.base + ScaleRing::kBytes);
    if (threadIdx.x == 0)
        for (unsigned k = 0; k < ScaleRing::kStages; ++k) {
            mbar_init(scales.full(k), 32);
            mbar_init(scales.empty(k), kEpilogueWarps);
        }
    auto epilogue = [&](uint32_t tmem, int rank, int first, int stride) {
        more_registers<kEpilogueRegisters>();
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        const int quarter = warp & 3, part = (warp - kFirstEpilogueWarp) / 4;
        const uint32_t empty = map_to_cta(b.acc_empty, Joins ? cluster_cta_rank() & ~1u : 0u);
        const Product &product = p.launch.product[0];
        const int blocks = Joins ? unit_at(p.launch, first).count : product.blocks;
        unsigned acc = 0;
        bool ok = true;
        for (int t = first; t < p.launch.units && ok; t += stride) {
            unsigned long long sum[64];
#pragma unroll
            for (int j = 0; j < 64; ++j)
                sum[j] = 0;
#pragma unroll 1
            for (int kb = 0; kb < blocks; ++kb, ++acc) {
                if (!acquire(p.launch, b, acc,
                             mbar_wait_bounded(scales.full(acc), ScaleRing::parity(acc), p.launch.wait_limit_ns))) {
                    ok = false;
                    break;
                }
                const uint32_t at =
                    tmem + (static_cast<uint32_t>(quarter * 32) << 16) + (acc & 1u) * kCols + part * 128;
                uint32_t r[2][32];
                tmem_ld_32x32b_x32(at, r[0]);
                const uint32_t held = scales.stage(acc);
                const uint32_t columns = held + 512u + static_cast<uint32_t>(part) * 512u;
                float s;
                asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(s) : "r"(held + (quarter * 32 + lane) * 4) : "memory");
                if constexpr (!Vector) {
                    float sb;
                    asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(sb) : "r"(columns) : "memory");
                    s *= sb;
                }
                const unsigned long long ss = pair(s, s);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    // The next 32 columns come while these are added up.
                    tmem_ld_wait();
                    if (c < 3)
                        tmem_ld_32x32b_x32(at + (c + 1) * 32, r[(c + 1) & 1]);
                    else
                        release(empty, acc);
                    const uint32_t(&v)[32] = r[c & 1];
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        unsigned long long v0 = pair(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                        unsigned long long v1 = pair(__uint_as_float(v[2 * j + 2]), __uint_as_float(v[2 * j + 3]));
                        if constexpr (Vector) {
                            unsigned long long s0, s1;
                            asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];\n"
                                         : "=l"(s0), "=l"(s1)
                                         : "r"(columns + (c * 32 + 2 * j) * 4)
                                         : "memory");
                            v0 = mul2(v0, s0);
                            v1 = mul2(v1, s1);
                        }
                        add_scaled(sum[c * 16 + j], v0, ss);
                        add_scaled(sum[c * 16 + j + 1], v1, ss);
                    }
                }
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(scales.empty(acc));
            }
            if constexpr (Joins) {
                // Of its 128 columns each pair of the cluster finishes a share.
                // All sums go through the owner's ring, its own too, so that one
                // piece of code serves any share.
                // Worked out here, not kept through the loop: no register is free there.
                int u = t;
                asm volatile("" : "+r"(u)::"memory");
                const Unit unit = unit_at(p.launch, u);
                const int splits = product.splits;
                cluster_sync();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int owner = c * splits / 4;
                    const uint32_t to =
                        map_to_cta(base + left_sums(unit.split, c - owner * (4 / splits), splits), owner * 2 + rank);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float v[4];
                        split(sum[c * 16 + 2 * j], v[0], v[1]);
                        split(sum[c * 16 + 2 * j + 1], v[2], v[3]);
                        st_cluster_v4(to + j * 512, __float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                      __float_as_uint(v[3]));
                    }
                }
                cluster_sync();
                const Tile tile = tile_at(product, unit.tile);
                const long long row0 = tile.mb * kRows + rank * 128 + quarter * 32;
                if (!ok || row0 >= product.rows)
                    continue;
                const int share = 4 / splits;
                int col = tile.nb * kCols + part * 128 + unit.split * share * 32;
#pragma unroll 1
                for (int c = 0; c < share && col < product.cols; ++c, col += 32) {
                    float v[32] = {};
#pragma unroll 1
                    for (int k = 0; k < splits; ++k) { // in their order
                        const uint32_t from = base + left_sums(k, c, splits);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float q[4];
                            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];\n"
                                         : "=f"(q[0]), "=f"(q[1]), "=f"(q[2]), "=f"(q[3])
                                         : "r"(from + j * 512)
                                         : "memory");
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                v[4 * j + i] += q[i];
                        }
                    }
                    store_tile(static_cast<T *>(p.c), p.ldc, row0, product.rows, col, product.cols, v, p.access);
                }
                continue;
            }
            const Tile tile = tile_at(product, t);
            const long long row0 = tile.mb * kRows + rank * 128 + quarter * 32;
            const int col0 = tile.nb * kCols + part * 128;
            if (!ok || row0 >= product.rows)
                continue;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int col = col0 + c * 32;
                if (col < product.cols) {
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        split(sum[c * 16 + j], v[2 * j], v[2 * j + 1]);
                    store_tile(static_cast<T *>(p.c), p.ldc, row0, product.rows, col, product.cols, v, p.access);
                }
            }
        }
    };
    auto load_scales = [&](int rank, int first, int stride) {
        const int lane = threadIdx.x % 32;
        const Product &product = p.launch.product[0];
        unsigned f = 0;
        bool ok = true;
        for (int t = first; t < p.launch.units && ok; t += stride) {
            int at = t, begin = 0, blocks = product.blocks;
            if constexpr (Joins) {
                const Unit unit = unit_at(p.launch, t);
                at = unit.tile;
                begin = unit.first;
                blocks = unit.count;
            }
            const Tile tile = tile_at(product, at);
            // Rows and columns outside take the last one's scales.  A lane has
            // four rows, and eight columns or none (Vector) or a block of 128.
            const float *from_a[4], *from_b[Vector ? 8 : 1];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                from_a[i] = p.a_scale + min(tile.mb * kRows + rank * 128 + i * 32 + lane, product.rows - 1) / p.a_group *
                                            p.a_scale_m +
                            begin * p.a_scale_k;
            if constexpr (Vector) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    from_b[i] = p.b_scale + min(tile.nb * kCols + i * 32 + lane, product.cols - 1) * p.b_scale_n +
                                begin * p.b_scale_k;
            } else {
                from_b[0] = p.b_scale +
                            min(tile.nb * kCols + (lane & 1) * 128, product.cols - 1) / kBlock * p.b_scale_n +
                            begin * p.b_scale_k;
            }
            for (int kb = 0; kb < blocks; ++kb, ++f) {
                if (!mbar_wait_bounded(scales.empty(f), ScaleRing::parity(f) ^ 1u, p.launch.wait_limit_ns)) {
                    // Each lane for itself: nothing here needs all of them.
                    record_error(p.launch.status, p.launch.family | kErrRoleProducer);
                    ok = false;
                    break;
                }
                const uint32_t to = scales.stage(f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    cp_async_ca4(to + (i * 32 + lane) * 4, from_a[i], 4);
                    from_a[i] += p.a_scale_k;
                }
                if constexpr (Vector) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        cp_async_ca4(to + 512 + (i * 32 + lane) * 4, from_b[i], 4);
                        from_b[i] += p.b_scale_k;
                    }
                } else {
                    if (lane < 2)
                        cp_async_ca4(to + 512 + lane * 512, from_b[0], 4);
                    from_b[0] += p.b_scale_k;
                }
                if (static_cast<int>(f) != p.withhold_scales)
                    cp_async_mbar_arrive_noinc(scales.full(f));
            }
        }
        cp_async_wait_all();
    };
    run<kMmaF8, true, kOtherRegisters, Joins>(p.launch, maps, base, b, epilogue, load_scales);
}

template <class Kernel, class... Args>
int launch_clusters(Kernel kernel, int ctas, int of, int smem, cudaStream_t s, const Args &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(of);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

template <class T, bool Vector, bool Joins>
int launch(const Maps &maps, const Call &p, int dev, unsigned long long ctx, int sms, cudaStream_t s)
{
    constexpr int kSmem = smem_bytes(ScaleRing::kBytes);
    static std::atomic<unsigned long long> limit_set[kMaxDevices];
    if (ensure_smem_limit(gemm_fp8_kernel<T, Vector, Joins>, kSmem, dev, ctx, limit_set) != GEMM_OK)
        return GEMM_ERR_CUDA;
    // The shares come out of what the launch gives: asked for more, the warps
    // would wait for good.
    static std::atomic<bool> enough{false};
    if (!enough.load(std::memory_order_relaxed)) {
        cudaFuncAttributes a = {};
        if (cudaFuncGetAttributes(&a, gemm_fp8_kernel<T, Vector, Joins>) != cudaSuccess ||
            a.numRegs * kThreads < kEpilogueWarps * 32 * kEpilogueRegisters +
                                       (kThreads - kEpilogueWarps * 32) * kOtherRegisters)
            return GEMM_ERR_CUDA;
        enough.store(true, std::memory_order_relaxed);
    }
    const int splits = p.launch.product[0].splits;
    const int pairs = Joins ? p.launch.units : std::max(1, std::min(p.launch.units, sms / 2));
    return launch_clusters(gemm_fp8_kernel<T, Vector, Joins>, 2 * pairs, 2 * splits, kSmem, s, maps, p);
}

// ---------------------------------------------------------------- few rows
struct FewCall {
    few_rows::Launch launch;
    const float *a_scale, *b_scale;
    long long a_scale_m, a_scale_k, b_scale_k, b_scale_n;
    int a_group, b_group;
    void *c;
    long long ldc;
    int c_bf16;
};

template <int Tokens>
__global__ void __launch_bounds__(few_rows::kThreads, 2)
    gemm_fp8_few_rows_kernel(const __grid_constant__ few_rows::Maps maps, const __grid_constant__ FewCall p)
{
    using S = few_rows::Shape<kMmaF8, Tokens>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = align_smem(smem_u32(smem_raw), 1024);
    few_rows::run<kMmaF8, Tokens>(
        p.launch, maps, base,
        [&](uint32_t tmem, const auto &b, int first, int count, int token0, int feature, auto put) {
            const few_rows::Launch &l = p.launch;
            const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
            // This warp's tokens' scales of two K blocks.
            const uint32_t scales = base + S::kStages * S::kStageBytes + few_rows::kBarrierBytes +
                                    static_cast<uint32_t>(warp - 2) * (2 * few_rows::kMaxTokens * 4);
            constexpr int kPerLane = (Tokens + 31) / 32;
            // Tokens and features outside take the last one's scales.
            const float *from_b =
                p.b_scale + min(feature, l.features - 1) / p.b_group * p.b_scale_n + first * p.b_scale_k;
            const float *from_a[kPerLane];
#pragma unroll
            for (int i = 0; i < kPerLane; ++i)
                from_a[i] = p.a_scale + min(token0 + lane + 32 * i, l.rows - 1) / p.a_group * p.a_scale_m +
                            first * p.a_scale_k;
            unsigned long long sum[Tokens / 2];
#pragma unroll
            for (int j = 0; j < Tokens / 2; ++j)
                sum[j] = 0;
            float next_a[kPerLane], next_b;
            auto fetch = [&](int f) {
                next_b = __ldg(from_b + f * p.b_scale_k);
#pragma unroll
                for (int i = 0; i < kPerLane; ++i)
                    next_a[i] = __ldg(from_a[i] + f * p.a_scale_k);
            };
            fetch(0);
            for (int f = 0; f < count; ++f) {
                const uint32_t held = scales + (f & 1) * (few_rows::kMaxTokens * 4);
#pragma unroll
                for (int i = 0; i < kPerLane; ++i)
                    if (lane + 32 * i < Tokens)
                        asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(held + (lane + 32 * i) * 4), "f"(next_a[i])
                                     : "memory");
                const unsigned long long sb = pair(next_b, next_b);
                __syncwarp();
                if (f + 1 < count)
                    fetch(f + 1);
                const uint32_t acc = static_cast<uint32_t>(f & 1);
                const bool ok = mbar_wait_bounded(b.acc_full + 8u * acc, (static_cast<uint32_t>(f) >> 1) & 1u,
                                                  l.wait_limit_ns);
                if (!__all_sync(0xffffffffu, ok)) {
                    if (lane == 0)
                        record_error(l.status, l.family | kErrRoleEpilogue);
                    return;
                }
                tc_fence_after_sync();
#pragma unroll
                for (int c = 0; c < Tokens; c += 16) {
                    uint32_t r[16];
                    tmem_ld_32x32b_x16(tmem + acc * Tokens + c, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        unsigned long long s0, s1;
                        asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];\n"
                                     : "=l"(s0), "=l"(s1)
                                     : "r"(held + (c + j) * 4)
                                     : "memory");
                        const unsigned long long v0 = pair(__uint_as_float(r[j]), __uint_as_float(r[j + 1]));
                        const unsigned long long v1 = pair(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3]));
                        const int at = (c + j) / 2;
                        sum[at] = fma2(mul2(v0, s0), sb, sum[at]);
                        sum[at + 1] = fma2(mul2(v1, s1), sb, sum[at + 1]);
                    }
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(b.acc_empty + 8u * acc);
            }
#pragma unroll
            for (int j = 0; j < Tokens / 2; ++j) {
                float lo, hi;
                split(sum[j], lo, hi);
                put(2 * j, lo);
                put(2 * j + 1, hi);
            }
        },
        [&](int token, int feature, const float(&sum)[1]) {
            store_f32(p.c, p.c_bf16, token * p.ldc + feature, sum[0]);
        });
}

// Of few_rows::faster; more than 64 tokens go in tiles of 64 (of 128: 25 us for
// 128 x 8192 x 4096 where these take 21).
// With a scale per 128 columns of B, and with one for each.
constexpr few_rows::Times kTimes{0.4, 5.0, 0.43}, kVectorTimes{0.4, 5.0, 0.63};

// How many pairs share a tile's K blocks, where there are few tiles, and what they
// take. A join costs the ring's end, a cluster's barriers and the sums' way: 4 us
// for two pairs, 5.5 for four. Clusters of two pairs fill 36 * 4 of 152 SMs, of
// four at least 12 * 8 (16 tiles took two rounds: 1024 x 4096 x 1024 26.9 us). us
// with one, two and four pairs a tile:
//   1024 x 4096 x 1024         18.8  15.9
//   768 x 4096 x 1024          18.7  15.9  15.4
//   256 x 8192 x 4096          30.7  22.1  33.6
//   1536 x 4096 x 1536         19.3  17.9
//   512 x 1024 x 512            8.7  10.4  11.0
// and with a scale for each column
//   512 x 4096 x 512           24.9  18.9  15.3
//   1000 x 8000 x 1000         44.9  29.8  40.6
//   1280 x 2048 x 1280         15.8  15.3
inline int splits_for(const few_rows::Times &t, long long tiles, int blocks, int sms, double *us)
{
    *us = few_rows::pairs_time(t, tiles, blocks, sms);
    int best = 1;
    for (int s = 2; s <= 4; s *= 2) {
        if (tiles > (s == 2 ? sms / 4 - 2 : sms / 12) || blocks < s)
            break;
        const double with = t.pair_start + t.pair_block * ((blocks + s - 1) / s) + (s == 2 ? 4.0 : 5.5);
        if (with < *us) {
            best = s;
            *us = with;
        }
    }
    return best;
}

template <int Tokens>
int launch_few(const few_rows::Maps &maps, FewCall &p, int dev, unsigned long long ctx, int sms, cudaStream_t s)
{
    using S = few_rows::Shape<kMmaF8, Tokens>;
    static std::atomic<unsigned long long> limit_set[kMaxDevices];
    if (ensure_smem_limit(gemm_fp8_few_rows_kernel<Tokens>, S::kSmem, dev, ctx, limit_set) != GEMM_OK)
        return GEMM_ERR_CUDA;
    few_rows::Launch &l = p.launch;
    l.feature_tiles = (l.features + few_rows::kFeatures - 1) / few_rows::kFeatures;
    const long long tiles = static_cast<long long>(l.feature_tiles) * ((l.rows + Tokens - 1) / Tokens);
    l.ranks = few_rows::ranks_for(tiles, l.blocks, sms);
    return few_rows::launch(gemm_fp8_few_rows_kernel<Tokens>, static_cast<unsigned>(tiles * l.ranks), l.ranks, S::kSmem,
                            s, maps, p);
}

constexpr int kMaxSide = 1 << 30;

bool valid_format(int f) { return f == GEMM_FP8_E4M3 || f == GEMM_FP8_E5M2; }
bool valid_group(int g) { return g == 1 || g == kBlock; }

// rows x cols: as stored.
int check_operand(const void *p, int rows, int cols, long long pitch)
{
    if (!p || (rows > 1 && pitch < cols))
        return GEMM_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0 || (rows > 1 && pitch % 16 != 0))
        return GEMM_ERR_MISALIGNED;
    return GEMM_OK;
}

} // namespace fp8
} // namespace pg

using namespace pg;

extern "C" int gemm_fp8(int M, int N, int K, const void *A, long long lda, int a_format, int a_transposed,
                        const float *a_scale, long long a_scale_m, long long a_scale_k, int a_group, const void *B,
                        long long ldb, int b_format, int b_transposed, const float *b_scale, long long b_scale_k,
                        long long b_scale_n, int b_group, void *C, long long ldc, int dtype, void *stream)
{
    using namespace fp8;
    if (M < 0 || N < 0 || K < 0 || !valid_format(a_format) || !valid_format(b_format) || !valid_group(a_group) ||
        !valid_group(b_group) || (dtype != GEMM_DTYPE_F32 && dtype != GEMM_DTYPE_BF16))
        return GEMM_ERR_INVALID_ARG;
    if (M > kMaxSide || N > kMaxSide || K > kMaxSide)
        return GEMM_ERR_UNSUPPORTED;
    const long long tiles = (static_cast<long long>(M) + kRows - 1) / kRows * ((N + kCols - 1) / kCols);
    if (tiles > 1ll << 30)
        return GEMM_ERR_UNSUPPORTED;
    const bool empty = M == 0 || N == 0;
    const size_t size = dtype == GEMM_DTYPE_F32 ? 4 : 2;
    int st;
    if (!empty) {
        if (!C || (M > 1 && ldc < N))
            return GEMM_ERR_INVALID_ARG;
        if (K > 0) {
            if ((st = check_operand(A, a_transposed ? K : M, a_transposed ? M : K, lda)) != GEMM_OK ||
                (st = check_operand(B, b_transposed ? N : K, b_transposed ? K : N, ldb)) != GEMM_OK)
                return st;
            if (!a_scale || !b_scale)
                return GEMM_ERR_INVALID_ARG;
            if (((reinterpret_cast<uintptr_t>(a_scale) | reinterpret_cast<uintptr_t>(b_scale)) & 3u) != 0)
                return GEMM_ERR_MISALIGNED;
        }
        if ((reinterpret_cast<uintptr_t>(C) & (size - 1)) != 0)
            return GEMM_ERR_MISALIGNED;
    }
    int dev;
    st = device_checked(&dev);
    if (st != GEMM_OK || empty)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (K == 0) {
        const size_t row = static_cast<size_t>(N) * size;
        return cudaMemset2DAsync(C, M > 1 ? static_cast<size_t>(ldc) * size : row, 0, row, M, s) == cudaSuccess
                   ? GEMM_OK
                   : GEMM_ERR_CUDA;
    }
    const unsigned long long ctx = current_context_id();
    unsigned int *const status = device_status_word(dev, ctx);
    if (!status)
        return GEMM_ERR_CUDA;
    const int sms = device_sms();
    const int blocks = (K + kBlock - 1) / kBlock;
    const few_rows::Times &times = b_group == 1 ? kVectorTimes : kTimes;
    double pairs;
    const int splits = splits_for(times, tiles, blocks, sms, &pairs);
    const int tokens = M <= 16 ? 16 : M <= 32 ? 32 : 64;
    if (!a_transposed && few_rows::time_of(times, tokens, M, N, blocks, sms) < pairs) {
        const int weight_mn = b_transposed ? 0 : 1;
        few_rows::Maps few;
        std::memset(&few, 0, sizeof few);
        if ((st = few_rows::encode_tokens(&few.tokens, kMmaF8, A, M, K, lda, tokens)) != GEMM_OK ||
            (st = encode_operand(&few.weight[0], kMmaF8, B, weight_mn ? K : N, weight_mn ? N : K, ldb,
                                 weight_mn ? across(kMmaF8, N) : kAlongK)) != GEMM_OK)
            return st;
        FewCall p = {};
        p.launch.rows = M;
        p.launch.features = N;
        p.launch.blocks = blocks;
        p.launch.weight_mn = weight_mn;
        p.launch.idesc = few_rows::instruction(b_format == GEMM_FP8_E5M2, a_format == GEMM_FP8_E5M2, weight_mn, tokens);
        p.launch.family = kErrFamilyFp8;
        p.launch.status = status;
        p.launch.wait_limit_ns = call_wait_limit_ns();
        p.launch.withhold = call_withhold();
        p.a_scale = a_scale;
        p.b_scale = b_scale;
        p.a_scale_m = a_scale_m;
        p.a_scale_k = a_scale_k;
        p.b_scale_k = b_scale_k;
        p.b_scale_n = b_scale_n;
        p.a_group = a_group;
        p.b_group = b_group;
        p.c = C;
        p.ldc = ldc;
        p.c_bf16 = dtype == GEMM_DTYPE_BF16;
        return tokens == 16   ? launch_few<16>(few, p, dev, ctx, sms, s)
               : tokens == 32 ? launch_few<32>(few, p, dev, ctx, sms, s)
                              : launch_few<64>(few, p, dev, ctx, sms, s);
    }
    Call p = {};
    p.launch.status = status;
    p.launch.family = kErrFamilyFp8;
    p.launch.wait_limit_ns = call_wait_limit_ns();
    p.launch.withhold = call_withhold();
    const int a_mn = a_transposed ? 1 : 0, b_mn = b_transposed ? 0 : 1;
    const Layout a_layout = a_mn ? across(kMmaF8, M) : kAlongK, b_layout = b_mn ? across(kMmaF8, N) : kAlongK;
    Product &product = p.launch.product[0];
    product.rows = M;
    product.cols = N;
    product.tiles_m = (M + kRows - 1) / kRows;
    product.tiles_n = (N + kCols - 1) / kCols;
    product.blocks = blocks;
    product.segments = 1;
    product.splits = splits;
    product.a_layout = a_layout;
    product.b_layout = b_layout;
    product.b_map = 1;
    product.idesc = instruction(a_format == GEMM_FP8_E5M2, b_format == GEMM_FP8_E5M2, a_layout, b_layout);
    p.launch.units = p.launch.first_units = product.units();
    p.launch.maps = 2;
    Maps maps;
    std::memset(&maps, 0, sizeof maps);
    if ((st = encode_operand(&maps.map[0], kMmaF8, A, a_mn ? K : M, a_mn ? M : K, lda, a_layout)) != GEMM_OK ||
        (st = encode_operand(&maps.map[1], kMmaF8, B, b_mn ? K : N, b_mn ? N : K, ldb, b_layout)) != GEMM_OK)
        return st;
    p.a_scale = a_scale;
    p.b_scale = b_scale;
    p.a_scale_m = a_scale_m;
    p.a_scale_k = a_scale_k;
    p.b_scale_k = b_scale_k;
    p.b_scale_n = b_scale_n;
    p.a_group = a_group;
    p.c = C;
    p.ldc = ldc;
    p.access = row_access(C, ldc, M, size);
    p.withhold_scales = call_withhold_scales();
    auto go = [&](auto type, auto vector) {
        using T = decltype(type);
        constexpr bool kVector = decltype(vector)::value;
        return splits > 1 ? launch<T, kVector, true>(maps, p, dev, ctx, sms, s)
                          : launch<T, kVector, false>(maps, p, dev, ctx, sms, s);
    };
    if (dtype == GEMM_DTYPE_F32)
        return b_group == 1 ? go(float(), std::true_type()) : go(float(), std::false_type());
    return b_group == 1 ? go(__nv_bfloat16(), std::true_type()) : go(__nv_bfloat16(), std::false_type());
}
