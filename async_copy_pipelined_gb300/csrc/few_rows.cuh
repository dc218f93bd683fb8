// Products of a few rows (tokens) by a weight, where the weight's bytes bound
// the time: the loop that the gated projection and the 8-bit product share.
//
// The tensor core's 128 rows are 128 of the weight's columns (features) and its
// N columns are the tokens, 16 to 64 of them, so that nothing is padded to 128
// rows of tokens.  The contraction is split over the CTAs of a cluster, as many
// as fill the GPU with two CTAs on each SM; their float32 sums meet in shared
// memory, where each CTA adds up some of the tokens over the cluster, in the
// order of the ranks.
//
//   warp 0      TMA producer: a ring of stages of one 128-byte K block: the
//               weight's 16 KiB (of both weights of a gated projection) and the
//               tokens' rows of 128 bytes.
//   warp 1      allocates tensor memory, issues the MMAs.
//   warps 2-5   epilogue: warp w has features 32 (w % 4) .. +31, a lane each.
//
// Operands lie in shared memory as in pair_product.cuh.
#pragma once

#include <cstdint>

#include "gemm_internal.h"
#include "ptx.cuh"
#include "tma_ring.cuh"
#include "vector_io.cuh"

namespace pg {
namespace few_rows {

constexpr int kFeatures = 128;
constexpr int kThreads = 192;
constexpr int kEpilogueThreads = 128;
constexpr uint32_t kWeightBytes = 128 * 128; // of one weight's K block
constexpr int kMaxRanks = 8;
constexpr int kAtOnce = 4;
constexpr int kMaxTokens = 64;
// Shared memory of one of two CTAs of an SM.  All of it is asked for: it keeps
// the library's other tensor-core kernels (116 KiB and more) off an SM that has
// one of these.  Two kernels of clusters, on two streams, that took tensor memory
// on each other's SMs could otherwise wait for each other in its allocation.
constexpr int kBudget = 112 * 1024;
constexpr int kBarrierBytes = 256;
constexpr int kScaleBytes = 4 * 2 * kMaxTokens * 4; // each epilogue warp's tokens' scales of two K blocks

template <MmaKind Kind, int Tokens>
struct Shape {
    static_assert(Tokens <= kMaxTokens, "as many as there is room for scales");
    static constexpr int kWeights = Kind == kMmaF16 ? 2 : 1;
    static constexpr uint32_t kStageBytes = kWeights * kWeightBytes + Tokens * 128;
    static constexpr int kExtra = kBarrierBytes + (Kind == kMmaF8 ? kScaleBytes : 0) + 1024;
    static constexpr int kFit = (kBudget - kExtra) / static_cast<int>(kStageBytes);
    static constexpr int kStages = kFit < 6 ? kFit : 6;
    static constexpr int kSmem = kBudget;
    static_assert(kStages * static_cast<int>(kStageBytes) + kExtra <= kBudget, "the ring fits");
    // Sums of the CTA's features: columns of 128 floats, a token's (and weight's) each.
    static constexpr int kColumns = kWeights * Tokens;
    static_assert(kStages >= 2 && kColumns * 512 <= kStages * static_cast<int>(kStageBytes), "the sums fit the ring");
    // Gated: both accumulators.  8-bit: one for each of two K blocks.
    static constexpr uint32_t kTmemCols = 2 * Tokens < 32 ? 32 : 2 * Tokens;
    static constexpr int kBlockK = Kind == kMmaF16 ? 64 : 128;
};

struct Maps {
    CUtensorMap tokens, weight[2];
};

struct Launch {
    int rows, features; // of the result
    int blocks;         // K blocks
    int feature_tiles;
    int ranks;          // CTAs of a cluster
    int weight_mn;      // the weight is stored with its features contiguous
    uint32_t idesc;
    unsigned int family;
    unsigned int *status;
    unsigned long long wait_limit_ns;
    int withhold;
};

constexpr uint32_t instruction(uint32_t weight_format, uint32_t token_format, int weight_mn, int tokens)
{
    return (1u << 4) | (weight_format << 7) | (token_format << 10) | (static_cast<uint32_t>(weight_mn) << 15) |
           (static_cast<uint32_t>(tokens >> 3) << 17) | (static_cast<uint32_t>(kFeatures >> 4) << 24);
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

template <int S>
struct Barriers {
    TmaRing<S> ring;
    uint32_t acc_full, acc_empty, mma_done, tmem_slot;
    __device__ __forceinline__ explicit Barriers(uint32_t at)
        : ring{at, at + 8u * S}, acc_full(at + 16u * S), acc_empty(acc_full + 16u), mma_done(acc_empty + 16u),
          tmem_slot(mma_done + 8u)
    {
    }
};

// One CTA.  `accumulate(tmem, barriers, first, count, put)` is the epilogue
// warps' work on K blocks first .. first + count - 1: it calls put(column, value)
// for its feature's sums; `finish(token, feature, sum)` gets sum[weight], the
// cluster's sums of one element.
template <MmaKind Kind, int Tokens, class Accumulate, class Finish>
__device__ __forceinline__ void run(const Launch &l, const Maps &maps, uint32_t base, Accumulate accumulate,
                                    Finish finish)
{
    using S = Shape<Kind, Tokens>;
    constexpr int kWeights = S::kWeights;
    constexpr int kBoxMn = Kind == kMmaF16 ? 64 : 128; // elements of 128 bytes along the features
    constexpr uint32_t kMnStep = Kind == kMmaF16 ? 2048 : 4096;
    const Barriers<S::kStages> b(base + S::kStages * S::kStageBytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = static_cast<int>(cluster_cta_rank());
    const int tile = static_cast<int>(blockIdx.x) / l.ranks;
    const int feature0 = tile % l.feature_tiles * kFeatures;
    const int token0 = tile / l.feature_tiles * Tokens;
    // This rank's K blocks: at least one (the launcher sees to it).
    const int first = static_cast<int>(static_cast<long long>(l.blocks) * rank / l.ranks);
    const int count = static_cast<int>(static_cast<long long>(l.blocks) * (rank + 1) / l.ranks) - first;

    if (threadIdx.x == 0) {
        b.ring.init(1);
        for (int k = 0; k < 2; ++k) {
            mbar_init(b.acc_full + 8u * k, 1);
            mbar_init(b.acc_empty + 8u * k, kEpilogueThreads / 32);
        }
        mbar_init(b.mma_done, 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(b.tmem_slot, S::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(tmem) : "r"(b.tmem_slot) : "memory");

    if (warp == 0) {
        const uint32_t on = lane == 0; // issues for the warp, as in pair_product.cuh
        if (on) {
            tma_prefetch_map(&maps.tokens);
            for (int w = 0; w < kWeights; ++w)
                tma_prefetch_map(&maps.weight[w]);
        }
        int f = 0;
        for (; f < count; ++f) {
            if (f == l.withhold)
                continue; // test hook: this position is never filled
            // Each lane by itself, as in pair_product.cuh.
            if (!b.ring.producer_acquire(f, l.wait_limit_ns)) {
                if (on)
                    record_error(l.status, l.family | kErrRoleProducer);
                break;
            }
            const uint32_t to = base + static_cast<uint32_t>(f % S::kStages) * S::kStageBytes;
            const uint32_t full = b.ring.full_bar(f);
            mbar_arrive_expect_tx_if(on, full, S::kStageBytes);
            const int k = (first + f) * S::kBlockK;
#pragma unroll
            for (int w = 0; w < kWeights; ++w) {
                if (l.weight_mn) {
#pragma unroll
                    for (int j = 0; j < kFeatures / kBoxMn; ++j)
                        tma_load_2d_if(on, to + w * kWeightBytes + j * 8192, &maps.weight[w], full,
                                       feature0 + j * kBoxMn, k);
                } else {
                    tma_load_2d_if(on, to + w * kWeightBytes, &maps.weight[w], full, k, feature0);
                }
            }
            tma_load_2d_if(on, to + kWeights * kWeightBytes, &maps.tokens, full, k, token0);
        }
        // Only the last kStages positions can still be in flight.
        bool drained = true;
        for (int g = f > S::kStages ? f - S::kStages : 0; g < f; ++g)
            if (g != l.withhold && !b.ring.consumer_wait(g, l.wait_limit_ns))
                drained = false;
        if (!drained && on)
            record_error(l.status, l.family | kErrRoleDrain);
    } else if (warp == 1) {
        const uint32_t on = lane == 0;
        const uint32_t step = (l.weight_mn ? kMnStep : 32u) >> 4;
        const uint64_t w0 = smem_desc_sw128(base, l.weight_mn ? 8192 : 16, 1024);
        const uint64_t t0 = smem_desc_sw128(base + kWeights * kWeightBytes, 16, 1024);
        bool ok = true;
        for (int f = 0; f < count; ++f) {
            const uint32_t acc = Kind == kMmaF8 ? static_cast<uint32_t>(f & 1) : 0u;
            if (Kind == kMmaF8 &&
                !mbar_wait_bounded(b.acc_empty + 8u * acc, ((static_cast<uint32_t>(f) >> 1) & 1u) ^ 1u,
                                   l.wait_limit_ns)) {
                ok = false;
                break;
            }
            if (!b.ring.consumer_wait(f, l.wait_limit_ns)) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            const uint32_t stage = static_cast<uint32_t>(f % S::kStages) * (S::kStageBytes >> 4);
#pragma unroll
            for (uint32_t ks = 0; ks < 4; ++ks)
#pragma unroll
                for (int w = 0; w < kWeights; ++w) {
                    const uint32_t d = tmem + (Kind == kMmaF8 ? acc : static_cast<uint32_t>(w)) * Tokens;
                    mma_if<Kind>(on, d, w0 + stage + w * (kWeightBytes >> 4) + ks * step, t0 + stage + ks * 2, l.idesc,
                                 (Kind == kMmaF16 && f != 0) || ks != 0);
                }
            mma_commit_if(on, b.ring.empty_bar(f));
            if (Kind == kMmaF8 || f == count - 1)
                mma_commit_if(on, b.acc_full + 8u * acc);
        }
        if (!ok && on)
            record_error(l.status, l.family | kErrRoleMma);
        // Every MMA issued must finish before tensor memory is freed.
        mma_commit_if(on, b.mma_done);
        if (!mbar_wait_bounded(b.mma_done, 0, l.wait_limit_ns) && on)
            record_error(l.status, l.family | kErrRoleDrain);
    } else {
        // The MMAs have read every stage once the last accumulator is full, and
        // the ring takes the sums.
        const int feature = (warp & 3) * 32 + lane;
        accumulate(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16), b, first, count, token0, feature0 + feature,
                   [&](int column, float v) {
                       asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(base + static_cast<uint32_t>(column * 512 +
                                                                                                  feature * 4)),
                                    "f"(v)
                                    : "memory");
                   });
    }
    tc_fence_before_sync();
    cluster_sync();
    tc_fence_after_sync();
    if (warp == 1) {
        tmem_dealloc(tmem, S::kTmemCols);
    } else if (warp >= 2) {
        const int feature = static_cast<int>(threadIdx.x) - 64;
        uint32_t from[kMaxRanks];
#pragma unroll
        for (int r = 0; r < kMaxRanks; ++r)
            from[r] = map_to_cta(base + static_cast<uint32_t>(feature) * 4u, r < l.ranks ? r : 0);
        const int tokens = min(Tokens, l.rows - token0);
        if (feature0 + feature < l.features)
            // kAtOnce tokens' sums are on their way together.
            for (int t = rank; t < tokens; t += kAtOnce * l.ranks) {
                float v[kAtOnce][kWeights][kMaxRanks];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
                    for (int w = 0; w < kWeights; ++w) {
                        const uint32_t at = static_cast<uint32_t>(w * Tokens + min(t + k * l.ranks, Tokens - 1)) * 512u;
#pragma unroll
                        for (int r = 0; r < kMaxRanks; ++r)
                            if (r < l.ranks)
                                v[k][w][r] = ld_cluster_f32(from[r] + at);
                    }
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    if (t + k * l.ranks >= tokens)
                        break;
                    float sum[kWeights];
#pragma unroll
                    for (int w = 0; w < kWeights; ++w) {
                        sum[w] = v[k][w][0];
#pragma unroll
                        for (int r = 1; r < kMaxRanks; ++r)
                            if (r < l.ranks)
                                sum[w] += v[k][w][r];
                    }
                    finish(token0 + t + k * l.ranks, feature0 + feature, sum);
                }
            }
    }
    cluster_sync(); // no CTA leaves while another reads its sums
}

// -------------------------------------------------------------------- host
// How many CTAs share a contraction: a power of two, as clusters of others leave
// SMs of a processing cluster empty (384 x 1000 x 2700 in 8 bits: 16 us with
// six, where 512 take 12 with four).  Two CTAs fit an SM; a wave of them takes
// its K blocks and about four blocks' time to start, join and write.
inline int ranks_for(long long tiles, int blocks, int sms)
{
    const long long slots = 2ll * sms;
    int best = 1;
    double least = 0.0;
    for (int r = 1; r <= kMaxRanks && r <= blocks; r *= 2) {
        const long long waves = (tiles * r + slots - 1) / slots;
        const double cost = static_cast<double>(waves) * ((blocks + r - 1) / r + 4);
        if (r == 1 || cost < least) {
            best = r;
            least = cost;
        }
    }
    return best;
}

// What the choice between this kernel and pairs of CTAs on 256 x 256 tiles goes
// by: microseconds to start, join and write, and for a K block while each SM has
// one CTA (or pair) at work.  Fitted to 26 sizes with both kernels at each; the
// faster one is chosen at all but a few, where they differ by 5 % (us, this
// kernel / pairs, each at a tile of its own; 8-bit M x N x K and gated rows x
// width -> hidden):
//   8-bit 64 x 8192 x 4096   13.5 / 19.1    gated 32 x 4096 -> 8192  26.3 / 27.2
//         128                19.4 / 19.8          33                 31.3 / 27.3
//         192                31.4 / 20.0          128 x 1024 -> 2048  9.9 / 11.4
//         512 x 1000 x 2700  10.7 / 17.4          256                13.1 / 11.5
//         1000               15.8 / 17.5          256 x 8192 -> 512  16.0 / 43.6
struct Times {
    double block, pair_start, pair_block;
};

inline double start_time(int tokens) { return tokens == 16 ? 4.3 : tokens == 32 ? 5.0 : 6.0; }

// What `rows` in tiles of `tokens` take here.
inline double time_of(const Times &t, int tokens, int rows, int features, int blocks, int sms)
{
    const long long tiles =
        (static_cast<long long>(rows) + tokens - 1) / tokens * ((features + kFeatures - 1) / kFeatures);
    const int ranks = ranks_for(tiles, blocks, sms);
    const long long per_sm = (tiles * ranks + sms - 1) / sms;
    return start_time(tokens) + t.block * static_cast<double>(per_sm) * ((blocks + ranks - 1) / ranks);
}

// What `tiles` of 256 x 256 take pairs of CTAs.
inline double pairs_time(const Times &t, long long tiles, int blocks, int sms)
{
    const long long waves = (tiles + sms / 2 - 1) / (sms / 2);
    return t.pair_start + t.pair_block * static_cast<double>(waves) * blocks;
}

// Whether they are faster here; pair_tiles: of 256 x 256.
inline bool faster(const Times &t, int tokens, int rows, int features, int blocks, long long pair_tiles, int sms)
{
    return time_of(t, tokens, rows, features, blocks, sms) < pairs_time(t, pair_tiles, blocks, sms);
}

int encode_tokens(CUtensorMap *map, MmaKind kind, const void *x, int rows, int cols, long long pitch, int tokens);

template <class Kernel, class... Args>
int launch(Kernel kernel, unsigned ctas, int ranks, int smem, cudaStream_t s, const Args &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(ranks);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

} // namespace few_rows
} // namespace pg
