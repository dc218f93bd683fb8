// The orthogonalisation of small matrices in one kernel: everything stays in
// shared and tensor memory from G to the result.
//
// The iteration is that of orthogonalize.cu, bfloat16 results only, for
// matrices whose shorter side r is at most 128.  There a product takes a
// microsecond and the rest of a launch, a round through L2 and the wait for the
// kernel before take six.  One CTA holds up to 256 columns of X (two
// float16 planes, 128 KiB), and A and then Q in two planes (64 KiB); 1, 2, 4
// or 8 CTAs, a cluster, hold a matrix.  The square and Q X need no exchange:
// every CTA has all of A.  X X^T is summed over the CTAs' columns, each rank
// adding the others' partial sums of its part in rank order and sending the
// finished planes to all, in 4 KiB bulk copies.
//
// X lies as 64-column blocks of 128 rows of 128 bytes in the 128-byte swizzle:
// K-major for X X^T, and the same bytes are the MN-major right operand of Q X.
//
// What bounds it is latency: five steps of three dependent products, each a
// barrier, 8 to 24 MMAs, a wait and the accumulator's way through registers
// back to shared memory, about 2.5 us together, and between the CTAs of a
// cluster two exchanges a step.  The tensor cores work for a tenth of it.
//
// Measured on GB300, five steps, bfloat16 (microseconds a call; in brackets
// orthogonalize.cu's kernels): 64 x 64 35 (70), 128 x 128 43 (90), 128 x 256 51
// (94), 100 x 512 66 (107), 128 x 1024 72 to 76 (113), 2048 x 128 84 to 88
// (117); 16 of 100 x 300 82.
#include <algorithm>

#include "orthogonalize_internal.h"

namespace pg {

namespace orth {

constexpr int kSmallRows = 128;
constexpr int kSlab = 256;     // columns of X that a CTA holds
constexpr int kMaxRanks = 8;
constexpr int kSmallThreads = 512;
constexpr uint32_t kColumnBlock = kSmallRows * 128; // 64 columns: 16 KiB
constexpr uint32_t kUnit = 32 * 32 * 4;             // a warp's share of a 128 x 128 sum
constexpr uint32_t kStrip = 32 * 128;               // 32 rows of a column block: one piece of a plane

// Shared memory, from a 1024-byte boundary: A's planes and then Q's, the other
// ranks' sums, X's planes.  Four column blocks of X leave no room for the sums
// beside A; they then arrive where A and Q are not yet, with two more meetings
// of the cluster.
constexpr uint32_t kA0 = 0, kA1 = 2 * kColumnBlock;
constexpr uint32_t kBeside = 4 * kColumnBlock;
constexpr int kRoomyBlocks = 3;
constexpr uint32_t kSmallSmem = 14 * kColumnBlock + 1024;
static_assert(16 * kUnit <= 4 * kColumnBlock, "the sums take no more than A's planes");
static_assert(8 * kColumnBlock + kRoomyBlocks * 2 * kColumnBlock <= kSmallSmem - 1024, "X fits behind the sums");

struct Small {
    Matrix g;
    int r, c, tall;
    int ranks, blocks; // CTAs of a matrix; 64-column blocks that each holds
    void *out;
    long long ldo, out_batch;
    int out_vec; // rows of out can be written eight elements at a time
    int steps;
    float eps;
    unsigned int *status;
    unsigned long long wait_limit_ns;
    int withhold;
    float coefficients[3 * kMaxSteps];
    Slow slow[kMaxSteps];
};

constexpr uint32_t instruction(int n, bool right_mn)
{
    return (1u << 4) | (right_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(kSmallRows >> 4) << 24);
}

// 32 columns of this lane's row as one plane; what it leaves over stays in v.
__device__ __forceinline__ void make_plane(unsigned long long (&v)[16], uint32_t (&w)[16])
{
    const unsigned long long minus = pair(-1.0f, -1.0f);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        float lo, hi;
        split(v[j], lo, hi);
        w[j] = pack_f16(lo, hi);
        const float2 kept = unpack_f16(w[j]);
        v[j] = fma2(pair(kept.x, kept.y), minus, v[j]);
    }
}

// The same to `row`, a row's 128 bytes of a column block, its first or second
// half, in the 128-byte swizzle.
__device__ __forceinline__ void store_plane(uint32_t row, int lane, int second, const uint32_t (&w)[16])
{
#pragma unroll
    for (int j = 0; j < 4; ++j)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(
                         row + static_cast<uint32_t>(((second * 4 + j) ^ (lane & 7)) << 4)),
                     "r"(w[4 * j]), "r"(w[4 * j + 1]), "r"(w[4 * j + 2]), "r"(w[4 * j + 3])
                     : "memory");
}

__global__ void __launch_bounds__(kSmallThreads, 1) small_kernel(const __grid_constant__ Small p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[3];
    __shared__ uint32_t tmem_slot;
    __shared__ float4 warp_sums[kSmallThreads / 32];
    __shared__ float4 rank_sums[kMaxRanks];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = align_smem(raw, 1024); // the same offset in every CTA of the cluster
    const uint32_t done = smem_u32(&bars[0]), drained = smem_u32(&bars[1]), arrived = smem_u32(&bars[2]);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = p.ranks > 1 ? static_cast<int>(cluster_cta_rank()) : 0;
    const int b = static_cast<int>(blockIdx.x) / p.ranks;
    const int width = p.blocks * 64, col0 = rank * width; // this CTA's columns of X
    const int quarter = warp & 3, part = warp >> 2;       // of the accumulators' rows and 32-column parts
    const int row = quarter * 32 + lane;
    const bool roomy = p.blocks <= kRoomyBlocks;
    const uint32_t receive = base + (roomy ? kBeside : kA0);
    const uint32_t x0 = base + (roomy && p.ranks > 1 ? 2 * kBeside : kBeside);
    const uint32_t x1 = x0 + static_cast<uint32_t>(p.blocks) * kColumnBlock;
    auto sync = [&]() {
        if (p.ranks > 1)
            cluster_sync();
        else
            __syncthreads();
    };

    if (threadIdx.x == 0) {
        mbar_init(done, 1);
        mbar_init(drained, 1);
        mbar_init(arrived, 1);
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(&tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    sync(); // also: every CTA of the cluster has started
    tc_fence_after_sync();
    const uint32_t tmem = *static_cast<volatile uint32_t *>(&tmem_slot);

    // ------------------------------------------------ G's columns, twice
    // Eight elements at a time: of a wide G a row's, lane l columns 8 l ..; of
    // a tall one (X is its transpose) a column of X, neighbouring lanes'
    // columns neighbours, so that the transposed stores do not collide.
    const long long g0 = b * p.g.batch_pitch;
    auto visit = [&](auto take) {
        float v[8];
        if (!p.tall) {
            const int j = lane * 8;
            if (j < width)
                for (int i = warp; i < kSmallRows; i += kSmallThreads / 32) {
                    const bool in = i < p.r && col0 + j < p.c;
                    if (in)
                        load8(p.g, g0 + i * p.g.ld, col0 + j, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = in ? v[e] : 0.0f;
                    take(v, i, j);
                }
        } else {
            for (int u = warp; u < p.blocks * 2 * (kSmallRows / 8); u += kSmallThreads / 32) {
                const int i = u % (kSmallRows / 8) * 8, j = u / (kSmallRows / 8) * 32 + lane;
                const bool in = i < p.r && col0 + j < p.c;
                if (in)
                    load8(p.g, g0 + (col0 + j) * p.g.ld, i, v);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = in ? v[e] : 0.0f;
                take(v, i, j);
            }
        }
    };
    Squares sum;
    visit([&](const float (&v)[8], int, int) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum.add(v[e]);
    });
    sum.add_up_warp();
    if (lane == 0)
        warp_sums[warp] = sum.sums();
    __syncthreads();
    if (threadIdx.x < p.ranks) { // this CTA's sums to rank threadIdx.x
        Squares cta;
        for (int w = 0; w < kSmallThreads / 32; ++w)
            cta.add(warp_sums[w]);
        const float4 q = cta.sums();
        if (p.ranks > 1)
            st_cluster_v4(map_to_cta(smem_u32(&rank_sums[rank]), threadIdx.x), __float_as_uint(q.x),
                          __float_as_uint(q.y), __float_as_uint(q.z), __float_as_uint(q.w));
        else
            rank_sums[0] = q;
    }
    sync();
    Squares all;
    for (int k = 0; k < p.ranks; ++k)
        all.add(rank_sums[k]);
    int e2;
    float g = split_scale(all, p.eps, &e2);
    const float s0 = power_of_two(e2 / 2), s1 = power_of_two(e2 - e2 / 2);
    const bool exact = p.g.bf16 != 0; // one plane holds a bfloat16 G
    visit([&](const float (&v)[8], int i, int j) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = v[e] * s0 * s1;
        for (int q = 0; q < (exact ? 1 : 2); ++q) {
            const uint32_t plane = (q == 0 ? x0 : x1) + static_cast<uint32_t>(j / 64) * kColumnBlock;
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[e] = pack_f16(x[2 * e], x[2 * e + 1]);
                const float2 kept = unpack_f16(w[e]);
                x[2 * e] -= kept.x;
                x[2 * e + 1] -= kept.y;
            }
            if (!p.tall) {
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(
                                 plane + static_cast<uint32_t>(i * 128 + ((((j % 64) / 8) ^ (i & 7)) << 4))),
                             "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                             : "memory");
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    asm volatile("st.shared.b16 [%0], %1;\n" ::"r"(
                                     plane + static_cast<uint32_t>((i + e) * 128 + ((((j % 64) / 8) ^ e) << 4) +
                                                                   (j % 8) * 2)),
                                 "h"(static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1))))
                                 : "memory");
            }
        }
    });

    // ------------------------------------------------ the iteration
    uint32_t parity = 0;
    int product = 0;
    bool failed = false;
    // What the threads have written is there for the tensor core; one thread
    // issues the product, all wait for it.  After a wait that ran out nobody
    // waits again and the barriers stay matched.
    auto multiply = [&](auto issue) {
        fence_proxy_async_smem();
        tc_fence_before_sync();
        __syncthreads();
        if (warp == 0) { // one lane's instructions, the warp's addresses
            tc_fence_after_sync();
            issue(lane == 0 ? 1u : 0u);
            if (product != p.withhold) // test hook: this product is never announced
                mma_commit_if(lane == 0 ? 1u : 0u, done);
        }
        ++product;
        __syncwarp();
        if (!failed && !mbar_wait_bounded(done, parity, p.wait_limit_ns)) {
            failed = true;
            record_error(p.status, kErrFamilyOrthogonalize | kErrRoleMma);
        }
        parity ^= 1u;
        tc_fence_after_sync();
        __syncwarp();
    };
    // 32 columns of this thread's row of the accumulator at `column`.
    auto read = [&](int column, unsigned long long (&v)[16]) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(column), r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j)
            v[j] = pair(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
    };
    // v alpha + diag I, for columns part * 32 .. of a 128 x 128 matrix.
    auto scale = [&](unsigned long long (&v)[16], float alpha, float diag) {
        const unsigned long long a = pair(alpha, alpha);
        const int at = row < p.r ? row - part * 32 : -1; // where the diagonal is among these columns
#pragma unroll
        for (int j = 0; j < 16; ++j)
            v[j] = fma2(v[j], a, pair(2 * j == at ? diag : 0.0f, 2 * j + 1 == at ? diag : 0.0f));
    };
    const int k_blocks = p.r > 64 ? 2 : 1; // of A and Q
    // Descriptors of the first block; others add to the address field
    // (16-byte units).  K-major: a K step is 32 bytes, a K block 16 KiB; the
    // MN-major right operand of Q X: 16 rows and 64 rows of 128 bytes.
    constexpr uint64_t kBlockStep = kColumnBlock >> 4, kStep = 32 >> 4, kRowStep = (16 * 128) >> 4;
    const uint64_t k_major = smem_desc_sw128(base, 16, 1024), mn_major = smem_desc_sw128(base, kColumnBlock, 1024);
    const uint32_t square_form = instruction(128, false), result_form = instruction(width, true);
    auto square_pass = [&](uint32_t on, uint32_t left, uint32_t right, int blocks, bool first) {
        uint64_t l = k_major + ((left - base) >> 4), q = k_major + ((right - base) >> 4);
        for (int kb = 0; kb < blocks; ++kb, l += kBlockStep, q += kBlockStep) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_f16_ss_if(on, tmem, l + ks * kStep, q + ks * kStep, square_form,
                              !first || kb != 0 || ks != 0 ? 1u : 0u);
        }
    };
    constexpr int kResult = 128; // accumulator of Q X, beside that of X X^T and the square
    auto result_pass = [&](uint32_t on, uint32_t left, uint32_t right, bool first) {
        uint64_t l = k_major + ((left - base) >> 4), q = mn_major + ((right - base) >> 4);
        for (int kb = 0; kb < k_blocks; ++kb, l += kBlockStep, q += 4 * kRowStep) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_f16_ss_if(on, tmem + kResult, l + ks * kStep, q + ks * kRowStep, result_form,
                              !first || kb != 0 || ks != 0 ? 1u : 0u);
        }
    };

    for (int step = 0; step < p.steps; ++step) {
        const float ca = p.coefficients[3 * step], cb = p.coefficients[3 * step + 1],
                    cc = p.coefficients[3 * step + 2];
        const bool first = step == 0, last = step == p.steps - 1;
        const Factors f = step_factors(g, p.slow[step]);
        unsigned long long v[16];
        uint32_t w[16];

        // X X^T, over all ranks' columns.
        multiply([&](uint32_t on) { square_pass(on, x0, x0, p.blocks, true); });
        read(part * 32, v);
        // Ranks own 128 / ranks columns' worth of rows: strips of 32 rows by
        // 64 columns, eight of them, two warps each.
        const int strip = quarter * 2 + part / 2, owner = strip * p.ranks / 8;
        if (p.ranks > 1) {
            const uint32_t mine = static_cast<uint32_t>(strip % (8 / p.ranks) * 2 + (part & 1));
            const uint32_t slots = receive + mine * static_cast<uint32_t>(p.ranks) * kUnit;
            if (!roomy)
                cluster_sync(); // no rank still multiplies by the Q that lies there
            if (owner != rank) {
                const uint32_t to = map_to_cta(slots + static_cast<uint32_t>(rank) * kUnit,
                                               static_cast<uint32_t>(owner)) + static_cast<uint32_t>(lane) * 16u;
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    float q0, q1, q2, q3;
                    split(v[j], q0, q1);
                    split(v[j + 1], q2, q3);
                    st_cluster_v4(to + static_cast<uint32_t>(j) * 256u, __float_as_uint(q0), __float_as_uint(q1),
                                  __float_as_uint(q2), __float_as_uint(q3));
                }
            }
            cluster_sync(); // also: no rank still multiplies by Q
            if (owner == rank) {
                for (int src = 0; src < p.ranks; ++src) {
                    if (src == rank)
                        continue;
                    const uint8_t *from = smem_raw + (slots - raw) + src * kUnit + lane * 16;
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float4 q = *reinterpret_cast<const float4 *>(from + j * 256);
                        v[j] = add2(v[j], pair(q.x, q.y));
                        v[j + 1] = add2(v[j + 1], pair(q.z, q.w));
                    }
                }
            }
            if (!roomy)
                cluster_sync(); // the sums have been taken: A (or Q) may lie there
            if (threadIdx.x == 0) // the strips the other ranks send, both planes
                mbar_arrive_expect_tx(arrived, static_cast<uint32_t>(8 - 8 / p.ranks) * 2u * kStrip);
        }
        if (cc != 0.0f)
            scale(v, kScaleA / (kScaleX * kScaleX) * f.g * f.g, kScaleA * (cb / (2.0f * cc)));
        else
            scale(v, kScaleQ * cb / (kScaleX * kScaleX) * f.g * f.g * f.rho, kScaleQ * ca * f.rho);
        const uint32_t row_at = static_cast<uint32_t>(part / 2) * kColumnBlock + static_cast<uint32_t>(row) * 128u;
        if (owner == rank) {
            for (int q = 0; q < 2; ++q) {
                make_plane(v, w);
                store_plane(base + (q == 0 ? kA0 : kA1) + row_at, lane, part & 1, w);
            }
        }
        if (p.ranks > 1) {
            // Each strip, 4 KiB in one piece, to every other rank.
            fence_proxy_async_smem();
            __syncthreads();
            if (owner == rank && (part & 1) == 0 && lane < 2 * p.ranks) {
                const uint32_t at = base + (lane & 1 ? kA1 : kA0) + static_cast<uint32_t>(part / 2) * kColumnBlock +
                                    static_cast<uint32_t>(quarter * 32) * 128u;
                const uint32_t to = static_cast<uint32_t>(lane / 2);
                if (to != static_cast<uint32_t>(rank))
                    bulk_copy_to_cta(map_to_cta(at, to), at, kStrip, map_to_cta(arrived, to));
            }
            // Also after a product's wait ran out: no rank leaves before the
            // copies to it have landed.
            if (!mbar_wait_bounded(arrived, static_cast<uint32_t>(step & 1), p.wait_limit_ns) && !failed) {
                failed = true;
                record_error(p.status, kErrFamilyOrthogonalize | kErrRoleConsumer);
            }
            cluster_arrive(); // this rank has them: the copies to it no longer read their source
        }

        if (cc != 0.0f) {
            // The square, in every rank, and Q in A's place.
            multiply([&](uint32_t on) {
                square_pass(on, base + kA1, base + kA0, k_blocks, true);
                square_pass(on, base + kA0, base + kA1, k_blocks, false);
                square_pass(on, base + kA0, base + kA0, k_blocks, false);
            });
            read(part * 32, v);
            scale(v, kScaleQ * cc / (kScaleA * kScaleA) * f.rho,
                  kScaleQ * static_cast<float>(ca - static_cast<double>(cb) * cb / (4.0 * cc)) * f.rho);
            if (p.ranks > 1)
                cluster_wait(); // before Q replaces the strips this rank has sent
            for (int q = 0; q < 2; ++q) {
                make_plane(v, w);
                store_plane(base + (q == 0 ? kA0 : kA1) + row_at, lane, part & 1, w);
            }
        } else if (p.ranks > 1) {
            cluster_wait();
        }

        // Q X: this rank's columns, in X's place or to the result.
        multiply([&](uint32_t on) {
            result_pass(on, base + kA1, x0, true);
            if (!last && !(first && exact))
                result_pass(on, base + kA0, x1, false);
            result_pass(on, base + kA0, x0, false);
        });
        for (int k = part; k < 2 * p.blocks; k += 4) { // 32 columns each
            read(kResult + k * 32, v);
            const float alpha = last ? 1.0f / (kScaleQ * kScaleX) * g : 1.0f / kScaleQ;
            const unsigned long long a2 = pair(alpha, alpha);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                v[j] = mul2(v[j], a2);
            if (!last) {
                for (int q = 0; q < 2; ++q) {
                    make_plane(v, w);
                    store_plane((q == 0 ? x0 : x1) + static_cast<uint32_t>(k / 2) * kColumnBlock +
                                    static_cast<uint32_t>(row) * 128u, lane, k & 1, w);
                }
            } else if (row < p.r) {
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + b * p.out_batch;
                const int j0 = col0 + k * 32;
                if (p.tall) { // neighbouring lanes write neighbours
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        float lo, hi;
                        split(v[j / 2], lo, hi);
                        if (j0 + j < p.c)
                            out[(j0 + j) * p.ldo + row] = __float2bfloat16_rn(j & 1 ? hi : lo);
                    }
                } else {
                    __nv_bfloat16 *o = out + row * p.ldo + j0;
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        float q[8];
#pragma unroll
                        for (int e = 0; e < 8; e += 2)
                            split(v[(j + e) / 2], q[e], q[e + 1]);
                        if (p.out_vec && j0 + j + 8 <= p.c) {
                            *reinterpret_cast<uint4 *>(o + j) =
                                make_uint4(pack_bf16(q[0], q[1]), pack_bf16(q[2], q[3]), pack_bf16(q[4], q[5]),
                                           pack_bf16(q[6], q[7]));
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (j0 + j + e < p.c)
                                    o[j + e] = __float2bfloat16_rn(q[e]);
                        }
                    }
                }
            }
        }
    }

    // Every product has finished before tensor memory is freed, and no rank
    // leaves while another may still write to it.
    if (threadIdx.x == 0) {
        mma_commit(drained);
        if (!mbar_wait_bounded(drained, 0, p.wait_limit_ns))
            record_error(p.status, kErrFamilyOrthogonalize | kErrRoleDrain);
    }
    __syncwarp();
    tc_fence_before_sync();
    sync();
    tc_fence_after_sync();
    if (warp == 0)
        tmem_dealloc(tmem, 512);
}

// CTAs of a matrix whose longer side is c, and 64-column blocks of each.  A
// cluster whose CTAs hold at most three blocks saves two meetings a step: one
// 128 x 1024 matrix takes 71.9 us on eight CTAs, 78.1 on four.  So a cluster
// grows to that where all matrices still run at once; 64 such matrices, which
// would take five rounds of eight CTAs, take 361 us so and 167 on four.
static int ranks_for(int c, int batch, const Device &d, int *blocks)
{
    int ranks = 1;
    while (ranks < kMaxRanks && c > ranks * kSlab)
        ranks *= 2;
    int more = ranks;
    while (more > 1 && more < kMaxRanks && c > more * kRoomyBlocks * 64)
        more *= 2;
    if (more > ranks && batch <= cluster_room(more, d))
        ranks = more;
    *blocks = (c + 64 * ranks - 1) / (64 * ranks);
    return ranks;
}

bool fits_small(int m, int n, int out_dtype)
{
    const int r = std::min(m, n), c = std::max(m, n);
    return out_dtype == GEMM_DTYPE_BF16 && r <= kSmallRows && c <= kMaxRanks * kSlab;
}

int run_small(const Call &call, const Device &d, unsigned int *status, cudaStream_t s)
{
    Small p = {};
    p.g = call.matrix();
    p.r = std::min(call.m, call.n);
    p.c = std::max(call.m, call.n);
    p.tall = call.m > call.n;
    p.ranks = ranks_for(p.c, call.batch, d, &p.blocks);
    p.out = call.out;
    p.ldo = call.ldo;
    p.out_batch = call.o_batch;
    p.out_vec = (reinterpret_cast<uintptr_t>(call.out) & 15u) == 0 && call.ldo % 8 == 0 &&
                (call.batch == 1 || call.o_batch % 8 == 0);
    p.steps = call.steps;
    p.eps = call.eps;
    p.status = status;
    p.wait_limit_ns = call_wait_limit_ns();
    p.withhold = call_withhold();
    for (int k = 0; k < 3 * call.steps; ++k)
        p.coefficients[k] = call.coefficients[k];
    for (int k = 0; k < call.steps; ++k)
        p.slow[k] = slow_step(call.coefficients + 3 * k);
    static std::atomic<unsigned long long> limit_set[kMaxDevices];
    if (ensure_smem_limit(small_kernel, kSmallSmem, d.index, d.ctx, limit_set) != GEMM_OK)
        return GEMM_ERR_CUDA;
    return launch(small_kernel, dim3(static_cast<unsigned>(call.batch * p.ranks)), kSmallThreads, kSmallSmem, false,
                  p.ranks, s, p);
}

} // namespace orth

} // namespace pg
