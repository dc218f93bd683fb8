// The gated projection h = act(x Wg) * (x Wu) and its gradient.
//
//   G = x Wg, U = x Wu, h = act(G) U
//   dG = dh U act'(G), dU = dh act(G)
//   dx = dG Wg^T + dU Wu^T,  dWg = x^T dG,  dWu = x^T dU
//
// Both are products on the tensor cores (pair_product.cuh) and bound by their
// rate from a few hundred rows on.  Forward: a tile's 256 columns are 128 of Wg
// and the same 128 of Wu, one loaded by each CTA of the pair, so that the
// epilogue finds G and U of an element in one lane's tensor memory and G and U
// never leave the chip unless they are to be kept.  Backward: one pass over
// dh, gate and up makes dG and dU, then one launch computes all three products:
// dx with two segments of K blocks (dG Wg^T, then dU Wu^T, one sum), dWg and
// dWu as one product whose tile takes 128 columns of each.
//
// Measured, call after call for seconds, where the power limit holds: 8192 x 4096 ->
// 8192 in 667 us (1.65 PFLOP/s), 698 with G and U kept, where a library product of that
// size takes 622; its gradient in 1500 (2.2 TFLOP; 95 us of them dG and dU, 7 TB/s),
// where library products of its sizes take 1305.  In a burst of six calls 604, 630
// (570), 1370 (1196).  One token 23 us on the device, 5.8 TB/s of the weights.
#include <algorithm>
#include <cstdint>
#include <cstring>

#include "few_rows.cuh"
#include "pair_product.cuh"
#include "pipelined_ffn.h"

namespace pg {
namespace gated {

using namespace pair_product;

// ------------------------------------------------------------- activations
// The fast exponential and reciprocal: their few units in float32's last place
// do not reach a bfloat16 result.  The exponential is taken of -|v|, which
// cannot overflow, so that the far tail keeps its precision down to float32's
// subnormal numbers.
__device__ __forceinline__ float reciprocal(float v)
{
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float sigmoid(float v)
{
    const float z = __expf(-fabsf(v));
    return (v >= 0.0f ? 1.0f : z) * reciprocal(1.0f + z);
}

// The normal distribution's function, given e = exp(-g^2 / 2): with z = |g| /
// sqrt 2, its tail is exp(-z^2) times erfc(z) exp(z^2) / 2 = t Q(t), t = 1 / (1 +
// 0.3 z).  Q is a polynomial of degree 8 fitted to that function (least relative
// error over z from 0 to 14: 4e-8, in float32 9 units), so the tail keeps its
// relative precision, where 1 + erf cancels.  normcdff takes twice the
// instructions, and this shares the exponential with the density: the slopes of
// 1000 x 2700 went from 11.4 to 7 us.
__device__ __forceinline__ float normal(float g, float e)
{
    const float t = reciprocal(fmaf(0.3f * 0.70710678f, fabsf(g), 1.0f));
    float q = -0.0633113384f;
    q = fmaf(q, t, 0.235927477f);
    q = fmaf(q, t, -0.242374599f);
    q = fmaf(q, t, 0.258556098f);
    q = fmaf(q, t, -0.037045639f);
    q = fmaf(q, t, 0.10320121f);
    q = fmaf(q, t, 0.0752323121f);
    q = fmaf(q, t, 0.0852121413f);
    q = fmaf(q, t, 0.0846023634f);
    const float tail = e * (t * q);
    return g < 0.0f ? tail : 1.0f - tail;
}

constexpr float kTanhScale = 0.7978845608028654f; // sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;

template <int Act>
__device__ __forceinline__ float activate(float g)
{
    if constexpr (Act == GEMM_ACT_SILU)
        return g * sigmoid(g);
    else if constexpr (Act == GEMM_ACT_GELU)
        return g * normal(g, __expf(-0.5f * g * g));
    else
        // (1 + tanh z) / 2 = sigmoid(2 z)
        return g * sigmoid(2.0f * kTanhScale * g * fmaf(kTanhCubic * g, g, 1.0f));
}

// act(g) and act'(g).
template <int Act>
__device__ __forceinline__ void activate_with_slope(float g, float &value, float &slope)
{
    if constexpr (Act == GEMM_ACT_SILU) {
        const float s = sigmoid(g);
        value = g * s;
        slope = fmaf(value, 1.0f - s, s);
    } else if constexpr (Act == GEMM_ACT_GELU) {
        const float e = __expf(-0.5f * g * g), c = normal(g, e);
        value = g * c;
        slope = fmaf(g * 0.3989422804014327f, e, c);
    } else {
        const float s = sigmoid(2.0f * kTanhScale * g * fmaf(kTanhCubic * g, g, 1.0f));
        value = g * s;
        // Beyond 32 the first factor is zero; the other one's g^2 is kept finite for it.
        const float c = fminf(fabsf(g), 32.0f);
        slope = fmaf(value * (1.0f - s), 2.0f * kTanhScale * fmaf(3.0f * kTanhCubic * c, c, 1.0f), s);
    }
}

// ----------------------------------------------------------------- forward
struct Forward {
    Launch launch;
    __nv_bfloat16 *h, *gate, *up;
    long long ldh, ldgate, ldup;
    int h_access, gate_access, up_access;
};

template <int Act>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gated_forward_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Forward p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = align_smem(smem_u32(smem_raw), 1024);
    const Barriers b(base + kStages * kStageBytes);
    run<kMmaF16, false, 0, false>(p.launch, maps, base, b, [&](uint32_t tmem, int rank, int first, int stride) {
        const int warp = threadIdx.x / 32;
        const int quarter = warp & 3, part = (warp - kFirstEpilogueWarp) / 4;
        const uint32_t empty = map_to_cta(b.acc_empty, 0);
        const Product &product = p.launch.product[0];
        unsigned acc = 0;
        for (int t = first; t < p.launch.units; t += stride, ++acc) {
            if (!acquire(p.launch, b, acc))
                break;
            const Tile tile = tile_at(product, t);
            const long long row0 = tile.mb * kRows + rank * 128 + quarter * 32;
            const uint32_t at = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + (acc & 1u) * kCols;
#pragma unroll 1
            for (int c = part * 2; c < part * 2 + 2; ++c) {
                const int col = tile.nb * 128 + c * 32;
                uint32_t g[32], u[32];
                __syncwarp();
                tmem_ld_32x32b_x32(at + c * 32, g);
                tmem_ld_32x32b_x32(at + 128 + c * 32, u);
                tmem_ld_wait();
                if (c % 2 == 1)
                    release(empty, acc); // all of it is in registers
                if (row0 >= product.rows || col >= product.cols)
                    continue; // warp-uniform
                float v[32];
                if (p.gate) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = __uint_as_float(g[j]);
                    store_tile(p.gate, p.ldgate, row0, product.rows, col, product.cols, v, p.gate_access);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = __uint_as_float(u[j]);
                    store_tile(p.up, p.ldup, row0, product.rows, col, product.cols, v, p.up_access);
                }
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    v[j] = activate<Act>(__uint_as_float(g[j])) * __uint_as_float(u[j]);
                store_tile(p.h, p.ldh, row0, product.rows, col, product.cols, v, p.h_access);
            }
        }
    }, [](int, int, int) {});
}

// ------------------------------------------------------ forward of few rows
struct ForwardFew {
    few_rows::Launch launch;
    int activation;
    __nv_bfloat16 *h, *gate, *up;
    long long ldh, ldgate, ldup;
};

template <int Tokens>
__global__ void __launch_bounds__(few_rows::kThreads, 2)
    gated_few_rows_kernel(const __grid_constant__ few_rows::Maps maps, const __grid_constant__ ForwardFew p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = align_smem(smem_u32(smem_raw), 1024);
    few_rows::run<kMmaF16, Tokens>(
        p.launch, maps, base,
        [&](uint32_t tmem, const auto &b, int, int, int token0, int, auto put) {
            const bool ok = mbar_wait_bounded(b.acc_full, 0, p.launch.wait_limit_ns);
            if (!__all_sync(0xffffffffu, ok)) {
                if (threadIdx.x % 32 == 0)
                    record_error(p.launch.status, p.launch.family | kErrRoleEpilogue);
                return;
            }
            tc_fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < 2 * Tokens; c += 16) {
                if (token0 + c % Tokens >= p.launch.rows)
                    continue; // warp-uniform
                uint32_t r[16];
                tmem_ld_32x32b_x16(tmem + static_cast<uint32_t>(c), r);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    put(c + j, __uint_as_float(r[j]));
            }
        },
        [&](int token, int feature, const float(&sum)[2]) {
            const float g = sum[0], u = sum[1];
            if (p.gate) {
                p.gate[token * p.ldgate + feature] = __float2bfloat16_rn(g);
                p.up[token * p.ldup + feature] = __float2bfloat16_rn(u);
            }
            const float a = p.activation == GEMM_ACT_SILU   ? activate<GEMM_ACT_SILU>(g)
                            : p.activation == GEMM_ACT_GELU ? activate<GEMM_ACT_GELU>(g)
                                                            : activate<GEMM_ACT_GELU_TANH>(g);
            p.h[token * p.ldh + feature] = __float2bfloat16_rn(a * u);
        });
}

// ---------------------------------------------------------------- backward
struct Slopes {
    int rows, hidden;
    const __nv_bfloat16 *dh, *gate, *up;
    long long lddh, ldgate, ldup;
    __nv_bfloat16 *dgate, *dup;
    long long pitch; // of dgate and dup, a multiple of 8
    unsigned int *arrived; // counters of the products' cut tiles, set to zero here
    int counters;
};

// dG and dU, eight columns a thread, computed in float32 and rounded to bfloat16: they
// are operands of the tensor cores.  With the result's own rounding a gradient is off
// by 0.0024 of its norm, where one rounding alone gives 0.0017.
constexpr int kSlopeThreads = 256;

// Eight elements in pieces of Bytes, to which their address is aligned.
template <int Bytes>
__device__ __forceinline__ void load8(const __nv_bfloat16 *from, float (&v)[8])
{
    if constexpr (Bytes == 16) {
        Vec16<__nv_bfloat16>::unpack(__ldcs(reinterpret_cast<const uint4 *>(from)), v);
    } else if constexpr (Bytes == 8) {
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            const uint2 q = __ldcs(reinterpret_cast<const uint2 *>(from + e));
            unpack_bf16(q.x, v + e);
            unpack_bf16(q.y, v + e + 2);
        }
    } else if constexpr (Bytes == 4) {
#pragma unroll
        for (int e = 0; e < 8; e += 2)
            unpack_bf16(__ldcs(reinterpret_cast<const unsigned int *>(from + e)), v + e);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = to_f32(from[e]);
    }
}

// Bytes: what the rows of dh, gate and up are all aligned to.
template <int Act, int Bytes>
__global__ void __launch_bounds__(kSlopeThreads) slopes_kernel(const Slopes p)
{
    grid_launch_next(); // the products' CTAs start as these leave, and wait for the last
    for (int i = blockIdx.x * kSlopeThreads + threadIdx.x; i < p.counters; i += gridDim.x * kSlopeThreads)
        p.arrived[i] = 0;
    const int pieces = (p.hidden + 7) / 8;
    const long long total = static_cast<long long>(p.rows) * pieces;
    for (long long i = blockIdx.x * static_cast<long long>(kSlopeThreads) + threadIdx.x; i < total;
         i += static_cast<long long>(gridDim.x) * kSlopeThreads) {
        const long long row = i / pieces;
        const int col = static_cast<int>(i - row * pieces) * 8;
        float d[8], g[8], u[8];
        const __nv_bfloat16 *pd = p.dh + row * p.lddh + col, *pgt = p.gate + row * p.ldgate + col,
                            *pu = p.up + row * p.ldup + col;
        if (col + 8 <= p.hidden) {
            load8<Bytes>(pd, d);
            load8<Bytes>(pgt, g);
            load8<Bytes>(pu, u);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool in = col + e < p.hidden;
                d[e] = in ? to_f32(pd[e]) : 0.0f;
                g[e] = in ? to_f32(pgt[e]) : 0.0f;
                u[e] = in ? to_f32(pu[e]) : 0.0f;
            }
        }
        float dg[8], du[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float value, slope;
            activate_with_slope<Act>(g[e], value, slope);
            dg[e] = d[e] * u[e] * slope;
            du[e] = d[e] * value;
        }
        // The pitch leaves room for a last piece's columns beyond `hidden`,
        // which the products do not read.
        *reinterpret_cast<uint4 *>(p.dgate + row * p.pitch + col) = Vec16<__nv_bfloat16>::pack(dg);
        *reinterpret_cast<uint4 *>(p.dup + row * p.pitch + col) = Vec16<__nv_bfloat16>::pack(du);
    }
}

struct Results {
    __nv_bfloat16 *out[2]; // of a dual product's halves (else the first)
    long long ld[2];
    int access[2];
    // Of tiles whose K blocks are cut: float32 sums of each unit, and how many of
    // a tile's units have left theirs, for each epilogue warp of the pair.
    float4 *partial;
    unsigned int *arrived;
};

struct Backward {
    Launch launch;
    Results results[kMaxProducts];
};

constexpr int kWarpsOfPair = 2 * kEpilogueWarps;
constexpr int kPartialQuads = 32 * 128 / 4; // of a warp's 32 x 128 sums

// A unit's sums come to memory, and the warp that is last at its part of the
// tile adds up all units' in their order: the same sums whichever is last.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gated_backward_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Backward p)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = align_smem(smem_u32(smem_raw), 1024);
    const Barriers b(base + kStages * kStageBytes);
    run<kMmaF16, false, 0, false>(p.launch, maps, base, b, [&](uint32_t tmem, int rank, int first, int stride) {
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        const int quarter = warp & 3, part = (warp - kFirstEpilogueWarp) / 4;
        const int warp_of_pair = rank * kEpilogueWarps + warp - kFirstEpilogueWarp;
        const uint32_t empty = map_to_cta(b.acc_empty, 0);
        unsigned acc = 0;
        for (int t = first; t < p.launch.units; t += stride, ++acc) {
            if (!acquire(p.launch, b, acc))
                break;
            const Unit unit = unit_at(p.launch, t);
            const Product &product = p.launch.product[unit.which];
            const Tile tile = tile_at(product, unit.tile);
            const Results &to = p.results[unit.which];
            const int half = product.dual ? part : 0, splits = product.splits;
            const long long row0 = tile.mb * kRows + rank * 128 + quarter * 32;
            const int col0 = product.dual ? tile.nb * 128 : tile.nb * kCols + part * 128;
            const uint32_t at = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + (acc & 1u) * kCols + part * 128;
            float4 *const parts = to.partial + static_cast<size_t>(unit.tile) * splits * kWarpsOfPair * kPartialQuads +
                                  static_cast<size_t>(warp_of_pair) * kPartialQuads + lane;
            bool last = true;
            if (splits > 1) {
                float4 *const mine = parts + static_cast<size_t>(unit.split) * kWarpsOfPair * kPartialQuads;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(at + c * 32, r);
                    tmem_ld_wait();
                    if (c == 3)
                        release(empty, acc);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        __stcg(mine + (c * 8 + j) * 32,
                               make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                                           __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3])));
                }
                __threadfence();
                __syncwarp();
                unsigned int before = 0;
                if (lane == 0)
                    before = atomicAdd(to.arrived + unit.tile * kWarpsOfPair + warp_of_pair, 1u);
                last = __shfl_sync(0xffffffffu, before, 0) == static_cast<unsigned int>(splits - 1);
                __threadfence();
            }
            if (!last)
                continue;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                const int col = col0 + c * 32;
                float v[32];
                __syncwarp();
                if (splits > 1) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = 0.0f;
                    // The sums of kAtOnce units are on their way together: one at
                    // a time, a unit's way from L2 was waited for 4 * splits times.
                    constexpr int kAtOnce = 3;
#pragma unroll 1
                    for (int k = 0; k < splits; k += kAtOnce) {
                        float4 q[kAtOnce][8];
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                q[i][j] = __ldcg(parts +
                                                 static_cast<size_t>(min(k + i, splits - 1)) * kWarpsOfPair *
                                                     kPartialQuads +
                                                 (c * 8 + j) * 32);
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i)
                            if (k + i < splits) {
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    v[4 * j] += q[i][j].x;
                                    v[4 * j + 1] += q[i][j].y;
                                    v[4 * j + 2] += q[i][j].z;
                                    v[4 * j + 3] += q[i][j].w;
                                }
                            }
                    }
                } else {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(at + c * 32, r);
                    tmem_ld_wait();
                    if (c == 3)
                        release(empty, acc); // all of it is in registers
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = __uint_as_float(r[j]);
                }
                if (row0 >= product.rows || col >= product.cols)
                    continue; // warp-uniform
                store_tile(to.out[half], to.ld[half], row0, product.rows, col, product.cols, v, to.access[half]);
            }
        }
    }, [](int, int, int) {});
}

// -------------------------------------------------------------------- host
constexpr int kMaxSide = 1 << 30;
constexpr int kSmem = smem_bytes(0);

struct Device {
    int index, sms;
    unsigned long long ctx;
    unsigned int *status;
};

int enter(Device *d)
{
    const int st = device_checked(&d->index);
    if (st != GEMM_OK)
        return st;
    d->sms = device_sms();
    d->ctx = current_context_id();
    d->status = device_status_word(d->index, d->ctx);
    return d->status ? GEMM_OK : GEMM_ERR_CUDA;
}

long long tiles_of(long long rows, long long cols, int tile_cols)
{
    return (rows + kRows - 1) / kRows * ((cols + tile_cols - 1) / tile_cols);
}

// Sizes whose tiles, and pieces of a row, are counted in an int.
int check_sizes(int rows, int width, int hidden)
{
    if (rows < 0 || width < 0 || hidden < 0)
        return GEMM_ERR_INVALID_ARG;
    if (rows > kMaxSide || width > kMaxSide || hidden > kMaxSide)
        return GEMM_ERR_UNSUPPORTED;
    const long long most = 1ll << 30;
    if (tiles_of(rows, hidden, 128) > most || tiles_of(rows, width, kCols) + tiles_of(width, hidden, 128) > most)
        return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

bool odd(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 1u) != 0; }

// An operand that TMA reads.
int check_operand(const void *p, int rows, int cols, long long pitch)
{
    if (!p || (rows > 1 && pitch < cols))
        return GEMM_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0 || (rows > 1 && pitch % 8 != 0))
        return GEMM_ERR_MISALIGNED;
    return GEMM_OK;
}

int check_plain(const void *p, int rows, int cols, long long pitch)
{
    if (!p || (rows > 1 && pitch < cols))
        return GEMM_ERR_INVALID_ARG;
    return odd(p) ? GEMM_ERR_MISALIGNED : GEMM_OK;
}

int zero_matrix(void *p, int rows, int cols, long long pitch, cudaStream_t s)
{
    const size_t row = static_cast<size_t>(cols) * 2;
    return cudaMemset2DAsync(p, rows > 1 ? static_cast<size_t>(pitch) * 2 : row, 0, row, rows, s) == cudaSuccess
               ? GEMM_OK
               : GEMM_ERR_CUDA;
}

Launch make_launch(const Device &d)
{
    Launch l = {};
    l.family = kErrFamilyGated;
    l.status = d.status;
    l.wait_limit_ns = call_wait_limit_ns();
    l.withhold = call_withhold();
    return l;
}

Product make_product(int rows, int cols, int k, int segments, int dual, Layout a, Layout b, int a_map, int b_map)
{
    Product p = {};
    p.splits = 1;
    p.rows = rows;
    p.cols = cols;
    p.tiles_m = (rows + kRows - 1) / kRows;
    p.tiles_n = (cols + (dual ? 128 : kCols) - 1) / (dual ? 128 : kCols);
    p.blocks = (k + 63) / 64;
    p.segments = segments;
    p.dual = dual;
    p.a_layout = a;
    p.b_layout = b;
    p.a_map = a_map;
    p.b_map = b_map;
    p.idesc = instruction(1, 1, a, b); // bfloat16
    return p;
}

// One pair per two SMs, or one per unit where there are fewer.
int grid_of(int units, const Device &d) { return 2 * std::max(1, std::min(units, d.sms / 2)); }

template <int Act>
int launch_forward(const Maps &maps, const Forward &p, const Device &d, cudaStream_t s)
{
    static std::atomic<unsigned long long> limit_set[kMaxDevices];
    if (ensure_smem_limit(gated_forward_kernel<Act>, kSmem, d.index, d.ctx, limit_set) != GEMM_OK)
        return GEMM_ERR_CUDA;
    gated_forward_kernel<Act><<<grid_of(p.launch.units, d), kThreads, kSmem, s>>>(maps, p);
    return cudaGetLastError() == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

// Of few_rows::faster; more than 32 tokens go in tiles of 32 (of 64: 27 us for 64
// x 2000 -> 5461 where these take 21).
constexpr few_rows::Times kTimes{0.5, 5.0, 0.31};

template <int Tokens>
int launch_few(const few_rows::Maps &maps, ForwardFew &p, const Device &d, cudaStream_t s)
{
    using S = few_rows::Shape<kMmaF16, Tokens>;
    static std::atomic<unsigned long long> limit_set[kMaxDevices];
    if (ensure_smem_limit(gated_few_rows_kernel<Tokens>, S::kSmem, d.index, d.ctx, limit_set) != GEMM_OK)
        return GEMM_ERR_CUDA;
    few_rows::Launch &l = p.launch;
    l.blocks = (l.blocks + S::kBlockK - 1) / S::kBlockK;
    l.feature_tiles = (l.features + few_rows::kFeatures - 1) / few_rows::kFeatures;
    const long long tiles = static_cast<long long>(l.feature_tiles) * ((l.rows + Tokens - 1) / Tokens);
    l.ranks = few_rows::ranks_for(tiles, l.blocks, d.sms);
    l.weight_mn = 1;
    l.idesc = few_rows::instruction(1, 1, 1, Tokens);
    return few_rows::launch(gated_few_rows_kernel<Tokens>, static_cast<unsigned>(tiles * l.ranks), l.ranks, S::kSmem, s,
                            maps, p);
}

template <int Act>
int launch_slopes(const Slopes &p, const Device &d, cudaStream_t s)
{
    const long long threads = static_cast<long long>(p.rows) * ((p.hidden + 7) / 8);
    const long long blocks = std::min<long long>((threads + kSlopeThreads - 1) / kSlopeThreads, 64ll * d.sms);
    const unsigned grid = static_cast<unsigned>(blocks);
    uintptr_t low = reinterpret_cast<uintptr_t>(p.dh) | reinterpret_cast<uintptr_t>(p.gate) |
                    reinterpret_cast<uintptr_t>(p.up);
    if (p.rows > 1)
        low |= static_cast<uintptr_t>(p.lddh | p.ldgate | p.ldup) * 2u;
    if ((low & 15u) == 0)
        slopes_kernel<Act, 16><<<grid, kSlopeThreads, 0, s>>>(p);
    else if ((low & 7u) == 0)
        slopes_kernel<Act, 8><<<grid, kSlopeThreads, 0, s>>>(p);
    else if ((low & 3u) == 0)
        slopes_kernel<Act, 4><<<grid, kSlopeThreads, 0, s>>>(p);
    else
        slopes_kernel<Act, 2><<<grid, kSlopeThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

bool valid_activation(int a) { return a >= GEMM_ACT_SILU && a <= GEMM_ACT_GELU_TANH; }

// Cuts the tiles' K blocks where there are too few tiles to keep the pairs
// equally busy.  Every pair takes the units its own number of pairs apart; the
// one with most work, a block's time to begin each unit, and what the last pair
// at a cut tile has to add up (in blocks' time, 0.31 us: a unit's sums are 128 KiB
// for each CTA, and come back from L2 in about 1.1 us) are what a choice costs.
// 1000 x 1000 -> 2700: dx has 16 tiles of 86 blocks and the weights' gradients 88
// of 16; with dx cut in four 34 us, whole 49.
constexpr int kMaxSplits = 16;
constexpr int kLeastBlocks = 8; // of a unit

double cost_of(const Product *product, int products, int pairs, const int (&splits)[kMaxProducts])
{
    long long units[kMaxProducts] = {};
    double time[kMaxProducts] = {}, tail = 0.0;
    for (int k = 0; k < products; ++k) {
        units[k] = static_cast<long long>(product[k].tiles()) * splits[k];
        time[k] = static_cast<double>(product[k].blocks) * product[k].segments / splits[k] + 1.0;
        if (splits[k] > 1)
            tail = std::max(tail, 6.0 + 3.5 * splits[k]);
    }
    const int longer = time[0] >= time[1] ? 0 : 1; // its units come first
    const long long u0 = units[longer], all = units[0] + units[1];
    double most = 0.0;
    // The counts change only where either product's units end.
    for (const long long i : {0ll, u0 % pairs, all % pairs}) {
        const long long n0 = u0 > i ? (u0 - 1 - i) / pairs + 1 : 0, n = all > i ? (all - 1 - i) / pairs + 1 : 0;
        most = std::max(most, n0 * time[longer] + (n - n0) * time[1 - longer]);
    }
    return most + tail;
}

void cut(Product *product, int products, int sms)
{
    const int pairs = std::max(1, sms / 2);
    long long work = 0, longest = 0;
    for (int k = 0; k < products; ++k) {
        const long long blocks = static_cast<long long>(product[k].blocks) * product[k].segments;
        work += product[k].tiles() * blocks;
        longest = std::max(longest, blocks);
    }
    if (work >= 4 * longest * pairs)
        return; // no unit is more than a quarter of a pair's share
    static const int tried[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, kMaxSplits};
    int best[kMaxProducts] = {1, 1};
    double least = cost_of(product, products, pairs, best);
    for (const int s0 : tried)
        for (const int s1 : tried) {
            if ((products < 2 && s1 > 1) || (s0 > 1 && product[0].blocks * product[0].segments < kLeastBlocks * s0) ||
                (s1 > 1 && product[1].blocks * product[1].segments < kLeastBlocks * s1))
                continue;
            const int splits[kMaxProducts] = {s0, s1};
            const double c = cost_of(product, products, pairs, splits);
            if (c < least) {
                least = c;
                best[0] = s0;
                best[1] = s1;
            }
        }
    for (int k = 0; k < products; ++k)
        product[k].splits = best[k];
}

// Counters and sums of a product's cut tiles.
size_t counters_of(const Product &p) { return p.splits > 1 ? static_cast<size_t>(p.tiles()) * kWarpsOfPair : 0; }
size_t partial_bytes(const Product &p)
{
    return p.splits > 1 ? static_cast<size_t>(p.units()) * kWarpsOfPair * kPartialQuads * sizeof(float4) : 0;
}

// The gradient's products: dx, and both weights' gradients.
Product input_product(int rows, int width, int hidden, int map)
{
    return make_product(rows, width, hidden, 2, 0, kAlongK, kAlongK, map, map + 2);
}
Product weight_product(int rows, int width, int hidden, int map)
{
    return make_product(width, hidden, rows, 1, 1, across(kMmaF16, width), across(kMmaF16, hidden), map, map + 1);
}

size_t matrix_bytes(int rows, int hidden)
{
    return (static_cast<size_t>(rows) * ((static_cast<size_t>(hidden) + 7) / 8 * 16) + 255) / 256 * 256;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// What the products of one call need beside dG and dU.
size_t split_bytes(const Product *product, int products)
{
    size_t counters = 0, bytes = 0;
    for (int k = 0; k < products; ++k) {
        counters += counters_of(product[k]);
        bytes += partial_bytes(product[k]);
    }
    return align256(counters * 4) + bytes;
}

} // namespace gated
} // namespace pg

using namespace pg;

extern "C" {

int gated_projection(int rows, int width, int hidden, const void *x, long long ldx, const void *w_gate, long long ldwg,
                     const void *w_up, long long ldwu, void *h, long long ldh, void *gate, long long ldgate, void *up,
                     long long ldup, int activation, void *stream)
{
    using namespace gated;
    int st = check_sizes(rows, width, hidden);
    if (st != GEMM_OK)
        return st;
    if (!valid_activation(activation) || (gate == nullptr) != (up == nullptr))
        return GEMM_ERR_INVALID_ARG;
    const bool empty = rows == 0 || hidden == 0;
    if (!empty) {
        if ((st = check_plain(h, rows, hidden, ldh)) != GEMM_OK ||
            (gate && ((st = check_plain(gate, rows, hidden, ldgate)) != GEMM_OK ||
                      (st = check_plain(up, rows, hidden, ldup)) != GEMM_OK)))
            return st;
        if (width > 0 && ((st = check_operand(x, rows, width, ldx)) != GEMM_OK ||
                          (st = check_operand(w_gate, width, hidden, ldwg)) != GEMM_OK ||
                          (st = check_operand(w_up, width, hidden, ldwu)) != GEMM_OK))
            return st;
    }
    Device d;
    st = enter(&d);
    if (st != GEMM_OK || empty)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (width == 0) {
        st = zero_matrix(h, rows, hidden, ldh, s);
        if (st == GEMM_OK && gate)
            st = zero_matrix(gate, rows, hidden, ldgate, s);
        return st == GEMM_OK && up ? zero_matrix(up, rows, hidden, ldup, s) : st;
    }
    const int tokens = rows <= 16 ? 16 : 32;
    if (few_rows::faster(kTimes, tokens, rows, hidden, (width + 63) / 64, tiles_of(rows, hidden, 128), d.sms)) {
        few_rows::Maps few;
        std::memset(&few, 0, sizeof few);
        if ((st = few_rows::encode_tokens(&few.tokens, kMmaF16, x, rows, width, ldx, tokens)) != GEMM_OK ||
            (st = encode_operand(&few.weight[0], kMmaF16, w_gate, width, hidden, ldwg, kAcrossRagged)) != GEMM_OK ||
            (st = encode_operand(&few.weight[1], kMmaF16, w_up, width, hidden, ldwu, kAcrossRagged)) != GEMM_OK)
            return st;
        ForwardFew p = {};
        p.launch.rows = rows;
        p.launch.features = hidden;
        p.launch.blocks = width; // in elements until the launcher knows the block
        p.launch.family = kErrFamilyGated;
        p.launch.status = d.status;
        p.launch.wait_limit_ns = call_wait_limit_ns();
        p.launch.withhold = call_withhold();
        p.activation = activation;
        p.h = static_cast<__nv_bfloat16 *>(h);
        p.gate = static_cast<__nv_bfloat16 *>(gate);
        p.up = static_cast<__nv_bfloat16 *>(up);
        p.ldh = ldh;
        p.ldgate = ldgate;
        p.ldup = ldup;
        return tokens == 16 ? launch_few<16>(few, p, d, s) : launch_few<32>(few, p, d, s);
    }
    Maps maps;
    std::memset(&maps, 0, sizeof maps);
    const Layout across_w = across(kMmaF16, hidden);
    if ((st = encode_operand(&maps.map[0], kMmaF16, x, rows, width, ldx, kAlongK)) != GEMM_OK ||
        (st = encode_operand(&maps.map[1], kMmaF16, w_gate, width, hidden, ldwg, across_w)) != GEMM_OK ||
        (st = encode_operand(&maps.map[2], kMmaF16, w_up, width, hidden, ldwu, across_w)) != GEMM_OK)
        return st;
    Forward p = {};
    p.launch = make_launch(d);
    p.launch.product[0] = make_product(rows, hidden, width, 1, 1, kAlongK, across_w, 0, 1);
    p.launch.units = p.launch.first_units = p.launch.product[0].units();
    p.launch.maps = 3;
    p.h = static_cast<__nv_bfloat16 *>(h);
    p.gate = static_cast<__nv_bfloat16 *>(gate);
    p.up = static_cast<__nv_bfloat16 *>(up);
    p.ldh = ldh;
    p.ldgate = ldgate;
    p.ldup = ldup;
    p.h_access = row_access(h, ldh, rows, 2);
    p.gate_access = row_access(gate, ldgate, rows, 2);
    p.up_access = row_access(up, ldup, rows, 2);
    return activation == GEMM_ACT_SILU   ? launch_forward<GEMM_ACT_SILU>(maps, p, d, s)
           : activation == GEMM_ACT_GELU ? launch_forward<GEMM_ACT_GELU>(maps, p, d, s)
                                         : launch_forward<GEMM_ACT_GELU_TANH>(maps, p, d, s);
}

int gated_projection_backward_workspace(int rows, int width, int hidden, size_t *bytes)
{
    const int st = gated::check_sizes(rows, width, hidden);
    if (st != GEMM_OK || !bytes)
        return st != GEMM_OK ? st : GEMM_ERR_INVALID_ARG;
    using namespace gated;
    // Whichever of the gradients is wanted.
    size_t most = 0;
    if (rows > 0 && hidden > 0 && width > 0)
        for (int wanted = 1; wanted <= 3; ++wanted) {
            Product product[kMaxProducts];
            int n = 0;
            if (wanted & 1)
                product[n++] = input_product(rows, width, hidden, 0);
            if (wanted & 2)
                product[n++] = weight_product(rows, width, hidden, 0);
            cut(product, n, device_sms());
            most = std::max(most, split_bytes(product, n));
        }
    *bytes = 2 * matrix_bytes(rows, hidden) + most;
    return GEMM_OK;
}

int gated_projection_backward(int rows, int width, int hidden, const void *dh, long long lddh, const void *x,
                              long long ldx, const void *w_gate, long long ldwg, const void *w_up, long long ldwu,
                              const void *gate, long long ldgate, const void *up, long long ldup, void *dx,
                              long long lddx, void *dw_gate, long long lddwg, void *dw_up, long long lddwu,
                              int activation, void *workspace, size_t workspace_bytes, void *stream)
{
    using namespace gated;
    int st = check_sizes(rows, width, hidden);
    if (st != GEMM_OK)
        return st;
    if (!valid_activation(activation) || (dw_gate == nullptr) != (dw_up == nullptr))
        return GEMM_ERR_INVALID_ARG;
    const bool want_x = dx && rows > 0 && width > 0, want_w = dw_gate && width > 0 && hidden > 0;
    const bool any = rows > 0 && hidden > 0; // dG and dU have elements
    if (want_x && (st = check_plain(dx, rows, width, lddx)) != GEMM_OK)
        return st;
    if (want_w && ((st = check_plain(dw_gate, width, hidden, lddwg)) != GEMM_OK ||
                   (st = check_plain(dw_up, width, hidden, lddwu)) != GEMM_OK))
        return st;
    if (any && (want_x || want_w)) {
        if ((st = check_plain(dh, rows, hidden, lddh)) != GEMM_OK ||
            (st = check_plain(gate, rows, hidden, ldgate)) != GEMM_OK ||
            (st = check_plain(up, rows, hidden, ldup)) != GEMM_OK)
            return st;
        if (want_x && ((st = check_operand(w_gate, width, hidden, ldwg)) != GEMM_OK ||
                       (st = check_operand(w_up, width, hidden, ldwu)) != GEMM_OK))
            return st;
        if (want_w && (st = check_operand(x, rows, width, ldx)) != GEMM_OK)
            return st;
        if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
            return GEMM_ERR_MISALIGNED;
        if (!workspace || workspace_bytes < 2 * matrix_bytes(rows, hidden))
            return GEMM_ERR_INVALID_ARG;
    }
    Device d;
    st = enter(&d);
    if (st != GEMM_OK)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!any) {
        if (want_x)
            st = zero_matrix(dx, rows, width, lddx, s);
        if (st == GEMM_OK && want_w)
            st = zero_matrix(dw_gate, width, hidden, lddwg, s);
        return st == GEMM_OK && want_w ? zero_matrix(dw_up, width, hidden, lddwu, s) : st;
    }
    if (!want_x && !want_w)
        return GEMM_OK;

    uint8_t *const ws = static_cast<uint8_t *>(workspace);
    Slopes sl = {};
    sl.rows = rows;
    sl.hidden = hidden;
    sl.dh = static_cast<const __nv_bfloat16 *>(dh);
    sl.gate = static_cast<const __nv_bfloat16 *>(gate);
    sl.up = static_cast<const __nv_bfloat16 *>(up);
    sl.lddh = lddh;
    sl.ldgate = ldgate;
    sl.ldup = ldup;
    sl.dgate = reinterpret_cast<__nv_bfloat16 *>(ws);
    sl.dup = reinterpret_cast<__nv_bfloat16 *>(ws + matrix_bytes(rows, hidden));
    sl.pitch = (static_cast<long long>(hidden) + 7) / 8 * 8;

    Maps maps;
    std::memset(&maps, 0, sizeof maps);
    Backward p = {};
    p.launch = make_launch(d);
    Product *const product = p.launch.product;
    int n = 0, products = 0, of_x = -1, of_w = -1;
    if (want_x) {
        product[products] = input_product(rows, width, hidden, n);
        of_x = products++;
        n += 4;
    }
    if (want_w) {
        product[products] = weight_product(rows, width, hidden, n);
        of_w = products++;
        n += 3;
    }
    cut(product, products, d.sms);
    if (workspace_bytes < 2 * matrix_bytes(rows, hidden) + split_bytes(product, products))
        return GEMM_ERR_INVALID_ARG;
    // The product with the longer units comes first.
    if (products == 2 && 2.0 * product[0].blocks / product[0].splits < 1.0 * product[1].blocks / product[1].splits) {
        std::swap(product[0], product[1]);
        std::swap(of_x, of_w);
    }
    if (want_x) {
        const int m = product[of_x].a_map;
        if ((st = encode_operand(&maps.map[m], kMmaF16, sl.dgate, rows, hidden, sl.pitch, kAlongK)) != GEMM_OK ||
            (st = encode_operand(&maps.map[m + 1], kMmaF16, sl.dup, rows, hidden, sl.pitch, kAlongK)) != GEMM_OK ||
            (st = encode_operand(&maps.map[m + 2], kMmaF16, w_gate, width, hidden, ldwg, kAlongK)) != GEMM_OK ||
            (st = encode_operand(&maps.map[m + 3], kMmaF16, w_up, width, hidden, ldwu, kAlongK)) != GEMM_OK)
            return st;
        Results &to = p.results[of_x];
        to.out[0] = static_cast<__nv_bfloat16 *>(dx);
        to.ld[0] = lddx;
        to.access[0] = row_access(dx, lddx, rows, 2);
    }
    if (want_w) {
        const Product &w = product[of_w];
        const int m = w.a_map;
        if ((st = encode_operand(&maps.map[m], kMmaF16, x, rows, width, ldx, w.a_layout)) != GEMM_OK ||
            (st = encode_operand(&maps.map[m + 1], kMmaF16, sl.dgate, rows, hidden, sl.pitch, w.b_layout)) != GEMM_OK ||
            (st = encode_operand(&maps.map[m + 2], kMmaF16, sl.dup, rows, hidden, sl.pitch, w.b_layout)) != GEMM_OK)
            return st;
        Results &to = p.results[of_w];
        void *const out[2] = {dw_gate, dw_up};
        const long long ld[2] = {lddwg, lddwu};
        for (int k = 0; k < 2; ++k) {
            to.out[k] = static_cast<__nv_bfloat16 *>(out[k]);
            to.ld[k] = ld[k];
            to.access[k] = row_access(out[k], ld[k], width, 2);
        }
    }
    // Counters of both products, then their sums.
    sl.arrived = reinterpret_cast<unsigned int *>(ws + 2 * matrix_bytes(rows, hidden));
    for (int k = 0; k < products; ++k) {
        p.results[k].arrived = sl.arrived + sl.counters;
        sl.counters += static_cast<int>(counters_of(product[k]));
    }
    uint8_t *sums = reinterpret_cast<uint8_t *>(sl.arrived) + align256(static_cast<size_t>(sl.counters) * 4);
    for (int k = 0; k < products; ++k) {
        p.results[k].partial = reinterpret_cast<float4 *>(sums);
        sums += partial_bytes(product[k]);
    }
    p.launch.maps = n;
    p.launch.first_units = product[0].units();
    p.launch.units = p.launch.first_units + (products > 1 ? product[1].units() : 0);
    // Ahead of the first launch: a call that fails has enqueued nothing.
    static std::atomic<unsigned long long> limit_set[kMaxDevices];
    if (ensure_smem_limit(gated_backward_kernel, kSmem, d.index, d.ctx, limit_set) != GEMM_OK)
        return GEMM_ERR_CUDA;
    st = activation == GEMM_ACT_SILU   ? launch_slopes<GEMM_ACT_SILU>(sl, d, s)
         : activation == GEMM_ACT_GELU ? launch_slopes<GEMM_ACT_GELU>(sl, d, s)
                                       : launch_slopes<GEMM_ACT_GELU_TANH>(sl, d, s);
    if (st != GEMM_OK)
        return st;
    // Started while the slopes end, for which all but the setting up waits: 45 us
    // to 43 for 1000 x 1000 -> 2700.  Not behind many slopes: 1380 us to 1345 for
    // 8192 x 4096 -> 8192.
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid_of(p.launch.units, d)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = static_cast<long long>(rows) * hidden <= 8ll * 16 * kSlopeThreads * d.sms ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, gated_backward_kernel, maps, p) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

} // extern "C"
