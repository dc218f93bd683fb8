// Layer norm of rows that a group of threads holds in registers: x is read
// once, y written once.  Mean first, then squared differences to it, from the
// same registers.  With a ring, weight and bias wait in shared memory as
// float32 from row to row; otherwise they are loaded beside x.
//
// Measured on GB300 (bytes of x and y; a device copy of as many bytes runs at
// 6.1 TB/s): 16384 x 4096 bfloat16 47 to 50 us, 5.7 to 5.4 TB/s; 8192 x 8192
// bfloat16 58 us, 4.6 TB/s; 16384 x 4096 float32 94 us, 5.7 TB/s.  Neither DRAM
// (56 % of its cycles at 16384 x 4096 bfloat16) nor the schedulers (1.5 of 4
// instructions a clock) are full: a group waits for its row's two sums, one
// after the other, and the few rows at a time that registers allow hide that in
// part.  (One sum would do, of each thread's mean and squared differences put
// together; not tried.)  Longer rows: 4096 x 16384 bfloat16 60 us; float32 has
// room for two rows in the ring up to 14336 columns, 4096 of them 86 us, of
// 16384, without, 115; beyond that three passes, 2048 x 32768 bfloat16 131 and
// float32 219.  One row is the launch: 4096 bfloat16 take about 3 us on the
// device.
#include "layer_norm_internal.h"

namespace pg {

namespace ln {

template <class T, int E, Source S>
__global__ void __launch_bounds__(forward_threads(E), 1) forward_rows_kernel(const Forward p, const Shape shape)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[kMaxWarps * kMaxSlots];
    __shared__ GroupScratch scratch;
    constexpr bool kRing = from_ring(S);
    Group g(threadIdx.x, shape.tpr, &scratch);
    const Spread<T, E, S> at(g.t, p.cols);
    constexpr int kPiece = at.kPiece, kPieces = at.kPieces;
    float *weight = reinterpret_cast<float *>(smem), *bias = weight + parameter_floats(p.cols);
    uint8_t *slots = smem + (kRing ? 2 * parameter_floats(p.cols) * 4 : 0);
    Ring<1> ring(smem_u32(bars), smem_u32(slots), shape, g, p.cols * static_cast<int>(sizeof(T)), p.rows);
    uint8_t *own = slots + (ring.slots_at - smem_u32(slots));
    if constexpr (kRing) {
        ring.in[0] = Stream{static_cast<const uint8_t *>(p.x), p.ldx * static_cast<long long>(sizeof(T))};
        ring.init();
        ring.start(); // a thread's own copies on its own mbarriers; the others meet them past the barrier
        at.copy_parameter(weight, p.weight, p.weight_bf16, 1.0f);
        at.copy_parameter(bias, p.bias, p.weight_bf16, 0.0f);
    }
    const long long step = static_cast<long long>(gridDim.x) * shape.groups;
    const long long first = static_cast<long long>(blockIdx.x) * shape.groups + g.index;
    Edges<T, 1> edges;
    if constexpr (S == kRingShifted) {
        edges.load(ring, g, first);
        edges.place(ring, own, 0);
        edges.load(ring, g, first + step);
    }
    __syncthreads();
    const float n = static_cast<float>(p.cols), inv = 1.0f / n;

    // The bound is the same in the whole group.
    for (long long row = first; row < p.rows; row += step) {
        if constexpr (S == kRingShifted) {
            edges.place(ring, own, ring.slot + 1 == ring.slots ? 0 : ring.slot + 1);
            edges.load(ring, g, row + 2 * step);
        }
        unsigned long long d[E / 2];
        // Without a ring, and while registers allow, weight and bias are loaded
        // beside x: a single row waits for memory once.
        constexpr bool kEarly = !kRing && E <= 16;
        float w[kEarly ? E : 1], b[kEarly ? E : 1];
        {
            float x[E];
            if constexpr (kRing) {
                ring.wait();
                at.load(ring.template view<T>(own, 0, row), x);
            } else {
                const T *from = static_cast<const T *>(p.x) + row * p.ldx;
                at.load(Row<T>{from, 0}, x);
                if constexpr (kEarly) {
#pragma unroll
                    for (int k = 0; k < kPieces; ++k) {
                        at.load_parameter_piece(p.weight, p.weight_bf16, 1.0f, k, w + k * kPiece);
                        at.load_parameter_piece(p.bias, p.weight_bf16, 0.0f, k, b + k * kPiece);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < E / 2; ++i)
                d[i] = pair(x[2 * i], x[2 * i + 1]);
        }
        // Two chains of paired additions: one would cost a latency each.
        unsigned long long part[2] = {0ull, 0ull};
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            part[i & 1] = add2(part[i & 1], d[i]);
        const float mean = divided(g.sum(both(add2(part[0], part[1]))), n, inv);
        if constexpr (kRing) // the group has met in the sum, past its loads
            ring.next();
        const unsigned long long minus = pair(-mean, -mean);
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            d[i] = add2(d[i], minus);
        at.clear_absent(d);
        part[0] = part[1] = 0ull;
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            part[i & 1] = fma2(d[i], d[i], part[i & 1]);
        const float rstd = rsqrtf(fmaf(g.sum(both(add2(part[0], part[1]))), inv, p.eps));
        const unsigned long long scale = pair(rstd, rstd);
        RowOut<T, E, S> y(at, static_cast<T *>(p.y) + row * p.ldy);
        auto parameters = [&](int k, float *wk, float *bk) {
            if constexpr (kRing) {
                at.load_copy_piece(weight, p.cols, k, wk);
                at.load_copy_piece(bias, p.cols, k, bk);
            } else if constexpr (kEarly) {
#pragma unroll
                for (int e = 0; e < kPiece; ++e) {
                    wk[e] = w[k * kPiece + e];
                    bk[e] = b[k * kPiece + e];
                }
            } else {
                at.load_parameter_piece(p.weight, p.weight_bf16, 1.0f, k, wk);
                at.load_parameter_piece(p.bias, p.weight_bf16, 0.0f, k, bk);
            }
        };
        if constexpr (kPiece == 1) {
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
                float wk, bk, lo, hi;
                parameters(k, &wk, &bk);
                split(d[k / 2], lo, hi);
                const float v = fmaf((k & 1 ? hi : lo) * rstd, wk, bk);
                y.put(k, &v);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
                float wk[kPiece], bk[kPiece], v[kPiece];
                parameters(k, wk, bk);
#pragma unroll
                for (int e = 0; e < kPiece; e += 2) {
                    const unsigned long long r = fma2(mul2(d[(k * kPiece + e) / 2], scale), pair(wk[e], wk[e + 1]),
                                                      pair(bk[e], bk[e + 1]));
                    split(r, v[e], v[e + 1]);
                }
                y.put(k, v);
            }
            y.finish();
        }
        if (p.mean && g.t == 0) {
            p.mean[row] = mean;
            p.rstd[row] = rstd;
        }
    }
    if constexpr (kRing)
        ring.drain();
}

template <class T, int E, Source S>
static int launch(const Forward &p, const Plan &plan, const Device &d, cudaStream_t s)
{
    if constexpr (from_ring(S)) {
        static std::atomic<unsigned long long> limit_set[kMaxDevices];
        if (ensure_smem_limit(forward_rows_kernel<T, E, S>, kSmemBytes, d.index, d.ctx, limit_set) != GEMM_OK)
            return GEMM_ERR_CUDA;
    }
    const int threads = plan.shape.groups * plan.shape.tpr;
    forward_rows_kernel<T, E, S><<<plan.grid, threads, plan.smem, s>>>(p, plan.shape);
    return cudaGetLastError() == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

template <class T, int E>
static int launch_source(const Forward &p, const Plan &plan, const Device &d, cudaStream_t s)
{
    switch (plan.source) {
    case kRingFull: return launch<T, E, kRingFull>(p, plan, d, s);
    case kRingVector: return launch<T, E, kRingVector>(p, plan, d, s);
    case kRingShifted: return launch<T, E, kRingShifted>(p, plan, d, s);
    case kVector: return launch<T, E, kVector>(p, plan, d, s);
    default: return launch<T, E, kScalar>(p, plan, d, s);
    }
}

int launch_forward_rows(const Forward &p, bool bf16, const Plan &plan, const Device &d, cudaStream_t s)
{
    if (plan.elements == 16)
        return bf16 ? launch_source<__nv_bfloat16, 16>(p, plan, d, s) : launch_source<float, 16>(p, plan, d, s);
    return bf16 ? launch_source<__nv_bfloat16, 32>(p, plan, d, s) : launch_source<float, 32>(p, plan, d, s);
}

} // namespace ln

} // namespace pg
