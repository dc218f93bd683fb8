// Gradient of layer norm for rows that a group of threads holds in registers:
// dy and x are read once and dx written once, and each thread sums dweight and
// dbias of its columns over all its rows in registers.  What remains of those
// is one partial sum per column and CTA, added up by a second small kernel.
//
// Measured on GB300 (bytes of dy, x and dx): 16384 x 4096 bfloat16 84 us, 4.8
// TB/s; 3000 x 5000 float32 41 us, 4.4 TB/s; 16384 x 4096 float32 137 us, 5.9
// TB/s.  In bfloat16 nothing is full: DRAM is busy 55 % of the time, two of four
// issue slots a clock are used.  The sixteen warps that the column sums'
// registers leave wait, a group at a time, for their loads from the ring and
// for a row's sums.  Above 8192 columns a CTA holds one row of 32 elements a
// thread and reads it twice from shared memory: 4096 x 16384 bfloat16 127 us.
// From 11469 float32 columns on no two rows of x and dy fit the ring, and
// nothing runs ahead: 5461 x 11468 156 us, x 12288 300.
#include "layer_norm_internal.h"

namespace pg {

namespace ln {

template <class T, int E, Source S>
__global__ void __launch_bounds__(kBackwardThreads, 1) backward_rows_kernel(const Backward p, const Shape shape)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[kMaxWarps * kMaxSlots];
    __shared__ GroupScratch scratch;
    constexpr bool kRing = from_ring(S);
    // Up to 16 elements a thread keeps a row's between its two passes; with
    // 32 the column sums take those registers, and the second pass reads the
    // row again where it is.
    constexpr bool kKeep = E <= 16;
    grid_launch_next(); // the kernel that adds the partial sums waits for this one's end
    Group g(threadIdx.x, shape.tpr, &scratch);
    using Columns = Spread<T, E, S>;
    const Columns at(g.t, p.cols);
    constexpr int kPiece = Columns::kPiece, kPieces = Columns::kPieces;
    float *weight = reinterpret_cast<float *>(smem);
    uint8_t *slots = smem + (kRing ? parameter_floats(p.cols) * 4 : 0);
    Ring<2> ring(smem_u32(bars), smem_u32(slots), shape, g, p.cols * static_cast<int>(sizeof(T)), p.rows);
    uint8_t *own = slots + (ring.slots_at - smem_u32(slots));
    if constexpr (kRing) {
        ring.in[0] = Stream{static_cast<const uint8_t *>(p.x), p.ldx * static_cast<long long>(sizeof(T))};
        ring.in[1] = Stream{static_cast<const uint8_t *>(p.dy), p.lddy * static_cast<long long>(sizeof(T))};
        ring.init();
        ring.start(); // a thread's own copies on its own mbarriers; the others meet them past the barrier
        at.copy_parameter(weight, p.weight, p.weight_bf16, 1.0f);
    }
    const long long step = static_cast<long long>(gridDim.x) * shape.groups;
    const long long first = static_cast<long long>(blockIdx.x) * shape.groups + g.index;
    Edges<T, 2> edges;
    if constexpr (unaligned(S)) {
        edges.load(ring, g, first);
        edges.place(ring, own, 0);
        edges.load(ring, g, first + step);
    }
    __syncthreads();
    unsigned long long dw[E / 2], db[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i)
        dw[i] = db[i] = 0ull;
    const float inv = -1.0f / static_cast<float>(p.cols);
    auto weight_piece = [&](int k, float *v) {
        if constexpr (kRing)
            at.load_copy_piece(weight, p.cols, k, v);
        else
            at.load_parameter_piece(p.weight, p.weight_bf16, 1.0f, k, v);
    };

    float next_mean = 0.0f, next_rstd = 0.0f; // loaded a row ahead
    if (first < p.rows) {
        next_mean = p.mean[first];
        next_rstd = p.rstd[first];
    }
    // The bound is the same in the whole group.
    for (long long row = first; row < p.rows; row += step) {
        if constexpr (unaligned(S)) {
            edges.place(ring, own, ring.slot + 1 == ring.slots ? 0 : ring.slot + 1);
            edges.load(ring, g, row + 2 * step);
        }
        const float mean = next_mean, rstd = next_rstd;
        if (row + step < p.rows) {
            next_mean = p.mean[row + step];
            next_rstd = p.rstd[row + step];
        }
        Row<T> x, dy;
        if constexpr (kRing) {
            ring.wait();
            x = ring.template view<T>(own, 0, row);
            dy = ring.template view<T>(own, 1, row);
        } else {
            x.at = static_cast<const T *>(p.x) + row * p.ldx;
            dy.at = static_cast<const T *>(p.dy) + row * p.lddy;
        }
        RowOut<T, E, S> dx(at, static_cast<T *>(p.dx) + row * p.lddx);
        const unsigned long long minus = pair(-mean, -mean), scale = pair(rstd, rstd);
        // Two chains of paired additions for each sum.
        unsigned long long s1[2] = {0ull, 0ull}, s2[2] = {0ull, 0ull};
        // xhat and t = dy weight of pairs 2j, 2j + 1 of the thread, added to
        // the row's and the columns' sums.  Absent elements: dy and so t are 0.
        auto first_pass = [&](int j, unsigned long long xv, unsigned long long gv, unsigned long long wv,
                              unsigned long long &xhat, unsigned long long &t) {
            xhat = mul2(add2(xv, minus), scale);
            t = mul2(gv, wv);
            s1[j & 1] = add2(s1[j & 1], t);
            s2[j & 1] = fma2(t, xhat, s2[j & 1]);
            dw[j] = fma2(gv, xhat, dw[j]);
            db[j] = add2(db[j], gv);
        };
        if constexpr (kKeep) {
            unsigned long long xhat[E / 2], t[E / 2];
            {
                float xv[E], gv[E], wv[E];
                at.load(x, xv);
                at.load(dy, gv);
#pragma unroll
                for (int k = 0; k < kPieces; ++k)
                    weight_piece(k, wv + k * kPiece);
#pragma unroll
                for (int j = 0; j < E / 2; ++j)
                    first_pass(j, pair(xv[2 * j], xv[2 * j + 1]), pair(gv[2 * j], gv[2 * j + 1]),
                               pair(wv[2 * j], wv[2 * j + 1]), xhat[j], t[j]);
            }
            const float2 c = g.sum(both(add2(s1[0], s1[1])), both(add2(s2[0], s2[1])));
            if constexpr (kRing) // the group has met in the sum, past its loads
                ring.next();
            const float c1 = c.x * inv, c2 = c.y * inv; // negated means
            const unsigned long long m1 = pair(c1, c1), m2 = pair(c2, c2);
            float v[E];
#pragma unroll
            for (int j = 0; j < E / 2; ++j)
                split(mul2(add2(fma2(xhat[j], m2, t[j]), m1), scale), v[2 * j], v[2 * j + 1]);
#pragma unroll
            for (int k = 0; k < kPieces; ++k)
                dx.put(k, v + k * kPiece);
            dx.finish();
        } else {
            constexpr int kStep = kPiece == 1 ? 2 : kPiece; // elements at a time: whole pairs
            auto load = [&](int i, float (&xv)[kStep], float (&gv)[kStep], float (&wv)[kStep]) {
#pragma unroll
                for (int e = 0; e < kStep; e += kPiece) {
                    const int k = (i + e) / kPiece;
                    at.load_piece(x, k, xv + e);
                    at.load_piece(dy, k, gv + e);
                    weight_piece(k, wv + e);
                }
            };
#pragma unroll
            for (int i = 0; i < E; i += kStep) {
                float xv[kStep], gv[kStep], wv[kStep];
                load(i, xv, gv, wv);
#pragma unroll
                for (int e = 0; e < kStep; e += 2) {
                    unsigned long long xhat, t;
                    first_pass((i + e) / 2, pair(xv[e], xv[e + 1]), pair(gv[e], gv[e + 1]), pair(wv[e], wv[e + 1]),
                               xhat, t);
                }
            }
            const float2 c = g.sum(both(add2(s1[0], s1[1])), both(add2(s2[0], s2[1])));
            const float c1 = c.x * inv, c2 = c.y * inv; // negated means
            const unsigned long long m1 = pair(c1, c1), m2 = pair(c2, c2);
#pragma unroll
            for (int i = 0; i < E; i += kStep) {
                float xv[kStep], gv[kStep], wv[kStep], v[kStep];
                load(i, xv, gv, wv);
#pragma unroll
                for (int e = 0; e < kStep; e += 2) {
                    const unsigned long long xhat = mul2(add2(pair(xv[e], xv[e + 1]), minus), scale);
                    const unsigned long long t = mul2(pair(gv[e], gv[e + 1]), pair(wv[e], wv[e + 1]));
                    split(mul2(add2(fma2(xhat, m2, t), m1), scale), v[e], v[e + 1]);
                }
#pragma unroll
                for (int e = 0; e < kStep; e += kPiece)
                    dx.put((i + e) / kPiece, v + e);
            }
            dx.finish();
            if constexpr (kRing) {
                g.barrier();
                ring.next();
            }
        }
    }
    if constexpr (kRing)
        ring.drain();

    if (!p.dweight && !p.dbias)
        return;
    if constexpr (!kKeep) {
        // At these lengths a CTA has one group, whose threads write their own
        // columns.  Inside a loop that runs once, the columns worked out anew
        // from what the compiler cannot trace back, so that none of this takes
        // registers from the loop over the rows, where they would be spilled:
        // 4096 x 16384 bfloat16 127 us, written straight on 187; 7456 x 9000
        // float32 162 and 213.
        for (int k = g.index; k < shape.groups; k += shape.groups) {
            int t = g.t, cols = p.cols;
            asm volatile("" : "+r"(t), "+r"(cols));
            const Columns own_columns(t, cols);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if (!own_columns.has(i / kPiece, i % kPiece))
                    break;
                const int j = own_columns.column(i / kPiece) + i % kPiece;
                float lo, hi;
                split(dw[i / 2], lo, hi);
                const float vw = i & 1 ? hi : lo;
                split(db[i / 2], lo, hi);
                const float vb = i & 1 ? hi : lo;
                if (gridDim.x == 1) {
                    if (p.dweight)
                        store_f32(p.dweight, p.weight_bf16, j, vw);
                    if (p.dbias)
                        store_f32(p.dbias, p.weight_bf16, j, vb);
                } else {
                    float *out = p.partial + static_cast<long long>(blockIdx.x) * 2 * p.cols;
                    out[j] = vw;
                    out[p.cols + j] = vb;
                }
            }
        }
        return;
    }
    // Every group's sums to shared memory (the ring's: all of its rows have
    // been taken), added up in group order and written by neighbouring threads.
    // (One group after the other adding to one copy, and each thread writing
    // its own columns, took 1000 x 1024 bfloat16 4 us longer.)
    const int pitch = parameter_floats(p.cols);
    float *sums = reinterpret_cast<float *>(smem); // [groups][2][pitch]
    __syncthreads();
    float *mine = sums + g.index * 2 * pitch;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        if (!at.has(k))
            break;
        const int j = at.column(k);
        float vw[kPiece], vb[kPiece];
#pragma unroll
        for (int e = 0; e < kPiece; ++e) {
            const int i = k * kPiece + e;
            float lo, hi;
            split(dw[i / 2], lo, hi);
            vw[e] = i & 1 ? hi : lo;
            split(db[i / 2], lo, hi);
            vb[e] = i & 1 ? hi : lo;
        }
        if constexpr (kPiece == 1) {
            mine[j] = vw[0];
            mine[pitch + j] = vb[0];
        } else {
#pragma unroll
            for (int e = 0; e < kPiece; e += 4) {
                *reinterpret_cast<uint4 *>(mine + j + e) = Vec16<float>::pack(vw + e);
                *reinterpret_cast<uint4 *>(mine + pitch + j + e) = Vec16<float>::pack(vb + e);
            }
        }
    }
    __syncthreads();
    float *out = p.partial + static_cast<long long>(blockIdx.x) * 2 * p.cols;
    for (int u = threadIdx.x; u < 2 * p.cols; u += blockDim.x) {
        const int which = u >= p.cols, j = u - which * p.cols;
        const float *from = sums + which * pitch + j;
        float v = from[0];
        for (int k = 1; k < shape.groups; ++k)
            v += from[k * 2 * pitch];
        if (gridDim.x > 1)
            out[u] = v;
        else if (void *to = which == 0 ? p.dweight : p.dbias)
            store_f32(to, p.weight_bf16, j, v);
    }
}

template <class T, int E, Source S>
static int launch(const Backward &p, const Plan &plan, const Device &d, cudaStream_t s)
{
    const int sums = E <= 16 ? plan.shape.groups * 2 * parameter_floats(p.cols) * 4 : 0; // the groups' column sums
    static std::atomic<unsigned long long> limit_set[kMaxDevices];
    if (ensure_smem_limit(backward_rows_kernel<T, E, S>, kSmemBytes, d.index, d.ctx, limit_set) != GEMM_OK)
        return GEMM_ERR_CUDA;
    const int threads = plan.shape.groups * plan.shape.tpr;
    backward_rows_kernel<T, E, S><<<plan.grid, threads, std::max(plan.smem, sums), s>>>(p, plan.shape);
    return cudaGetLastError() == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

template <class T, int E>
static int launch_source(const Backward &p, const Plan &plan, const Device &d, cudaStream_t s)
{
    if constexpr (E == 16)
        if (plan.source == kRingFull)
            return launch<T, E, kRingFull>(p, plan, d, s);
    // What spread() was given for unaligned rows.
    constexpr Source kUnaligned = backward_unaligned(sizeof(T));
    switch (plan.source) {
    case kRingVector: return launch<T, E, kRingVector>(p, plan, d, s);
    case kUnaligned: return launch<T, E, kUnaligned>(p, plan, d, s);
    case kVector: return launch<T, E, kVector>(p, plan, d, s);
    default: return launch<T, E, kScalar>(p, plan, d, s);
    }
}

int launch_backward_rows(const Backward &p, bool bf16, const Plan &plan, const Device &d, cudaStream_t s)
{
    if (plan.elements == 16)
        return bf16 ? launch_source<__nv_bfloat16, 16>(p, plan, d, s) : launch_source<float, 16>(p, plan, d, s);
    return bf16 ? launch_source<__nv_bfloat16, 32>(p, plan, d, s) : launch_source<float, 32>(p, plan, d, s);
}

} // namespace ln

} // namespace pg
