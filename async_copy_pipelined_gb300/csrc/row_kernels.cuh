// What the layer norm kernels share: how a row is spread over threads, how
// its sums are formed, and the ring through which rows reach shared memory.
//
// A group of `tpr` threads (whole warps) takes a row, each thread E of its
// elements in registers; a CTA holds `groups` groups.  Rows that are 16-byte
// aligned move in 16-byte vectors, others element by element.
//
// Ring: the first thread of each group copies the group's rows into shared
// memory (bulk copies completing on mbarriers), several ahead of the one being
// computed, so that the bytes in flight do not depend on how many registers
// the computation leaves.  A slot is refilled once a barrier of the group's
// sums shows that its threads have taken their elements.  With no more than a
// row or two to a group there is nothing to run ahead of, and threads load
// their elements themselves.
//
// Beside DRAM it is the instructions issued per element that bound these
// kernels, so additions and multiplications run on pairs (one instruction for
// two float32 values), and a thread has enough elements to spread the cost of
// a row's reductions over.
#pragma once

#include "gemm_internal.h"
#include "ptx.cuh"
#include "vector_io.cuh"

namespace pg {

namespace ln {

constexpr int kMaxWarps = 24; // of a CTA
constexpr int kMaxSlots = 8;
constexpr int kSmemBytes = 224 * 1024; // dynamic, at most
// Of it the ring's slots, where two of them fit: enough bytes in flight (16384
// rows of 4096 bfloat16, forward: 49.4 us with 80 KiB, 49.5 with 128, 51.8 with
// 192, whose first copies take longer to arrive).
constexpr int kRingBytes = 128 * 1024;

// Where a row's elements come from and in what pieces: the ring, or loads of
// the thread's own; 16-byte vectors, or single elements.
// kRingFull: vectors from the ring in rows of exactly tpr E elements, so that
// no piece needs asking whether it is there.
enum Source { kRingFull, kRingVector, kRingScalar, kVector, kScalar };
constexpr bool from_ring(Source s) { return s == kRingFull || s == kRingVector || s == kRingScalar; }
constexpr bool in_vectors(Source s) { return s == kRingFull || s == kRingVector || s == kVector; }

struct Shape {
    int tpr, groups; // threads per row; rows at a time in a CTA
    int slots;       // of a group's ring
    int slot_bytes;  // one row of one matrix, with room for its alignment
    unsigned int *status;
    unsigned long long wait_limit_ns;
    int withhold;
};

// a / n for a positive n whose reciprocal is `inv`: the product, corrected by
// what it is off (exact where the quotient is, as a constant row's mean).
__device__ __forceinline__ float divided(float a, float n, float inv)
{
    const float q = a * inv;
    return isfinite(q) ? fmaf(fmaf(-q, n, a), inv, q) : q;
}
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ------------------------------------------------------------ a row's elements
// A row where a thread finds it: elements head .. tail-1 at `near` (shared
// memory, or the row itself), the others at `far` (the row in global memory).
template <class T>
struct Row {
    const T *near, *far;
    int head, tail;
};

// Where a thread has its elements: warp w of a group takes 32 E columns in a
// row, piece k (a vector, or one element) of its lane l starting at column
// 32 E w + (32 k + l) kPiece, a constant distance from piece to piece.
template <class T, int E, Source S>
struct Spread {
    static constexpr int kPiece = in_vectors(S) ? Vec16<T>::kElements : 1;
    static constexpr int kPieces = E / kPiece;
    int first;  // column of piece 0
    int pieces; // of this thread that lie in the row (a vector row has whole vectors only)
    bool full;  // every lane of the warp has all of them

    __device__ __forceinline__ Spread(int t, int cols) : first(t / 32 * 32 * E + t % 32 * kPiece)
    {
        const int left = (cols - first + 32 * kPiece - 1) / (32 * kPiece);
        pieces = cols > first ? (left < kPieces ? left : kPieces) : 0;
        full = __all_sync(0xffffffffu, pieces == kPieces);
    }
    __device__ __forceinline__ int column(int k) const { return first + k * (32 * kPiece); }
    __device__ __forceinline__ bool has(int k) const { return S == kRingFull || k < pieces; }

    __device__ __forceinline__ void load_piece(const Row<T> &row, int k, float *v) const
    {
        if (has(k)) {
            const int j = column(k);
            if constexpr (S == kRingScalar)
                v[0] = to_f32(j >= row.head && j < row.tail ? row.near[j] : row.far[j]);
            else if constexpr (S == kScalar)
                v[0] = to_f32(row.near[j]);
            else
                Vec16<T>::unpack(*reinterpret_cast<const uint4 *>(row.near + j), v);
        } else {
#pragma unroll
            for (int e = 0; e < kPiece; ++e)
                v[e] = 0.0f;
        }
    }
    __device__ __forceinline__ void load(const Row<T> &row, float (&v)[E]) const
    {
#pragma unroll
        for (int k = 0; k < kPieces; ++k)
            load_piece(row, k, v + k * kPiece);
    }
    // v with zeros where there is no element.
    __device__ __forceinline__ void clear_absent(unsigned long long (&v)[E / 2]) const
    {
        if (S == kRingFull || full)
            return;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            float a, b;
            split(v[i], a, b);
            if (2 * i / kPiece >= pieces)
                a = 0.0f;
            if ((2 * i + 1) / kPiece >= pieces)
                b = 0.0f;
            v[i] = pair(a, b);
        }
    }
    __device__ __forceinline__ void store_piece(T *row, int k, const float *v) const
    {
        if (has(k)) {
            if constexpr (in_vectors(S))
                *reinterpret_cast<uint4 *>(row + column(k)) = Vec16<T>::pack(v);
            else
                row[column(k)] = from_f32<T>(v[0]);
        }
    }

    // A parameter vector of run-time type in global memory (null: `absent`
    // everywhere).  The planner has checked that vectors can be read from it.
    __device__ __forceinline__ void load_parameter_piece(const void *p, bool bf16, float absent, int k, float *v) const
    {
        if (!has(k) || !p) {
#pragma unroll
            for (int e = 0; e < kPiece; ++e)
                v[e] = absent;
        } else if constexpr (!in_vectors(S)) {
            v[0] = load_f32(p, bf16, column(k));
        } else if (bf16) {
            const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p) + column(k);
            if constexpr (kPiece == 8) {
                Vec16<__nv_bfloat16>::unpack(*reinterpret_cast<const uint4 *>(q), v);
            } else {
                const uint2 h = *reinterpret_cast<const uint2 *>(q);
                v[0] = __uint_as_float(h.x << 16);
                v[1] = __uint_as_float(h.x & 0xFFFF0000u);
                v[2] = __uint_as_float(h.y << 16);
                v[3] = __uint_as_float(h.y & 0xFFFF0000u);
            }
        } else {
            const float *q = static_cast<const float *>(p) + column(k);
#pragma unroll
            for (int e = 0; e < kPiece; e += 4)
                Vec16<float>::unpack(*reinterpret_cast<const uint4 *>(q + e), v + e);
        }
    }
    // The same from its float32 copy in shared memory (copy_parameter()).
    // Absent pieces read the first.
    __device__ __forceinline__ void load_copy_piece(const float *copy, int cols, int k, float *v) const
    {
        const int j = has(k) ? column(k) : 0;
        if constexpr (kPiece == 8) {
            Vec16<float>::unpack(*reinterpret_cast<const uint4 *>(copy + j / 2), v);
            Vec16<float>::unpack(*reinterpret_cast<const uint4 *>(copy + cols / 2 + j / 2), v + 4);
        } else if constexpr (kPiece == 4) {
            Vec16<float>::unpack(*reinterpret_cast<const uint4 *>(copy + j), v);
        } else {
            v[0] = copy[j];
        }
    }
    // A parameter vector as float32 in shared memory, by the whole CTA.  For
    // pieces of eight the first halves of all pieces come before the second
    // halves, so that neighbouring threads' 16-byte reads are neighbours.
    static __device__ __forceinline__ void copy_parameter(float *copy, const void *p, bool bf16, float absent, int cols)
    {
        // Several loads of a thread in flight: the first rows wait for them.
        constexpr int kUnit = in_vectors(S) ? 4 : 1, kBatch = 8;
        const int units = cols / kUnit;
        for (int u0 = threadIdx.x; u0 < units; u0 += kBatch * blockDim.x) {
            float v[kBatch][kUnit];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int j = (u0 + k * static_cast<int>(blockDim.x)) * kUnit;
#pragma unroll
                for (int e = 0; e < kUnit; ++e)
                    v[k][e] = absent;
                if (j < cols && p) {
                    if constexpr (kUnit == 1) {
                        v[k][0] = load_f32(p, bf16, j);
                    } else if (bf16) {
                        const uint2 h = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p) + j);
                        v[k][0] = __uint_as_float(h.x << 16);
                        v[k][1] = __uint_as_float(h.x & 0xFFFF0000u);
                        v[k][2] = __uint_as_float(h.y << 16);
                        v[k][3] = __uint_as_float(h.y & 0xFFFF0000u);
                    } else {
                        Vec16<float>::unpack(*reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + j), v[k]);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int j = (u0 + k * static_cast<int>(blockDim.x)) * kUnit;
                if (j < cols) {
                    if constexpr (kUnit == 1)
                        copy[j] = v[k][0];
                    else
                        *reinterpret_cast<uint4 *>(copy + (kPiece == 8 ? (j & 4 ? cols / 2 : 0) + j / 8 * 4 : j)) =
                            Vec16<float>::pack(v[k]);
                }
            }
        }
    }
};

// ------------------------------------------------------------ a row's threads
// One group's place in the CTA, and sums over its threads.
struct GroupScratch {
    float warp[2][2][64]; // double-buffered, so that a sum takes one barrier; two values
};

struct Group {
    int tpr, warps;    // threads, warps of a group
    int index;         // this group
    int t, warp, lane; // this thread in it
    int span;          // warps rounded up to a multiple of four: this group's part of the scratch
    int buffer = 0;
    GroupScratch *scratch;

    // Every thread of the CTA; __syncthreads() before the first sum.
    __device__ __forceinline__ Group(int thread, int tpr_, GroupScratch *s)
        : tpr(tpr_), warps(tpr_ / 32), index(thread / tpr_), t(thread % tpr_), warp(t / 32), lane(t % 32),
          span((warps + 3) / 4 * 4), scratch(s)
    {
        for (int k = thread; k < 64; k += blockDim.x)
            scratch->warp[0][0][k] = scratch->warp[0][1][k] = scratch->warp[1][0][k] = scratch->warp[1][1][k] = 0.0f;
    }
    // The sum of a group's values in the scratch (those past its warps are zero).
    __device__ __forceinline__ float add_up(const float *mine) const
    {
        const float4 *q = reinterpret_cast<const float4 *>(mine);
        float4 v = q[0];
        for (int k = 1; k < span / 4; ++k) {
            const float4 w = q[k];
            v.x += w.x;
            v.y += w.y;
            v.z += w.z;
            v.w += w.w;
        }
        return (v.x + v.y) + (v.z + v.w);
    }
    __device__ __forceinline__ void barrier() const
    {
        if (warps > 1)
            named_barrier(1 + index, tpr);
        else
            __syncwarp();
    }
    // Sums over the group, the same in all its threads.
    __device__ __forceinline__ float2 sum(float a, float b)
    {
        a = warp_sum(a);
        b = warp_sum(b);
        if (warps > 1) {
            float *mine = scratch->warp[buffer][0] + index * span;
            if (lane == 0) {
                mine[warp] = a;
                mine[64 + warp] = b;
            }
            named_barrier(1 + index, tpr);
            a = add_up(mine);
            b = add_up(mine + 64);
            buffer ^= 1;
        }
        return make_float2(a, b);
    }
    __device__ __forceinline__ float sum(float a)
    {
        a = warp_sum(a);
        if (warps > 1) {
            float *mine = scratch->warp[buffer][0] + index * span;
            if (lane == 0)
                mine[warp] = a;
            named_barrier(1 + index, tpr);
            a = add_up(mine);
            buffer ^= 1;
        }
        return a;
    }
};

// ------------------------------------------------------------ the ring
// One matrix the ring's rows come from.
struct Stream {
    const uint8_t *base;
    long long pitch; // bytes
};

// A group's ring: position i (its row first + i step) uses slot i % slots.
// Only whole 16-byte granules of a row are copied, to the offset in the slot
// that they have in global memory; what is left of an unaligned row at its two
// ends its threads read themselves.  A wait that runs out is recorded once;
// from then on the thread neither waits nor fills, and its group's barriers
// stay matched.
template <int Streams>
struct Ring {
    uint32_t bars, slots_at; // of this group
    int row_bytes, slot_bytes;
    int slots, rows;
    long long row, step; // the next position to fill
    unsigned int *status;
    unsigned long long limit;
    int withhold;
    bool filler;
    Stream in[Streams];
    int slot = 0; // of the position being computed
    uint32_t phase = 0;
    int ahead = 0;    // positions filled and not waited for
    int position = 0; // the next to fill
    bool failed = false;

    __device__ __forceinline__ Ring(uint32_t bars_at, uint32_t slots_base, const Shape &s, const Group &g, int row_bytes_,
                                    int rows_)
        : bars(bars_at + 8u * kMaxSlots * g.index),
          slots_at(slots_base + static_cast<uint32_t>(g.index * s.slots * Streams * s.slot_bytes)),
          row_bytes(row_bytes_), slot_bytes(s.slot_bytes), slots(s.slots), rows(rows_),
          row(static_cast<long long>(blockIdx.x) * s.groups + g.index),
          step(static_cast<long long>(gridDim.x) * s.groups), status(s.status), limit(s.wait_limit_ns),
          withhold(s.withhold), filler(g.t == 0)
    {
    }
    // Before the CTA barrier that publishes the mbarriers.
    __device__ __forceinline__ void init() const
    {
        if (filler) {
            for (int k = 0; k < slots; ++k)
                mbar_init(bars + 8u * k, 1);
            fence_barrier_init();
        }
    }
    __device__ __forceinline__ void start()
    {
        for (int k = 0; k < slots; ++k)
            fill(k);
    }
    // The next row, if there is one, into slot k, which nobody reads any more.
    __device__ __forceinline__ void fill(int k)
    {
        if (!filler || failed || row >= rows)
            return;
        if (position++ != withhold) { // test hook: this position is never filled
            const uint32_t bar = bars + 8u * k;
            uint64_t from[Streams];
            uint32_t bytes[Streams], total = 0;
#pragma unroll
            for (int i = 0; i < Streams; ++i) {
                const uint64_t first = reinterpret_cast<uint64_t>(in[i].base + row * in[i].pitch);
                const uint64_t end = (first + static_cast<uint64_t>(row_bytes)) & ~15ull;
                from[i] = (first + 15ull) & ~15ull;
                bytes[i] = end > from[i] ? static_cast<uint32_t>(end - from[i]) : 0u;
                total += bytes[i];
                from[i] |= first & 15ull ? 1ull : 0ull; // whether the first granule is only part of the row
            }
            mbar_arrive_expect_tx(bar, total);
#pragma unroll
            for (int i = 0; i < Streams; ++i)
                if (bytes[i] != 0)
                    bulk_load(slots_at + static_cast<uint32_t>((k * Streams + i) * slot_bytes) +
                                  (from[i] & 1ull ? 16u : 0u),
                              reinterpret_cast<const void *>(from[i] & ~1ull), bytes[i], bar);
            ++ahead;
        }
        row += step;
    }
    // Wait for the position to compute.
    __device__ __forceinline__ void wait()
    {
        if (failed)
            return;
        if (mbar_wait_bounded(bars + 8u * slot, phase, limit)) {
            --ahead;
        } else {
            failed = true;
            record_error(status, kErrFamilyLayerNorm | kErrRoleConsumer);
        }
    }
    // Row `r` of matrix i in the slot waited for; `own`: the group's slots.
    template <class T>
    __device__ __forceinline__ Row<T> view(const uint8_t *own, int i, long long r) const
    {
        const uint8_t *far = in[i].base + r * in[i].pitch;
        const int lead = static_cast<int>(reinterpret_cast<uint64_t>(far) & 15ull);
        const int size = static_cast<int>(sizeof(T));
        Row<T> v;
        v.near = reinterpret_cast<const T *>(own + (slot * Streams + i) * slot_bytes + lead);
        v.far = reinterpret_cast<const T *>(far);
        v.head = lead ? (16 - lead) / size : 0;
        v.tail = ((lead + row_bytes) / 16 * 16 - lead) / size; // at or before `head` when no granule is whole
        return v;
    }
    // Past a barrier of the group after its last read of the slot.
    __device__ __forceinline__ void next()
    {
        fill(slot);
        if (++slot == slots) {
            slot = 0;
            phase ^= 1u;
        }
    }
    // After a failure: what was filled and not waited for lands before the
    // CTA ends.
    __device__ __forceinline__ void drain()
    {
        if (!filler || !failed)
            return;
        for (int k = 0; k < slots && ahead > 0; ++k) {
            if (mbar_wait_bounded(bars + 8u * slot, phase, limit))
                --ahead;
            else
                record_error(status, kErrFamilyLayerNorm | kErrRoleDrain);
            if (++slot == slots) {
                slot = 0;
                phase ^= 1u;
            }
        }
    }
};

} // namespace ln

} // namespace pg
