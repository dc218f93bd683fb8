// What the layer norm kernels share: how a row is spread over threads, how
// its sums are formed, and the ring through which rows reach shared memory.
//
// A group of `tpr` threads (whole warps) takes a row, each thread E of its
// elements in registers; a CTA holds `groups` groups.  Elements move in 16-byte
// vectors: straight where the rows are 16-byte aligned; where they are not,
// through shared memory, there shifted (kRingShifted) or read one by one
// (kRingElement), or, when there are too few rows for a ring, one by one from
// where they are.
//
// Ring: the first thread of each group copies the group's rows into shared
// memory (bulk copies completing on mbarriers), several ahead of the one being
// computed, so that the bytes in flight do not depend on how many registers
// the computation leaves.  A slot is refilled once a barrier of the group's
// sums shows that its threads have taken their elements.  With no more than a
// row or two to a group there is nothing to run ahead of, and threads load
// their elements themselves.
//
// Beside DRAM these kernels spend their time on instructions per element and on
// waiting for a row's reductions, so additions and multiplications run on pairs
// (one instruction for two float32 values), and a thread has enough elements to
// spread the cost of the reductions over.
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
// kRingShifted: rows of any alignment and length.  A piece is cut out of the
// two 16-byte granules of shared memory it lies in, and a warp's pieces are
// shifted against each other to the granules of the output: 8192 rows of 8192
// bfloat16 at a pitch of 8195 take 68 us forward and 115 backward, 142 and 193
// element by element; in float32 the forward 89 and 128.
// kRingElement: the same rows element by element, which for the gradient of
// float32 rows, two rows read and one written, costs less than their
// selections: 8192 x 8192 at a pitch of 8195 takes 132 us, shifted 159 (134
// and 184 where the output has that pitch too); 16384 x 1000 at 1001 40 and
// 43, 40000 x 33 34 and 50.
enum Source { kRingFull, kRingVector, kRingShifted, kRingElement, kVector, kScalar };
constexpr bool unaligned(Source s) { return s == kRingShifted || s == kRingElement; }
constexpr bool from_ring(Source s) { return s == kRingFull || s == kRingVector || unaligned(s); }
constexpr bool in_vectors(Source s) { return s != kScalar && s != kRingElement; }

// Floats that a parameter's copy in shared memory takes: whole pieces.
__host__ __device__ constexpr int parameter_floats(int cols) { return (cols + 7) / 8 * 8; }

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
// A row where a thread finds it: in shared memory or in global memory.
template <class T>
struct Row {
    const T *at;
    int lead; // bytes of its first granule before it (kRingShifted)
};

// The sixteen bytes at byte s of a and b in a row; s below 16, a whole number
// of T.  By selections: branching on the row's s instead took a third longer
// in float32, whose registers then spill.
template <class T>
__device__ __forceinline__ uint4 window(const uint4 &a, const uint4 &b, int s)
{
    const bool two = s & 8, one = s & 4;
    const uint32_t c0 = two ? a.z : a.x, c1 = two ? a.w : a.y, c2 = two ? b.x : a.z, c3 = two ? b.y : a.w,
                   c4 = two ? b.z : b.x, c5 = two ? b.w : b.y;
    const uint32_t d0 = one ? c1 : c0, d1 = one ? c2 : c1, d2 = one ? c3 : c2, d3 = one ? c4 : c3;
    if constexpr (sizeof(T) == 4)
        return make_uint4(d0, d1, d2, d3);
    const uint32_t d4 = one ? c5 : c4, bits = (s & 2) * 8;
    return make_uint4(__funnelshift_r(d0, d1, bits), __funnelshift_r(d1, d2, bits), __funnelshift_r(d2, d3, bits),
                      __funnelshift_r(d3, d4, bits));
}

// Where a thread has its elements: warp w of a group takes 32 E columns in a
// row, piece k (a vector, or one element) of its lane l starting at column
// 32 E w + (32 k + l) kPiece, a constant distance from piece to piece.
template <class T, int E, Source S>
struct Spread {
    static constexpr int kPiece = in_vectors(S) ? Vec16<T>::kElements : 1;
    static constexpr int kPieces = E / kPiece;
    int first;  // column of piece 0
    int cols;
    int pieces; // of this thread that lie in the row (kRingShifted: the last perhaps in part)
    bool full;  // every lane of the warp has all of them, whole

    __device__ __forceinline__ Spread(int t, int cols_) : first(t / 32 * 32 * E + t % 32 * kPiece), cols(cols_)
    {
        const int left = (cols - first + 32 * kPiece - 1) / (32 * kPiece);
        pieces = cols > first ? (left < kPieces ? left : kPieces) : 0;
        const bool whole = S != kRingShifted || column(kPieces - 1) + kPiece <= cols;
        full = __all_sync(0xffffffffu, pieces == kPieces && whole);
    }
    __device__ __forceinline__ int column(int k) const { return first + k * (32 * kPiece); }
    __device__ __forceinline__ bool has(int k) const { return S == kRingFull || k < pieces; }
    // Element e of piece k.
    __device__ __forceinline__ bool has(int k, int e) const
    {
        return S == kRingShifted ? column(k) + e < cols : has(k);
    }

    __device__ __forceinline__ void load_piece(const Row<T> &row, int k, float *v) const
    {
        if constexpr (S == kRingShifted) {
            const uint4 *q = reinterpret_cast<const uint4 *>(
                reinterpret_cast<const uint8_t *>(row.at + (has(k) ? column(k) : 0)) - row.lead);
            Vec16<T>::unpack(window<T>(q[0], q[1], row.lead), v);
            if (!full) {
#pragma unroll
                for (int e = 0; e < kPiece; ++e)
                    v[e] = has(k, e) ? v[e] : 0.0f;
            }
        } else if (has(k)) {
            const int j = column(k);
            if constexpr (!in_vectors(S))
                v[0] = to_f32(row.at[j]);
            else
                Vec16<T>::unpack(*reinterpret_cast<const uint4 *>(row.at + j), v);
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
            if (!has(2 * i / kPiece, 2 * i % kPiece))
                a = 0.0f;
            if (!has((2 * i + 1) / kPiece, (2 * i + 1) % kPiece))
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
                unpack_bf16(h.x, v);
                unpack_bf16(h.y, v + 2);
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
        const int j = has(k) ? column(k) : 0, half = S == kRingShifted ? parameter_floats(cols) / 2 : cols / 2;
        if constexpr (kPiece == 8) {
            Vec16<float>::unpack(*reinterpret_cast<const uint4 *>(copy + j / 2), v);
            Vec16<float>::unpack(*reinterpret_cast<const uint4 *>(copy + half + j / 2), v + 4);
        } else if constexpr (kPiece == 4) {
            Vec16<float>::unpack(*reinterpret_cast<const uint4 *>(copy + j), v);
        } else {
            v[0] = copy[j];
        }
    }
    // A parameter vector as float32 in shared memory, by the whole CTA.  For
    // pieces of eight the first halves of all pieces come before the second
    // halves, so that neighbouring threads' 16-byte reads are neighbours.  What
    // a last piece has beyond the row is `absent` too: it meets zeros, and must
    // be finite.
    __device__ __forceinline__ void copy_parameter(float *copy, const void *p, bool bf16, float absent) const
    {
        // Several loads of a thread in flight: the first rows wait for them.
        constexpr int kUnit = unaligned(S) ? 1 : 4, kBatch = 8;
        const int half = parameter_floats(cols) / 2, there = unaligned(S) ? 2 * half : cols;
        for (int u0 = threadIdx.x; u0 < there / kUnit; u0 += kBatch * blockDim.x) {
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
                        unpack_bf16(h.x, v[k]);
                        unpack_bf16(h.y, v[k] + 2);
                    } else {
                        Vec16<float>::unpack(*reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + j), v[k]);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int j = (u0 + k * static_cast<int>(blockDim.x)) * kUnit;
                if (j < there) {
                    float *to = copy + (kPiece == 8 ? (j & 4 ? half : 0) + j / 8 * 4 + j % 4 : j);
                    if constexpr (kUnit == 1)
                        *to = v[k][0];
                    else
                        *reinterpret_cast<uint4 *>(to) = Vec16<float>::pack(v[k]);
                }
            }
        }
    }
};

// A row of the output, written piece by piece: put() for every piece in turn,
// then finish(), by whole warps.  kRingShifted: where the row starts `off`
// bytes into a granule, a lane writes the granule in which its piece begins,
// whose first `off` bytes are the end of the piece before: the lane's before
// it, or for the first lane the last lane's of the round before.  What lies in
// granules that two warps share goes element by element.
template <class T, int E, Source S>
struct RowOut {
    using At = Spread<T, E, S>;
    const At &at;
    T *row;
    int off;
    uint4 edge = {}; // the first lane's first piece, the last lane's last

    __device__ __forceinline__ RowOut(const At &at_, T *row_)
        : at(at_), row(row_), off(static_cast<int>(reinterpret_cast<uintptr_t>(row_) & 15u))
    {
    }
    // Elements from .. to-1 of q, whose element 0 belongs to column j.
    __device__ __forceinline__ void elements(const uint4 &q, int j, int from, int to) const
    {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < At::kPiece; ++e) {
            if (e < from || e >= to)
                continue;
            if constexpr (sizeof(T) == 4)
                row[j + e] = __uint_as_float(w[e]);
            else
                row[j + e] = __ushort_as_bfloat16(static_cast<unsigned short>(w[e / 2] >> (16 * (e & 1))));
        }
    }
    __device__ __forceinline__ void put(int k, const float *v)
    {
        if constexpr (S != kRingShifted) {
            at.store_piece(row, k, v);
        } else {
            const uint4 q = Vec16<T>::pack(v);
            const int lane = static_cast<int>(threadIdx.x) & 31;
            int j = at.column(k), from = 0;
            uint4 out = q;
            if (off != 0) {
                const uint4 sent = lane == 31 ? edge : q;
                uint4 before;
                before.x = __shfl_sync(0xffffffffu, sent.x, (lane + 31) & 31);
                before.y = __shfl_sync(0xffffffffu, sent.y, (lane + 31) & 31);
                before.z = __shfl_sync(0xffffffffu, sent.z, (lane + 31) & 31);
                before.w = __shfl_sync(0xffffffffu, sent.w, (lane + 31) & 31);
                out = window<T>(before, q, 16 - off);
                j -= off / static_cast<int>(sizeof(T));
                if (lane == 0 ? k == 0 : lane == 31)
                    edge = q;
                if (k == 0 && lane == 0)
                    from = At::kPiece; // finish() writes it
            }
            const int to = at.cols - j;
            if (from == 0 && to >= At::kPiece)
                *reinterpret_cast<uint4 *>(row + j) = out;
            else if (from == 0 && to > 0)
                elements(out, j, 0, to);
        }
    }
    __device__ __forceinline__ void finish() const
    {
        if constexpr (S == kRingShifted) {
            const int lane = static_cast<int>(threadIdx.x) & 31;
            if (off != 0 && (lane == 0 || lane == 31)) {
                const int cut = At::kPiece - off / static_cast<int>(sizeof(T));
                const int j = at.column(lane == 0 ? 0 : At::kPieces - 1), left = at.cols - j;
                elements(edge, j, lane == 0 ? 0 : cut, lane == 0 ? min(cut, left) : left);
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
// ends follows through registers (Edges).  A wait that runs out is recorded once;
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

    __device__ __forceinline__ Ring(uint32_t bars_at, uint32_t slots_base, const Shape &s, const Group &g,
                                    int row_bytes_, int rows_)
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
        const int lead = static_cast<int>(reinterpret_cast<uint64_t>(in[i].base + r * in[i].pitch) & 15ull);
        return Row<T>{reinterpret_cast<const T *>(own + (slot * Streams + i) * slot_bytes + lead), lead};
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

// The elements of unaligned rows in granules that are not wholly the row's, at
// most seven at each end.  Eight lanes of a group's first warp hold each end
// of each matrix's row, loaded a row before it is written into its slot, which
// is a row before it is read: no row waits for them.
template <class T, int Streams>
struct Edges {
    static_assert(16 * Streams <= 32, "a warp holds a row's edges");
    T value{};
    int at = -1; // its byte in the slot, if this lane holds one

    __device__ __forceinline__ void load(const Ring<Streams> &ring, const Group &g, long long r)
    {
        at = -1;
        const int i = g.lane / 16;
        if (g.warp != 0 || i >= Streams || r >= ring.rows)
            return;
        const int size = static_cast<int>(sizeof(T)), cols = ring.row_bytes / size;
        const Stream in = i == 0 ? ring.in[0] : ring.in[Streams - 1]; // in registers
        const T *row = reinterpret_cast<const T *>(in.base + r * in.pitch);
        const int lead = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15u);
        const int head = lead ? min((16 - lead) / size, cols) : 0;
        const int tail = max(((lead + ring.row_bytes) / 16 * 16 - lead) / size, head);
        const int j = g.lane % 8 + (g.lane & 8 ? tail : 0);
        if (j < (g.lane & 8 ? cols : head)) {
            value = row[j];
            at = i * ring.slot_bytes + lead + j * size;
        }
    }
    // Into the group's slot k, which nobody reads any more.
    __device__ __forceinline__ void place(const Ring<Streams> &ring, uint8_t *own, int k) const
    {
        if (at >= 0)
            *reinterpret_cast<T *>(own + k * Streams * ring.slot_bytes + at) = value;
        __syncwarp();
    }
};

} // namespace ln

} // namespace pg
