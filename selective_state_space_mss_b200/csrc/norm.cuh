// norm.cuh -- residual add and layer norm (mss_norm_fwd, mss_norm_bwd).
//
//   s = x + residual, y = (s - mean) rstd w + b
//   ds = rstd (g - avg(g) - x^ avg(g x^)), g = dy w, x^ = (s - mean) rstd
//
// Bound by memory: every element is read and written once, with a few
// operations between, so a row is kept in the registers of the threads that
// share it -- a group of one to 32 warps (backward 16).
//
// Rows of whole 16-byte words are taken word by word.  Other rows begin anywhere
// in a word, but all tensors are dense and flat element k lies in the word that
// begins at element k - k % 8 (two words with fp32) of each of them: a row then
// has up to 7 elements in front of its first whole word and up to 7 behind its
// last one, which one warp takes with an element a lane.  Rows 8 apart begin at
// the same place in a word, so a group that strides over rows by a multiple of 8
// keeps its columns.
#pragma once

#include <cstdint>
#include <type_traits>

#include "mss_device.cuh"
#include "mss_params.h"
#include "ring.h"
#include "tma.cuh"

namespace mss {

constexpr int kNormStages = 4;  // slots of a group's ring at most
constexpr int kNormGroups = 18;  // groups of a block at most; 15 where they need a named barrier each
// How the rows lie: whole 16-byte words, parts of them behind aligned addresses,
// or anything.
enum NormRows { kRowsWide, kRowsShifted, kRowsStrided };
// Threads of a block of the backward pass at most.  One piece a thread through
// the ring: 576 leave the registers that 768 would spill (16384 x 768: 38 against 44
// us).  Strided loads, which tensors take that begin between words, need the
// threads of 768 although they spill (16384 x 1023 bf16 with a fp32 residual: 91 against
// 122 us).
template <int kRows, int kPieces> constexpr int kNormThreads = kPieces == 2 ? 512 : kRows == kRowsStrided ? 768 : 576;

// Eight elements of a row as four pairs, for packed two-wide arithmetic.
struct Octet {
    float2 v[4];
    __device__ __forceinline__ float& at(int i) { return i & 1 ? v[i >> 1].y : v[i >> 1].x; }
};

__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// Eight neighbouring elements (wide rows) as 16-byte words.
template <typename T> struct Raw;
template <> struct Raw<bf16_t> {
    uint4 a = {0u, 0u, 0u, 0u};
    __device__ __forceinline__ void load(const bf16_t* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ Octet get() const {
        return {{make_float2(bf16_lo(a.x), bf16_hi(a.x)), make_float2(bf16_lo(a.y), bf16_hi(a.y)),
                 make_float2(bf16_lo(a.z), bf16_hi(a.z)), make_float2(bf16_lo(a.w), bf16_hi(a.w))}};
    }
    static __device__ __forceinline__ void store(bf16_t* p, const Octet& o) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(o.v[0].x, o.v[0].y), pack_bf16x2(o.v[1].x, o.v[1].y),
                                                  pack_bf16x2(o.v[2].x, o.v[2].y), pack_bf16x2(o.v[3].x, o.v[3].y));
    }
};
template <> struct Raw<float> {
    float4 a = {0.f, 0.f, 0.f, 0.f}, b = {0.f, 0.f, 0.f, 0.f};
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ Octet get() const {
        return {{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
    }
    static __device__ __forceinline__ void store(float* p, const Octet& o) {
        reinterpret_cast<float4*>(p)[0] = make_float4(o.v[0].x, o.v[0].y, o.v[1].x, o.v[1].y);
        reinterpret_cast<float4*>(p)[1] = make_float4(o.v[2].x, o.v[2].y, o.v[3].x, o.v[3].y);
    }
};
// The same of a row that is not whole 16-byte words: element i lies G behind
// element i - 1, `n` of them inside the row.
template <typename T> struct Strided {
    T a[8];
    __device__ __forceinline__ void load(const T* p, int G, int n) {
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = i < n ? p[i * G] : T{};
    }
    __device__ __forceinline__ Octet get() const {
        Octet o;
#pragma unroll
        for (int i = 0; i < 8; ++i) o.at(i) = to_f32(a[i]);
        return o;
    }
};

// A thread's piece j of a row of `dim` elements shared by G threads: eight
// neighbours from column (j G + t) 8 on, with kRowsShifted from `front` columns
// further and whole words only, or columns 8 j G + t + i G, i < 8 (kRowsStrided).
// What lies behind the row is 0 and not stored.
template <int kRows>
struct Piece {
    int at;  // first column
    int n;   // elements of it inside the row (0 or 8 unless kRowsStrided)
    int G;
    __device__ __forceinline__ Piece(int j, int t, int G_, int dim, int front = 0) : G(G_) {
        if constexpr (kRows == kRowsStrided) {
            at = j * 8 * G + t;
            n = at >= dim ? 0 : min((dim - at + G - 1) / G, 8);
        } else {
            at = (j * G + t) * 8 + front;
            n = at + 8 <= dim ? 8 : 0;
        }
    }
    template <typename T> using Held = std::conditional_t<kRows == kRowsStrided, Strided<T>, Raw<T>>;
    template <typename T>
    __device__ __forceinline__ Held<T> load(const T* row) const {
        Held<T> r;
        if constexpr (kRows == kRowsStrided) {
            r.load(row + at, G, n);
        } else {
            if (n) r.load(row + at);
        }
        return r;
    }
    // of the weight or bias, which lie where the rows do not
    __device__ __forceinline__ Octet load_param(const float* v) const {
        if constexpr (kRows != kRowsShifted) {
            return load(v).get();
        } else {
            Octet o;
#pragma unroll
            for (int i = 0; i < 8; ++i) o.at(i) = n ? v[at + i] : 0.f;
            return o;
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T* row, Octet o) const {
        if constexpr (kRows == kRowsStrided) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) row[at + i * G] = from_f32<T>(o.at(i));
        } else {
            if (n) Raw<T>::store(row + at, o);
        }
    }
    __device__ __forceinline__ void store_sums(float* v, Octet o) const {
        if constexpr (kRows != kRowsShifted) {
            store(v, o);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (n) v[at + i] = o.at(i);
        }
    }
};

// A group's rows, which all begin `shift` elements into a word (kRowsShifted).
struct Edges {
    int front, count;  // elements in front of the whole words; those and the ones behind
    int64_t whole;     // elements in words that the tensors fill
    __device__ __forceinline__ Edges(int64_t row, int64_t rows, int dim, int& shift) : whole(rows * dim / 8 * 8) {
        shift = int(uint32_t(row) * uint32_t(dim) % 8u);
        front = min(-shift & 7, dim);
        count = front + ((dim - front) & 7);
    }
    __device__ __forceinline__ int column(int t, int dim) const { return t < front ? t : dim - count + t; }
    // first element and number of those to copy for a row; the last word of the
    // tensors, where they do not fill it, is left out
    __device__ __forceinline__ int64_t words(int64_t row, int dim, int shift, int& n) const {
        const int64_t at = row * dim - shift, end = (at + shift + dim + 7) / 8 * 8;
        n = int((end < whole ? end : whole) - at);
        return at;
    }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// Rows in registers: groups of G threads (a multiple of 32), a row each, kPieces
// pieces a thread; a block is one group or more.  A row's loads are all on their
// way before the first store.  The mean is taken first, then the squares about
// it.  16384 x 2048 bf16 with a fp32 residual: 66 us, 6.1 TB/s; 8 x 2560: 2.5 us.
template <typename T, typename R, int kRows, int kPieces>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const NormParams p, int G) {
    __shared__ float part[2][32];
    const int t = threadIdx.x % G, group = threadIdx.x / G, warps = G >> 5;
    const int64_t r = int64_t(blockIdx.x) * (blockDim.x / G) + group;
    const bool live = r < p.rows;
    const int64_t o = (live ? r : 0) * p.dim;
    const int dim = live ? int(p.dim) : 0;
    const float inv = 1.f / float(p.dim);
    typename Piece<kRows>::template Held<T> hx[kPieces];
    typename Piece<kRows>::template Held<R> hr[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        const Piece<kRows> q(j, t, G, dim);
        hx[j] = q.load(static_cast<const T*>(p.x) + o);
        if (p.residual) hr[j] = q.load(static_cast<const R*>(p.residual) + o);
    }
    Octet s[kPieces];
    float2 sum = both(0.f);
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        s[j] = hx[j].get();
        if (p.residual) {
            const Octet v = hr[j].get();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 a = __fadd2_rn(s[j].v[i], v.v[i]);
                s[j].v[i] = make_float2(to_f32(from_f32<R>(a.x)), to_f32(from_f32<R>(a.y)));
            }
        }
        if (p.residual_out) Piece<kRows>(j, t, G, dim).store(static_cast<R*>(p.residual_out) + o, s[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = __fadd2_rn(sum, s[j].v[i]);
    }
    const auto total = [&](float2 v2, float* tmp) {
        float v = warp_sum(v2.x + v2.y);
        if (warps > 1) {
            if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
            __syncthreads();
            v = 0.f;
#pragma unroll 4
            for (int k = 0; k < warps; ++k) v += tmp[group * warps + k];
        }
        return v;
    };
    const float mean = p.rms ? 0.f : total(sum, part[0]) * inv;
    sum = both(0.f);
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        const int n = Piece<kRows>(j, t, G, dim).n;
        if (kRows == kRowsWide && n == 0) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[j].v[i] = __fadd2_rn(s[j].v[i], both(-mean));
            if (kRows == kRowsStrided) {  // what lies behind the row adds nothing
                if (2 * i >= n) s[j].v[i].x = 0.f;
                if (2 * i + 1 >= n) s[j].v[i].y = 0.f;
            }
            sum = __ffma2_rn(s[j].v[i], s[j].v[i], sum);
        }
    }
    const float rstd = 1.f / sqrtf(total(sum, part[1]) * inv + p.eps);
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        const Piece<kRows> q(j, t, G, dim);
        const Octet w = q.load(p.weight).get();
        Octet y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y.v[i] = __fmul2_rn(__fmul2_rn(s[j].v[i], both(rstd)), w.v[i]);
        if (p.bias) {
            const Octet b = q.load(p.bias).get();
#pragma unroll
            for (int i = 0; i < 4; ++i) y.v[i] = __fadd2_rn(y.v[i], b.v[i]);
        }
        q.store(static_cast<T*>(p.y) + o, y);
    }
    if (live && t == 0) {
        if (p.mean) p.mean[r] = mean;
        if (p.rstd) p.rstd[r] = rstd;
    }
}

// Threads of a block of the forward pass over kRowsShifted at most.
template <int kPieces> constexpr int kNormRingThreads = kPieces == 2 ? 640 : 768;

// Forward pass over rows that begin anywhere in a word: as the backward pass
// below, each group of G threads takes every (blocks * groups)-th row, streamed
// through a ring in shared memory, and keeps its columns' weight and bias in
// registers.  16384 x 1023 bf16 with a fp32 residual: 38 us,
// 5.3 TB/s (by strides: 67 us); 1003 x 769 fp32 4.8 us.
template <typename T, typename R, int kPieces>
__global__ void __launch_bounds__(kNormRingThreads<kPieces>) norm_fwd_ring_kernel(const NormParams p, int G, int stages) {
    extern __shared__ __align__(128) unsigned char ring_mem[];
    __shared__ uint64_t full[kNormGroups * kNormStages];
    __shared__ float part[4][24];
    __shared__ int gave_up[2][kNormGroups];  // a bounded wait ran out: the group leaves behind the row
    using Row = Piece<kRowsShifted>;
    const int t = threadIdx.x % G, group = threadIdx.x / G, groups = blockDim.x / G, warps = G >> 5;
    const int64_t stride = int64_t(gridDim.x) * groups;
    int64_t r = int64_t(blockIdx.x) * groups + group;
    const int dim = int(p.dim);
    const float inv = 1.f / float(dim);
    int shift = 0;
    const Edges edges(r, p.rows, dim, shift);
    const bool edge = t < edges.count;  // this thread takes column ec too
    const int front = edges.front, ec = edge ? edges.column(t, dim) : 0;
    const int room = (dim + 14) / 8 * 8, tb = room * int(sizeof(T)), slot_bytes = tb + (p.residual ? room * int(sizeof(R)) : 0);
    unsigned char* ring = ring_mem + group * stages * slot_bytes;
    uint64_t* bar = full + group * kNormStages;
    const auto issue = [&](int slot, int64_t row) {  // one thread of the group
        if (row >= p.rows) return;
        unsigned char* to = ring + slot * slot_bytes;
        int count;
        const int64_t at = edges.words(row, dim, shift, count);
        const uint32_t tn = uint32_t(count * int(sizeof(T))), rn = p.residual ? uint32_t(count * int(sizeof(R))) : 0u;
        mbar_arrive_expect_tx(bar + slot, tn + rn);
        if (count == 0) return;
        bulk_load(to, static_cast<const T*>(p.x) + at, tn, bar + slot);
        if (p.residual) bulk_load(to + tb, static_cast<const R*>(p.residual) + at, rn, bar + slot);
    };
    if (t == 0) {
        gave_up[0][group] = gave_up[1][group] = 0;
        for (int k = 0; k < stages; ++k) mbar_init(bar + k, 1 + p.selftest);
        fence_barrier_init();
    }
    __syncthreads();
    if (t == 0)
        for (int k = 0; k < stages; ++k) issue(k, r + k * stride);
    Octet w[kPieces], b[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        w[j] = Row(j, t, G, dim, front).load_param(p.weight);
        if (p.bias) {
            b[j] = Row(j, t, G, dim, front).load_param(p.bias);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) b[j].v[i] = both(0.f);
        }
    }
    const float ew = edge ? p.weight[ec] : 0.f, eb = edge && p.bias ? p.bias[ec] : 0.f;
    const auto total = [&](float v, float* tmp) {  // over the group
        v = warp_sum(v);
        if (warps > 1) {
            if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(G) : "memory");
            v = 0.f;
#pragma unroll 4
            for (int k = 0; k < warps; ++k) v += tmp[group * warps + k];
        } else {
            __syncwarp();
        }
        return v;
    };
    int slot = 0, buf = 0;
    uint32_t parity = 0;
    for (; r < p.rows; r += stride, buf ^= 1) {
        const T* x = reinterpret_cast<const T*>(ring + slot * slot_bytes) + shift;
        const R* res = reinterpret_cast<const R*>(ring + slot * slot_bytes + tb) + shift;
        R* out = p.residual_out ? static_cast<R*>(p.residual_out) + r * p.dim : nullptr;
        if (!mbar_wait_bounded(bar + slot, parity, p.err, p.wait_ns)) gave_up[buf][group] = 1;
        Octet s[kPieces];
        float2 sum = both(0.f);
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const Row q(j, t, G, dim, front);
            s[j] = q.load(x).get();
            if (p.residual) {
                const Octet v = q.load(res).get();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 a = __fadd2_rn(s[j].v[i], v.v[i]);
                    s[j].v[i] = make_float2(to_f32(from_f32<R>(a.x)), to_f32(from_f32<R>(a.y)));
                }
            }
            if (out) q.store(out, s[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) sum = __fadd2_rn(sum, s[j].v[i]);
        }
        float es = 0.f;
        if (edge) {
            const bool loose = r * p.dim + ec >= edges.whole;  // not in the ring
            es = loose ? ld(static_cast<const T*>(p.x) + r * p.dim + ec) : ld(x + ec);
            if (p.residual) es = to_f32(from_f32<R>(es + (loose ? ld(static_cast<const R*>(p.residual) + r * p.dim + ec) : ld(res + ec))));
            if (out) out[ec] = from_f32<R>(es);
            sum.x += es;
        }
        const float mean = p.rms ? 0.f : total(sum.x + sum.y, part[buf]) * inv;
        sum = both(0.f);
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            if (Row(j, t, G, dim, front).n == 0) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[j].v[i] = __fadd2_rn(s[j].v[i], both(-mean));
                sum = __ffma2_rn(s[j].v[i], s[j].v[i], sum);
            }
        }
        if (edge) {
            es -= mean;
            sum.x = fmaf(es, es, sum.x);
        }
        const float rstd = 1.f / sqrtf(total(sum.x + sum.y, part[2 + buf]) * inv + p.eps);
        // the whole group has read the slot
        if (gave_up[buf][group]) {  // no more copies; those in flight are waited for
            drain_ring(slot, parity, stages, stages, [&](int k, int at, uint32_t phase) {
                if (r + k * stride >= p.rows) return;
                if (p.selftest && t == 0) mbar_arrive(bar + at);  // what the wait was for comes late
                mbar_wait_bounded(bar + at, phase, p.err);
            });
            break;
        }
        if (t == 0) issue(slot, r + stages * stride);
        if (++slot == stages) slot = 0, parity ^= 1;
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j].v[i] = __ffma2_rn(__fmul2_rn(s[j].v[i], both(rstd)), w[j].v[i], b[j].v[i]);
            Row(j, t, G, dim, front).store(static_cast<T*>(p.y) + r * p.dim, s[j]);
        }
        if (edge) static_cast<T*>(p.y)[r * p.dim + ec] = from_f32<T>(fmaf(es * rstd, ew, eb));
        if (t == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.rstd) p.rstd[r] = rstd;
        }
    }
}

// Backward pass, rows in registers.  A block is one group of G threads or more,
// each taking every (blocks * groups)-th row and keeping its columns' sums for
// dweight and dbias in registers; at the end the groups' sums are added in
// shared memory in order and the block writes its row of the partial sums.
// Unless kRowsStrided, each group streams its rows through a ring in shared
// memory, a row of s, dy and dresidual_out per slot (bulk copies, an mbarrier per
// slot).  dresidual_out is read from there again where it is added, which saves the
// registers of two pieces; a slot is filled anew once the whole group has come to
// the sums of the next row.  kRowsShifted: gridDim.x * groups * dim is a multiple of 8, or every group
// has one row.
// kMean: with avg(g) and dbias.  With the sum over the blocks, 16384 x 2048 bf16: 48
// us, 5.6 TB/s; 16384 x 768 with a fp32 residual: 38 us, 5.3 TB/s; 16384 x 1023: 55
// us, 4.9 TB/s (strided: 91 us).
template <typename T, typename S, int kRows, bool kMean, int kPieces>
__global__ void __launch_bounds__(kNormThreads<kRows, kPieces>) norm_bwd_kernel(const NormParams p, int G, int stages) {
    extern __shared__ __align__(128) unsigned char ring_mem[];
    __shared__ uint64_t full[kNormGroups * kNormStages];
    __shared__ float2 part[2][24];
    __shared__ int gave_up[2][kNormGroups];  // a bounded wait ran out: the group leaves behind the row
    const int t = threadIdx.x % G, group = threadIdx.x / G, groups = blockDim.x / G, warps = G >> 5;
    const int64_t stride = int64_t(gridDim.x) * groups;
    int64_t r = int64_t(blockIdx.x) * groups + group;
    const int dim = int(p.dim);
    const float inv = 1.f / float(dim);
    constexpr bool kRing = kRows != kRowsStrided;
    int shift = 0;
    const Edges edges(r, p.rows, dim, shift);
    const bool edge = kRows == kRowsShifted && t < edges.count;  // this thread takes column ec too
    const int front = kRows == kRowsShifted ? edges.front : 0, ec = edge ? edges.column(t, dim) : 0;
    const int64_t room = kRows == kRowsShifted ? (p.dim + 14) / 8 * 8 : p.dim;
    const int64_t sb = room * int64_t(sizeof(S)), tb = room * int64_t(sizeof(T));
    const int64_t slot_bytes = (p.residual ? 2 : 1) * sb + tb;
    unsigned char* ring = ring_mem + group * stages * slot_bytes;
    uint64_t* bar = full + group * kNormStages;
    const auto issue = [&](int slot, int64_t row) {  // one thread of the group
        if (row >= p.rows) return;
        unsigned char* to = ring + slot * slot_bytes;
        int count = dim;
        const int64_t at = kRows == kRowsShifted ? edges.words(row, dim, shift, count) : row * dim;
        const uint32_t sn = uint32_t(count * int(sizeof(S))), tn = uint32_t(count * int(sizeof(T)));
        mbar_arrive_expect_tx(bar + slot, (p.residual ? 2 : 1) * sn + tn);
        if (kRows == kRowsShifted && count == 0) return;
        bulk_load(to, static_cast<const S*>(p.x) + at, sn, bar + slot);
        bulk_load(to + sb, static_cast<const T*>(p.dy) + at, tn, bar + slot);
        if (p.residual) bulk_load(to + sb + tb, static_cast<const S*>(p.residual) + at, sn, bar + slot);
    };
    if (kRing) {
        if (t == 0) {
            gave_up[0][group] = gave_up[1][group] = 0;
            for (int k = 0; k < stages; ++k) mbar_init(bar + k, 1 + p.selftest);
            fence_barrier_init();
        }
        __syncthreads();
        if (t == 0)
            for (int k = 0; k < stages; ++k) issue(k, r + k * stride);
    }
    Octet w[kPieces], dw[kPieces], db[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        w[j] = Piece<kRows>(j, t, G, dim, front).load_param(p.weight);
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[j].v[i] = db[j].v[i] = both(0.f);
    }
    const float ew = edge ? p.weight[ec] : 0.f;
    float edw = 0.f, edb = 0.f;
    int slot = 0, used = -1, buf = 0;  // used: the slot of the row before
    uint32_t parity = 0;
    float next_mean = 0.f, next_rstd = 0.f;
    const auto fetch = [&](int64_t row) {
        if (row < p.rows) next_rstd = p.rstd[row];
        if (kMean && row < p.rows && p.mean) next_mean = p.mean[row];
    };
    fetch(r);
    for (; r < p.rows; r += stride, buf ^= 1) {
        const S* s = static_cast<const S*>(p.x) + r * p.dim;
        const T* dy = static_cast<const T*>(p.dy) + r * p.dim;
        const S* dres = p.residual ? static_cast<const S*>(p.residual) + r * p.dim : nullptr;
        const float rstd = next_rstd, mean = next_mean;
        fetch(r + stride);
        const S* const s_in = s;
        const T* const dy_in = dy;
        const S* const dres_in = dres;
        if (kRing) {
            s = reinterpret_cast<const S*>(ring + slot * slot_bytes) + shift;
            dy = reinterpret_cast<const T*>(ring + slot * slot_bytes + sb) + shift;
            if (dres) dres = reinterpret_cast<const S*>(ring + slot * slot_bytes + sb + tb) + shift;
            if (!mbar_wait_bounded(bar + slot, parity, p.err, p.wait_ns)) gave_up[buf][group] = 1;
        }
        Octet hat[kPieces], g[kPieces];
        typename Piece<kRows>::template Held<S> add[kRing ? 1 : kPieces];
        float2 a2 = both(0.f), b2 = both(0.f);
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const Piece<kRows> q(j, t, G, dim, front);
            hat[j] = q.load(s).get();
            g[j] = q.load(dy).get();
            if (!kRing && dres) add[j] = q.load(dres);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // the difference first: -mean rstd rounded would not cancel where the mean is far above the spread
                if (kMean) hat[j].v[i] = __fadd2_rn(hat[j].v[i], both(-mean));
                hat[j].v[i] = __fmul2_rn(hat[j].v[i], both(rstd));
                dw[j].v[i] = __ffma2_rn(g[j].v[i], hat[j].v[i], dw[j].v[i]);
                if (kMean) db[j].v[i] = __fadd2_rn(db[j].v[i], g[j].v[i]);
                g[j].v[i] = __fmul2_rn(g[j].v[i], w[j].v[i]);
                if (kMean) a2 = __fadd2_rn(a2, g[j].v[i]);
                b2 = __ffma2_rn(g[j].v[i], hat[j].v[i], b2);
            }
        }
        float ehat = 0.f, eg = 0.f;
        const bool loose = edge && r * dim + ec >= edges.whole;  // not in the ring
        if (edge) {
            const float d = loose ? ld(dy_in + ec) : ld(dy + ec);
            ehat = loose ? ld(s_in + ec) : ld(s + ec);
            ehat = (kMean ? ehat - mean : ehat) * rstd;
            edw = fmaf(d, ehat, edw);
            edb += d;
            eg = d * ew;
            a2.x += eg;
            b2.x = fmaf(eg, ehat, b2.x);
        }
        float a = a2.x + a2.y, b = b2.x + b2.y;
        // both sums at once: the lower half warp ends with a, the upper one with b
        const bool upper = threadIdx.x & 16;
        float v = (upper ? b : a) + __shfl_xor_sync(~0u, upper ? a : b, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
        if (warps > 1) {
            if ((threadIdx.x & 15) == 0) reinterpret_cast<float*>(&part[buf][threadIdx.x >> 5])[upper] = v;
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(G) : "memory");
            a = b = 0.f;
            const float2* all = part[buf] + group * warps;
#pragma unroll 4
            for (int k = 0; k < warps; ++k) {
                a += all[k].x;
                b += all[k].y;
            }
        } else {
            a = __shfl_sync(~0u, v, 0);
            b = __shfl_sync(~0u, v, 16);
            __syncwarp();
        }
        if (kRing) {  // the whole group is done with the slot of the row before
            if (gave_up[buf][group]) {  // no more copies; those in flight are waited for (`used` is not filled anew yet)
                drain_ring(slot, parity, stages, used < 0 ? stages : stages - 1, [&](int k, int at, uint32_t phase) {
                    if (r + k * stride >= p.rows) return;
                    if (p.selftest && t == 0) mbar_arrive(bar + at);  // what the wait was for comes late
                    mbar_wait_bounded(bar + at, phase, p.err);
                });
                break;
            }
            if (t == 0 && used >= 0) issue(used, r + (stages - 1) * stride);
            used = slot;
            if (++slot == stages) slot = 0, parity ^= 1;
        }
        // rstd (g - a - hat b)
        const float ra = kMean && p.mean ? -rstd * a * inv : 0.f, rb = -rstd * b * inv;
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const Piece<kRows> q(j, t, G, dim, front);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                g[j].v[i] = __ffma2_rn(g[j].v[i], both(rstd), __ffma2_rn(hat[j].v[i], both(rb), both(ra)));
            if (dres) {
                Octet more;
                if constexpr (kRing) {
                    more = q.load(dres).get();
                } else {
                    more = add[j].get();
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) g[j].v[i] = __fadd2_rn(g[j].v[i], more.v[i]);
            }
            if (p.y) q.store(static_cast<T*>(p.y) + r * p.dim, g[j]);
            if (p.residual_out) q.store(static_cast<S*>(p.residual_out) + r * p.dim, g[j]);
        }
        if (edge) {
            float d = fmaf(eg, rstd, fmaf(ehat, rb, ra));
            if (dres) d += loose ? ld(dres_in + ec) : ld(dres + ec);
            if (p.y) static_cast<T*>(p.y)[r * p.dim + ec] = from_f32<T>(d);
            if (p.residual_out) static_cast<S*>(p.residual_out)[r * p.dim + ec] = from_f32<S>(d);
        }
    }
    if (!p.part) return;
    launch_dependents();
    // the groups' sums, in order; every copy into the ring has arrived
    __syncthreads();
    float* all = reinterpret_cast<float*>(ring_mem);
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        const Piece<kRows> q(j, t, G, dim, front);
        q.store_sums(all + int64_t(group) * 2 * p.dim, dw[j]);
        q.store_sums(all + int64_t(group) * 2 * p.dim + p.dim, db[j]);
    }
    if (edge) {
        all[int64_t(group) * 2 * p.dim + ec] = edw;
        all[int64_t(group) * 2 * p.dim + p.dim + ec] = edb;
    }
    __syncthreads();
    for (int64_t i = threadIdx.x; i < 2 * p.dim; i += blockDim.x) {
        float v = 0.f;
        for (int k = 0; k < groups; ++k) v += all[int64_t(k) * 2 * p.dim + i];
        p.part[int64_t(blockIdx.x) * 2 * p.dim + i] = v;
    }
}

// Sum over the block (at most 32 warps), the same value in every thread;
// `tmp` may be used again behind the next block barrier.
__device__ __forceinline__ float block_sum(float v, float* tmp) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int k = 0; k < warps; ++k) s += tmp[k];
    __syncthreads();
    return s;
}

// s of one element: the sum rounded to the residual's type.
template <typename T, typename R>
__device__ __forceinline__ float norm_input(const T* x, const R* res, int64_t i) {
    const float v = ld(x + i);
    return res ? to_f32(from_f32<R>(v + ld(res + i))) : v;
}

// Rows past 16384 elements, one block per row: the row is read three times
// (2048 x 20000 bf16 with a fp32 residual 328 us, 1.5 TB/s).
template <typename T, typename R>
__global__ void norm_fwd_long_kernel(const NormParams p) {
    __shared__ float tmp[32];
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(p.x) + r * p.dim;
        const R* res = p.residual ? static_cast<const R*>(p.residual) + r * p.dim : nullptr;
        R* out = p.residual_out ? static_cast<R*>(p.residual_out) + r * p.dim : nullptr;
        T* y = static_cast<T*>(p.y) + r * p.dim;
        float mean = 0.f, acc = 0.f;
        if (!p.rms) {
            for (int64_t i = threadIdx.x; i < p.dim; i += blockDim.x) acc += norm_input(x, res, i);
            mean = block_sum(acc, tmp) / float(p.dim);
        }
        acc = 0.f;
        for (int64_t i = threadIdx.x; i < p.dim; i += blockDim.x) {
            const float s = norm_input(x, res, i);
            if (out) out[i] = from_f32<R>(s);
            acc = fmaf(s - mean, s - mean, acc);
        }
        const float rstd = 1.f / sqrtf(block_sum(acc, tmp) / float(p.dim) + p.eps);
        for (int64_t i = threadIdx.x; i < p.dim; i += blockDim.x) {
            const float v = (norm_input(x, res, i) - mean) * rstd * p.weight[i];
            y[i] = from_f32<T>(p.bias ? v + p.bias[i] : v);
        }
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.rstd) p.rstd[r] = rstd;
        }
    }
}

// Rows past 8192 elements.  A block takes every gridDim.x-th row; its sums for
// dweight and dbias stay in its own row of the partial sums, each column in one
// thread's hands.  Element loads, and the sums go through memory with every row:
// 4096 x 12288 bf16 with a fp32 residual 852 us, 0.9 TB/s (8192 columns, in registers: 4.4).
template <typename T, typename S>
__global__ void norm_bwd_long_kernel(const NormParams p) {
    __shared__ float tmp[32];
    float* dw = p.part ? p.part + int64_t(blockIdx.x) * 2 * p.dim : nullptr;
    float* db = dw ? dw + p.dim : nullptr;
    if (dw)
        for (int64_t i = threadIdx.x; i < p.dim; i += blockDim.x) dw[i] = db[i] = 0.f;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const S* s = static_cast<const S*>(p.x) + r * p.dim;
        const T* dy = static_cast<const T*>(p.dy) + r * p.dim;
        const S* dres = p.residual ? static_cast<const S*>(p.residual) + r * p.dim : nullptr;
        T* dx = p.y ? static_cast<T*>(p.y) + r * p.dim : nullptr;
        S* dro = p.residual_out ? static_cast<S*>(p.residual_out) + r * p.dim : nullptr;
        const float mean = p.mean ? p.mean[r] : 0.f, rstd = p.rstd[r];
        float a = 0.f, b = 0.f;
        for (int64_t i = threadIdx.x; i < p.dim; i += blockDim.x) {
            const float d = ld(dy + i), hat = (ld(s + i) - mean) * rstd, g = d * p.weight[i];
            a += g;
            b = fmaf(g, hat, b);
            if (dw) {
                dw[i] += d * hat;
                db[i] += d;
            }
        }
        a = p.mean ? block_sum(a, tmp) / float(p.dim) : 0.f;
        b = block_sum(b, tmp) / float(p.dim);
        for (int64_t i = threadIdx.x; i < p.dim; i += blockDim.x) {
            const float hat = (ld(s + i) - mean) * rstd, g = ld(dy + i) * p.weight[i];
            float d = rstd * (g - a - hat * b);
            if (dres) d += ld(dres + i);
            if (dx) dx[i] = from_f32<T>(d);
            if (dro) dro[i] = from_f32<S>(d);
        }
    }
}

}  // namespace mss
