// glr.cuh -- the gated linear recurrence (mss_glr_fwd, mss_glr_bwd,
// mss_glr_update).
//
//   f_t = sigmoid(s_t), h_t = f_t h_{t-1} + (1 - f_t) x_t, y_t = h_t silu(z_t)
//
// One pass over the data.  A token maps the state h to P h + H, and such maps
// compose to (P2 P1, P2 H1 + H2), so a span of tokens reduces to one pair.  A
// block owns 64 channels and walks the sequence in tiles of 64 tokens; each of
// its warps takes 8 tokens of a tile (two channels per lane, packed two-wide
// arithmetic), keeps their gates and inputs in registers and reduces them to a
// pair.  One warp composes the warps' pairs from shared memory and hands each
// warp the state before its first token, from which the warp runs its tokens
// in order.  Every warp streams its own tokens into its own ring in shared
// memory (TMA boxes of 8 tokens x 64 channels), a tile or more ahead.  With few
// channels a cluster of blocks shares the sequence: block r takes tiles r, r +
// S, ..., and the blocks send each other their tiles' pairs (st.async into the
// peers' shared memory, counted by an mbarrier), so that the sequence still
// goes by in one pass.
//
// Packed sequences are one scan over all tokens in which the first token of a
// sequence takes its state from initial_state.  A pair that holds such a token
// does not depend on the state before it; its P is then the mark kGlrCut, and the
// state is dropped instead of multiplied by zero, so that an infinity or NaN
// of one sequence does not reach another.
//
// Backward, E_t = f_t dh_t is handed from a token to the one before it, and
// dh_t = u_t + E_{t+1} with u_t = dy_t silu(z_t): E_t = f_t E_{t+1} + f_t u_t is the
// same scan in the other direction, with the same products of gates, and
// over a warp's tokens sum_t (f_0 .. f_t) u_t is its constant term.  The states
// are recomputed from the one saved before every 64 tokens.
#pragma once

#include <cstdint>
#include <type_traits>

#include "mss_device.cuh"
#include "mss_params.h"
#include "ring.h"
#include "tma.cuh"

namespace mss {

constexpr int kGlrLanes = 2;                        // channels per lane
constexpr int kGlrCols = 32 * kGlrLanes;            // channels per block
constexpr int kGlrRun = 8;                          // tokens per warp and tile
constexpr int kGlrWarps = 8;
constexpr int kGlrThreads = 32 * kGlrWarps;
constexpr int kGlrTile = kGlrRun * kGlrWarps;       // tokens per tile; a saved state before every tile
constexpr int kGlrMaxCluster = 16;

// Slots of a ring.  fp32 boxes are twice as large: where two slots would leave
// an SM one block instead of two, one slot and the other block's work hide the
// loads better (1 x 3001 x 1001 fp32 with z forward: 24 against 31 us, backward
// 36 against 44 us; 4 x 4096 x 4096 fp32 backward 331 against 395 us).
template <typename T, bool kTma, bool kBwd> constexpr int kGlrStages = sizeof(T) == 4 && (kBwd || !kTma) ? 1 : 2;
constexpr int kGlrSlotBytes = 32 * 16;              // a block's pair of each of its channels

// Elements of a token's row in a box: 64 channels, without TMA the 16-byte
// pieces that 64 channels can touch.
template <typename T, bool kTma> constexpr int kGlrPitch = kGlrCols + (kTma ? 0 : 16 / int(sizeof(T)));
template <typename T, bool kTma> constexpr int kGlrBox = kGlrRun * kGlrPitch<T, kTma>;  // elements of a box
// Bytes of a block's rings of `arrays` tensors, and of its shared memory in all.
template <typename T, bool kTma, bool kBwd> __host__ __device__ constexpr int glr_ring(int arrays) {
    return kGlrWarps * kGlrStages<T, kTma, kBwd> * arrays * kGlrBox<T, kTma> * int(sizeof(T));
}
template <typename T, bool kTma, bool kBwd> constexpr int glr_smem(int arrays, int cluster) {
    return glr_ring<T, kTma, kBwd>(arrays) + (cluster > 1 ? 2 * cluster * kGlrSlotBytes : 0);
}

struct GlrMaps {
    CUtensorMap gate, x, z, dy;
};

// ---------------------------------------------------------------------------
// Arithmetic on the two channels of a lane.

__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }

// min(a, cap) that keeps a NaN
__device__ __forceinline__ float glr_cap(float a, float cap) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(cap));
    return r;
}

// max(a, low) that keeps a NaN
__device__ __forceinline__ float glr_floor(float a, float low) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(low));
    return r;
}

// e^-s of the argument -s (fp32 io) or -s log2(e) (bf16 io, the
// single-instruction exponential; with fp32 io its error would add up over a
// long memory, and expf and the rounded reciprocal are used).  kGlrScale turns
// a gate into the argument.  Capped at 2^124, which leaves 1 + e a reciprocal.
template <typename T> constexpr float kGlrScale = -1.f;
template <> constexpr float kGlrScale<bf16_t> = -kLog2e;
template <typename T> constexpr float kGlrCap = 124.f / kLog2e;
template <> constexpr float kGlrCap<bf16_t> = 124.f;

template <typename T>
__device__ __forceinline__ float2 glr_exp(float2 a) {
    if constexpr (sizeof(T) == 2) return make_float2(ex2_approx(a.x), ex2_approx(a.y));
    else return make_float2(expf(a.x), expf(a.y));
}
template <typename T>
__device__ __forceinline__ float2 glr_rcp(float2 a) {
    if constexpr (sizeof(T) == 2) return make_float2(rcp_approx(a.x), rcp_approx(a.y));
    else return make_float2(__frcp_rn(a.x), __frcp_rn(a.y));
}

// f, an approximation of 1 / d, after one step of Newton's method.  A gate that
// holds its state has f next to 1 for thousands of tokens, over which an error
// of the approximation adds up; with the step f is within its rounding, and
// exactly 1 at d = 1.
__device__ __forceinline__ float2 glr_refine(float2 f, float2 d) {
    return __ffma2_rn(f, __ffma2_rn(make_float2(-d.x, -d.y), f, splat(1.f)), f);
}

// f = sigmoid(s) = 1 / (1 + e) and w = 1 - f = e / (1 + e) with e = e^-s: no
// subtraction, so both keep their precision.  The cap on e keeps w finite and
// f at least 2^-124.
template <typename T>
__device__ __forceinline__ void sigmoid2(float2 arg, float2& f, float2& w) {
    const float2 e = glr_exp<T>(make_float2(glr_cap(arg.x, kGlrCap<T>), glr_cap(arg.y, kGlrCap<T>)));
    const float2 d = __fadd2_rn(e, splat(1.f));
    f = glr_rcp<T>(d);
    if (sizeof(T) == 2) f = glr_refine(f, d);
    w = __fmul2_rn(e, f);
}

// The same for the forget gate (f, w) and the output gate (g, n) of a token, and
// silu(z) = z g, with one reciprocal for both: the kernels run into the rate of the
// multi-function unit, 3 instead of 4 of its instructions per element.  The
// output gate's 1 + e is held times 2^-124, so that the product of both
// denominators has a reciprocal although either e goes up to 2^124.  Below the z
// where e has reached its cap the product takes that z: silu(z) is then -86 x 2^-124,
// and not z times a g that has stopped falling (4 x 4096 x 4096 forward 110 us, with e^-|z|
// and selections, which go on to 0, 113 us).
// A NaN must not cross over: the output gate's argument drops its NaN (the
// product with z has it), and a NaN forget gate makes NaN only what it
// makes NaN anyway, the token's state and what follows from it.
template <typename T>
__device__ __forceinline__ void sigmoid2_both(float2 arg, float2 z, float2& f, float2& w, float2& g, float2& n, float2& silu) {
    constexpr float kScaled = 0x1p-124f, kLowest = kGlrCap<T> / kGlrScale<T>;
    const float2 argz = __fmul2_rn(z, splat(kGlrScale<T>));
    const float2 e = glr_exp<T>(make_float2(glr_cap(arg.x, kGlrCap<T>), glr_cap(arg.y, kGlrCap<T>)));
    const float2 ez = glr_exp<T>(make_float2(fminf(argz.x, kGlrCap<T>), fminf(argz.y, kGlrCap<T>)));
    const float2 d = __fadd2_rn(e, splat(1.f)), dz = __ffma2_rn(ez, splat(kScaled), splat(kScaled));
    const float2 r = glr_rcp<T>(__fmul2_rn(d, dz));
    f = glr_refine(__fmul2_rn(r, dz), d);
    w = __fmul2_rn(e, f);
    g = __fmul2_rn(__fmul2_rn(r, d), splat(kScaled));
    n = __fmul2_rn(ez, g);
    silu = __fmul2_rn(make_float2(glr_floor(z.x, kLowest), glr_floor(z.y, kLowest)), g);
}

// A lane's two channels of one token, in shared and in global memory.
__device__ __forceinline__ float2 glr_get(const bf16_t* box, int at) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(box + at);
    return make_float2(bf16_lo(v), bf16_hi(v));
}
__device__ __forceinline__ float2 glr_get(const float* box, int at) { return *reinterpret_cast<const float2*>(box + at); }

__device__ __forceinline__ void glr_put(bf16_t* p, float2 v) { *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(v.x, v.y); }
__device__ __forceinline__ void glr_put(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }

// P of a span in which a sequence begins has its sign set, in the first channel
// of a lane; the sign of any other, which may be a NaN, is cleared.
constexpr float kGlrCut = -1.f;
__device__ __forceinline__ bool glr_cut(float P) { return __float_as_int(P) < 0; }
template <bool kCuts>
__device__ __forceinline__ float2 glr_apply(float2 P, float2 H, float2 h) {
    const float2 r = __ffma2_rn(P, h, H);
    if (!kCuts) return r;
    const bool cut = glr_cut(P.x);  // one of the whole row
    return make_float2(cut ? H.x : r.x, cut ? H.y : r.y);
}

// The sequences of packed tokens that begin or end among a warp's kGlrRun
// tokens.  Each lane holds the offsets of one of 32 neighbouring sequences from s0
// on; behind them a 32-way search finds the next ones.  Tiles without a border
// cost one comparison with the next border's place.  Every index is checked
// against nseq and the tile, so offsets of any content stay inside the arrays.
template <bool kBackward>
struct GlrCursor {
    int s0 = -1, a = 0, b = 0;
    int border = kBackward ? INT32_MAX : INT32_MIN;  // no border before it in the scan's order

    // A bit for every token from t0 on that begins a sequence, from bit 8 on for
    // those that end one; start[i], end[i] are then the sequences' numbers.
    __device__ __forceinline__ uint32_t borders(const int* offsets, int64_t nseq, int64_t t0, int lane, int* start, int* end) {
        if (kBackward ? t0 > border : t0 + kGlrRun <= border) return 0;
        if (lane < kGlrRun) start[lane] = end[lane] = -1;
        __syncwarp();
        if (!covers(nseq, t0)) {
            const int64_t first = search(offsets, nseq, t0, lane);
            load(offsets, nseq, kBackward && first > 24 ? first - 24 : first, lane);
            if (!covers(nseq, t0)) {  // more than 32 sequences about these few tokens
                for (int64_t s = first; s < nseq; s += 32) {
                    load(offsets, nseq, s, lane);
                    put(t0, lane, start, end);
                    if (__shfl_sync(~0u, a, 31) >= t0 + kGlrRun) break;
                }
            }
        }
        put(t0, lane, start, end);
        // the next border among the held sequences, which is also where they stop serving
        if (kBackward) {
            int last = a < b && b - 1 < t0 ? b - 1 : a < b && a < t0 ? a : INT32_MIN;
            if (lane == 0 && s0 > 0 && a > last) last = a;
            border = __reduce_max_sync(~0u, last);
        } else {
            const int64_t t1 = t0 + kGlrRun;
            int next = a < b && a >= t1 ? a : a < b && b > t1 ? b - 1 : INT32_MAX;
            if (lane == 31 && s0 + 32 < nseq && a < next) next = a;
            if (lane == 0 && s0 > 0 && a > t1) next = a - 1 < next ? a - 1 : next;  // the one before may end there
            border = __reduce_min_sync(~0u, next);
        }
        __syncwarp();
        return __ballot_sync(~0u, lane < 2 * kGlrRun && (lane < kGlrRun ? start[lane] : end[lane - kGlrRun]) >= 0);
    }

  private:
    // the held sequences are all that can touch the tokens from t0 on
    __device__ __forceinline__ bool covers(int64_t nseq, int64_t t0) const {
        return s0 >= 0 && (s0 == 0 || __shfl_sync(~0u, a, 0) <= t0) &&
               (s0 + 32 >= nseq || __shfl_sync(~0u, a, 31) >= t0 + kGlrRun);
    }
    __device__ __forceinline__ void load(const int* offsets, int64_t nseq, int64_t s, int lane) {
        s0 = int(s);
        s += lane;
        a = b = INT32_MAX;
        if (s < nseq) {
            a = __ldg(offsets + s);
            b = __ldg(offsets + s + 1);
        }
    }
    __device__ __forceinline__ void put(int64_t t0, int lane, int* start, int* end) const {
        if (a >= b) return;
        if (a >= t0 && a < t0 + kGlrRun) start[a - t0] = s0 + lane;
        if (b > t0 && b <= t0 + kGlrRun) end[b - 1 - t0] = s0 + lane;
    }
    // the first sequence that ends behind t0
    __device__ __forceinline__ static int64_t search(const int* offsets, int64_t nseq, int64_t t0, int lane) {
        int64_t lo = 0, hi = nseq;
        while (lo < hi) {
            const int64_t stride = (hi - lo + 31) / 32, s = lo + lane * stride;
            const unsigned m = __ballot_sync(~0u, s >= hi || __ldg(offsets + s + 1) > t0);
            if (m & 1u) break;
            const int k = m ? __ffs(m) - 1 : 32;  // lanes 0 .. k-1 end at or before t0
            const int64_t nhi = lo + k * stride;
            lo += (k - 1) * stride + 1;
            hi = nhi < hi ? nhi : hi;
        }
        return lo;
    }
};

// Checks the offsets and calls empty(s) for every sequence without tokens;
// the warps of all blocks of a channel range share the sequences.
template <typename F>
__device__ __forceinline__ void glr_empty_sequences(const GlrParams& p, int64_t first, int64_t step, F&& empty) {
    bool bad = p.offsets[0] < 0 || p.offsets[p.nseq] > p.seqlen;
    for (int64_t s = first; s < p.nseq; s += step) {
        const int a = __ldg(p.offsets + s), b = __ldg(p.offsets + s + 1);
        if (a > b) bad = true;
        if (a >= b) empty(s);
    }
    if (bad) raise_device_error(p.err, kDeviceErrOffsets);
}

// ---------------------------------------------------------------------------
// Exchange of the tiles' pairs in a cluster.

__device__ __forceinline__ uint32_t glr_cluster_size() {
    uint32_t n;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}
__device__ __forceinline__ uint32_t glr_cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void glr_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct GlrSlots {
    float4* slot;   // [2][S][32]: a peer's P and H of a lane's two channels
    uint64_t* bar;  // [2]
    uint32_t S, rank;
    __device__ __forceinline__ float4* at(int use, uint32_t r, int lane) const { return slot + ((use & 1) * S + r) * 32 + lane; }

    // Takes `state` over all blocks' tiles in the scan's order; `mine` is what
    // comes in at this block's.
    template <bool kCuts, bool kBackward>
    __device__ __forceinline__ void walk(int use, int lane, float2& state, float2& mine) const {
        for (uint32_t i = 0; i < S; ++i) {
            const uint32_t r = kBackward ? S - 1 - i : i;
            if (r == rank) mine = state;
            const float4 a = *at(use, r, lane);
            state = glr_apply<kCuts>(make_float2(a.x, a.y), make_float2(a.z, a.w), state);
        }
    }
};

// Called by one whole warp: sends this block's pair to every block of the
// cluster (itself too) and waits for all of theirs, for two seconds at most.  Each
// use flips the buffer: a peer overwrites a slot two exchanges later, which it
// reaches only with this block's next pair in hand, sent after the slot was read.
__device__ __forceinline__ bool glr_exchange(const GlrSlots& sl, int use, int lane, float4 pair, unsigned* err) {
    if (lane == 0) mbar_arrive_expect_tx(sl.bar + (use & 1), sl.S * kGlrSlotBytes);
    __syncwarp();
    const uint32_t mine = smem_addr(sl.at(use, sl.rank, lane)), bar = smem_addr(sl.bar + (use & 1));
    for (uint32_t r = 0; r < sl.S; ++r) {
        uint32_t dst, dbar;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(mine), "r"(r));
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dbar) : "r"(bar), "r"(r));
        asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
                     "f"(pair.x), "f"(pair.y), "f"(pair.z), "f"(pair.w), "r"(dbar)
                     : "memory");
    }
    const uint32_t parity = (use >> 1) & 1;
    uint32_t ok = 0;
    uint64_t t0 = 0;
    for (uint32_t i = 0; !ok; ++i) {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (!ok && (i & 255u) == 0) {
            if (i == 0) t0 = global_timer_ns();
            else if (global_timer_ns() - t0 > 2000000000ull) {
                raise_device_error(err, kDeviceErrTimeout);
                break;
            }
        }
    }
    return __all_sync(~0u, ok != 0);
}

// (P, H) of two neighbouring spans, the second one (Q, K), in place.
template <bool kCuts>
__device__ __forceinline__ void glr_compose(float2& P, float2& H, float2 Q, float2 K) {
    H = glr_apply<kCuts>(Q, K, H);
    const float2 r = __fmul2_rn(P, Q);
    const int marks = __float_as_int(P.x) | __float_as_int(Q.x);
    P = kCuts ? make_float2(__int_as_float((__float_as_int(r.x) & INT32_MAX) | (marks & INT32_MIN)), r.y) : r;
}

__device__ __forceinline__ float2 lo2(float4 v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 hi2(float4 v) { return make_float2(v.z, v.w); }
__device__ __forceinline__ float4 join(float2 a, float2 b) { return make_float4(a.x, a.y, b.x, b.y); }

// ---------------------------------------------------------------------------
// A thread's place, and the warp's ring of tiles.

template <bool kPacked>
struct GlrPlace {
    int lane, warp;
    uint32_t S, rank;
    int64_t b, c;
    int lo, hi;  // packed sequences: the tokens that belong to them
    bool on, both;
    __device__ __forceinline__ GlrPlace(const GlrParams& p) {
        lane = threadIdx.x & 31;
        warp = threadIdx.x >> 5;
        S = glr_cluster_size();
        rank = glr_cluster_rank();
        const unsigned nblk = unsigned((p.dim + kGlrCols - 1) / kGlrCols), unit = blockIdx.x / S;
        b = unit / nblk;
        c = int64_t(unit % nblk) * kGlrCols + lane * kGlrLanes;
        on = c < p.dim;
        both = c + 1 < p.dim;
        if (kPacked) {
            const int a = p.offsets[0], e = p.offsets[p.nseq];
            lo = a > 0 ? a : 0;
            hi = e < p.seqlen ? e : int(p.seqlen);
        }
    }
    // of the kGlrRun tokens from t0 on, the ones that belong to a sequence are [n0, n1)
    __device__ __forceinline__ void valid(const GlrParams& p, int64_t t0, int& n0, int& n1) const {
        const int64_t left = (kPacked ? int64_t(hi) : p.seqlen) - t0;
        n1 = left < 0 ? 0 : left < kGlrRun ? int(left) : kGlrRun;
        n0 = !kPacked || t0 >= lo ? 0 : lo - t0 < kGlrRun ? int(lo - t0) : kGlrRun;
    }
    // a row of states, one value per channel; zero without it
    __device__ __forceinline__ float2 read(const float* row) const {
        return make_float2(row && on ? row[c] : 0.f, row && both ? row[c + 1] : 0.f);
    }
    __device__ __forceinline__ void write(float* row, float2 v) const {
        if (on) row[c] = v.x;
        if (both) row[c + 1] = v.y;
    }
    // a token's two channels at q; `pairs`: dim is even and q aligned to both
    template <typename T>
    __device__ __forceinline__ void put(T* q, bool pairs, float2 v) const {
        if (pairs) {
            if (on) glr_put(q, v);
        } else {
            if (on) q[0] = from_f32<T>(v.x);
            if (both) q[1] = from_f32<T>(v.y);
        }
    }
};

// The ring of one warp: kStages slots of kArrays boxes.  With kTma one lane
// issues a box per tensor and an mbarrier per slot counts the bytes.  Rows that
// are not whole 16-byte pieces are copied by the lanes as the pieces that the 64
// channels touch (cp.async; the last piece of the tensor only as far as it
// goes), so a row begins `shift` elements into its place; tensors that do not
// begin on 16 bytes go element by element into the same places.
template <typename T, bool kTma, int kArrays, int kStages>
struct GlrRing {
    static constexpr int kPitch = kGlrPitch<T, kTma>, kBox = kGlrBox<T, kTma>;
    static constexpr int kPer = 16 / int(sizeof(T));  // elements of a piece
    T* base;
    uint64_t* bar;
    const CUtensorMap* map[kArrays];
    const T* src[kArrays];  // the tensors
    int64_t row0;           // of the batch row's first token
    int slot = 0;
    uint32_t parity = 0;

    // where token i of the tile at t0 begins in its row of the box
    __device__ __forceinline__ int shift(int64_t t0, int i, const GlrParams& p) const {
        return int((uint32_t(row0 + t0) + uint32_t(i)) * uint32_t(p.dim) % uint32_t(kPer));  // 64 channels are whole pieces
    }

    // this lane's channels of token i of the current slot's tile
    __device__ __forceinline__ float2 get(int array, int i, int64_t t0, const GlrParams& p, int lane) const {
        const T* row = base + (slot * kArrays + array) * kBox + i * kPitch;
        if constexpr (kTma) return glr_get(row, lane * kGlrLanes);
        const int at = shift(t0, i, p) + lane * kGlrLanes;
        if constexpr (sizeof(T) == 4) {
            return make_float2(row[at], row[at + 1]);
        } else {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(row) + (at >> 1);
            const uint32_t v = at & 1 ? __byte_perm(w[0], w[1], 0x5432) : w[0];
            return make_float2(bf16_lo(v), bf16_hi(v));
        }
    }

    template <typename Place>
    __device__ __forceinline__ void issue(int s, int64_t t0, const GlrParams& p, const Place& me) {
        T* dst = base + s * kArrays * kBox;
        if constexpr (kTma) {
            if (me.lane == 0) {  // without tokens the slot's phase completes all the same
                const bool any = t0 < p.seqlen;
                mbar_arrive_expect_tx(bar + s, any ? kArrays * kBox * uint32_t(sizeof(T)) : 0);
#pragma unroll
                for (int a = 0; a < kArrays; ++a)
                    if (any) tma_load_3d(dst + a * kBox, map[a], int(me.c), int(t0), int(me.b), bar + s);
            }
        } else {
            const int n = t0 >= p.seqlen ? 0 : int(p.seqlen - t0 < kGlrRun ? p.seqlen - t0 : kGlrRun);
            const int64_t c0 = me.c - me.lane * kGlrLanes;
            const int cols = int(p.dim - c0 < kGlrCols ? p.dim - c0 : kGlrCols);
            if (p.pairs < 0) {
                for (int i = 0; i < n; ++i)
#pragma unroll
                    for (int a = 0; a < kArrays; ++a) {
                        T* to = dst + a * kBox + i * kPitch + shift(t0, i, p) + me.lane * kGlrLanes;
                        const T* q = src[a] + (row0 + t0 + i) * p.dim + me.c;
                        if (me.on) to[0] = q[0];
                        if (me.both) to[1] = q[1];
                    }
            } else {
                constexpr int kPieces = kPitch / kPer;  // of a row
                const int64_t end = p.batch * p.seqlen * p.dim;
#pragma unroll
                for (int k = 0; k < (kGlrRun * kPieces + 31) / 32; ++k) {
                    const int piece = k * 32 + me.lane, i = piece / kPieces, col = (piece % kPieces) * kPer;
                    const int sh = shift(t0, i, p);
                    if (i >= n || col >= sh + cols) continue;
                    const int64_t e = (row0 + t0 + i) * p.dim + c0 - sh + col;
                    const int64_t left = (end - e) * int64_t(sizeof(T));
                    const int bytes = left < 16 ? int(left) : 16;
#pragma unroll
                    for (int a = 0; a < kArrays; ++a)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                         smem_addr(dst + a * kBox + i * kPitch + col)),
                                     "l"(src[a] + e), "r"(bytes)
                                     : "memory");
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }

    // The tile in the current slot has arrived; false when its wait gave up.
    __device__ __forceinline__ bool wait(const GlrParams& p) {
        if constexpr (kTma) {
            return mbar_wait_bounded(bar + slot, parity, p.err, p.wait_ns);
        } else {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            __syncwarp();
            return true;
        }
    }

    // After a wait that gave up: waits once more for the boxes in flight.
    __device__ __forceinline__ void drain(const GlrParams& p) {
        if constexpr (kTma) {
            drain_ring(slot, parity, kStages, kStages, [&](int, int at, uint32_t phase) {
                if (p.selftest && (threadIdx.x & 31) == 0) mbar_arrive(bar + at);  // what the wait was for comes late
                mbar_wait_bounded(bar + at, phase, p.err);
            });
        } else {
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    }

    // The current slot has been read: fills it for the tile at t_next and moves on.
    template <typename Place>
    __device__ __forceinline__ void advance(int64_t t_next, const GlrParams& p, const Place& me) {
        __syncwarp();
        issue(slot, t_next, p, me);
        if (++slot == kStages) slot = 0, parity ^= 1;
    }
};

// Of the borders among a warp's tokens, those where sequences begin and end.
__device__ __forceinline__ uint32_t glr_starts(uint32_t marks) { return marks & ((1u << kGlrRun) - 1u); }
__device__ __forceinline__ uint32_t glr_ends(uint32_t marks) { return marks >> kGlrRun; }

__device__ __forceinline__ int glr_first(uint32_t bits) { return bits ? __ffs(bits) - 1 : kGlrRun; }
// How a warp runs its tokens: 0 all belong to one sequence, 1 some lie outside
// or one begins and one ends at most (selections instead of branches), 2 more
// borders than that.
__device__ __forceinline__ int glr_mode(int n0, int n1, uint32_t marks) {
    if (__popc(glr_starts(marks)) > 1 || __popc(glr_ends(marks)) > 1) return 2;
    return marks || n0 > 0 || n1 < kGlrRun ? 1 : 0;
}

// A row of per-sequence states; `first`: that of the first token of `bits`, read ahead.
template <typename Place>
__device__ __forceinline__ float2 glr_row(const Place& me, const GlrParams& p, const float* states, int s) {
    return me.read(states ? states + int64_t(s) * p.dim : nullptr);
}
template <typename Place>
__device__ __forceinline__ float2 glr_row(const Place& me, const GlrParams& p, const float* states, const int* seq, int i,
                                          uint32_t bits, float2 first) {
    return (bits & ((1u << i) - 1u)) == 0 ? first : glr_row(me, p, states, seq[i]);
}

// ---------------------------------------------------------------------------
// The kernels.  Two blocks of eight warps per SM: a third would leave a thread 80
// registers, too few for eight tokens of two channels.

// Bound by memory: 8 bytes per element (bf16, with z).  4 x 4096 x 4096: 110 us, 4.9
// TB/s.  In clusters the exchange between a tile's two barriers costs a fifth: 1
// x 131072 x 2048, 9 blocks a cluster, 541 us, 4.0 TB/s.  12289 x 1536 without z:
// the dense kernel 38 us, the packed one 46 us with one sequence and 53 us with 37.
template <typename T, bool kTma, bool kPacked, bool kZ>
__global__ void __launch_bounds__(kGlrThreads, 2)
    glr_fwd_kernel(const __grid_constant__ GlrMaps maps, const GlrParams p) {
    extern __shared__ __align__(128) unsigned char ring_mem[];
    // P and H of a warp's tokens, then in their place the state before them
    __shared__ float4 agg[kGlrWarps][32];
    __shared__ uint64_t slot_bar[2];
    __shared__ int gave_up, stop;  // a bounded wait ran out; every warp leaves behind the tile
    __shared__ int starts[2][kGlrWarps][kGlrRun], ends[2][kGlrWarps][kGlrRun];
    constexpr int kStages = kGlrStages<T, kTma, false>;
    constexpr int kArrays = kZ ? 3 : 2;
    __shared__ uint64_t full[kGlrWarps][kStages];
    const GlrPlace<kPacked> me(p);
    const int lane = me.lane, warp = me.warp;
    const GlrSlots sl{reinterpret_cast<float4*>(ring_mem + glr_ring<T, kTma, false>(kArrays)), slot_bar, me.S, me.rank};
    if (threadIdx.x == 0) {
        gave_up = stop = 0;
        mbar_init(slot_bar, 1);
        mbar_init(slot_bar + 1, 1);
        for (int i = 0; i < kGlrWarps * kStages; ++i) mbar_init(&full[0][0] + i, 1 + p.selftest);
        fence_barrier_init();
    }
    __syncthreads();
    if (me.S > 1) glr_cluster_sync();

    const int64_t base = me.b * p.seqlen * p.dim + me.c;
    GlrRing<T, kTma, kArrays, kStages> ring;
    ring.base = reinterpret_cast<T*>(ring_mem) + warp * kStages * kArrays * kGlrBox<T, kTma>;
    ring.row0 = me.b * p.seqlen;
    ring.bar = full[warp];
    ring.map[0] = &maps.gate, ring.src[0] = static_cast<const T*>(p.gate);
    ring.map[1] = &maps.x, ring.src[1] = static_cast<const T*>(p.x);
    if constexpr (kZ) ring.map[2] = &maps.z, ring.src[2] = static_cast<const T*>(p.z);

    const int64_t strip = int64_t(me.S) * kGlrTile, strips = (p.seqlen + strip - 1) / strip;
    int64_t t0 = int64_t(me.rank) * kGlrTile + warp * kGlrRun;
#pragma unroll
    for (int s = 0; s < kStages; ++s) ring.issue(s, t0 + s * strip, p, me);

    T* y = p.y ? static_cast<T*>(p.y) + base + t0 * p.dim : nullptr;
    const int64_t step = strip * p.dim;
    const float2 bias = __fmul2_rn(me.read(p.bias), splat(kGlrScale<T>));
    float2 carry = make_float2(0.f, 0.f);  // warp 0: the state before the strip of S tiles
    if (!kPacked && p.init) carry = me.read(p.init + me.b * p.dim);
    if (kPacked)
        glr_empty_sequences(p, me.rank * kGlrWarps + warp, me.S * kGlrWarps, [&](int64_t s) {
            if (p.last) me.write(p.last + s * p.dim, me.read(p.init ? p.init + s * p.dim : nullptr));
        });

    GlrCursor<false> cursor;
    // the next tile's borders, and the state that its first sequence begins with; all
    // warps but the composing one look for them while that one composes
    uint32_t next = 0;
    float2 next_start = splat(0.f);
    const auto look = [&](int64_t t, int par) {
        next = t >= me.lo - kGlrRun && t < me.hi ? cursor.borders(p.offsets, p.nseq, t, lane, starts[par][warp], ends[par][warp]) : 0;
        if (glr_starts(next)) next_start = glr_row(me, p, p.init, starts[par][warp][__ffs(next) - 1]);
    };
    for (int64_t k = 0; k < strips; ++k, t0 += strip, y += step) {
        int n0, n1;
        me.valid(p, t0, n0, n1);
        const int par = int(k & 1);
        if (kPacked && (warp == 0 || k == 0)) look(t0, par);
        const uint32_t marks = next;
        const float2 at_start = next_start;
        const int i_start = glr_first(glr_starts(marks)), i_end = glr_first(glr_ends(marks));
        const int mode = glr_mode(n0, n1, marks);
        if (!ring.wait(p)) gave_up = 1;
        float2 f[kGlrRun], v[kGlrRun], g[kGlrRun];  // the gates, (1 - f) x, and silu(z)
        float2 P = splat(1.f), H = splat(0.f);
        const auto get = [&](int array, int i) { return ring.get(array, i, t0, p, lane); };
        const auto gates = [&](int i) {
            const float2 arg = __ffma2_rn(get(0, i), splat(kGlrScale<T>), bias);
            if constexpr (kZ) {
                float2 sg, sn;
                sigmoid2_both<T>(arg, get(kArrays - 1, i), f[i], v[i], sg, sn, g[i]);
            } else {
                sigmoid2<T>(arg, f[i], v[i]);
            }
            v[i] = __fmul2_rn(v[i], get(1, i));
        };
        const auto reduce = [&](auto m) {
            constexpr int kMode = decltype(m)::value;
            if (kMode) {
#pragma unroll
                for (int i = 0; i < kGlrRun; ++i) gates(i);
            }
#pragma unroll
            for (int i = 0; i < kGlrRun; ++i) {
                if (!kMode) gates(i);
                if (kMode) {  // outside the sequences: hands the state on
                    const bool in = i >= n0 && i < n1;
                    f[i] = in ? f[i] : splat(1.f);
                    v[i] = in ? v[i] : splat(0.f);
                }
                if (kMode == 1 && kPacked) H = i == i_start ? at_start : H;
                if (kMode == 2 && (marks >> i & 1u)) H = glr_row(me, p, p.init, starts[par][warp], i, glr_starts(marks), at_start);
                P = __fmul2_rn(P, f[i]);
                H = __ffma2_rn(f[i], H, v[i]);
            }
        };
        if (mode == 0) reduce(std::integral_constant<int, 0>{});
        else if (!kPacked || mode == 1) reduce(std::integral_constant<int, 1>{});
        else reduce(std::integral_constant<int, kPacked ? 2 : 1>{});
        const bool cut = kPacked && i_start < kGlrRun;  // a sequence begins among these tokens
        if (kPacked) P.x = cut ? kGlrCut : fabsf(P.x);
        agg[warp][lane] = join(P, H);
        __syncthreads();
        if (warp == 0) {
            float2 h = carry;
            if (me.S > 1) {
                float2 Pt = lo2(agg[0][lane]), Ht = hi2(agg[0][lane]);
#pragma unroll
                for (int j = 1; j < kGlrWarps; ++j) glr_compose<kPacked>(Pt, Ht, lo2(agg[j][lane]), hi2(agg[j][lane]));
                if (!glr_exchange(sl, int(k & 3), lane, join(Pt, Ht), p.err)) gave_up = 1;
                sl.walk<kPacked, false>(int(k & 1), lane, carry, h);
            }
            float2 s[kGlrWarps];  // stored behind the chain, so that its loads need not wait for the stores
#pragma unroll
            for (int j = 0; j < kGlrWarps; ++j) {
                s[j] = h;
                h = glr_apply<kPacked>(lo2(agg[j][lane]), hi2(agg[j][lane]), h);
            }
#pragma unroll
            for (int j = 0; j < kGlrWarps; ++j) *reinterpret_cast<float2*>(&agg[j][lane]) = s[j];
            if (me.S == 1) carry = h;
            if (lane == 0) stop = gave_up;
        } else if (kPacked) {
            look(t0 + strip, par ^ 1);
        }
        __syncthreads();
        if (stop) break;
        float2 h = lo2(agg[warp][lane]);
        if (warp == 0 && p.states && t0 < p.seqlen)
            me.write(p.states + (me.b * ((p.seqlen + kGlrTile - 1) / kGlrTile) + t0 / kGlrTile) * p.dim, h);
        const auto emit = [&](auto m) {
            constexpr int kMode = decltype(m)::value;
            T* out = y;
            float2 at_end = h;
#pragma unroll
            for (int i = 0; i < kGlrRun; ++i, out += p.dim) {
                if (kMode == 1 && kPacked) h = i == i_start ? at_start : h;
                if (kMode == 2 && (marks >> i & 1u)) h = glr_row(me, p, p.init, starts[par][warp], i, glr_starts(marks), at_start);
                h = __ffma2_rn(f[i], h, v[i]);
                if (p.y) {
                    float2 o = h;
                    if constexpr (kZ) o = __fmul2_rn(o, g[i]);
                    if (!kMode || (i >= n0 && i < n1)) me.put(out, kTma || p.pairs > 0, o);
                }
                if (kMode == 1 && kPacked) at_end = i == i_end ? h : at_end;
                if (kMode == 2 && p.last && (glr_ends(marks) >> i & 1u)) me.write(p.last + int64_t(ends[par][warp][i]) * p.dim, h);
            }
            if (kMode == 1 && kPacked && p.last && i_end < kGlrRun) me.write(p.last + int64_t(ends[par][warp][i_end]) * p.dim, at_end);
        };
        if (mode == 0) emit(std::integral_constant<int, 0>{});
        else if (!kPacked || mode == 1) emit(std::integral_constant<int, 1>{});
        else emit(std::integral_constant<int, kPacked ? 2 : 1>{});
        ring.advance(t0 + kStages * strip, p, me);
    }
    if (stop) ring.drain(p);
    if (!kPacked && p.last && warp == 0 && me.rank == 0) me.write(p.last + me.b * p.dim, carry);
    if (me.S > 1) glr_cluster_sync();  // no block leaves while a peer may still send to it
}

// The strips run from the last to the first.  One warp runs both chains of a tile:
// the states from the saved one, the gradients from behind.  The states are run
// through again in place of being kept for the second loop, which would cost
// 16 registers.  Bound by memory, 14 bytes per element (bf16, with z): 4 x 4096 x
// 4096 in 188 us, 5.0 TB/s.
template <typename T, bool kTma, bool kPacked, bool kZ>
__global__ void __launch_bounds__(kGlrThreads, 2)
    glr_bwd_kernel(const __grid_constant__ GlrMaps maps, const GlrParams p) {
    extern __shared__ __align__(128) unsigned char ring_mem[];
    __shared__ float4 agg[kGlrWarps][32];     // P and H of a warp's tokens
    __shared__ float2 agge[kGlrWarps][32];    // the constant term of E over them
    __shared__ float2 before[kGlrWarps][32];  // the state before a warp's tokens
    __shared__ float2 behind[kGlrWarps][32];  // E behind them
    __shared__ uint64_t slot_bar[2];
    __shared__ int gave_up, stop;  // a bounded wait ran out; every warp leaves behind the tile
    __shared__ int starts[kGlrWarps][kGlrRun], ends[kGlrWarps][kGlrRun];
    constexpr int kStages = kGlrStages<T, kTma, true>;
    constexpr int kArrays = kZ ? 4 : 3;
    __shared__ uint64_t full[kGlrWarps][kStages];
    const GlrPlace<kPacked> me(p);
    const int lane = me.lane, warp = me.warp;
    const GlrSlots sl{reinterpret_cast<float4*>(ring_mem + glr_ring<T, kTma, true>(kArrays)), slot_bar, me.S, me.rank};
    if (threadIdx.x == 0) {
        gave_up = stop = 0;
        mbar_init(slot_bar, 1);
        mbar_init(slot_bar + 1, 1);
        for (int i = 0; i < kGlrWarps * kStages; ++i) mbar_init(&full[0][0] + i, 1 + p.selftest);
        fence_barrier_init();
    }
    __syncthreads();
    if (me.S > 1) glr_cluster_sync();

    const int64_t base = me.b * p.seqlen * p.dim + me.c;
    GlrRing<T, kTma, kArrays, kStages> ring;
    ring.base = reinterpret_cast<T*>(ring_mem) + warp * kStages * kArrays * kGlrBox<T, kTma>;
    ring.row0 = me.b * p.seqlen;
    ring.bar = full[warp];
    ring.map[0] = &maps.gate, ring.src[0] = static_cast<const T*>(p.gate);
    ring.map[1] = &maps.x, ring.src[1] = static_cast<const T*>(p.x);
    ring.map[2] = &maps.dy, ring.src[2] = static_cast<const T*>(p.dy);
    if constexpr (kZ) ring.map[3] = &maps.z, ring.src[3] = static_cast<const T*>(p.z);

    // the strips from the last to the first; a last strip's tiles may lie behind the tokens
    const int64_t strip = int64_t(me.S) * kGlrTile, strips = (p.seqlen + strip - 1) / strip;
    const int64_t tiles = (p.seqlen + kGlrTile - 1) / kGlrTile;
    int64_t tile = (strips - 1) * me.S + me.rank, t0 = tile * kGlrTile + warp * kGlrRun;
#pragma unroll
    for (int s = 0; s < kStages; ++s)
        ring.issue(s, t0 - s * strip >= 0 ? t0 - s * strip : p.seqlen, p, me);  // seqlen: nothing

    int64_t o = base + t0 * p.dim;
    const int64_t step = strip * p.dim;
    const float2 bias = __fmul2_rn(me.read(p.bias), splat(kGlrScale<T>));
    float2 E = make_float2(0.f, 0.f);  // warp 0: the gradient handed to the strip's last token from behind
    if (!kPacked && p.dlast) E = me.read(p.dlast + me.b * p.dim);
    if (kPacked)
        glr_empty_sequences(p, me.rank * kGlrWarps + warp, me.S * kGlrWarps, [&](int64_t s) {
            if (p.dinit) me.write(p.dinit + s * p.dim, me.read(p.dlast ? p.dlast + s * p.dim : nullptr));
        });

    float2 sum = splat(0.f);  // dgate over this warp's tokens
    GlrCursor<true> cursor;
    int use = 0;
    for (int64_t k = strips - 1; k >= 0; --k, use = (use + 1) & 3, tile -= me.S, t0 -= strip, o -= step) {
        int n0, n1;
        me.valid(p, t0, n0, n1);
        const uint32_t marks = kPacked && n0 < n1 ? cursor.borders(p.offsets, p.nseq, t0, lane, starts[warp], ends[warp]) : 0;
        const int i_start = glr_first(glr_starts(marks)), i_end = glr_first(glr_ends(marks));
        const int mode = glr_mode(n0, n1, marks);
        float2 at_start = splat(0.f), at_end = at_start;
        if (kPacked && i_start < kGlrRun) at_start = glr_row(me, p, p.init, starts[warp][i_start]);
        if (kPacked && i_end < kGlrRun) at_end = glr_row(me, p, p.dlast, ends[warp][i_end]);
        float2 h = splat(0.f);
        if (warp == 0 && tile < tiles) h = me.read(p.states + (me.b * tiles + tile) * p.dim);
        if (!ring.wait(p)) gave_up = 1;
        // u: dy silu(z) (+ dlast); v: dy silu'(z), later the factor of dgate
        float2 f[kGlrRun], w[kGlrRun], u[kGlrRun], v[kGlrRun];
        float2 P = splat(1.f), H = splat(0.f), G = splat(0.f);
        const auto get = [&](int array, int i) { return ring.get(array, i, t0, p, lane); };
        const auto gates = [&](int i) {
            const float2 arg = __ffma2_rn(get(0, i), splat(kGlrScale<T>), bias);
            u[i] = get(2, i);
            if constexpr (!kZ) {
                sigmoid2<T>(arg, f[i], w[i]);
            } else {
                float2 sg, sn, si;
                sigmoid2_both<T>(arg, get(kArrays - 1, i), f[i], w[i], sg, sn, si);
                v[i] = __fmul2_rn(u[i], __ffma2_rn(si, sn, sg));
                u[i] = __fmul2_rn(u[i], si);
            }
        };
        const auto reduce = [&](auto m) {
            constexpr int kMode = decltype(m)::value;
            if (kMode) {
#pragma unroll
                for (int i = 0; i < kGlrRun; ++i) gates(i);
            }
#pragma unroll
            for (int i = 0; i < kGlrRun; ++i) {
                if (!kMode) gates(i);
                float2 x = get(1, i);
                if (kMode) {  // outside the sequences: hands both on
                    const bool in = i >= n0 && i < n1;
                    f[i] = in ? f[i] : splat(1.f);
                    w[i] = in ? w[i] : splat(0.f);
                    u[i] = in ? u[i] : splat(0.f);
                    x = in ? x : splat(0.f);
                }
                if (kMode == 1 && kPacked) {
                    u[i] = i == i_end ? __fadd2_rn(u[i], at_end) : u[i];
                    H = i == i_start ? at_start : H;
                }
                if (kMode == 2 && p.dlast && (glr_ends(marks) >> i & 1u))
                    u[i] = __fadd2_rn(u[i], glr_row(me, p, p.dlast, ends[warp], i, glr_ends(marks), at_end));
                if (kMode == 2 && (marks >> i & 1u)) H = glr_row(me, p, p.init, starts[warp], i, glr_starts(marks), at_start);
                P = __fmul2_rn(P, f[i]);
                H = __ffma2_rn(f[i], H, __fmul2_rn(w[i], x));
                const float2 more = __ffma2_rn(P, u[i], G);
                G = !kMode || !kPacked || i < i_start ? more : G;  // nothing goes in front of a first token
            }
        };
        if (mode == 0) reduce(std::integral_constant<int, 0>{});
        else if (!kPacked || mode == 1) reduce(std::integral_constant<int, 1>{});
        else reduce(std::integral_constant<int, kPacked ? 2 : 1>{});
        const bool cut = kPacked && i_start < kGlrRun;  // a sequence begins among these tokens
        if (kPacked) P.x = cut ? kGlrCut : fabsf(P.x);
        agg[warp][lane] = join(P, H);
        agge[warp][lane] = G;
        __syncthreads();
        if (warp == 0) {
            float2 e = E;
            if (me.S > 1) {
                float2 Pt = lo2(agg[kGlrWarps - 1][lane]), Gt = agge[kGlrWarps - 1][lane];
#pragma unroll
                for (int j = kGlrWarps - 2; j >= 0; --j) glr_compose<kPacked>(Pt, Gt, lo2(agg[j][lane]), agge[j][lane]);
                if (!glr_exchange(sl, use, lane, join(Pt, Gt), p.err)) gave_up = 1;
                sl.walk<kPacked, true>(use, lane, E, e);
            }
            float2 s[kGlrWarps];  // stored behind the chain, so that its loads need not wait for the stores
#pragma unroll
            for (int j = 0; j < kGlrWarps; ++j) {
                s[j] = h;
                h = glr_apply<kPacked>(lo2(agg[j][lane]), hi2(agg[j][lane]), h);
            }
#pragma unroll
            for (int j = 0; j < kGlrWarps; ++j) before[j][lane] = s[j];
#pragma unroll
            for (int j = kGlrWarps - 1; j >= 0; --j) {
                s[j] = e;
                e = glr_apply<kPacked>(lo2(agg[j][lane]), agge[j][lane], e);
            }
#pragma unroll
            for (int j = 0; j < kGlrWarps; ++j) behind[j][lane] = s[j];
            if (me.S == 1) E = e;
            if (lane == 0) stop = gave_up;
        }
        __syncthreads();
        if (stop) break;
        h = before[warp][lane];
        float2 e = behind[warp][lane];
        const auto emit = [&](auto m) {
            constexpr int kMode = decltype(m)::value;
            // forward: the states, dz, and the factor (h_{t-1} - x_t) f_t (1 - f_t) of dgate
            T* out = static_cast<T*>(p.dz) + o;
#pragma unroll
            for (int i = 0; i < kGlrRun; ++i, out += p.dim) {
                const bool in = !kMode || (i >= n0 && i < n1);
                if (kMode == 1 && kPacked) h = i == i_start ? at_start : h;
                if (kMode == 2 && (marks >> i & 1u)) h = glr_row(me, p, p.init, starts[warp], i, glr_starts(marks), at_start);
                const float2 x = in ? get(1, i) : splat(0.f);
                const float2 q = __fmul2_rn(__ffma2_rn(x, splat(-1.f), h), __fmul2_rn(f[i], w[i]));
                h = __ffma2_rn(f[i], h, __fmul2_rn(w[i], x));
                if constexpr (kZ)
                    if (in) me.put(out, kTma || p.pairs > 0, __fmul2_rn(v[i], h));
                v[i] = q;
            }
            // backward: dh, dx, dgate
            float2 part = splat(0.f), first = splat(0.f);
            T* ox = static_cast<T*>(p.dx) + o + (kGlrRun - 1) * p.dim;
            T* og = static_cast<T*>(p.dgate) + o + (kGlrRun - 1) * p.dim;
#pragma unroll
            for (int i = kGlrRun - 1; i >= 0; --i, ox -= p.dim, og -= p.dim) {
                const bool in = !kMode || (i >= n0 && i < n1);
                const float2 d = __fadd2_rn(u[i], e), dg = __fmul2_rn(d, v[i]);
                if (in) {
                    me.put(ox, kTma || p.pairs > 0, __fmul2_rn(w[i], d));
                    me.put(og, kTma || p.pairs > 0, dg);
                }
                const float2 sofar = __fadd2_rn(part, dg);
                part = in ? sofar : part;
                e = __fmul2_rn(f[i], d);
                if (kMode == 1 && kPacked) {
                    first = i == i_start ? e : first;
                    e = i == i_start ? splat(0.f) : e;
                }
                if (kMode == 2 && (marks >> i & 1u)) {
                    if (p.dinit) me.write(p.dinit + int64_t(starts[warp][i]) * p.dim, e);
                    e = splat(0.f);
                }
            }
            if (kMode == 1 && kPacked && p.dinit && i_start < kGlrRun)
                me.write(p.dinit + int64_t(starts[warp][i_start]) * p.dim, first);
            sum = __fadd2_rn(sum, part);
        };
        if (mode == 0) emit(std::integral_constant<int, 0>{});
        else if (!kPacked || mode == 1) emit(std::integral_constant<int, 1>{});
        else emit(std::integral_constant<int, kPacked ? 2 : 1>{});
        const int64_t later = t0 - kStages * strip;
        ring.advance(later >= 0 ? later : p.seqlen, p, me);
    }
    if (stop) ring.drain(p);
    if (!kPacked && p.dinit && warp == 0 && me.rank == 0) me.write(p.dinit + me.b * p.dim, E);
    if (p.dbias_part) {
        launch_dependents();
        __syncthreads();
        agge[warp][lane] = sum;
        __syncthreads();
        if (warp == 0) {
            sum = splat(0.f);
#pragma unroll
            for (int j = 0; j < kGlrWarps; ++j) sum = __fadd2_rn(sum, agge[j][lane]);
            me.write(p.dbias_part + (me.b * me.S + me.rank) * p.dim, sum);
        }
    }
    if (me.S > 1) glr_cluster_sync();  // no block leaves while a peer may still send to it
}

// kN neighbouring elements (1, or as many as fill 8 or 16 bytes) in one access.
template <typename T, int kN>
struct Lanes {
    struct __align__(kN * sizeof(T)) Pack {
        T v[kN];
    } p;
    __device__ __forceinline__ void load(const T* q) { p = *reinterpret_cast<const Pack*>(q); }
    __device__ __forceinline__ void store(T* q) const { *reinterpret_cast<Pack*>(q) = p; }
    __device__ __forceinline__ float get(int i) const { return to_f32(p.v[i]); }
    __device__ __forceinline__ void set(int i, float f) { p.v[i] = from_f32<T>(f); }
};

// One token: a thread takes kN neighbouring channels of one batch row.  Bound by
// the state's two passes (256 x 5120 bf16 3.6 us, from L2) or by the launch (1 x
// 2048 1.9 us).
template <typename T, int kN>
__global__ void glr_update_kernel(const float* state, float* state_out, const T* x, const T* gate, const T* z,
                                  const float* bias, T* y, int64_t batch, int64_t dim) {
    const int64_t c = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) * kN;
    if (c >= dim) return;
    float bv[kN];
    Lanes<float, kN> raw;
    if (bias) raw.load(bias + c);
#pragma unroll
    for (int i = 0; i < kN; ++i) bv[i] = bias ? raw.get(i) * kGlrScale<T> : 0.f;
    for (int64_t b = blockIdx.y; b < batch; b += gridDim.y) {
        const int64_t o = b * dim + c;
        Lanes<float, kN> h;
        Lanes<T, kN> vx, vg, vz;
        h.load(state + o);
        vx.load(x + o);
        vg.load(gate + o);
        if (z) vz.load(z + o);
#pragma unroll
        for (int i = 0; i < kN; i += 2) {
            // a single channel rides along twice
            const int k = i + 1 < kN ? i + 1 : i;
            const float2 arg = make_float2(fmaf(vg.get(i), kGlrScale<T>, bv[i]), fmaf(vg.get(k), kGlrScale<T>, bv[k]));
            float2 f, w, g, n, out = splat(1.f);
            if (z) {
                sigmoid2_both<T>(arg, make_float2(vz.get(i), vz.get(k)), f, w, g, n, out);
            } else {
                sigmoid2<T>(arg, f, w);
            }
            const float2 v = __ffma2_rn(f, make_float2(h.get(i), h.get(k)), __fmul2_rn(w, make_float2(vx.get(i), vx.get(k))));
            h.set(i, v.x);
            vx.set(i, v.x * out.x);
            if (k != i) {
                h.set(k, v.y);
                vx.set(k, v.y * out.y);
            }
        }
        h.store(state_out + o);
        vx.store(y + o);
    }
}

}  // namespace mss
