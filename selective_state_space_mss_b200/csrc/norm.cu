// norm.cu -- residual add and layer norm behind the C ABI: argument checks and
// launches (kernels in norm.cuh).
#include <algorithm>
#include <cmath>

#include "host_common.h"
#include "launch.h"

#include "norm.cuh"
#include "sum_rows.cuh"

namespace mss_host {
namespace {

using mss::bf16_t;
using mss::NormParams;

// Partial sums of dweight and dbias: one per SM of a B200.
constexpr int64_t kNormParts = 148;

bool known_dtype(int d) { return d == MSS_DTYPE_F32 || d == MSS_DTYPE_BF16; }

// Elements of the rows x dim matrix; false on a negative size or overflow.
bool norm_elems(int64_t rows, int64_t dim, int64_t* n) {
    int64_t bytes;
    return rows >= 0 && dim >= 0 && mul_ok(rows, dim, n) && mul_ok(*n, 8, &bytes) && dim <= (int64_t(1) << 40);
}

// Threads that share a row of the forward pass, and the pieces of eight
// elements that each holds: two (one where a row is taken by strides, whose loads
// need more registers, and while the rows alone would leave SMs idle).  16384 x 2048
// with a fp32 residual: two pieces 66 us, one 69 us, four 75 us; 16384 x 1023 by
// strides: one 65 us, two 78 us, four 94 us.
struct NormShape {
    int G, pieces;
};

NormShape norm_fwd_shape(int64_t rows, int64_t dim, bool wide) {
    const int64_t warps = (dim + 255) / 256;  // at one piece a thread
    const int64_t half = (warps + 1) / 2;
    const bool one = warps <= 32 && (!wide || warps == 1 || rows * half * 32 < 148 * 1024);
    return {32 * int(one ? warps : half), one ? 1 : 2};
}

template <typename T, typename R, int kRows>
void launch_norm_fwd(const NormParams& p, NormShape sh, cudaStream_t s) {
    const int64_t per = std::max(1, 256 / sh.G);
    const unsigned grid = unsigned((p.rows + per - 1) / per), threads = unsigned(per * sh.G);
    if (sh.pieces == 1)
        mss::norm_fwd_kernel<T, R, kRows, 1><<<grid, threads, 0, s>>>(p, sh.G);
    else
        mss::norm_fwd_kernel<T, R, kRows, 2><<<grid, threads, 0, s>>>(p, sh.G);
}

constexpr int64_t kNormSmem = 224 * 1024;  // of a block that streams rows

template <typename T, typename R, int kPieces>
int launch_norm_fwd_ring(const NormParams& p, cudaStream_t s) {
    const int G = int(((p.dim + 7) / 8 + 32 * kPieces - 1) / (32 * kPieces) * 32);
    const int64_t slot = (p.dim + 14) / 8 * 8 * int64_t(sizeof(T) + (p.residual ? sizeof(R) : 0));
    int64_t blocks = std::min(p.rows, kNormParts);
    int64_t groups = std::min<int64_t>({mss::kNormRingThreads<kPieces> / G, G == 32 ? mss::kNormGroups : 15, (p.rows + blocks - 1) / blocks});
    groups = std::min(groups, kNormSmem / (2 * slot));
    if (groups < 1) return MSS_ERR_PATH;
    if (p.rows > blocks * groups && blocks * groups * (p.dim % 8) % 8 != 0) blocks -= blocks % 8;  // a group's rows have one shift
    const int stages = int(std::min<int64_t>(mss::kNormStages, kNormSmem / (groups * slot)));
    const auto kern = mss::norm_fwd_ring_kernel<T, R, kPieces>;
    static std::mutex mu;
    static int done[kMaxDevices] = {};
    if (!per_device(done, mu, [&](int) {
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kNormSmem)) == cudaSuccess ? 1 : 0;
        }))
        return MSS_ERR_CUDA;
    kern<<<unsigned(blocks), unsigned(groups * G), size_t(groups * stages * slot), s>>>(p, G, stages);
    return launch_status();
}

template <typename T, typename R>
int run_norm_fwd(const NormParams& p, bool wide, bool aligned, cudaStream_t s) {
    // One piece a thread where a warp takes the row, else two: 16384 x 769 bf16 with a
    // fp32 residual two 33, one 39 us.  Strided loads would take 63 us, and at 148 x
    // 1001 4.6 against 4.2 us.
    if (!wide && aligned && p.dim <= 8192)
        return p.dim <= 256 ? launch_norm_fwd_ring<T, R, 1>(p, s) : launch_norm_fwd_ring<T, R, 2>(p, s);
    if (p.selftest) return MSS_ERR_FLAGS;  // no waits for rows to test
    const NormShape sh = norm_fwd_shape(p.rows, p.dim, wide);
    if (sh.G > 1024 || p.rows > 0x7fffffffLL)
        mss::norm_fwd_long_kernel<T, R><<<unsigned(std::min<int64_t>(p.rows, 148 * 8)), 256, 0, s>>>(p);
    else if (wide)
        launch_norm_fwd<T, R, mss::kRowsWide>(p, sh, s);
    else
        launch_norm_fwd<T, R, mss::kRowsStrided>(p, sh, s);
    return launch_status();
}

// `blocks`: at most so many on entry, those launched on return.
template <typename T, typename S, int kRows, bool kMean, int kPieces>
int launch_norm_bwd(const NormParams& p, int G, int64_t* blocks, cudaStream_t s) {
    constexpr bool kRing = kRows != mss::kRowsStrided;
    const int64_t room = kRows == mss::kRowsShifted ? (p.dim + 14) / 8 * 8 : p.dim;
    const int64_t slot = kRing ? room * int64_t(sizeof(T) + sizeof(S) * (p.residual ? 2 : 1)) : 0;
    const int64_t sums = p.part ? p.dim * 8 : 0;  // of one group, at the end
    int64_t groups = std::min<int64_t>({mss::kNormThreads<kRows, kPieces> / G, G == 32 ? mss::kNormGroups : 15, (p.rows + *blocks - 1) / *blocks});
    groups = std::min(groups, kNormSmem / std::max(2 * slot, std::max<int64_t>(sums, 1)));
    if (groups < 1) return MSS_ERR_PATH;
    if (kRows == mss::kRowsShifted && p.rows > *blocks * groups && *blocks * groups * (p.dim % 8) % 8 != 0)
        *blocks -= *blocks % 8;  // a group's rows have one shift; more rows than blocks: 148 blocks
    const int stages = kRing ? int(std::min<int64_t>(mss::kNormStages, kNormSmem / (groups * slot))) : 0;
    const int smem = int(groups * std::max(stages * slot, sums));
    const auto kern = mss::norm_bwd_kernel<T, S, kRows, kMean, kPieces>;
    static std::mutex mu;
    static int done[kMaxDevices] = {};
    if (!per_device(done, mu, [&](int) {
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kNormSmem)) == cudaSuccess ? 1 : 0;
        }))
        return MSS_ERR_CUDA;
    kern<<<unsigned(*blocks), unsigned(groups * G), size_t(smem), s>>>(p, G, stages);
    return launch_status();
}

template <typename T, typename S, int kRows, bool kMean>
int launch_norm_bwd(const NormParams& p, int64_t* blocks, cudaStream_t s) {
    const int64_t pieces = (p.dim + 7) / 8;
    const auto group = [&](int per) { return int((pieces + 32 * per - 1) / (32 * per) * 32); };
    // One piece a thread where a warp takes the row, else two, which halve the work per
    // row that is not per element; with fp32 rows of middle length the memory sets
    // the time and one piece leaves more loads in flight.  16384 x 1024 bf16: two
    // 31, one 38 us; fp32: 47 both; 16384 x 1531 fp32: 78, 73 us.
    if (pieces <= 32 || (sizeof(S) == 4 && pieces > 64 && pieces <= 288)) return launch_norm_bwd<T, S, kRows, kMean, 1>(p, group(1), blocks, s);
    return launch_norm_bwd<T, S, kRows, kMean, 2>(p, group(2), blocks, s);
}

template <typename T, typename S>
int run_norm_bwd(const NormParams& p, mss::NormRows rows, bool mean, int64_t* blocks, cudaStream_t s) {
    if (p.selftest && (p.dim > 8192 || rows == mss::kRowsStrided)) return MSS_ERR_FLAGS;  // no waits for rows to test
    if (p.dim > 8192) {
        mss::norm_bwd_long_kernel<T, S><<<unsigned(*blocks), 512, 0, s>>>(p);
        return launch_status();
    }
    const auto go = [&](auto kRows) {
        constexpr int k = decltype(kRows)::value;
        return mean ? launch_norm_bwd<T, S, k, true>(p, blocks, s) : launch_norm_bwd<T, S, k, false>(p, blocks, s);
    };
    if (rows == mss::kRowsWide) return go(std::integral_constant<int, mss::kRowsWide>{});
    if (rows == mss::kRowsShifted) return go(std::integral_constant<int, mss::kRowsShifted>{});
    return go(std::integral_constant<int, mss::kRowsStrided>{});
}

}  // namespace
}  // namespace mss_host

using namespace mss_host;

extern "C" {

int64_t mss_norm_bwd_workspace_size(int64_t rows, int64_t dim) {
    int64_t n, bytes;
    if (!norm_elems(rows, dim, &n) || !mul_ok(std::min(rows, kNormParts), dim * 8, &bytes)) return MSS_ERR_SHAPE;
    return bytes;
}

int mss_norm_fwd(const void* x, const void* residual, const float* weight, const float* bias, float eps, void* y,
                 void* residual_out, float* mean, float* rstd, int64_t rows, int64_t dim, int dtype,
                 int residual_dtype, unsigned flags, void* stream) {
    if (flags & ~unsigned(MSS_NORM_FLAG_RMS)) return MSS_ERR_FLAGS;
    if (!known_dtype(dtype)) return MSS_ERR_DTYPE;
    if (!residual && !residual_out) residual_dtype = dtype;
    if (residual_dtype != MSS_DTYPE_F32 && residual_dtype != dtype) return MSS_ERR_DTYPE;
    int64_t n;
    if (!norm_elems(rows, dim, &n) || !(eps >= 0.f) || std::isinf(eps)) return MSS_ERR_SHAPE;
    if (n == 0) return MSS_OK;
    if (!x || !weight || !y) return MSS_ERR_NULL;
    const size_t esz = dtype == MSS_DTYPE_BF16 ? 2 : 4, rsz = residual_dtype == MSS_DTYPE_BF16 ? 2 : 4;
    const void* const io[] = {x, y};
    const void* const rs[] = {residual, residual_out};
    const void* const fl[] = {weight, bias, mean, rstd};
    if (!all_aligned(io, esz) || !all_aligned(rs, rsz) || !all_aligned(fl, 4)) return MSS_ERR_ALIGN;
    const int64_t nb = n * int64_t(esz), rb = n * int64_t(rsz);
    const Range ins[] = {{x, nb}, {residual, rb}, {weight, dim * 4}, {bias, dim * 4}};
    const Range outs[] = {{y, nb}, {residual_out, rb}, {mean, rows * 4}, {rstd, rows * 4}};
    if (any_overlap(outs, ins)) return MSS_ERR_ALIAS;
    NormParams p{};
    p.x = x, p.residual = residual, p.weight = weight, p.bias = bias, p.y = y, p.residual_out = residual_out;
    p.mean = mean, p.rstd = rstd, p.rows = rows, p.dim = dim, p.eps = eps, p.rms = (flags & MSS_NORM_FLAG_RMS) != 0;
    p.wait_ns = wait_limit_ns(), p.selftest = selftest_timeout();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool begins = all_aligned(io, 16) && all_aligned(rs, 16);
    const bool wide = begins && dim % 8 == 0 && aligned(weight, 16) && aligned(bias, 16);
    if (!(p.err = device_error_word())) return MSS_ERR_CUDA;
    if (dtype == MSS_DTYPE_F32) return run_norm_fwd<float, float>(p, wide, begins, s);
    return residual_dtype == MSS_DTYPE_F32 ? run_norm_fwd<bf16_t, float>(p, wide, begins, s) : run_norm_fwd<bf16_t, bf16_t>(p, wide, begins, s);
}

int mss_norm_bwd(const void* s_in, const float* weight, const float* mean, const float* rstd, const void* dy,
                 const void* dresidual_out, void* dx, void* dresidual, float* dweight, float* dbias, int64_t rows,
                 int64_t dim, int dtype, int s_dtype, void* workspace, int64_t workspace_bytes, void* stream) {
    if (!known_dtype(dtype) || (s_dtype != MSS_DTYPE_F32 && s_dtype != dtype)) return MSS_ERR_DTYPE;
    int64_t n;
    if (!norm_elems(rows, dim, &n) || workspace_bytes < 0) return MSS_ERR_SHAPE;
    if (dim == 0) return MSS_OK;
    if (rows > 0 && (!s_in || !weight || !rstd || !dy || (!dx && !dresidual))) return MSS_ERR_NULL;
    const size_t esz = dtype == MSS_DTYPE_BF16 ? 2 : 4, ssz = s_dtype == MSS_DTYPE_BF16 ? 2 : 4;
    const void* const io[] = {dy, dx};
    const void* const ss[] = {s_in, dresidual_out, dresidual};
    const void* const fl[] = {weight, mean, rstd, dweight, dbias};
    const void* const ws[] = {workspace};
    if (!all_aligned(io, esz) || !all_aligned(ss, ssz) || !all_aligned(fl, 4) || !all_aligned(ws, 16))
        return MSS_ERR_ALIGN;
    const int64_t need = dweight || dbias ? mss_norm_bwd_workspace_size(rows, dim) : 0;
    if (need < 0) return int(need);
    if (need > 0 && (!workspace || workspace_bytes < need)) return MSS_ERR_WORKSPACE;
    const int64_t nb = n * int64_t(esz), sb = n * int64_t(ssz);
    const Range ins[] = {{s_in, sb}, {weight, dim * 4}, {mean, rows * 4}, {rstd, rows * 4}, {dy, nb}, {dresidual_out, sb}};
    const Range outs[] = {{dx, nb}, {dresidual, sb}, {dweight, dim * 4}, {dbias, dim * 4}, {workspace, need}};
    if (any_overlap(outs, ins)) return MSS_ERR_ALIAS;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {
        if (dweight && cudaMemsetAsync(dweight, 0, size_t(dim) * 4, s) != cudaSuccess) return MSS_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, size_t(dim) * 4, s) != cudaSuccess) return MSS_ERR_CUDA;
        return MSS_OK;
    }
    NormParams p{};
    p.x = s_in, p.weight = weight, p.mean = const_cast<float*>(mean), p.rstd = const_cast<float*>(rstd), p.dy = dy;
    p.residual = dresidual_out, p.y = dx, p.residual_out = dresidual, p.rows = rows, p.dim = dim;
    p.part = need > 0 ? static_cast<float*>(workspace) : nullptr;
    p.wait_ns = wait_limit_ns(), p.selftest = selftest_timeout();
    if (!(p.err = device_error_word())) return MSS_ERR_CUDA;
    const mss::NormRows lie = !all_aligned(io, 16) || !all_aligned(ss, 16) ? mss::kRowsStrided
                              : dim % 8 == 0 && aligned(weight, 16)       ? mss::kRowsWide
                                                                          : mss::kRowsShifted;
    int64_t blocks = std::min(rows, kNormParts);
    const bool with_mean = mean || dbias;
    const int rc = dtype == MSS_DTYPE_F32    ? run_norm_bwd<float, float>(p, lie, with_mean, &blocks, s)
                   : s_dtype == MSS_DTYPE_F32 ? run_norm_bwd<bf16_t, float>(p, lie, with_mean, &blocks, s)
                                              : run_norm_bwd<bf16_t, bf16_t>(p, lie, with_mean, &blocks, s);
    if (rc != MSS_OK || need == 0) return rc;
    return launch_behind(mss::sum_rows_kernel, unsigned((2 * dim + 31) / 32), mss::kSumThreads, s, p.part, dweight, dbias, blocks,
                         2 * dim, dim);
}

}  // extern "C"
