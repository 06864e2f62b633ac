// glr.cu -- the gated linear recurrence behind the C ABI: argument checks and
// launches (kernels in glr.cuh).
#include <algorithm>
#include <iterator>

#include "host_common.h"
#include "launch.h"

#include "glr.cuh"
#include "sum_rows.cuh"
#include "tensor_map.h"

namespace mss_host {
namespace {

using mss::bf16_t;
using mss::GlrParams;

// Sizes in bytes of one call's arrays; false on a negative size or overflow.
struct GlrSizes {
    int64_t io, state, saved, units;  // units: blocks of 64 channels of one batch row
};

bool glr_sizes(int64_t batch, int64_t seqlen, int64_t dim, int64_t nstates, int64_t esz, GlrSizes* s) {
    int64_t tok, n, st, sv;
    if (batch < 0 || seqlen < 0 || dim < 0 || nstates < 0) return false;
    if (!mul_ok(batch, seqlen, &tok) || !mul_ok(tok, dim, &n) || !mul_ok(n, esz, &s->io)) return false;
    if (!mul_ok(nstates, dim, &st) || !mul_ok(st, 4, &s->state)) return false;
    const int64_t saves = seqlen / mss::kGlrTile + (seqlen % mss::kGlrTile != 0);
    if (!mul_ok(batch, saves, &sv) || !mul_ok(sv, dim, &sv) || !mul_ok(sv, 4, &s->saved)) return false;
    const int64_t nblk = dim / mss::kGlrCols + (dim % mss::kGlrCols != 0);
    return mul_ok(batch, nblk, &s->units) && s->units <= 0x7fffffffLL / mss::kGlrMaxCluster && tok <= (int64_t(1) << 40);
}

int copy_or_zero(float* dst, const float* src, int64_t bytes, cudaStream_t s) {
    if (!dst || bytes == 0) return MSS_OK;
    const cudaError_t e = src ? cudaMemcpyAsync(dst, src, size_t(bytes), cudaMemcpyDeviceToDevice, s)
                              : cudaMemsetAsync(dst, 0, size_t(bytes), s);
    return e == cudaSuccess ? MSS_OK : MSS_ERR_CUDA;
}

// A tensor [batch][seqlen][dim] as boxes of 8 tokens x 64 channels; tokens and
// channels behind the end read as zero.
bool encode_glr(CUtensorMap* m, const void* base, const GlrParams& p, int esz) {
    if (!base) return true;
    const cuuint64_t dims[3] = {cuuint64_t(p.dim), cuuint64_t(p.seqlen), cuuint64_t(p.batch)};
    const cuuint64_t strides[2] = {cuuint64_t(p.dim * esz), cuuint64_t(p.seqlen * p.dim * esz)};
    const cuuint32_t box[3] = {cuuint32_t(mss::kGlrCols), cuuint32_t(mss::kGlrRun), 1u};
    return encode_tiled(m, esz == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims,
                        strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <typename T, bool kTma, bool kPacked, bool kZ>
auto glr_kernel(bool bwd) -> void (*)(mss::GlrMaps, GlrParams) {
    return bwd ? mss::glr_bwd_kernel<T, kTma, kPacked, kZ> : mss::glr_fwd_kernel<T, kTma, kPacked, kZ>;
}

template <typename T, bool kTma>
constexpr int glr_smem_bytes(bool bwd, bool z, int cluster) {
    return bwd ? mss::glr_smem<T, kTma, true>(z ? 4 : 3, cluster) : mss::glr_smem<T, kTma, false>(z ? 3 : 2, cluster);
}

// The kernel may use its largest shared memory and clusters past 8 blocks on
// the current device; set once per device.
template <typename T, bool kTma, bool kPacked, bool kZ>
bool glr_allow(bool bwd) {
    static std::mutex mu[2];
    static int done[2][kMaxDevices] = {};
    return per_device(done[bwd], mu[bwd], [&](int) {
               const auto kern = glr_kernel<T, kTma, kPacked, kZ>(bwd);
               return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           glr_smem_bytes<T, kTma>(bwd, kZ, mss::kGlrMaxCluster)) == cudaSuccess &&
                              cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess
                          ? 1
                          : 0;
           }) > 0;
}

cudaLaunchConfig_t glr_config(cudaLaunchAttribute* at, int64_t units, int cluster, int smem, cudaStream_t s) {
    at->id = cudaLaunchAttributeClusterDimension;
    at->val.clusterDim.x = unsigned(cluster);
    at->val.clusterDim.y = at->val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(units * cluster));
    cfg.blockDim = dim3(mss::kGlrThreads);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    return cfg;
}

// Blocks that share the sequence of one unit (64 channels of a batch row): the
// most that still run all units at once and all have a tile.  Measured (bf16
// forward, with z) for 1 x 12288 x 1536 (24 units): 10 blocks 48 us, 8 53 us, 12
// (two rounds) 66 us; 2 x 8192 x 2560 (80 units): 3 blocks 92 us, 2 128 us, 4 113
// us; 1 x 65536 x 256 (4 units): 16 blocks 120 us, 8 205 us.
constexpr int kGlrClusters[] = {16, 14, 12, 10, 9, 8, 7, 6, 5, 4, 3, 2};
constexpr int64_t kGlrBlocks = 2 * 148;  // at most two blocks per SM of a B200 run at once

template <typename T, bool kTma>
int glr_cluster(bool bwd, int64_t units, int64_t seqlen) {
    static std::mutex mu[2][std::size(kGlrClusters)];
    static int active[2][std::size(kGlrClusters)][kMaxDevices] = {};  // 1 + how many run at once
    const int64_t tiles = (seqlen + mss::kGlrTile - 1) / mss::kGlrTile;
    for (size_t i = 0; i < std::size(kGlrClusters); ++i) {
        const int c = kGlrClusters[i];
        if (c > tiles || units * c > kGlrBlocks) continue;
        const int n = per_device(active[bwd][i], mu[bwd][i], [&](int) {
            if (!glr_allow<T, kTma, false, true>(bwd)) return 0;
            cudaLaunchAttribute at{};
            const cudaLaunchConfig_t cfg = glr_config(&at, 1, c, glr_smem_bytes<T, kTma>(bwd, true, c), nullptr);
            int k = 0;
            if (cudaOccupancyMaxActiveClusters(&k, glr_kernel<T, kTma, false, true>(bwd), &cfg) != cudaSuccess) {
                cudaGetLastError();
                k = 0;
            }
            return 1 + k;
        });
        if (units < n) return c;
    }
    return 1;
}

template <typename T, bool kTma, bool kPacked, bool kZ>
int launch_glr_variant(const mss::GlrMaps& maps, const GlrParams& p, bool bwd, int cluster, int64_t units, cudaStream_t s) {
    if (!glr_allow<T, kTma, kPacked, kZ>(bwd)) return MSS_ERR_CUDA;
    cudaLaunchAttribute at{};
    const cudaLaunchConfig_t cfg = glr_config(&at, units, cluster, glr_smem_bytes<T, kTma>(bwd, kZ, cluster), s);
    return cudaLaunchKernelEx(&cfg, glr_kernel<T, kTma, kPacked, kZ>(bwd), maps, p) == cudaSuccess ? launch_status() : MSS_ERR_CUDA;
}

template <typename T>
int launch_update(bool wide, const float* state, float* state_out, const void* x, const void* gate, const void* z,
                  const float* bias, void* y, int64_t batch, int64_t dim, cudaStream_t s) {
    const int64_t threads = wide ? dim / 4 : dim;
    const dim3 grid(unsigned((threads + 127) / 128), unsigned(std::min<int64_t>(batch, 65535)));
    const auto kern = wide ? mss::glr_update_kernel<T, 4> : mss::glr_update_kernel<T, 1>;
    kern<<<grid, 128, 0, s>>>(state, state_out, static_cast<const T*>(x), static_cast<const T*>(gate), static_cast<const T*>(z),
                              bias, static_cast<T*>(y), batch, dim);
    return launch_status();
}

// Rows of whole 16-byte pieces go by TMA, other rows by the 16-byte pieces that
// they touch, and tensors that begin off 16 bytes element by element.
template <typename T>
int launch_glr(GlrParams p, bool bwd, int64_t units, int* cluster, cudaStream_t s) {
    constexpr int esz = int(sizeof(T));
    const void* const in[] = {p.x, p.gate, p.z, p.dy};
    const void* const out[] = {p.y, p.dx, p.dgate, p.dz};
    const bool begins = all_aligned(in, 16);
    p.pairs = !begins ? -1 : p.dim % mss::kGlrLanes == 0 && all_aligned(out, esz * mss::kGlrLanes) ? 1 : 0;
    constexpr int64_t kMaxCoordinate = int64_t(1) << 31;
    const bool tma = p.pairs > 0 && p.dim * esz % 16 == 0 && p.batch < kMaxCoordinate &&
                     p.seqlen < kMaxCoordinate - mss::kGlrTile && p.dim < kMaxCoordinate - mss::kGlrCols;
    p.wait_ns = wait_limit_ns();
    p.selftest = selftest_timeout();
    if (p.selftest && !tma) return MSS_ERR_FLAGS;  // no waits for tiles to test
    *cluster = tma ? glr_cluster<T, true>(bwd, units, p.seqlen) : glr_cluster<T, false>(bwd, units, p.seqlen);
    mss::GlrMaps maps{};
    if (tma && (!encode_glr(&maps.gate, p.gate, p, esz) || !encode_glr(&maps.x, p.x, p, esz) ||
                !encode_glr(&maps.z, p.z, p, esz) || !encode_glr(&maps.dy, p.dy, p, esz)))
        return MSS_ERR_CUDA;
    const auto go = [&](auto t, auto k, auto z) {
        return launch_glr_variant<T, decltype(t)::value, decltype(k)::value, decltype(z)::value>(maps, p, bwd, *cluster, units, s);
    };
    const auto with_z = [&](auto t, auto k) { return p.z ? go(t, k, std::true_type{}) : go(t, k, std::false_type{}); };
    const auto with_k = [&](auto t) { return p.offsets ? with_z(t, std::true_type{}) : with_z(t, std::false_type{}); };
    return tma ? with_k(std::true_type{}) : with_k(std::false_type{});
}

}  // namespace
}  // namespace mss_host

using namespace mss_host;

extern "C" {

int64_t mss_glr_states_size(int64_t batch, int64_t seqlen, int64_t dim) {
    GlrSizes z;
    return glr_sizes(batch, seqlen, dim, batch, 4, &z) ? z.saved : int64_t(MSS_ERR_SHAPE);
}

int64_t mss_glr_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int dtype) {
    if (dtype != MSS_DTYPE_F32 && dtype != MSS_DTYPE_BF16) return MSS_ERR_DTYPE;
    GlrSizes z;
    if (!glr_sizes(batch, seqlen, dim, batch, dtype == MSS_DTYPE_BF16 ? 2 : 4, &z)) return MSS_ERR_SHAPE;
    if (seqlen == 0 || z.units == 0) return 0;
    // a row of sums for every block of a channel; the blocks per unit follow from
    // the device, at most these
    const int64_t tiles = (seqlen + mss::kGlrTile - 1) / mss::kGlrTile;
    const int64_t cluster = std::max<int64_t>(1, std::min<int64_t>({mss::kGlrMaxCluster, tiles, kGlrBlocks / z.units}));
    return batch * cluster < 2 ? 0 : z.state * cluster;
}

int mss_glr_fwd(const void* x, const void* gate, const void* z, const float* gate_bias, const float* initial_state,
                const int32_t* seq_offsets, int64_t nseq, void* y, float* last_state, float* states,
                int64_t states_bytes, int64_t batch, int64_t seqlen, int64_t dim, int dtype, void* stream) {
    if (dtype != MSS_DTYPE_F32 && dtype != MSS_DTYPE_BF16) return MSS_ERR_DTYPE;
    const size_t esz = dtype == MSS_DTYPE_BF16 ? 2 : 4;
    if (states_bytes < 0) return MSS_ERR_SHAPE;
    if (seq_offsets && (batch != 1 || nseq < 0 || seqlen >= 0x7fffffffLL || nseq >= 0x7fffffffLL)) return MSS_ERR_SHAPE;
    GlrSizes n;
    if (!glr_sizes(batch, seqlen, dim, seq_offsets ? nseq : batch, int64_t(esz), &n)) return MSS_ERR_SHAPE;
    if (batch == 0 || dim == 0) return MSS_OK;
    if (seqlen > 0 && (!x || !gate || (!y && !last_state && !states))) return MSS_ERR_NULL;
    const void* const io[] = {x, gate, z, y};
    const void* const fl[] = {gate_bias, initial_state, seq_offsets, last_state, states};
    if (!all_aligned(io, esz) || !all_aligned(fl, 4)) return MSS_ERR_ALIGN;
    if (states && states_bytes < n.saved) return MSS_ERR_WORKSPACE;
    const Range ins[] = {{x, n.io}, {gate, n.io}, {z, n.io}, {gate_bias, dim * 4}, {initial_state, n.state},
                         {seq_offsets, seq_offsets ? (nseq + 1) * 4 : 0}};
    const Range outs[] = {{y, n.io}, {last_state, n.state}, {states, n.saved}};
    if (any_overlap(outs, ins)) return MSS_ERR_ALIAS;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (seqlen == 0) return copy_or_zero(last_state, initial_state, n.state, s);
    GlrParams p{};
    p.x = x, p.gate = gate, p.z = y ? z : nullptr, p.bias = gate_bias, p.init = initial_state, p.offsets = seq_offsets;
    p.y = y, p.last = last_state, p.states = states;
    p.batch = batch, p.seqlen = seqlen, p.dim = dim, p.nseq = nseq;
    if (!(p.err = device_error_word())) return MSS_ERR_CUDA;
    int cluster;
    return dtype == MSS_DTYPE_BF16 ? launch_glr<bf16_t>(p, false, n.units, &cluster, s)
                                   : launch_glr<float>(p, false, n.units, &cluster, s);
}

int mss_glr_bwd(const void* x, const void* gate, const void* z, const float* gate_bias, const float* initial_state,
                const int32_t* seq_offsets, int64_t nseq, const float* states, int64_t states_bytes, const void* dy,
                const float* dlast, void* dx, void* dgate, void* dz, float* dbias, float* dinit, int64_t batch,
                int64_t seqlen, int64_t dim, int dtype, void* workspace, int64_t workspace_bytes, void* stream) {
    if (dtype != MSS_DTYPE_F32 && dtype != MSS_DTYPE_BF16) return MSS_ERR_DTYPE;
    const size_t esz = dtype == MSS_DTYPE_BF16 ? 2 : 4;
    if (states_bytes < 0 || workspace_bytes < 0) return MSS_ERR_SHAPE;
    if (seq_offsets && (batch != 1 || nseq < 0 || seqlen >= 0x7fffffffLL || nseq >= 0x7fffffffLL)) return MSS_ERR_SHAPE;
    GlrSizes n;
    if (!glr_sizes(batch, seqlen, dim, seq_offsets ? nseq : batch, int64_t(esz), &n)) return MSS_ERR_SHAPE;
    if (dim == 0) return MSS_OK;
    if (!z) dz = nullptr;
    if (batch > 0 && seqlen > 0 && (!x || !gate || !dy || !dx || !dgate || (z && !dz))) return MSS_ERR_NULL;
    const void* const io[] = {x, gate, z, dy, dx, dgate, dz};
    const void* const fl[] = {gate_bias, initial_state, seq_offsets, states, dlast, dbias, dinit, workspace};
    if (!all_aligned(io, esz) || !all_aligned(fl, 4)) return MSS_ERR_ALIGN;
    const int64_t need = dbias ? mss_glr_bwd_workspace_size(batch, seqlen, dim, dtype) : 0;
    if ((n.saved > 0 && (!states || states_bytes < n.saved)) || (need > 0 && (!workspace || workspace_bytes < need)))
        return MSS_ERR_WORKSPACE;
    const Range ins[] = {{x, n.io}, {gate, n.io}, {z, n.io}, {gate_bias, dim * 4}, {initial_state, n.state},
                         {seq_offsets, seq_offsets ? (nseq + 1) * 4 : 0}, {states, n.saved}, {dy, n.io}, {dlast, n.state}};
    const Range outs[] = {{dx, n.io}, {dgate, n.io}, {dz, n.io}, {dbias, dim * 4}, {dinit, n.state}, {workspace, need}};
    if (any_overlap(outs, ins)) return MSS_ERR_ALIAS;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (batch == 0 || seqlen == 0) {
        const int rc = copy_or_zero(dbias, nullptr, dim * 4, s);
        return rc != MSS_OK ? rc : copy_or_zero(dinit, dlast, n.state, s);
    }
    GlrParams p{};
    p.x = x, p.gate = gate, p.z = z, p.bias = gate_bias, p.init = initial_state, p.offsets = seq_offsets;
    p.states = const_cast<float*>(states), p.dy = dy, p.dlast = dlast, p.dx = dx, p.dgate = dgate, p.dz = dz;
    p.dinit = dinit, p.dbias_part = !dbias ? nullptr : need > 0 ? static_cast<float*>(workspace) : dbias;
    p.batch = batch, p.seqlen = seqlen, p.dim = dim, p.nseq = nseq;
    if (!(p.err = device_error_word())) return MSS_ERR_CUDA;
    int cluster;
    const int rc = dtype == MSS_DTYPE_BF16 ? launch_glr<bf16_t>(p, true, n.units, &cluster, s)
                                           : launch_glr<float>(p, true, n.units, &cluster, s);
    if (rc != MSS_OK || need == 0) return rc;
    return launch_behind(mss::sum_rows_kernel, unsigned((dim + 31) / 32), mss::kSumThreads, s, static_cast<const float*>(workspace),
                         dbias, static_cast<float*>(nullptr), batch * cluster, dim, dim);
}

int mss_glr_update(float* state, float* state_out, const void* x, const void* gate, const void* z,
                   const float* gate_bias, void* y, int64_t batch, int64_t dim, int dtype, void* stream) {
    if (dtype != MSS_DTYPE_F32 && dtype != MSS_DTYPE_BF16) return MSS_ERR_DTYPE;
    const size_t esz = dtype == MSS_DTYPE_BF16 ? 2 : 4;
    GlrSizes n;
    if (!glr_sizes(batch, 1, dim, batch, int64_t(esz), &n)) return MSS_ERR_SHAPE;
    if (batch == 0 || dim == 0) return MSS_OK;
    if (!state || !x || !gate || !y) return MSS_ERR_NULL;
    if (!state_out) state_out = state;
    const void* const io[] = {x, gate, z, y};
    const void* const fl[] = {gate_bias, state, state_out};
    if (!all_aligned(io, esz) || !all_aligned(fl, 4)) return MSS_ERR_ALIGN;
    const Range ins[] = {{x, n.io}, {gate, n.io}, {z, n.io}, {gate_bias, dim * 4}};
    const Range outs[] = {{y, n.io}, {state, n.state}, {state_out == state ? nullptr : state_out, n.state}};
    if (any_overlap(outs, ins)) return MSS_ERR_ALIAS;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool wide = dim % 4 == 0 && all_aligned(io, 4 * esz) && all_aligned(fl, 16);
    if (dtype == MSS_DTYPE_BF16) return launch_update<bf16_t>(wide, state, state_out, x, gate, z, gate_bias, y, batch, dim, s);
    return launch_update<float>(wide, state, state_out, x, gate, z, gate_bias, y, batch, dim, s);
}

}  // extern "C"
