// FlashAttention-2 forward and backward for GB300 (sm_103a): host side and C ABI.
//
// The kernels: fa2_fwd_sm103.cuh (16-bit forward), fa2_fwd_fp8_sm103.cuh (FP8
// forward), fa2_bwd_sm103.cuh (backward). This file plans the launches
// (tensor maps, persistent grid, work items), checks arguments and device,
// and exports the functions declared in include/fa2.h.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <chrono>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <type_traits>
#include <utility>

#include "fa2.h"
#include "fa2_bwd_sm103.cuh"
#include "fa2_fwd_fp8_sm103.cuh"
#include "fa2_fwd_sm103.cuh"
#include "fa2_fwd_d64_sm103.cuh"
#include "fa2_kv4_sm103.cuh"
#include "fa2_kv4_tc_sm103.cuh"
#include "fa2_rope_sm103.cuh"
#include "fa2_kv16_sm103.cuh"

// ==================================================================== host

namespace {

using fa2::Layout;
using fa2::Params;

std::atomic<long long> g_wait_limit_ns{2000000000LL};
std::atomic<int> g_debug_flags{0};

// The planner's kernel table has one shape with a choice: d = 64 with equal
// lengths runs fa2_fwd_d64_kernel (P in TMEM columns of its own, two MMA
// warps; the default, measured faster) or, with this bit set, the 16-bit
// kernel's d = 64 path (P written over S, one MMA warp).
constexpr int kTileCfgD64Shared = 1;
constexpr int kTileCfgMask = kTileCfgD64Shared;
std::atomic<int> g_tile_cfg{-1};   // -1: FA2_TILE_CFG not read yet

int tile_cfg() {
    const int c = g_tile_cfg.load(std::memory_order_acquire);
    if (c >= 0) return c;
    int v = 0;
    if (const char* e = std::getenv("FA2_TILE_CFG"))
        if (std::strcmp(e, "d64=shared") == 0) v = kTileCfgD64Shared;
    int expected = -1;
    g_tile_cfg.compare_exchange_strong(expected, v, std::memory_order_acq_rel);
    return g_tile_cfg.load(std::memory_order_acquire);
}
std::mutex g_mu;
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

constexpr int kMaxDevices = 64;
// Kernel slots: 16-bit forward 0-7, backward dK/dV 8-11, FP8 forward 12-13,
// backward dQ 14-17, d = 64 equal-length forward 18-19, attention over the
// 4-bit cache 20-43, over the 16-bit cache 44-47.
constexpr int kKernelSlots = 48;
// Per-device facts, read without a lock: every field is an atomic written
// with release and read with acquire, and two threads that probe the same
// device at once store the same values.
struct DeviceState {
    std::atomic<int> state;     // 0 = not probed, 1 = compute capability 10.3, 2 = other
    std::atomic<int> sm_count;
    std::atomic<bool> smem_set[kKernelSlots];  // dynamic shared-memory limit raised for kernel slot i
};
DeviceState g_dev[kMaxDevices];  // static storage: zero-initialised

// A CUDA call of this library failed: return FA2_ERR_CUDA and leave no
// (non-sticky) error of ours pending for the caller's next cudaGetLastError.
fa2_status cuda_fail() {
    (void)cudaGetLastError();
    return FA2_ERR_CUDA;
}

fa2_status get_encoder() {
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_encode) return FA2_OK;
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn)
        return cuda_fail();
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    return FA2_OK;
}

fa2_status check_device(int* dev_out) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return cuda_fail();
    if (dev < 0 || dev >= kMaxDevices) return FA2_ERR_UNSUPPORTED;
    DeviceState& st = g_dev[dev];
    int s = st.state.load(std::memory_order_acquire);
    if (s == 0) {
        int major = 0, minor = 0, sms = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return cuda_fail();
        st.sm_count.store(sms, std::memory_order_relaxed);
        s = (major == 10 && minor == 3) ? 1 : 2;
        st.state.store(s, std::memory_order_release);
    }
    *dev_out = dev;
    return s == 1 ? FA2_OK : FA2_ERR_UNSUPPORTED;
}

int sm_count(int dev) { return g_dev[dev].sm_count.load(std::memory_order_relaxed); }

// Raises the dynamic shared-memory limit of `kern` on device `dev` once.
template <typename K>
fa2_status set_smem(int dev, int slot, K kern, int bytes) {
    std::atomic<bool>& done = g_dev[dev].smem_set[slot];
    if (done.load(std::memory_order_acquire)) return FA2_OK;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return cuda_fail();
    done.store(true, std::memory_order_release);
    return FA2_OK;
}

// Queues one kernel and judges the launch by its own return code (not by
// cudaGetLastError, which would also report an error left pending earlier).
template <typename... Exp, typename... Act>
fa2_status launch_kernel(void (*kern)(Exp...), dim3 grid, int threads, int smem, cudaStream_t stream,
                         Act&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Act>(args)...) == cudaSuccess ? FA2_OK : cuda_fail();
}

// 2-D view [rows, d] of a 16-bit tensor, boxes of 128 rows x 64 elements
// (128 bytes, the widest box the 128-byte swizzle allows).
fa2_status encode_map(CUtensorMap* m, const void* ptr, uint64_t rows, int d) {
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), rows};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(d) * 2};
    cuuint32_t box[2] = {64, 128};
    cuuint32_t es[2] = {1, 1};
    CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(ptr), dims, strides, box,
                          es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FA2_OK : FA2_ERR_CUDA;
}

// 3-D view [mats, rows, d] of a 16-bit tensor (general mode): a box of 128
// rows never crosses into the next head, and rows past `rows` read as zero.
fa2_status encode_map_3d(CUtensorMap* m, const void* ptr, uint64_t mats, uint64_t rows, int d) {
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), rows, mats};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, rows * static_cast<cuuint64_t>(d) * 2};
    cuuint32_t box[3] = {64, 128, 1};
    cuuint32_t es[3] = {1, 1, 1};
    CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(ptr), dims, strides, box,
                          es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FA2_OK : FA2_ERR_CUDA;
}

template <int D, bool kBf16, bool kGen = false>
fa2_status launch(int dev, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                  const Params& p, dim3 grid, cudaStream_t stream) {
    constexpr int kSmem = Layout<D>::kSmemBytes;
    auto kern = fa2::fa2_fwd_kernel<D, kBf16, kGen>;
    const int slot = (D == 128 ? 0 : 2) + (kBf16 ? 0 : 1) + (kGen ? 4 : 0);
    const fa2_status st = set_smem(dev, slot, kern, kSmem);
    if (st != FA2_OK) return st;
    return launch_kernel(kern, grid, fa2::kThreads, kSmem, stream, mq, mk, mv, p);
}

// The d = 64 equal-length kernel (P in TMEM columns of its own).
template <bool kBf16>
fa2_status launch_d64(int dev, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                      const Params& p, dim3 grid, cudaStream_t stream) {
    constexpr int kSmem = fa2::d64::Lay::kSmemBytes;
    auto kern = fa2::fa2_fwd_d64_kernel<kBf16>;
    const fa2_status st = set_smem(dev, kBf16 ? 18 : 19, kern, kSmem);
    if (st != FA2_OK) return st;
    return launch_kernel(kern, grid, fa2::kThreads, kSmem, stream, mq, mk, mv, p);
}

// 2-D view [rows, 128] of an 8-bit tensor (FP8 kernel): boxes of 128 rows x
// 128 bytes, the full width of the 128-byte swizzle.
fa2_status encode_map_u8(CUtensorMap* m, const void* ptr, uint64_t rows) {
    cuuint64_t dims[2] = {128, rows};
    cuuint64_t strides[1] = {128};
    cuuint32_t box[2] = {128, 128};
    cuuint32_t es[2] = {1, 1};
    CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FA2_OK : FA2_ERR_CUDA;
}

// 3-D view [mats, rows, 128] of an 8-bit tensor (FP8 general mode): a box
// never crosses into the next head, and rows past `rows` read as zero.
fa2_status encode_map_u8_3d(CUtensorMap* m, const void* ptr, uint64_t mats, uint64_t rows) {
    cuuint64_t dims[3] = {128, rows, mats};
    cuuint64_t strides[2] = {128, rows * 128};
    cuuint32_t box[3] = {128, 128, 1};
    cuuint32_t es[3] = {1, 1, 1};
    CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FA2_OK : FA2_ERR_CUDA;
}

template <bool kGen>
fa2_status launch_fp8(int dev, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                      const Params& p, dim3 grid, cudaStream_t stream) {
    constexpr int kSmem = fa2::fp8::Lay::kSmemBytes;
    constexpr int kSlot = kGen ? 13 : 12;
    auto kern = fa2::fa2_fwd_fp8_kernel<kGen>;
    const fa2_status st = set_smem(dev, kSlot, kern, kSmem);
    if (st != FA2_OK) return st;
    return launch_kernel(kern, grid, fa2::kThreads, kSmem, stream, mq, mk, mv, p);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The general-mode kernel (any lengths, optional causal mask) on checked
// arguments. Also takes equal-length calls with N = 128, whose items have a
// single KV tile: the kernels' equal-length mode relies on every item
// having two or more.
fa2_status fwd_general(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H_q, int H_kv,
                       int N_q, int N_k, int d, float scale, int causal, fa2_dtype dtype, cudaStream_t stream) {
    const long long heads_q = static_cast<long long>(B) * H_q;
    const long long rows_q = heads_q * N_q;
    const long long rows_kv = static_cast<long long>(B) * H_kv * N_k;
    const long long tq = (N_q + fa2::kBM - 1) / fa2::kBM;
    const long long items = heads_q * ((tq + fa2::kNQ - 1) / fa2::kNQ);
    // Item indices stay below 2^31 - 4096 so that a CTA's next index (at most
    // two grids further) never overflows.
    if (rows_q > 0x7FFFFFFFLL || rows_kv > 0x7FFFFFFFLL || items > 0x7FFFFFFFLL - 4096) return FA2_ERR_UNSUPPORTED;

    int dev = 0;
    fa2_status st = check_device(&dev);
    if (st != FA2_OK) return st;
    if ((st = get_encoder()) != FA2_OK) return st;

    CUtensorMap mq, mk, mv;
    if (encode_map_3d(&mq, q, static_cast<uint64_t>(heads_q), static_cast<uint64_t>(N_q), d) != FA2_OK ||
        encode_map_3d(&mk, k, static_cast<uint64_t>(B) * H_kv, static_cast<uint64_t>(N_k), d) != FA2_OK ||
        encode_map_3d(&mv, v, static_cast<uint64_t>(B) * H_kv, static_cast<uint64_t>(N_k), d) != FA2_OK)
        return cuda_fail();

    Params p{};
    p.o = o;
    p.lse = lse;
    p.wait_limit_ns = g_wait_limit_ns.load();
    p.debug_flags = g_debug_flags.load();
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    p.nq = N_q;
    p.nk = N_k;
    p.causal = causal;
    p.heads_q = static_cast<int>(heads_q);
    p.hq = H_q;
    p.group = H_q / H_kv;
    p.tq = static_cast<int>(tq);
    p.pairs = static_cast<int>((tq + fa2::kNQ - 1) / fa2::kNQ);
    p.total_items = static_cast<int>(items);
    p.heads_kv = B * H_kv;
    p.rows_q = rows_q;
    p.rows_kv = rows_kv;
    const dim3 grid(static_cast<unsigned>(std::min<long long>(items, sm_count(dev))));

    const bool bf = dtype == FA2_BF16;
    if (d == 128)
        return bf ? launch<128, true, true>(dev, mq, mk, mv, p, grid, stream)
                  : launch<128, false, true>(dev, mq, mk, mv, p, grid, stream);
    return bf ? launch<64, true, true>(dev, mq, mk, mv, p, grid, stream)
              : launch<64, false, true>(dev, mq, mk, mv, p, grid, stream);
}

// FP8 counterpart of fwd_general (d = 128).
fa2_status fwd_fp8_general(const void* q, const void* k, const void* v, const float* q_descale,
                           const float* k_descale, const float* v_descale, void* o, float* lse, int B, int H_q,
                           int H_kv, int N_q, int N_k, float scale, int causal, cudaStream_t stream) {
    const long long heads_q = static_cast<long long>(B) * H_q;
    const long long rows_q = heads_q * N_q;
    const long long rows_kv = static_cast<long long>(B) * H_kv * N_k;
    const long long tq = (N_q + fa2::kBM - 1) / fa2::kBM;
    const long long items = heads_q * ((tq + fa2::kNQ - 1) / fa2::kNQ);
    // Item indices stay below 2^31 - 4096 so that a CTA's next index (at most
    // two grids further) never overflows.
    if (rows_q > 0x7FFFFFFFLL || rows_kv > 0x7FFFFFFFLL || items > 0x7FFFFFFFLL - 4096) return FA2_ERR_UNSUPPORTED;

    int dev = 0;
    fa2_status st = check_device(&dev);
    if (st != FA2_OK) return st;
    if ((st = get_encoder()) != FA2_OK) return st;

    CUtensorMap mq, mk, mv;
    const uint64_t hkv = static_cast<uint64_t>(B) * H_kv;
    if (encode_map_u8_3d(&mq, q, static_cast<uint64_t>(heads_q), static_cast<uint64_t>(N_q)) != FA2_OK ||
        encode_map_u8_3d(&mk, k, hkv, static_cast<uint64_t>(N_k)) != FA2_OK ||
        encode_map_u8_3d(&mv, v, hkv, static_cast<uint64_t>(N_k)) != FA2_OK)
        return cuda_fail();

    Params p{};
    p.o = o;
    p.lse = lse;
    p.wait_limit_ns = g_wait_limit_ns.load();
    p.debug_flags = g_debug_flags.load();
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    p.nq = N_q;
    p.nk = N_k;
    p.causal = causal;
    p.heads_q = static_cast<int>(heads_q);
    p.hq = H_q;
    p.group = H_q / H_kv;
    p.tq = static_cast<int>(tq);
    p.pairs = static_cast<int>((tq + fa2::kNQ - 1) / fa2::kNQ);
    p.total_items = static_cast<int>(items);
    p.heads_kv = B * H_kv;
    p.rows_q = rows_q;
    p.rows_kv = rows_kv;
    p.q_descale = q_descale;
    p.k_descale = k_descale;
    p.v_descale = v_descale;
    const dim3 grid(static_cast<unsigned>(std::min<long long>(items, sm_count(dev))));
    return launch_fp8<true>(dev, mq, mk, mv, p, grid, stream);
}

}  // namespace

extern "C" {

fa2_status fa2_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H_q,
                       int H_kv, int N, int d, float scale, fa2_dtype dtype, cudaStream_t stream) {
    if (!q || !k || !v || !o || !lse) return FA2_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return FA2_ERR_INVALID_ARG;
    if (B <= 0 || H_q <= 0 || H_kv <= 0 || N <= 0 || d <= 0) return FA2_ERR_INVALID_ARG;
    if (H_q % H_kv != 0) return FA2_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.0f)) return FA2_ERR_INVALID_ARG;
    if (dtype != FA2_BF16 && dtype != FA2_FP16) return FA2_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FA2_ERR_UNSUPPORTED;
    if (N % fa2::kBM != 0) return FA2_ERR_UNSUPPORTED;
    if (N == fa2::kBN) return fwd_general(q, k, v, o, lse, B, H_q, H_kv, N, N, d, scale, 0, dtype, stream);
    // TMA coordinates and row indices are 32-bit.
    const long long rows_q = static_cast<long long>(B) * H_q * N;
    const long long groups = static_cast<long long>(B) * H_kv;
    if (rows_q > 0x7FFFFFFFLL) return FA2_ERR_UNSUPPORTED;

    int dev = 0;
    fa2_status st = check_device(&dev);
    if (st != FA2_OK) return st;
    if ((st = get_encoder()) != FA2_OK) return st;

    CUtensorMap mq, mk, mv;
    const uint64_t rows_kv = static_cast<uint64_t>(B) * H_kv * N;
    if (encode_map(&mq, q, static_cast<uint64_t>(rows_q), d) != FA2_OK ||
        encode_map(&mk, k, rows_kv, d) != FA2_OK || encode_map(&mv, v, rows_kv, d) != FA2_OK)
        return cuda_fail();

    Params p{};
    p.o = o;
    p.lse = lse;
    p.wait_limit_ns = g_wait_limit_ns.load();
    p.n_kv_tiles = N / fa2::kBN;
    p.q_tiles = (H_q / H_kv) * (N / fa2::kBM);
    p.pairs = (p.q_tiles + fa2::kNQ - 1) / fa2::kNQ;
    p.total_items = static_cast<int>(p.pairs * groups);
    p.kv_rows = N;
    p.heads_kv = B * H_kv;
    p.rows_q = rows_q;
    p.rows_kv = static_cast<long long>(rows_kv);
    p.debug_flags = g_debug_flags.load();
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    // Persistent grid: one CTA per SM (shared memory and TMEM admit one).
    const dim3 grid(static_cast<unsigned>(std::min<long long>(p.total_items, sm_count(dev))));

    const bool bf = dtype == FA2_BF16;
    if (d == 128)
        return bf ? launch<128, true>(dev, mq, mk, mv, p, grid, stream)
                  : launch<128, false>(dev, mq, mk, mv, p, grid, stream);
    if (tile_cfg() & kTileCfgD64Shared)
        return bf ? launch<64, true>(dev, mq, mk, mv, p, grid, stream)
                  : launch<64, false>(dev, mq, mk, mv, p, grid, stream);
    return bf ? launch_d64<true>(dev, mq, mk, mv, p, grid, stream) : launch_d64<false>(dev, mq, mk, mv, p, grid, stream);
}

fa2_status fa2_fwd_fp8(const void* q, const void* k, const void* v, const float* q_descale,
                       const float* k_descale, const float* v_descale, void* o, float* lse, int B, int H_q,
                       int H_kv, int N, int d, float scale, cudaStream_t stream) {
    if (!q || !k || !v || !o || !lse || !q_descale || !k_descale || !v_descale) return FA2_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return FA2_ERR_INVALID_ARG;
    if (!aligned4(q_descale) || !aligned4(k_descale) || !aligned4(v_descale)) return FA2_ERR_INVALID_ARG;
    if (B <= 0 || H_q <= 0 || H_kv <= 0 || N <= 0 || d <= 0) return FA2_ERR_INVALID_ARG;
    if (H_q % H_kv != 0) return FA2_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.0f)) return FA2_ERR_INVALID_ARG;
    if (d != fa2::fp8::kD) return FA2_ERR_UNSUPPORTED;
    if (N % fa2::kBM != 0) return FA2_ERR_UNSUPPORTED;
    if (N == fa2::kBN)
        return fwd_fp8_general(q, k, v, q_descale, k_descale, v_descale, o, lse, B, H_q, H_kv, N, N, scale, 0, stream);
    const long long rows_q = static_cast<long long>(B) * H_q * N;
    const long long groups = static_cast<long long>(B) * H_kv;
    if (rows_q > 0x7FFFFFFFLL) return FA2_ERR_UNSUPPORTED;

    int dev = 0;
    fa2_status st = check_device(&dev);
    if (st != FA2_OK) return st;
    if ((st = get_encoder()) != FA2_OK) return st;

    CUtensorMap mq, mk, mv;
    const uint64_t rows_kv = static_cast<uint64_t>(B) * H_kv * N;
    if (encode_map_u8(&mq, q, static_cast<uint64_t>(rows_q)) != FA2_OK || encode_map_u8(&mk, k, rows_kv) != FA2_OK ||
        encode_map_u8(&mv, v, rows_kv) != FA2_OK)
        return cuda_fail();

    Params p{};
    p.o = o;
    p.lse = lse;
    p.wait_limit_ns = g_wait_limit_ns.load();
    p.n_kv_tiles = N / fa2::kBN;
    p.q_tiles = (H_q / H_kv) * (N / fa2::kBM);
    p.pairs = (p.q_tiles + fa2::kNQ - 1) / fa2::kNQ;
    p.total_items = static_cast<int>(p.pairs * groups);
    p.kv_rows = N;
    p.heads_kv = B * H_kv;
    p.rows_q = rows_q;
    p.rows_kv = static_cast<long long>(rows_kv);
    p.debug_flags = g_debug_flags.load();
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    p.q_descale = q_descale;
    p.k_descale = k_descale;
    p.v_descale = v_descale;
    const dim3 grid(static_cast<unsigned>(std::min<long long>(p.total_items, sm_count(dev))));
    return launch_fp8<false>(dev, mq, mk, mv, p, grid, stream);
}

fa2_status fa2_fwd_fp8_ex(const void* q, const void* k, const void* v, const float* q_descale,
                          const float* k_descale, const float* v_descale, void* o, float* lse, int B, int H_q,
                          int H_kv, int N_q, int N_k, int d, float scale, int causal, cudaStream_t stream) {
    if (!q || !k || !v || !o || !lse || !q_descale || !k_descale || !v_descale) return FA2_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return FA2_ERR_INVALID_ARG;
    if (!aligned4(q_descale) || !aligned4(k_descale) || !aligned4(v_descale)) return FA2_ERR_INVALID_ARG;
    if (B <= 0 || H_q <= 0 || H_kv <= 0 || N_q <= 0 || N_k <= 0 || d <= 0) return FA2_ERR_INVALID_ARG;
    if (H_q % H_kv != 0) return FA2_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.0f)) return FA2_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return FA2_ERR_INVALID_ARG;
    if (d != fa2::fp8::kD) return FA2_ERR_UNSUPPORTED;
    // The plain case is the multiple-of-128 kernel.
    if (!causal && N_q == N_k && N_q % fa2::kBM == 0)
        return fa2_fwd_fp8(q, k, v, q_descale, k_descale, v_descale, o, lse, B, H_q, H_kv, N_q, d, scale, stream);
    return fwd_fp8_general(q, k, v, q_descale, k_descale, v_descale, o, lse, B, H_q, H_kv, N_q, N_k, scale, causal,
                           stream);
}

fa2_status fa2_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N,
                   int d, float scale, fa2_dtype dtype, cudaStream_t stream) {
    return fa2_fwd_gqa(q, k, v, o, lse, B, H, H, N, d, scale, dtype, stream);
}

fa2_status fa2_fwd_ex(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H_q,
                      int H_kv, int N_q, int N_k, int d, float scale, int causal, fa2_dtype dtype,
                      cudaStream_t stream) {
    if (!q || !k || !v || !o || !lse) return FA2_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
        return FA2_ERR_INVALID_ARG;
    if (B <= 0 || H_q <= 0 || H_kv <= 0 || N_q <= 0 || N_k <= 0 || d <= 0) return FA2_ERR_INVALID_ARG;
    if (H_q % H_kv != 0) return FA2_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.0f)) return FA2_ERR_INVALID_ARG;
    if (dtype != FA2_BF16 && dtype != FA2_FP16) return FA2_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return FA2_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FA2_ERR_UNSUPPORTED;
    // The plain case is the multiple-of-128 kernel.
    if (!causal && N_q == N_k && N_q % fa2::kBM == 0)
        return fa2_fwd_gqa(q, k, v, o, lse, B, H_q, H_kv, N_q, d, scale, dtype, stream);
    return fwd_general(q, k, v, o, lse, B, H_q, H_kv, N_q, N_k, d, scale, causal, dtype, stream);
}

}  // extern "C"

namespace {

// The argument and size checks that fa2_bwd and fa2_bwd_noalloc share (every
// pointer but fa2_bwd's `delta`), in the order the header documents:
// FA2_ERR_INVALID_ARG before FA2_ERR_UNSUPPORTED.
fa2_status bwd_check_args(const void* q, const void* k, const void* v, const void* o, const float* lse,
                          const void* dout, void* dq, void* dk, void* dv, int B, int H_q, int H_kv, int N, int d,
                          float scale, int causal, fa2_dtype dtype) {
    const void* ptrs[] = {q, k, v, o, lse, dout, dq, dk, dv};
    for (const void* x : ptrs)
        if (!x || !aligned16(x)) return FA2_ERR_INVALID_ARG;
    if (B <= 0 || H_q <= 0 || H_kv <= 0 || N <= 0 || d <= 0) return FA2_ERR_INVALID_ARG;
    if (H_q % H_kv != 0) return FA2_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.0f)) return FA2_ERR_INVALID_ARG;
    if (dtype != FA2_BF16 && dtype != FA2_FP16) return FA2_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return FA2_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FA2_ERR_UNSUPPORTED;
    const long long rows_q = static_cast<long long>(B) * H_q * N;
    if (rows_q > 0x7FFFFFFFLL || static_cast<long long>(B) * H_q > 65535) return FA2_ERR_UNSUPPORTED;
    return FA2_OK;
}

// The backward's three launches on checked arguments and a checked device.
fa2_status bwd_launch(int dev, const void* q, const void* k, const void* v, const void* o, const float* lse,
                      const void* dout, void* dq, void* dk, void* dv, float* delta, int B, int H_q, int H_kv,
                      int N, int d, float scale, int causal, fa2_dtype dtype, cudaStream_t stream) {
    fa2_status st = get_encoder();
    if (st != FA2_OK) return st;
    const long long rows_q = static_cast<long long>(B) * H_q * N;
    // [heads, N, d] views: tiles never cross heads; rows past a ragged N read as 0
    CUtensorMap mq, mk, mv, mdo;
    const uint64_t hq = static_cast<uint64_t>(B) * H_q, hkv = static_cast<uint64_t>(B) * H_kv;
    const uint64_t n = static_cast<uint64_t>(N);
    if (encode_map_3d(&mq, q, hq, n, d) != FA2_OK || encode_map_3d(&mk, k, hkv, n, d) != FA2_OK ||
        encode_map_3d(&mv, v, hkv, n, d) != FA2_OK || encode_map_3d(&mdo, dout, hq, n, d) != FA2_OK)
        return FA2_ERR_CUDA;

    fa2::bwd::Params p{};
    p.o = o;
    p.lse = lse;
    p.dout = dout;
    p.delta = delta;
    p.dq = dq;
    p.dk = dk;
    p.dv = dv;
    p.wait_limit_ns = g_wait_limit_ns.load();
    p.debug_flags = g_debug_flags.load();
    p.n = N;
    p.n_tiles = (N + fa2::kBM - 1) / fa2::kBM;
    p.hq = H_q;
    p.group = H_q / H_kv;
    p.causal = causal;
    p.scale = scale;
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    p.heads_q = B * H_q;
    p.heads_kv = B * H_kv;
    p.rows_q = rows_q;
    p.rows_kv = static_cast<long long>(B) * H_kv * N;
    const bool bf = dtype == FA2_BF16;
    const dim3 gdelta(static_cast<unsigned>((rows_q + 15) / 16));
    // dK/dV and dQ: persistent, one CTA per SM over the key (query) tiles,
    // in pairs of equal total cost under the causal mask
    const long long kv_units = static_cast<long long>(causal ? (p.n_tiles + 1) / 2 : p.n_tiles) * B * H_kv;
    const dim3 gkv(static_cast<unsigned>(std::min<long long>(kv_units, sm_count(dev))));
    const long long q_units = static_cast<long long>(causal ? (p.n_tiles + 1) / 2 : p.n_tiles) * B * H_q;
    const dim3 gq(static_cast<unsigned>(std::min<long long>(q_units, sm_count(dev))));

    auto run = [&](auto delta_k, auto dkdv_k, auto dq_k, int smem_kv, int smem_q, int slot) -> fa2_status {
        fa2_status s = set_smem(dev, slot, dkdv_k, smem_kv);
        if (s == FA2_OK) s = set_smem(dev, slot + 6, dq_k, smem_q);
        if (s == FA2_OK) s = launch_kernel(delta_k, gdelta, 256, 0, stream, o, dout, delta, rows_q);
        if (s == FA2_OK) s = launch_kernel(dkdv_k, gkv, fa2::bwd::kThreads, smem_kv, stream, mq, mk, mv, mdo, p);
        if (s == FA2_OK) s = launch_kernel(dq_k, gq, fa2::bwd::kThreads, smem_q, stream, mq, mk, mv, mdo, p);
        return s;
    };
    using namespace fa2::bwd;
    if (d == 128)
        return bf ? run(fa2_bwd_delta_kernel<128, true>, fa2_bwd_dkdv_kernel<128, true>, fa2_bwd_dq_kernel<128, true>,
                        DkdvLayout<128>::kSmemBytes, DqLayout<128>::kSmemBytes, 8)
                  : run(fa2_bwd_delta_kernel<128, false>, fa2_bwd_dkdv_kernel<128, false>,
                        fa2_bwd_dq_kernel<128, false>, DkdvLayout<128>::kSmemBytes, DqLayout<128>::kSmemBytes, 9);
    return bf ? run(fa2_bwd_delta_kernel<64, true>, fa2_bwd_dkdv_kernel<64, true>, fa2_bwd_dq_kernel<64, true>,
                    DkdvLayout<64>::kSmemBytes, DqLayout<64>::kSmemBytes, 10)
              : run(fa2_bwd_delta_kernel<64, false>, fa2_bwd_dkdv_kernel<64, false>, fa2_bwd_dq_kernel<64, false>,
                    DkdvLayout<64>::kSmemBytes, DqLayout<64>::kSmemBytes, 11);
}

}  // namespace

extern "C" {

fa2_status fa2_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
                   const void* dout, void* dq, void* dk, void* dv, float* delta, int B, int H_q, int H_kv,
                   int N, int d, float scale, int causal, fa2_dtype dtype, cudaStream_t stream) {
    if (!delta || !aligned16(delta)) return FA2_ERR_INVALID_ARG;
    fa2_status st = bwd_check_args(q, k, v, o, lse, dout, dq, dk, dv, B, H_q, H_kv, N, d, scale, causal, dtype);
    if (st != FA2_OK) return st;
    int dev = 0;
    if ((st = check_device(&dev)) != FA2_OK) return st;
    return bwd_launch(dev, q, k, v, o, lse, dout, dq, dk, dv, delta, B, H_q, H_kv, N, d, scale, causal, dtype,
                      stream);
}

}  // extern "C"

// ---------------------------------------------------------------- backward without allocation

// Scratch for fa2_bwd_noalloc: the per-row D = rowsum(dO o O) of the
// backward, for at most kNoAllocMaxRows query rows (4 MiB of fp32). Every GPU
// that loads this library keeps this array until the process exits. In host
// code the name stands for the array but is not its device address: that
// comes from cudaGetSymbolAddress, asked on every call with the caller's
// device current, so the address always belongs to the context the kernels
// run in (after cudaDeviceReset, or under another context, the array may
// live elsewhere).
static constexpr long long kNoAllocMaxRows = 1LL << 20;
static __device__ __align__(256) float fa2_noalloc_delta[kNoAllocMaxRows];

extern "C" {

fa2_status fa2_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const float* lse,
                           const void* dout, void* dq, void* dk, void* dv, int B, int H_q, int H_kv, int N,
                           int d, float scale, int causal, fa2_dtype dtype, cudaStream_t stream) {
    // fa2_bwd's checks first, so the same arguments give the same errors.
    fa2_status st = bwd_check_args(q, k, v, o, lse, dout, dq, dk, dv, B, H_q, H_kv, N, d, scale, causal, dtype);
    if (st != FA2_OK) return st;
    int dev = 0;
    if ((st = check_device(&dev)) != FA2_OK) return st;
    if (static_cast<long long>(B) * H_q * N > kNoAllocMaxRows) return FA2_ERR_UNSUPPORTED;
    // The array's address in the current context (a host-side lookup; the
    // first one on a device may load this library's device code there).
    void* ptr = nullptr;
    if (cudaGetSymbolAddress(&ptr, fa2_noalloc_delta) != cudaSuccess || !ptr) return cuda_fail();
    // D is written in full by the first kernel of the backward before it is
    // read, so nothing left from an earlier call needs clearing.
    return bwd_launch(dev, q, k, v, o, lse, dout, dq, dk, dv, static_cast<float*>(ptr), B, H_q, H_kv, N, d, scale,
                      causal, dtype, stream);
}

}  // extern "C"

// ---------------------------------------------------------------- the paged 4-bit KV cache

namespace {

// Queues one kernel that waits itself for the one before it (programmatic
// dependent launch), in clusters of `cluster` CTAs.
template <typename P>
fa2_status kv4_launch_kernel(void (*kern)(P), long long grid, int threads, int smem, cudaStream_t stream, const P& p,
                             int cluster = 1) {
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? FA2_OK : cuda_fail();
}

// Launches a copy of `rows` rows with one row a thread where four would give
// fewer blocks than SMs, else with four.
template <typename F>
fa2_status kv4_rows(int dev, int rows, int d, F&& launch) {
    const int pass = 256 / (d / 8);
    const long long blocks = (static_cast<long long>(rows) + 4 * pass - 1) / (4 * pass);
    if (blocks < sm_count(dev)) return launch(std::true_type{}, (static_cast<long long>(rows) + pass - 1) / pass);
    return launch(std::false_type{}, blocks);
}

int log2_of(int x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

// Sizes that every cache entry point shares (INVALID_ARG before UNSUPPORTED).
constexpr long long kMaxTokens = 0x7FFFFFFFLL - 256;
fa2_status kv4_check_pages(int page_size, int num_pages, int max_pages) {
    if (page_size <= 0 || num_pages <= 0 || max_pages <= 0) return FA2_ERR_INVALID_ARG;
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return FA2_ERR_UNSUPPORTED;
    if (static_cast<long long>(num_pages) * page_size > kMaxTokens ||
        static_cast<long long>(max_pages) * page_size > kMaxTokens)
        return FA2_ERR_UNSUPPORTED;
    return FA2_OK;
}

// Query rows that a pass over the keys serves. Up to 24 (8, 16 or 24) by the
// kernel on mma.sync, beyond by the one on tcgen05 (32, 48 or 64): 38 sequences
// of 8192 tokens, heads of 128, take 89 and 110 us by the first for 16 and 24
// rows, 111 and 121 us by the second (its 32-row form for 24); for 32 rows 138 us
// by the first and 121 us by the second. More than 64 rows are cut into blocks
// of about equal size.
int kv4_block(long long rows) {
    if (rows <= 24) return static_cast<int>((rows + 7) / 8) * 8;
    const long long blocks = (rows + 63) / 64;
    return std::max(32, static_cast<int>((rows + 16 * blocks - 1) / (16 * blocks)) * 16);
}
constexpr bool kv4_on_tc(int block) { return block > 24; }
constexpr int kv4_ctas_per_sm(int block) { return block == 8 || kv4_on_tc(block) ? 2 : 1; }

// Sizes that the attention takes.
fa2_status kv4_check_sizes(int B, int H_q, int H_kv, int N_q, int d, int max_pages, int page_size) {
    if (B <= 0 || H_q <= 0 || H_kv <= 0 || N_q <= 0 || d <= 0 || H_q % H_kv != 0) return FA2_ERR_INVALID_ARG;
    const fa2_status st = kv4_check_pages(page_size, 1, max_pages);
    if (st != FA2_OK) return st;
    if (d != 64 && d != 128) return FA2_ERR_UNSUPPORTED;
    if (static_cast<long long>(B) * H_q > (0x7FFFFFFFLL - 64) / N_q) return FA2_ERR_UNSUPPORTED;   // row indices are 32-bit,
    if (H_kv > 65535 / 2) return FA2_ERR_UNSUPPORTED;                                             // and a page's bytes,
    // and units of the line of tiles, which padding can double
    const long long rows = static_cast<long long>(H_q / H_kv) * N_q, block = kv4_block(rows);
    const long long segments = static_cast<long long>(B) * H_kv * ((rows + block - 1) / block);
    if (segments * ((static_cast<long long>(max_pages) * page_size + 31) / 32) > (1LL << 30)) return FA2_ERR_UNSUPPORTED;
    return FA2_OK;
}

// The CTAs that can have work: runs have kMinRun tiles or more, and a padded
// line has at most one run for each segment beyond those.
long long kv4_ctas(long long segments, long long max_tokens, long long most) {
    const long long tiles = (max_tokens + 31) / 32;
    if (segments >= most) return most;
    return std::min(most, segments * (tiles / fa2::kv4::kMinRun + 1));
}

// Workspace: two partial results a CTA, then two counters a CTA; nothing where
// no segment can be split: each gets a CTA of its own (`locate`).
int64_t kv4_workspace(long long B, long long hkv, long long rows, int d, long long max_tokens) {
    const int block = kv4_block(rows);
    const long long segments = B * hkv * ((rows + block - 1) / block);
    // as many CTAs as a whole device runs at once have a segment each
    if (segments <= 128 * kv4_ctas_per_sm(block) && max_tokens <= 32LL * (fa2::kv4::kMinRun + fa2::kv4::kSpare)) return 0;
    return kv4_ctas(segments, max_tokens, fa2::kv4::kMaxCtas) *
           (2LL * block * (d + 2) * static_cast<int64_t>(sizeof(float)) + 2 * static_cast<int64_t>(sizeof(unsigned long long)));
}

// A number that no other launch of this process has, and that memory left
// by anything else holds only by a chance of 2^-48; low 16 bits 0.
unsigned long long kv4_nonce() {
    static const unsigned long long seed =
        static_cast<unsigned long long>(std::chrono::steady_clock::now().time_since_epoch().count()) * 0x9E3779B97F4A7C15ULL ^
        reinterpret_cast<uintptr_t>(&g_mu) * 0xD1B54A32D192ED03ULL;
    static std::atomic<unsigned long long> calls{seed};
    unsigned long long n = 0;
    while (n == 0) n = (calls.fetch_add(1, std::memory_order_relaxed) * 0x9E3779B97F4A7C15ULL) << 16;
    return n;
}

template <int D, int kRows, bool kBf16>
fa2_status kv4_launch(int dev, fa2::kv4::FwdParams p, cudaStream_t stream) {
    using namespace fa2::kv4;
    constexpr bool kTc = kv4_on_tc(kRows);
    constexpr int NR = kTc ? 1 : kRows / 8;
    constexpr int kThreads = kTc ? tc::kAll : Shape<NR>::kThreads;
    constexpr int kSmem = [] {
        if constexpr (kTc) return static_cast<int>(sizeof(tc::Smem<D, kRows>)) + 1024;
        else return static_cast<int>(sizeof(FwdSmem<D, NR>));
    }();
    constexpr int kPerSm = kv4_ctas_per_sm(kRows);
    static_assert(kTc || kPerSm == Shape<NR>::kCtas, "CTAs an SM");
    static_assert(kPerSm * (kSmem + 1024) <= 228 * 1024, "shared memory budget");
    auto kern = [] {
        if constexpr (kTc) return tc::fa2_kv4_fwd_tc_kernel<D, kRows, kBf16>;
        else return fa2_kv4_fwd_kernel<D, NR, kBf16>;
    }();
    const int slot = 20 + (D == 128 ? 0 : 12) + 2 * (kTc ? 1 + kRows / 16 : NR - 1) + (kBf16 ? 0 : 1);
    const fa2_status st = set_smem(dev, slot, kern, kSmem);
    if (st != FA2_OK) return st;
    p.rblocks = (p.rows + kRows - 1) / kRows;
    const long long segments = static_cast<long long>(p.B) * p.hkv * p.rblocks;
    p.ctas = static_cast<int>(kv4_ctas(segments, p.max_tokens, std::min(sm_count(dev) * kPerSm, fa2::kv4::kMaxCtas)));
    // Without a workspace every segment needs a CTA, also where they run in waves.
    if (!p.part_o) p.ctas = std::max(p.ctas, static_cast<int>(segments));
    if (p.part_o) {
        p.part_ml = p.part_o + 2LL * p.ctas * kRows * D;
        p.arrived = reinterpret_cast<unsigned long long*>(p.part_ml + 2LL * p.ctas * kRows * 2);
    }
    // 32 KB or more of zeros a CTA
    p.idle = static_cast<int>(std::min<long long>(std::max(1, p.ctas / p.B), static_cast<long long>(p.hkv) * p.rows * D / 16384 + 1));
    p.nonce = kv4_nonce();
    return kv4_launch_kernel(kern, p.ctas, kThreads, kSmem, stream, p);
}

template <int D, bool kBf16>
fa2_status kv4_launch_rows(int dev, const fa2::kv4::FwdParams& p, cudaStream_t stream) {
    switch (kv4_block(p.rows)) {
        case 8: return kv4_launch<D, 8, kBf16>(dev, p, stream);
        case 16: return kv4_launch<D, 16, kBf16>(dev, p, stream);
        case 24: return kv4_launch<D, 24, kBf16>(dev, p, stream);
        case 32: return kv4_launch<D, 32, kBf16>(dev, p, stream);
        case 48: return kv4_launch<D, 48, kBf16>(dev, p, stream);
        default: return kv4_launch<D, 64, kBf16>(dev, p, stream);
    }
}

}  // namespace

extern "C" {

fa2_status fa2_kv4_plan(const int32_t* seq_lens, const int32_t* new_lens, int32_t* block_table,
                        int32_t* free_pages, const int32_t* free_state, int32_t* seq_lens_out,
                        int32_t* accepted, int32_t* slots, int32_t* free_state_out, int B, int N,
                        int max_pages, int page_size, int num_pages, cudaStream_t stream) {
    const void* ptrs[] = {seq_lens, new_lens, block_table, free_pages, free_state, seq_lens_out, accepted, slots,
                          free_state_out};
    for (const void* x : ptrs)
        if (!x || !aligned4(x)) return FA2_ERR_INVALID_ARG;
    if (B <= 0 || N <= 0) return FA2_ERR_INVALID_ARG;
    fa2_status st = kv4_check_pages(page_size, num_pages, max_pages);
    if (st != FA2_OK) return st;
    // requests are counted in steps of up to 1024, slots in steps of 256
    if (static_cast<long long>(B) * N > 0x7FFFFFFFLL - 1024) return FA2_ERR_UNSUPPORTED;
    int dev = 0;
    if ((st = check_device(&dev)) != FA2_OK) return st;
    fa2::kv4::PlanParams p{};
    p.seq_lens = seq_lens;
    p.new_lens = new_lens;
    p.block_table = block_table;
    p.free_pages = free_pages;
    p.free_state = free_state;
    p.seq_lens_out = seq_lens_out;
    p.accepted = accepted;
    p.slots = slots;
    p.free_state_out = free_state_out;
    p.B = B;
    p.n = N;
    p.max_pages = max_pages;
    p.page = page_size;
    p.log2_page = log2_of(page_size);
    p.num_pages = num_pages;
    // 256 threads for a decoding step, whose scan is the shorter one: 256 requests of
    // one token take 2.9 us (3.8 with 1024 threads), of four 4.2 (3.9); 512 of one take
    // 4.6 us (4.0). One CTA up to 8192 slots: by a CTA for every 1024 slots 16 requests of
    // 512 take the same 4.4 us (512 of 16: 4.0 instead of 7.2); 32 of 512 take 5.8 by one
    // CTA and 4.4 by more. Above, a warp for every 256 slots: 48 prompts of 16384 take
    // 5.2 us (120 by one CTA; 20.9 by a cluster of eight, which writing in place asks for).
    const long long all = static_cast<long long>(B) * N;
    auto in = [](const void* a, const void* out, long long n) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(out);
        return x < y + 4 * n && y < x + 4 * n;
    };
    p.in_place = 0;
    for (const void* a : {static_cast<const void*>(seq_lens), static_cast<const void*>(new_lens)})
        p.in_place |= in(a, seq_lens_out, B) || in(a, accepted, B);
    p.in_place |= in(free_state, free_state_out, 2);
    if (B <= 256 && all <= 2048) return kv4_launch_kernel(fa2::kv4::fa2_kv4_plan_kernel<256>, 1, 256, 0, stream, p);
    if (all <= 8192) return kv4_launch_kernel(fa2::kv4::fa2_kv4_plan_kernel<1024>, 1, 1024, 0, stream, p);
    if (p.in_place)
        return kv4_launch_kernel(fa2::kv4::fa2_kv4_plan_kernel<1024>, fa2::kv4::kPlanCtas, 1024, 0, stream, p,
                                 fa2::kv4::kPlanCtas);
    return kv4_launch_kernel(fa2::kv4::fa2_kv4_plan_kernel<1024>,
                             std::min<long long>(sm_count(dev), (all + 8191) / 8192), 1024, 0, stream, p);
}

fa2_status fa2_kv4_append(const void* k, const void* v, const int32_t* slots, void* cache,
                          const float* k_descale, const float* v_descale, int B, int H_kv, int N, int d,
                          int64_t k_stride_b, int64_t k_stride_h, int64_t k_stride_n, int64_t v_stride_b,
                          int64_t v_stride_h, int64_t v_stride_n, int page_size, int num_pages,
                          fa2_dtype dtype, cudaStream_t stream) {
    if (!k || !v || !slots || !cache || !k_descale || !v_descale) return FA2_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(cache)) return FA2_ERR_INVALID_ARG;
    if (!aligned4(slots) || !aligned4(k_descale) || !aligned4(v_descale)) return FA2_ERR_INVALID_ARG;
    if (B <= 0 || H_kv <= 0 || N <= 0 || d <= 0) return FA2_ERR_INVALID_ARG;
    for (int64_t s : {k_stride_b, k_stride_h, k_stride_n, v_stride_b, v_stride_h, v_stride_n})
        if (s < 0 || s % 8 != 0) return FA2_ERR_INVALID_ARG;
    if (dtype != FA2_BF16 && dtype != FA2_FP16) return FA2_ERR_INVALID_ARG;
    fa2_status st = kv4_check_pages(page_size, num_pages, 1);
    if (st != FA2_OK) return st;
    if (d != 64 && d != 128) return FA2_ERR_UNSUPPORTED;
    for (int64_t s : {k_stride_b, k_stride_h, k_stride_n, v_stride_b, v_stride_h, v_stride_n})
        if (s > 0x7FFFFFFFLL) return FA2_ERR_UNSUPPORTED;
    const long long rows = static_cast<long long>(B) * H_kv;
    if (rows > 0x7FFFFFFFLL / N) return FA2_ERR_UNSUPPORTED;
    int dev = 0;
    if ((st = check_device(&dev)) != FA2_OK) return st;
    fa2::kv4::AppendParams p{};
    p.x[0] = k;
    p.x[1] = v;
    p.sb[0] = static_cast<int>(k_stride_b);
    p.sh[0] = static_cast<int>(k_stride_h);
    p.sn[0] = static_cast<int>(k_stride_n);
    p.sb[1] = static_cast<int>(v_stride_b);
    p.sh[1] = static_cast<int>(v_stride_h);
    p.sn[1] = static_cast<int>(v_stride_n);
    p.descale[0] = k_descale;
    p.descale[1] = v_descale;
    p.slots = slots;
    p.cache = static_cast<uint8_t*>(cache);
    p.rows = static_cast<int>(rows * N);
    p.hkv = H_kv;
    p.n = N;
    p.page = page_size;
    p.log2_page = log2_of(page_size);
    p.num_slots = num_pages * page_size;
    const bool bf = dtype == FA2_BF16;
    return kv4_rows(dev, p.rows, d, [&](auto few, long long grid) {
        using namespace fa2::kv4;
        constexpr int P = few ? 1 : 4;
        if (d == 128)
            return bf ? kv4_launch_kernel(fa2_kv4_append_kernel<128, true, P>, grid, 256, 0, stream, p)
                      : kv4_launch_kernel(fa2_kv4_append_kernel<128, false, P>, grid, 256, 0, stream, p);
        return bf ? kv4_launch_kernel(fa2_kv4_append_kernel<64, true, P>, grid, 256, 0, stream, p)
                  : kv4_launch_kernel(fa2_kv4_append_kernel<64, false, P>, grid, 256, 0, stream, p);
    });
}

fa2_status fa2_kv4_gather(const void* cache, const int32_t* block_table, const int32_t* seq_lens,
                          const int32_t* starts, const float* k_descale, const float* v_descale, void* k,
                          void* v, int B, int H_kv, int N, int d, int max_pages, int page_size, int num_pages,
                          fa2_dtype dtype, cudaStream_t stream) {
    if (!cache || !block_table || !seq_lens || !k_descale || !v_descale || !k || !v) return FA2_ERR_INVALID_ARG;
    if (!aligned16(cache) || !aligned16(k) || !aligned16(v)) return FA2_ERR_INVALID_ARG;
    if (!aligned4(block_table) || !aligned4(seq_lens) || !aligned4(starts) || !aligned4(k_descale) ||
        !aligned4(v_descale))
        return FA2_ERR_INVALID_ARG;
    if (B <= 0 || H_kv <= 0 || N <= 0 || d <= 0) return FA2_ERR_INVALID_ARG;
    if (dtype != FA2_BF16 && dtype != FA2_FP16) return FA2_ERR_INVALID_ARG;
    fa2_status st = kv4_check_pages(page_size, num_pages, max_pages);
    if (st != FA2_OK) return st;
    if (d != 64 && d != 128) return FA2_ERR_UNSUPPORTED;
    const long long rows = static_cast<long long>(B) * H_kv;
    if (rows > 0x7FFFFFFFLL / N) return FA2_ERR_UNSUPPORTED;
    int dev = 0;
    if ((st = check_device(&dev)) != FA2_OK) return st;
    fa2::kv4::GatherParams p{};
    p.cache = static_cast<const uint8_t*>(cache);
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.starts = starts;
    p.descale[0] = k_descale;
    p.descale[1] = v_descale;
    p.out[0] = k;
    p.out[1] = v;
    p.rows = static_cast<int>(rows * N);
    p.hkv = H_kv;
    p.n = N;
    p.page = page_size;
    p.log2_page = log2_of(page_size);
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    const bool bf = dtype == FA2_BF16;
    return kv4_rows(dev, p.rows, d, [&](auto few, long long grid) {
        using namespace fa2::kv4;
        constexpr int P = few ? 1 : 4;
        if (d == 128)
            return bf ? kv4_launch_kernel(fa2_kv4_gather_kernel<128, true, P>, grid, 256, 0, stream, p)
                      : kv4_launch_kernel(fa2_kv4_gather_kernel<128, false, P>, grid, 256, 0, stream, p);
        return bf ? kv4_launch_kernel(fa2_kv4_gather_kernel<64, true, P>, grid, 256, 0, stream, p)
                  : kv4_launch_kernel(fa2_kv4_gather_kernel<64, false, P>, grid, 256, 0, stream, p);
    });
}

int64_t fa2_fwd_kv4_workspace(int B, int H_q, int H_kv, int N_q, int d, int max_pages, int page_size) {
    if (kv4_check_sizes(B, H_q, H_kv, N_q, d, max_pages, page_size) != FA2_OK) return -1;
    return kv4_workspace(B, H_kv, static_cast<long long>(H_q / H_kv) * N_q, d,
                         static_cast<long long>(max_pages) * page_size);
}

fa2_status fa2_fwd_kv4(const void* q, const void* cache, const int32_t* block_table, const int32_t* seq_lens,
                       const float* k_descale, const float* v_descale, void* o, float* lse, void* workspace,
                       int64_t workspace_bytes, int B, int H_q, int H_kv, int N_q, int d, int max_pages,
                       int page_size, int num_pages, float scale, int causal, fa2_dtype dtype,
                       cudaStream_t stream) {
    if (!q || !cache || !block_table || !seq_lens || !k_descale || !v_descale || !o || !lse) return FA2_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(cache) || !aligned16(o) || !aligned16(lse) || !aligned16(workspace))
        return FA2_ERR_INVALID_ARG;
    if (!aligned4(block_table) || !aligned4(seq_lens) || !aligned4(k_descale) || !aligned4(v_descale))
        return FA2_ERR_INVALID_ARG;
    if (B <= 0 || H_q <= 0 || H_kv <= 0 || N_q <= 0 || d <= 0) return FA2_ERR_INVALID_ARG;
    if (H_q % H_kv != 0) return FA2_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.0f)) return FA2_ERR_INVALID_ARG;
    if (dtype != FA2_BF16 && dtype != FA2_FP16) return FA2_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return FA2_ERR_INVALID_ARG;
    fa2_status st = kv4_check_pages(page_size, num_pages, max_pages);
    if (st != FA2_OK) return st;
    if ((st = kv4_check_sizes(B, H_q, H_kv, N_q, d, max_pages, page_size)) != FA2_OK) return st;
    const int64_t need = fa2_fwd_kv4_workspace(B, H_q, H_kv, N_q, d, max_pages, page_size);
    if (need > 0 && (!workspace || workspace_bytes < need)) return FA2_ERR_INVALID_ARG;
    int dev = 0;
    if ((st = check_device(&dev)) != FA2_OK) return st;
    fa2::kv4::FwdParams p{};
    p.q = q;
    p.cache = static_cast<const uint8_t*>(cache);
    p.k_descale = k_descale;
    p.v_descale = v_descale;
    p.seq_lens = seq_lens;
    p.block_table = block_table;
    p.o = o;
    p.lse = lse;
    p.part_o = need > 0 ? static_cast<float*>(workspace) : nullptr;
    p.B = B;
    p.hkv = H_kv;
    p.nq = N_q;
    p.rows = H_q / H_kv * N_q;
    p.max_pages = max_pages;
    p.max_tokens = max_pages * page_size;
    p.page = page_size;
    p.log2_page = log2_of(page_size);
    p.num_pages = num_pages;
    p.wait_limit_ns = g_wait_limit_ns.load();
    p.debug_flags = g_debug_flags.load();
    p.part = page_size * (d / 2 + d / 16);
    p.page_bytes = H_kv * 2 * p.part;
    p.causal = causal;
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    const bool bf = dtype == FA2_BF16;
    if (d == 128)
        return bf ? kv4_launch_rows<128, true>(dev, p, stream) : kv4_launch_rows<128, false>(dev, p, stream);
    return bf ? kv4_launch_rows<64, true>(dev, p, stream) : kv4_launch_rows<64, false>(dev, p, stream);
}

}  // extern "C"

// ---------------------------------------------------------------- rotary positions, the paged 16-bit KV cache

namespace {

// The part of the arguments that the rotation and the append share.
fa2_status rope_check(const void* positions, const void* inv_freq, const void* axes, int d, int rot_dim, int n_axes,
                      int interleaved, fa2_dtype dtype) {
    if (!positions || !inv_freq || !aligned4(positions) || !aligned4(inv_freq) || !aligned4(axes)) return FA2_ERR_INVALID_ARG;
    if (d <= 0 || rot_dim <= 0 || n_axes <= 0 || (interleaved != 0 && interleaved != 1)) return FA2_ERR_INVALID_ARG;
    if (dtype != FA2_BF16 && dtype != FA2_FP16) return FA2_ERR_INVALID_ARG;
    return FA2_OK;
}
bool rope_sizes(int d, int rot_dim, int n_axes) { return (d == 64 || d == 128) && rot_dim <= d && rot_dim % 16 == 0 && n_axes <= 8; }

// Several tokens a block where that gives every SM four blocks or more: their
// angles are made together. Else one, which spreads few tokens wider.
template <bool kCache>
fa2_status rope_launch(int dev, const fa2::rope::Params& p, int d, bool bf, cudaStream_t stream) {
    using namespace fa2::rope;
    const long long blocks = (static_cast<long long>(p.tokens) + kTokens - 1) / kTokens;
    const bool many = blocks >= 4LL * sm_count(dev);
    const long long grid = many ? blocks : p.tokens;
    auto go = [&](auto few, auto many_k) { return kv4_launch_kernel(many ? +many_k : +few, grid, kThreads, 0, stream, p); };
    if (d == 128)
        return bf ? go(fa2_rope_kernel<128, true, kCache, 1>, fa2_rope_kernel<128, true, kCache, kTokens>)
                  : go(fa2_rope_kernel<128, false, kCache, 1>, fa2_rope_kernel<128, false, kCache, kTokens>);
    return bf ? go(fa2_rope_kernel<64, true, kCache, 1>, fa2_rope_kernel<64, true, kCache, kTokens>)
              : go(fa2_rope_kernel<64, false, kCache, 1>, fa2_rope_kernel<64, false, kCache, kTokens>);
}

fa2_status rope(const void* q, const void* k, void* q_out, void* k_out, const int32_t* positions, const float* inv_freq,
                const int32_t* axes, int B, int H_q, int H_kv, int N, int d, int rot_dim, int n_axes, int interleaved,
                int inverse, const int64_t* strides, fa2_dtype dtype, cudaStream_t stream) {
    if (!q || !q_out || !strides || !k != !k_out) return FA2_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out)) return FA2_ERR_INVALID_ARG;
    if (B <= 0 || H_q <= 0 || N <= 0 || (k ? H_kv <= 0 : H_kv != 0)) return FA2_ERR_INVALID_ARG;
    const int sizes[3] = {B, 0, N};
    for (int i = 0; i < 12; ++i) {
        if (!k && (i / 3) % 2) continue;
        const int64_t s = strides[i];
        if (s < 0 || s % 8 != 0) return FA2_ERR_INVALID_ARG;
        // what is written may not lie on itself
        const int n = i % 3 == 1 ? (i < 9 ? H_q : H_kv) : sizes[i % 3];
        if (i >= 6 && s == 0 && n > 1) return FA2_ERR_INVALID_ARG;
    }
    fa2_status st = rope_check(positions, inv_freq, axes, d, rot_dim, n_axes, interleaved, dtype);
    if (st != FA2_OK) return st;
    if (!rope_sizes(d, rot_dim, n_axes)) return FA2_ERR_UNSUPPORTED;
    for (int i = 0; i < 12; ++i)
        if ((k || !((i / 3) % 2)) && strides[i] > 0x7FFFFFFFLL) return FA2_ERR_UNSUPPORTED;
    // tokens, and a block's rows, are counted in 32 bits
    if (B > (0x7FFFFFFF - 1024) / N || static_cast<long long>(H_q) + H_kv > (1 << 24)) return FA2_ERR_UNSUPPORTED;
    int dev = 0;
    if ((st = check_device(&dev)) != FA2_OK) return st;
    fa2::rope::Params p{};
    const void* in[2] = {q, k};
    void* out[2] = {q_out, k_out};
    for (int i = 0; i < 2; ++i) {
        p.in[i] = in[i];
        p.out[i] = out[i];
        if (!in[i]) continue;
        p.in_b[i] = static_cast<int>(strides[3 * i]);
        p.in_h[i] = static_cast<int>(strides[3 * i + 1]);
        p.in_n[i] = static_cast<int>(strides[3 * i + 2]);
        p.out_b[i] = static_cast<int>(strides[6 + 3 * i]);
        p.out_h[i] = static_cast<int>(strides[6 + 3 * i + 1]);
        p.out_n[i] = static_cast<int>(strides[6 + 3 * i + 2]);
    }
    p.heads[0] = H_q;
    p.heads[1] = H_kv;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.axes = axes;
    p.tokens = B * N;
    p.n = N;
    p.n_axes = n_axes;
    p.rot = rot_dim;
    p.interleaved = interleaved;
    p.inverse = inverse;
    return rope_launch<false>(dev, p, d, dtype == FA2_BF16, stream);
}

// Pages of the 16-bit cache as matrices [page_size, d] in boxes of a whole one,
// in the order of shared memory (Tiles in fa2_kv16_sm103.cuh): columns of a block, tokens of a group of
// eight, blocks, groups. A coordinate past the last page reads as zeros.
fa2_status kv16_encode_cache(CUtensorMap* m, const void* ptr, uint64_t mats, int page_size, int d) {
    const cuuint64_t row = static_cast<cuuint64_t>(d) * 2;
    const cuuint32_t blocks = static_cast<cuuint32_t>(d / 64), groups = static_cast<cuuint32_t>(page_size / 8);
    cuuint64_t dims[5] = {64, 8, blocks, groups, mats};
    cuuint64_t strides[4] = {row, 128, 8 * row, static_cast<cuuint64_t>(page_size) * row};
    cuuint32_t box[5] = {64, 8, blocks, groups, 1};
    cuuint32_t es[5] = {1, 1, 1, 1, 1};
    CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 5, const_cast<void*>(ptr), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FA2_OK : FA2_ERR_CUDA;
}

// q [T, H_q, d] with boxes of the `group` heads that share a KV head and as
// many tokens as fill 128 rows.
fa2_status kv16_encode_q(CUtensorMap* m, const void* ptr, int T, int H_q, int d, int group, int64_t stride_t, int64_t stride_h) {
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H_q), static_cast<cuuint64_t>(T)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(stride_h) * 2, static_cast<cuuint64_t>(stride_t) * 2};
    cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(128 / group)};
    cuuint32_t es[3] = {1, 1, 1};
    CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(ptr), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FA2_OK : FA2_ERR_CUDA;
}

// Row blocks that T new tokens of B requests can have, for each KV head, and
// the units of all.
long long kv16_blocks(int T, int B, int H_q, int H_kv) { return T / (2 * (128 / (H_q / H_kv))) + std::min(T, B); }
long long kv16_units(int T, int B, int H_q, int H_kv, long long max_tokens) {
    return kv16_blocks(T, B, H_q, H_kv) * H_kv * (fa2::kv16::kStart + std::max(fa2::kv16::kPairUnits, fa2::kv16::kSingleUnits) * ((max_tokens + 127) / 128));
}

fa2_status kv16_check_sizes(int T, int B, int H_q, int H_kv, int d, int max_pages, int page_size) {
    if (T <= 0 || B <= 0 || H_q <= 0 || H_kv <= 0 || d <= 0 || H_q % H_kv != 0) return FA2_ERR_INVALID_ARG;
    const fa2_status st = kv4_check_pages(page_size, 1, max_pages);
    if (st != FA2_OK) return st;
    if ((d != 64 && d != 128) || H_q / H_kv > 128) return FA2_ERR_UNSUPPORTED;
    if (static_cast<long long>(T) * H_q > 0x7FFFFFFFLL || B > 0x7FFFFFFF - 1024) return FA2_ERR_UNSUPPORTED;
    if (kv16_blocks(T, B, H_q, H_kv) * H_kv > (1LL << 30) || kv16_units(T, B, H_q, H_kv, static_cast<long long>(max_pages) * page_size) > (1LL << 30))
        return FA2_ERR_UNSUPPORTED;
    return FA2_OK;
}

// Rows of a buffer of partial results: blocks are two tiles unless all tokens fit one.
int kv16_part_rows(int T, int group) { return T <= 128 / group ? (T * group + 31) / 32 * 32 : 256; }

int kv16_ctas(int T, int B, int H_q, int H_kv, long long max_tokens, int most) {
    const long long units = kv16_units(T, B, H_q, H_kv, max_tokens);
    return static_cast<int>(std::min<long long>(most, (units + fa2::kv16::kMinRun - 1) / fa2::kv16::kMinRun));
}

template <int D, bool kBf16>
fa2_status kv16_launch(int dev, const CUtensorMap& mq, const CUtensorMap& mkv, const fa2::kv16::Params& p, cudaStream_t stream) {
    using namespace fa2::kv16;
    constexpr int kSmem = Lay<D>::kSmemBytes;
    auto kern = fa2_kv16_fwd_kernel<D, kBf16>;
    constexpr int kSlot = 44 + (D == 128 ? 0 : 2) + (kBf16 ? 0 : 1);
    static_assert(kSlot < kKernelSlots, "a slot behind the array");
    const fa2_status st = set_smem(dev, kSlot, kern, kSmem);
    if (st != FA2_OK) return st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.ctas));
    cfg.blockDim = dim3(fa2::kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, mq, mkv, p) != cudaSuccess) return cuda_fail();
    cfg.gridDim = dim3(static_cast<unsigned>(p.ctas), kJoinY);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, fa2_kv16_join_kernel<D, kBf16>, p) == cudaSuccess ? FA2_OK : cuda_fail();
}

}  // namespace

extern "C" {

fa2_status fa2_rope(const void* q, const void* k, void* q_out, void* k_out, const int32_t* positions, const float* inv_freq,
                    const int32_t* axes, int B, int H_q, int H_kv, int N, int d, int rot_dim, int n_axes, int interleaved,
                    const int64_t* strides, fa2_dtype dtype, cudaStream_t stream) {
    return rope(q, k, q_out, k_out, positions, inv_freq, axes, B, H_q, H_kv, N, d, rot_dim, n_axes, interleaved, 0, strides,
                dtype, stream);
}

fa2_status fa2_rope_bwd(const void* dq_out, const void* dk_out, void* dq, void* dk, const int32_t* positions,
                        const float* inv_freq, const int32_t* axes, int B, int H_q, int H_kv, int N, int d, int rot_dim,
                        int n_axes, int interleaved, const int64_t* strides, fa2_dtype dtype, cudaStream_t stream) {
    return rope(dq_out, dk_out, dq, dk, positions, inv_freq, axes, B, H_q, H_kv, N, d, rot_dim, n_axes, interleaved, 1, strides,
                dtype, stream);
}

fa2_status fa2_kv16_append(const void* q, const void* k, const void* v, const int32_t* slots, const int32_t* positions,
                           const float* inv_freq, const int32_t* axes, void* cache, void* q_out, int T, int H_q, int H_kv, int d,
                           int rot_dim, int n_axes, int interleaved, const int64_t* strides, int page_size, int num_pages,
                           fa2_dtype dtype, cudaStream_t stream) {
    if (!k || !v || !slots || !cache || !strides || !q != !q_out) return FA2_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(cache) || !aligned16(q_out) || !aligned4(slots))
        return FA2_ERR_INVALID_ARG;
    if (T <= 0 || H_kv <= 0 || d <= 0 || (q ? H_q <= 0 : H_q != 0)) return FA2_ERR_INVALID_ARG;
    for (int i = q ? 0 : 2; i < 6; ++i)
        if (strides[i] < 0 || strides[i] % 8 != 0) return FA2_ERR_INVALID_ARG;
    fa2_status st = FA2_OK;
    if (positions) {
        if ((st = rope_check(positions, inv_freq, axes, d, rot_dim, n_axes, interleaved, dtype)) != FA2_OK) return st;
    } else if (q || rot_dim != 0 || (dtype != FA2_BF16 && dtype != FA2_FP16)) {
        return FA2_ERR_INVALID_ARG;   // without positions nothing is rotated, and there is nothing to do with q
    }
    if ((st = kv4_check_pages(page_size, num_pages, 1)) != FA2_OK) return st;
    if (positions ? !rope_sizes(d, rot_dim, n_axes) : d != 64 && d != 128) return FA2_ERR_UNSUPPORTED;
    for (int i = q ? 0 : 2; i < 6; ++i)
        if (strides[i] > 0x7FFFFFFFLL) return FA2_ERR_UNSUPPORTED;
    if (T > 0x7FFFFFFF - 1024 || H_kv > (1 << 23) || H_q > (1 << 23)) return FA2_ERR_UNSUPPORTED;
    int dev = 0;
    if ((st = check_device(&dev)) != FA2_OK) return st;
    fa2::rope::Params p{};
    const void* in[3] = {q, k, v};
    for (int i = 0; i < 3; ++i) {
        p.in[i] = in[i];
        if (!in[i]) continue;
        p.in_n[i] = static_cast<int>(strides[2 * i]);
        p.in_h[i] = static_cast<int>(strides[2 * i + 1]);
    }
    p.out[0] = q_out;
    p.out_n[0] = H_q * d;
    p.out_h[0] = d;
    p.heads[0] = H_q;
    p.heads[1] = p.heads[2] = H_kv;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.axes = axes;
    p.tokens = p.n = T;
    p.n_axes = n_axes;
    p.rot = rot_dim;
    p.interleaved = interleaved;
    p.slots = slots;
    p.cache = cache;
    p.page = page_size;
    p.log2_page = log2_of(page_size);
    p.num_slots = num_pages * page_size;
    return rope_launch<true>(dev, p, d, dtype == FA2_BF16, stream);
}

int64_t fa2_fwd_kv16_workspace(int T, int B, int H_q, int H_kv, int d, int max_pages, int page_size) {
    if (kv16_check_sizes(T, B, H_q, H_kv, d, max_pages, page_size) != FA2_OK) return -1;
    const int64_t ctas = kv16_ctas(T, B, H_q, H_kv, static_cast<long long>(max_pages) * page_size, fa2::kv16::kMaxCtas);
    // 16 more: the partial results begin at a multiple of 32 bytes
    return 16 + ctas * (2LL * kv16_part_rows(T, H_q / H_kv) * (d + 2) * static_cast<int64_t>(sizeof(float)) +
                        static_cast<int64_t>(sizeof(fa2::kv16::Begun)));
}

fa2_status fa2_fwd_kv16(const void* q, const void* cache, const int32_t* block_table, const int32_t* seq_lens,
                        const int32_t* q_starts, const int32_t* q_lens, void* o, float* lse, void* workspace,
                        int64_t workspace_bytes, int T, int B, int H_q, int H_kv, int d, int64_t q_stride_t, int64_t q_stride_h,
                        int max_pages, int page_size, int num_pages, float scale, int causal, fa2_dtype dtype,
                        cudaStream_t stream) {
    if (!q || !cache || !block_table || !seq_lens || !q_starts || !q_lens || !o || !lse || !workspace) return FA2_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(cache) || !aligned16(o) || !aligned16(lse) || !aligned16(workspace)) return FA2_ERR_INVALID_ARG;
    if (!aligned4(block_table) || !aligned4(seq_lens) || !aligned4(q_starts) || !aligned4(q_lens)) return FA2_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.0f)) return FA2_ERR_INVALID_ARG;
    if (dtype != FA2_BF16 && dtype != FA2_FP16) return FA2_ERR_INVALID_ARG;
    if (causal != 0 && causal != 1) return FA2_ERR_INVALID_ARG;
    if (T <= 0 || B <= 0 || H_q <= 0 || H_kv <= 0 || d <= 0 || H_q % H_kv != 0) return FA2_ERR_INVALID_ARG;
    if (q_stride_t <= 0 || q_stride_h <= 0 || q_stride_t % 8 != 0 || q_stride_h % 8 != 0) return FA2_ERR_INVALID_ARG;
    fa2_status st = kv4_check_pages(page_size, num_pages, max_pages);
    if (st != FA2_OK) return st;
    if ((st = kv16_check_sizes(T, B, H_q, H_kv, d, max_pages, page_size)) != FA2_OK) return st;
    if (q_stride_t > 0x7FFFFFFFLL || q_stride_h > 0x7FFFFFFFLL) return FA2_ERR_UNSUPPORTED;
    if (static_cast<long long>(num_pages) * H_kv > (0x7FFFFFFFLL - 2) / 2) return FA2_ERR_UNSUPPORTED;
    if (workspace_bytes < fa2_fwd_kv16_workspace(T, B, H_q, H_kv, d, max_pages, page_size)) return FA2_ERR_INVALID_ARG;
    int dev = 0;
    if ((st = check_device(&dev)) != FA2_OK) return st;
    if ((st = get_encoder()) != FA2_OK) return st;
    const int group = H_q / H_kv;
    CUtensorMap mq, mkv;
    if (kv16_encode_q(&mq, q, T, H_q, d, group, q_stride_t, q_stride_h) != FA2_OK ||
        kv16_encode_cache(&mkv, cache, static_cast<uint64_t>(num_pages) * H_kv * 2, page_size, d) != FA2_OK)
        return cuda_fail();
    fa2::kv16::Params p{};
    p.q_starts = q_starts;
    p.q_lens = q_lens;
    p.seq_lens = seq_lens;
    p.block_table = block_table;
    p.o = o;
    p.lse = lse;
    p.B = B;
    p.T = T;
    p.hq = H_q;
    p.hkv = H_kv;
    p.group = group;
    p.tok_tile = 128 / group;
    p.part_rows = kv16_part_rows(T, group);
    p.max_pages = max_pages;
    p.max_tokens = max_pages * page_size;
    p.page = page_size;
    p.log2_page = log2_of(page_size);
    p.num_pages = num_pages;
    p.causal = causal;
    p.ctas = kv16_ctas(T, B, H_q, H_kv, p.max_tokens, std::min(sm_count(dev), fa2::kv16::kMaxCtas));
    p.part_o = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(workspace) + 16) & ~static_cast<uintptr_t>(31));
    p.part_ml = p.part_o + 2LL * p.ctas * p.part_rows * d;
    p.begun = reinterpret_cast<fa2::kv16::Begun*>(p.part_ml + 4LL * p.ctas * p.part_rows);
    p.debug_flags = g_debug_flags.load();
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    p.wait_limit_ns = g_wait_limit_ns.load();
    const bool bf = dtype == FA2_BF16;
    if (d == 128) return bf ? kv16_launch<128, true>(dev, mq, mkv, p, stream) : kv16_launch<128, false>(dev, mq, mkv, p, stream);
    return bf ? kv16_launch<64, true>(dev, mq, mkv, p, stream) : kv16_launch<64, false>(dev, mq, mkv, p, stream);
}

fa2_status fa2_check_status(cudaStream_t stream) {
    // The status word read is that of the stream's device; the current
    // device is switched to it for the read and then restored.
    int sdev = 0, cur = 0;
    if (cudaStreamGetDevice(stream, &sdev) != cudaSuccess) return cuda_fail();
    if (cudaStreamSynchronize(stream) != cudaSuccess) return cuda_fail();
    if (cudaGetDevice(&cur) != cudaSuccess) return cuda_fail();
    if (sdev != cur && cudaSetDevice(sdev) != cudaSuccess) return cuda_fail();
    fa2_status result = FA2_OK;
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, fa2::g_fa2_status, sizeof(int)) != cudaSuccess) {
        result = cuda_fail();
    } else if (v != 0) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(fa2::g_fa2_status, &zero, sizeof(int)) != cudaSuccess)
            result = cuda_fail();
        else
            result = (v & 0xFF) == FA2_ERR_TIMEOUT || (v & 0xFF) == FA2_ERR_BOUNDS ? static_cast<fa2_status>(v & 0xFF)
                                                                                   : FA2_ERR_CUDA;
    }
    if (sdev != cur && cudaSetDevice(cur) != cudaSuccess) return cuda_fail();
    return result;
}

const char* fa2_status_string(fa2_status s) {
    switch (s) {
        case FA2_OK: return "FA2_OK";
        case FA2_ERR_INVALID_ARG: return "FA2_ERR_INVALID_ARG";
        case FA2_ERR_UNSUPPORTED: return "FA2_ERR_UNSUPPORTED";
        case FA2_ERR_CUDA: return "FA2_ERR_CUDA";
        case FA2_ERR_TIMEOUT: return "FA2_ERR_TIMEOUT";
        case FA2_ERR_BOUNDS: return "FA2_ERR_BOUNDS";
    }
    return "FA2_ERR_UNKNOWN";
}

int64_t fa2_set_wait_limit_ns(int64_t limit_ns) {
    if (limit_ns <= 0) limit_ns = 2000000000LL;
    return g_wait_limit_ns.exchange(limit_ns);
}

int fa2_set_debug_flags(int flags) { return g_debug_flags.exchange(flags); }

int fa2_set_tile_config(int config) {
    if (config < 0 || (config & ~kTileCfgMask) != 0) return -1;
    (void)tile_cfg();   // the environment's value first, so the previous value is the one in effect
    return g_tile_cfg.exchange(config, std::memory_order_acq_rel);
}

#ifdef FA2_DEBUG
const char* fa2_version(void) { return "fa2-sm103a 0.5.0 debug"; }
#else
const char* fa2_version(void) { return "fa2-sm103a 0.5.0"; }
#endif

}  // extern "C"
