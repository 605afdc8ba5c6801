// swa_api.cu -- host side of libswa: argument checks, TMA descriptors, launch
// configuration and the device status word.  All kernels are in the headers
// included below, compiled into this one translation unit.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/swa.h"
#include "decode_kernel.cuh"
#include "device_common.cuh"
#include "evict_kernel.cuh"
#include "prefill_kernel.cuh"
#include "q8_kernel.cuh"
#include "weights_kernel.cuh"

namespace {

thread_local int t_last_cuda_error = 0;

swa_status_t cuda_fail(cudaError_t e) {
    t_last_cuda_error = static_cast<int>(e);
    return SWA_ERR_CUDA;
}

#define SWA_CUDA_TRY(expr)                       \
    do {                                         \
        cudaError_t e_ = (expr);                 \
        if (e_ != cudaSuccess) return cuda_fail(e_); \
    } while (0)

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// ----------------------------------------------------------------- TMA descriptors
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// bf16 tensor [d3, d2, d1, d0] (d0 innermost, contiguous) as a 4-D TMA map
// with a (64, 1, 128, 1) box and 128-byte swizzle: one 128-row x 128-byte
// region of a K-major UMMA operand per load.  Out-of-range rows read as zero.
// box1 x box2 rows: of box1 heads and box2 positions, position-major.
swa_status_t make_operand_map(CUtensorMap *map, const void *base, uint64_t d0, uint64_t d1,
                              uint64_t d2, uint64_t d3, uint32_t box1 = 1, uint32_t box2 = 128) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return cuda_fail(cudaErrorNotSupported);
    const cuuint64_t dims[4] = {d0, d1, d2, d3};
    const cuuint64_t strides[3] = {d0 * 2, d0 * d1 * 2, d0 * d1 * d2 * 2};   // bytes, dims 1..3
    const cuuint32_t box[4] = {64, box1, box2, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims,
                    strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        t_last_cuda_error = static_cast<int>(r);
        return SWA_ERR_CUDA;
    }
    return SWA_OK;
}

// 8-bit tensor [d3, d2, d1, d0] (d0 = 64 or 128, innermost, contiguous) as a 4-D
// TMA map with a (d0, 1, rows, 1) box: `rows` consecutive rows of one head, in
// the swizzle of their width.  Out-of-range rows read as zero.
swa_status_t make_codes_map(CUtensorMap *map, const void *base, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t d3,
                            uint32_t rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return cuda_fail(cudaErrorNotSupported);
    const cuuint64_t dims[4] = {d0, d1, d2, d3};
    const cuuint64_t strides[3] = {d0, d0 * d1, d0 * d1 * d2};               // bytes, dims 1..3
    const cuuint32_t box[4] = {(cuuint32_t)d0, 1, rows, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE,
                    d0 == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        t_last_cuda_error = static_cast<int>(r);
        return SWA_ERR_CUDA;
    }
    return SWA_OK;
}

// ----------------------------------------------------------------- device info
constexpr int kMaxDevices = 64;

struct DeviceInfo {
    int sms = 0;
};
DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;
thread_local int t_device = 0;                      // the current device, as device_info found it in this call

swa_status_t device_info(DeviceInfo **out) {
    int dev = 0;
    SWA_CUDA_TRY(cudaGetDevice(&dev));
    if (dev < 0 || dev >= kMaxDevices) return SWA_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lk(g_dev_mu);
    DeviceInfo &d = g_dev[dev];
    if (d.sms == 0) SWA_CUDA_TRY(cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev));
    t_device = dev;
    *out = &d;
    return SWA_OK;
}

// Lets a kernel have `bytes` of dynamic shared memory (always the same for a
// kernel; after device_info): before its first launch on each device, because setting the attribute
// loads the kernel's code (of all kernels at the first call of the library: 3 ms).
template <auto KERNEL>
swa_status_t allow_smem(int bytes) {
    static std::atomic<uint64_t> done{0};
    static_assert(kMaxDevices <= 64, "a bit per device");
    const uint64_t bit = uint64_t(1) << t_device;
    if (done.load(std::memory_order_acquire) & bit) return SWA_OK;
    SWA_CUDA_TRY(cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    done.fetch_or(bit, std::memory_order_release);
    return SWA_OK;
}

// ----------------------------------------------------------------- common checks
swa_status_t check_heads(int Hq, int Hkv, int D) {
    if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return SWA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return SWA_ERR_UNSUPPORTED;
    return SWA_OK;
}

bool bad_scale(float s) { return !(std::isfinite(s) && s > 0.f); }

constexpr float kLog2e = 1.4426950408889634f;

template <int D>
// mks / mvs: sink-buffer maps (chunk mode with sinks), else any valid map.
swa_status_t launch_prefill(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                            const CUtensorMap &mkc, const CUtensorMap &mvc, const CUtensorMap &mks,
                            const CUtensorMap &mvs, const swa::PrefillParams &p, int sms, cudaStream_t s) {
    const int grid = p.num_units < sms ? p.num_units : sms;
    if (swa_status_t e = allow_smem<swa::swa_prefill_kernel<D>>(swa::PrefillCfg<D>::SMEM_ALLOC)) return e;
    swa::swa_prefill_kernel<D><<<grid, swa::PrefillCfg<D>::THREADS, swa::PrefillCfg<D>::SMEM_ALLOC, s>>>(
        mq, mk, mv, mkc, mvc, mks, mvs, p);
    SWA_CUDA_TRY(cudaGetLastError());
    return SWA_OK;
}

swa_status_t launch_append(const void *k_new, const void *v_new, void *k_cache, void *v_cache,
                           const int32_t *pos, int B, int T, int Hkv, int D, int W, int sms,
                           const swa::RopeTable *rope, cudaStream_t s, void *k_sink = nullptr,
                           void *v_sink = nullptr, int S = 0) {
    const int row_vec = Hkv * D * 2 / 16;
    const long long total = (long long)B * T * row_vec;
    long long blocks = (total + 255) / 256;
    const long long cap = (long long)sms * 8;
    if (blocks > cap) blocks = cap;
    if (blocks < 1) blocks = 1;
    swa::swa_append_kernel<<<(int)blocks, 256, 0, s>>>(
        static_cast<const uint4 *>(k_new), static_cast<const uint4 *>(v_new),
        static_cast<uint4 *>(k_cache), static_cast<uint4 *>(v_cache), pos, B, T, W, row_vec, D / 8,
        rope ? 1 : 0, rope ? *rope : swa::RopeTable{}, static_cast<uint4 *>(k_sink),
        static_cast<uint4 *>(v_sink), S);
    SWA_CUDA_TRY(cudaGetLastError());
    return SWA_OK;
}

// Keys per decode split for a launch over L = W (+ S) keys: kDecodeSplit, or
// fewer (multiples of 64, at least kDecodeMinSplit) when B * Hkv windows of
// kDecodeSplit keys would give fewer than ~256 blocks, so that a small batch
// still spreads over the GPU.  A function of the sizes only: the workspace
// size follows from it.
int decode_split_keys(int B, int Hkv, int L) {
    const long long pairs = (long long)B * Hkv;
    const long long want = (256 + pairs - 1) / pairs;       // splits per (sequence, kv head)
    long long split = ((L + want - 1) / want + 63) / 64 * 64;
    if (split < swa::kDecodeMinSplit) split = swa::kDecodeMinSplit;
    if (split > swa::kDecodeSplit) split = swa::kDecodeSplit;
    return (int)split;
}

// The decode kernel takes the Hq/Hkv query heads that share a K/V head as
// the rows of its MMA tile, at most 8 at a time: a group of G heads runs as
// rep = G / Gt groups of Gt heads, Gt the largest divisor of G up to 8 (each
// K/V head then read rep times).  Returns Gt.
int decode_group(int Hq, int Hkv, int *rep) {
    const int G = Hq / Hkv;
    int gt = G < 8 ? G : 8;
    while (G % gt != 0) --gt;
    *rep = G / gt;
    return gt;
}

int decode_nsplit_max(int B, int Hkv, int L) {
    const int split = decode_split_keys(B, Hkv, L);
    return (int)(((long long)L + split - 1) / split);
}

// Grid (kDecodeClusterSplits, Hkv, B) in clusters of kDecodeClusterSplits
// along x: the splits of each window are merged through distributed shared
// memory, with no workspace.  MODE kDecodeWindowCluster: the window of the
// cache (knew / vnew / cu unused, total = B); kDecodePackedRows: the
// one-row sequences of a packed batch.
template <int D, int G, int MODE>
swa_status_t launch_decode_cluster(const void *q, const void *kc, const void *vc, const int32_t *pos,
                                   void *out, int B, int Hkv, int W, float scale,
                                   const swa::RopeTable *rope, const void *knew, const void *vnew,
                                   const int32_t *cu, int total, int kv_rep, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(swa::kDecodeClusterSplits, Hkv, B);
    cfg.blockDim = dim3(swa::kDecodeWarps * 32);
    cfg.dynamicSmemBytes = swa::DecodeCfg<D, G>::SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = swa::kDecodeClusterSplits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (swa_status_t e = allow_smem<swa::swa_decode_kernel<D, G, MODE>>(swa::DecodeCfg<D, G>::SMEM_BYTES)) return e;
    float2 *no_ml = nullptr;
    float *no_o = nullptr;
    SWA_CUDA_TRY(cudaLaunchKernelEx(&cfg, swa::swa_decode_kernel<D, G, MODE>,
                                    static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(kc),
                                    static_cast<const __nv_bfloat16 *>(vc), pos, static_cast<__nv_bfloat16 *>(out),
                                    no_ml, no_o, Hkv, W, 1, scale * kLog2e, rope ? 1 : 0,
                                    rope ? *rope : swa::RopeTable{}, static_cast<const __nv_bfloat16 *>(knew),
                                    static_cast<const __nv_bfloat16 *>(vnew), 0, cu, total, 0, kv_rep));
    return SWA_OK;
}

// Hkv: groups of G query heads (kv_rep groups per K/V head in memory).
template <int D, int G>
swa_status_t launch_decode_dg(const void *q, const void *kc, const void *vc, const int32_t *pos,
                              void *out, int B, int Hkv, int W, float scale, void *ws,
                              const swa::RopeTable *rope, cudaStream_t s, const void *ksink,
                              const void *vsink, int S, int kv_rep) {
    const int nsm = decode_nsplit_max(B, Hkv, W + S);
    const int split = decode_split_keys(B, Hkv, W + S);
    const size_t o_elems = (size_t)B * Hkv * nsm * G * D;
    float *ws_o = static_cast<float *>(ws);
    float2 *ws_ml = ws ? reinterpret_cast<float2 *>(static_cast<char *>(ws) + ((o_elems * 4 + 255) & ~size_t(255)))
                       : nullptr;
    // a window of exactly kDecodeClusterSplits splits: merged in its cluster
    if (S == 0 && nsm == swa::kDecodeClusterSplits)
        return launch_decode_cluster<D, G, swa::kDecodeWindowCluster>(q, kc, vc, pos, out, B, Hkv, W, scale, rope,
                                                                      nullptr, nullptr, nullptr, B, kv_rep, s);
    dim3 grid(nsm, Hkv, B);
    constexpr int smem = swa::DecodeCfg<D, G>::SMEM_BYTES;
    auto kernel = S > 0 ? swa::swa_decode_kernel<D, G, swa::kDecodeSinks>
                        : swa::swa_decode_kernel<D, G, swa::kDecodeWindow>;
    if (swa_status_t e = S > 0 ? allow_smem<swa::swa_decode_kernel<D, G, swa::kDecodeSinks>>(smem)
                               : allow_smem<swa::swa_decode_kernel<D, G, swa::kDecodeWindow>>(smem))
        return e;
    kernel<<<grid, swa::kDecodeWarps * 32, smem, s>>>(
        static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(kc),
        static_cast<const __nv_bfloat16 *>(vc), pos, static_cast<__nv_bfloat16 *>(out), ws_ml, ws_o,
        Hkv, W, nsm, scale * kLog2e, rope ? 1 : 0, rope ? *rope : swa::RopeTable{},
        static_cast<const __nv_bfloat16 *>(ksink), static_cast<const __nv_bfloat16 *>(vsink), S,
        nullptr, 0, split, kv_rep);
    SWA_CUDA_TRY(cudaGetLastError());
    if (nsm > 1) {
        swa::swa_decode_combine_kernel<D, G><<<dim3(Hkv, B), G * D, 0, s>>>(
            pos, ws_ml, ws_o, static_cast<__nv_bfloat16 *>(out), Hkv, W, nsm, S, split);
        SWA_CUDA_TRY(cudaGetLastError());
    }
    return SWA_OK;
}

template <int D>
swa_status_t launch_decode_d(int G, int kv_rep, const void *q, const void *kc, const void *vc,
                             const int32_t *pos, void *out, int B, int Hkv, int W, float scale,
                             void *ws, const swa::RopeTable *rope, cudaStream_t s,
                             const void *ksink = nullptr, const void *vsink = nullptr, int S = 0) {
    switch (G) {
        case 1: return launch_decode_dg<D, 1>(q, kc, vc, pos, out, B, Hkv, W, scale, ws, rope, s, ksink, vsink, S, kv_rep);
        case 2: return launch_decode_dg<D, 2>(q, kc, vc, pos, out, B, Hkv, W, scale, ws, rope, s, ksink, vsink, S, kv_rep);
        case 3: return launch_decode_dg<D, 3>(q, kc, vc, pos, out, B, Hkv, W, scale, ws, rope, s, ksink, vsink, S, kv_rep);
        case 4: return launch_decode_dg<D, 4>(q, kc, vc, pos, out, B, Hkv, W, scale, ws, rope, s, ksink, vsink, S, kv_rep);
        case 5: return launch_decode_dg<D, 5>(q, kc, vc, pos, out, B, Hkv, W, scale, ws, rope, s, ksink, vsink, S, kv_rep);
        case 6: return launch_decode_dg<D, 6>(q, kc, vc, pos, out, B, Hkv, W, scale, ws, rope, s, ksink, vsink, S, kv_rep);
        case 7: return launch_decode_dg<D, 7>(q, kc, vc, pos, out, B, Hkv, W, scale, ws, rope, s, ksink, vsink, S, kv_rep);
        case 8: return launch_decode_dg<D, 8>(q, kc, vc, pos, out, B, Hkv, W, scale, ws, rope, s, ksink, vsink, S, kv_rep);
        default: return SWA_ERR_UNSUPPORTED;
    }
}

// The length-1 sequences of a packed chunk batch (q/k/v/out [total, H, D]):
// a cluster of kDecodeClusterSplits blocks per (sequence, kv head), merged in
// distributed shared memory; the other sequences' blocks return at once.
template <int D, int G>
swa_status_t launch_decode_packed_dg(const void *q, const void *k, const void *v, const void *kc,
                                     const void *vc, const int32_t *start_pos, const int32_t *cu,
                                     void *out, int B, int total, int Hkv, int W, float scale,
                                     cudaStream_t s, int kv_rep) {
    return launch_decode_cluster<D, G, swa::kDecodePackedRows>(q, kc, vc, start_pos, out, B, Hkv, W, scale, nullptr,
                                                               k, v, cu, total, kv_rep, s);
}

// false when the decode kernel has no instance for this head group
template <int D>
bool launch_decode_packed_d(int G, int kv_rep, swa_status_t *e, const void *q, const void *k, const void *v,
                            const void *kc, const void *vc, const int32_t *start_pos, const int32_t *cu,
                            void *out, int B, int total, int Hkv, int W, float scale, cudaStream_t s) {
    switch (G) {
        case 1: *e = launch_decode_packed_dg<D, 1>(q, k, v, kc, vc, start_pos, cu, out, B, total, Hkv, W, scale, s, kv_rep); return true;
        case 2: *e = launch_decode_packed_dg<D, 2>(q, k, v, kc, vc, start_pos, cu, out, B, total, Hkv, W, scale, s, kv_rep); return true;
        case 3: *e = launch_decode_packed_dg<D, 3>(q, k, v, kc, vc, start_pos, cu, out, B, total, Hkv, W, scale, s, kv_rep); return true;
        case 4: *e = launch_decode_packed_dg<D, 4>(q, k, v, kc, vc, start_pos, cu, out, B, total, Hkv, W, scale, s, kv_rep); return true;
        case 5: *e = launch_decode_packed_dg<D, 5>(q, k, v, kc, vc, start_pos, cu, out, B, total, Hkv, W, scale, s, kv_rep); return true;
        case 6: *e = launch_decode_packed_dg<D, 6>(q, k, v, kc, vc, start_pos, cu, out, B, total, Hkv, W, scale, s, kv_rep); return true;
        case 7: *e = launch_decode_packed_dg<D, 7>(q, k, v, kc, vc, start_pos, cu, out, B, total, Hkv, W, scale, s, kv_rep); return true;
        case 8: *e = launch_decode_packed_dg<D, 8>(q, k, v, kc, vc, start_pos, cu, out, B, total, Hkv, W, scale, s, kv_rep); return true;
        default: return false;
    }
}

__global__ void swa_selftest_wait_kernel() {
    __shared__ alignas(8) uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        swa::mbar_init(swa::smem_addr(&bar), 1);
        abort_flag = 0;
        swa::mbar_init_fence();
    }
    __syncthreads();
    // nothing ever arrives on `bar`: the wait must run out and record the status
    swa::mbar_wait_bounded(swa::smem_addr(&bar), 0, &abort_flag, swa::g_wait_limit_ns);
}

// Scratch of swa_decode_noalloc: reserved statically on every device that
// loads this library, shared by all its calls.  Host code must not pass the
// symbol itself to a kernel (on the host it names a host-side shadow); the
// device address is looked up once per device with cudaGetSymbolAddress.
constexpr size_t kNoallocScratchBytes = SWA_DECODE_NOALLOC_SCRATCH_BYTES;
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoallocScratchBytes];

void *g_noalloc_ptr[kMaxDevices] = {};
std::mutex g_noalloc_mu;

swa_status_t noalloc_scratch(void **out) {
    int dev = 0;
    SWA_CUDA_TRY(cudaGetDevice(&dev));
    if (dev < 0 || dev >= kMaxDevices) return SWA_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lk(g_noalloc_mu);
    if (!g_noalloc_ptr[dev]) {
        void *p = nullptr;
        SWA_CUDA_TRY(cudaGetSymbolAddress(&p, g_noalloc_scratch));   // device `dev` is current
        g_noalloc_ptr[dev] = p;
    }
    *out = g_noalloc_ptr[dev];
    return SWA_OK;
}

// FINE: the prompt weights' exponential, else the prefill's.
template <bool FINE>
__global__ void swa_selftest_exp2_kernel(const float *x, float *y, int n) {
    const int i = 2 * (blockIdx.x * blockDim.x + threadIdx.x);
    if (i >= n) return;
    const float2 v = make_float2(x[i], i + 1 < n ? x[i + 1] : 0.f);
    const float2 r = FINE ? swa::exp2_poly2_fine(v) : swa::exp2_poly2(v);
    y[i] = r.x;
    if (i + 1 < n) y[i + 1] = r.y;
}

// ----------------------------------------------------------------- implementations
// `rope` null: no rotary embedding; otherwise the frequency table.

bool bad_theta(float theta) { return !(std::isfinite(theta) && theta > 1.f); }

swa::RopeTable make_rope_table(float theta, int D) {
    swa::RopeTable t{};
    for (int i = 0; i < D / 2 && i < 64; ++i) t.f[i] = std::pow((double)theta, -2.0 * i / D);
    return t;
}

// cu_seqlens non-null: variable-length batch, tensors packed [N = total rows, H, D].
swa_status_t prefill_impl(const void *q, const void *k, const void *v, void *out, int B, int N,
                          int Hq, int Hkv, int D, int W, int window_mode, float scale,
                          const swa::RopeTable *rope, const int32_t *cu_seqlens, cudaStream_t s,
                          int sinks = 0) {
    if (!q || !k || !v || !out) return SWA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return SWA_ERR_INVALID_ARG;
    if (B < 1 || N < 1 || W < 1 || bad_scale(scale)) return SWA_ERR_INVALID_ARG;
    if (window_mode != SWA_WINDOW_EXCL_LEFT && window_mode != SWA_WINDOW_INCL_LEFT)
        return SWA_ERR_INVALID_ARG;
    if (swa_status_t e = check_heads(Hq, Hkv, D)) return e;
    long long Weff = (long long)W + (window_mode == SWA_WINDOW_INCL_LEFT ? 1 : 0);
    if (Weff > N) Weff = N;                       // the window never reaches before position 0
    const int G = Hq / Hkv;
    if (cu_seqlens && (B > swa::kMaxVarlenSeqs || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u)))
        return B > swa::kMaxVarlenSeqs ? SWA_ERR_UNSUPPORTED : SWA_ERR_INVALID_ARG;
    const long long nqb = (N + 127) / 128;
    // varlen: an upper bound (the kernel counts the real units from cu_seqlens)
    const long long units = cu_seqlens ? (long long)Hkv * ((G + 1) / 2) * (nqb + B)
                                       : (long long)B * Hkv * ((G + 1) / 2) * nqb;
    if (units > 0x7fffffffll) return SWA_ERR_UNSUPPORTED;
    DeviceInfo *dev = nullptr;
    if (swa_status_t e = device_info(&dev)) return e;

    const int mb = cu_seqlens ? 1 : B;              // packed tensors have one batch row
    CUtensorMap mq, mk, mv;
    if (swa_status_t e = make_operand_map(&mq, q, D, Hq, N, mb)) return e;
    if (swa_status_t e = make_operand_map(&mk, k, D, Hkv, N, mb)) return e;
    if (swa_status_t e = make_operand_map(&mv, v, D, Hkv, N, mb)) return e;

    swa::PrefillParams p{};
    swa::prefill_units(p, B, N, Hq, Hkv, (int)Weff, cu_seqlens != nullptr, false, dev->sms);
    p.scale_log2 = scale * kLog2e;
    p.start_pos = nullptr;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.out_v8 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
    p.rope = rope ? 1 : 0;
    if (rope) p.rope_freq = *rope;
    p.cu_seqlens = cu_seqlens;
    p.sinks = sinks;
    return D == 128 ? launch_prefill<128>(mq, mk, mv, mk, mv, mk, mv, p, dev->sms, s)
                    : launch_prefill<64>(mq, mk, mv, mk, mv, mk, mv, p, dev->sms, s);
}

// cu_seqlens non-null: variable-length batch; q/k/v/out packed [C = total rows,
// H, D], sequence b is rows cu[b]..cu[b+1]-1 (any length; one longer than W
// leaves its last W positions in the buffer).
// k_sink / v_sink, S > 0: S-slot sink buffers [B, S, Hkv, D] (fixed-length only).
// append false: the attention alone (fixed-length only).
swa_status_t prefill_chunk_impl(const void *q, const void *k, const void *v, void *k_cache,
                                void *v_cache, const int32_t *start_pos, void *out, int B, int C,
                                int Hq, int Hkv, int D, int W, float scale,
                                const swa::RopeTable *rope, const int32_t *cu_seqlens,
                                cudaStream_t s, void *k_sink = nullptr, void *v_sink = nullptr,
                                int S = 0, bool append = true) {
    if (!q || !k || !v || !k_cache || !v_cache || !start_pos || !out) return SWA_ERR_INVALID_ARG;
    if (S < 0 || (S > 0 && (!k_sink || !v_sink || !aligned16(k_sink) || !aligned16(v_sink) || cu_seqlens)))
        return SWA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(k_cache) ||
        !aligned16(v_cache) || !aligned16(out) || (reinterpret_cast<uintptr_t>(start_pos) & 3u))
        return SWA_ERR_INVALID_ARG;
    if (B < 1 || C < 1 || W < 1 || bad_scale(scale)) return SWA_ERR_INVALID_ARG;
    if (!cu_seqlens && C > W) return SWA_ERR_INVALID_ARG;
    if (cu_seqlens && (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u)) return SWA_ERR_INVALID_ARG;
    if (cu_seqlens && B > swa::kMaxVarlenSeqs) return SWA_ERR_UNSUPPORTED;
    if (swa_status_t e = check_heads(Hq, Hkv, D)) return e;
    const int G = Hq / Hkv;
    const long long nqb = (C + 127) / 128;
    const long long units = cu_seqlens ? (long long)Hkv * ((G + 1) / 2) * (nqb + B)
                                       : (long long)B * Hkv * ((G + 1) / 2) * nqb;
    if (units > 0x7fffffffll) return SWA_ERR_UNSUPPORTED;
    DeviceInfo *dev = nullptr;
    if (swa_status_t e = device_info(&dev)) return e;

    const int mb = cu_seqlens ? 1 : B;
    CUtensorMap mq, mk, mv, mkc, mvc;
    if (swa_status_t e = make_operand_map(&mq, q, D, Hq, C, mb)) return e;
    if (swa_status_t e = make_operand_map(&mk, k, D, Hkv, C, mb)) return e;
    if (swa_status_t e = make_operand_map(&mv, v, D, Hkv, C, mb)) return e;
    if (swa_status_t e = make_operand_map(&mkc, k_cache, D, Hkv, W, B)) return e;
    if (swa_status_t e = make_operand_map(&mvc, v_cache, D, Hkv, W, B)) return e;

    swa::PrefillParams p{};
    swa::prefill_units(p, B, C, Hq, Hkv, W, cu_seqlens != nullptr, true, dev->sms);
    p.scale_log2 = scale * kLog2e;
    p.start_pos = start_pos;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.out_v8 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
    p.rope = rope ? 1 : 0;
    if (rope) p.rope_freq = *rope;
    p.cu_seqlens = cu_seqlens;
    CUtensorMap mks = mkc, mvs = mvc;
    if (S > 0) {
        if (swa_status_t e = make_operand_map(&mks, k_sink, D, Hkv, S, B)) return e;
        if (swa_status_t e = make_operand_map(&mvs, v_sink, D, Hkv, S, B)) return e;
    }
    p.sink_buf = S;
    if (cu_seqlens) {
        // length-1 sequences (decode tokens) go to the decode kernel, which
        // reads their windows at memory speed instead of as 128-row tiles
        swa_status_t ed = SWA_OK;
        int rep = 1;
        const int gt = decode_group(Hq, Hkv, &rep);
        const bool fits = (long long)Hkv * rep <= 65535;
        const bool dec = fits && (D == 128 ? launch_decode_packed_d<128>(gt, rep, &ed, q, k, v, k_cache, v_cache,
                                                                         start_pos, cu_seqlens, out, B, C, Hkv * rep,
                                                                         W, scale, s)
                                           : launch_decode_packed_d<64>(gt, rep, &ed, q, k, v, k_cache, v_cache,
                                                                        start_pos, cu_seqlens, out, B, C, Hkv * rep,
                                                                        W, scale, s));
        if (ed) return ed;
        p.skip_len1 = dec ? 1 : 0;
    }
    swa_status_t e = D == 128 ? launch_prefill<128>(mq, mk, mv, mkc, mvc, mks, mvs, p, dev->sms, s)
                              : launch_prefill<64>(mq, mk, mv, mkc, mvc, mks, mvs, p, dev->sms, s);
    if (e || !append) return e;
    // attend first, then write the chunk (its keys already rotated) into the buffer
    if (!cu_seqlens)     // positions below S also go to the sink buffer
        return launch_append(k, v, k_cache, v_cache, start_pos, B, C, Hkv, D, W, dev->sms, nullptr, s,
                             k_sink, v_sink, S);
    const int row_vec = Hkv * D * 2 / 16;
    long long blocks = ((long long)C * row_vec + 255) / 256;
    if (blocks > (long long)dev->sms * 8) blocks = (long long)dev->sms * 8;
    swa::swa_append_varlen_kernel<<<(int)blocks, 256, 0, s>>>(
        static_cast<const uint4 *>(k), static_cast<const uint4 *>(v), static_cast<uint4 *>(k_cache),
        static_cast<uint4 *>(v_cache), start_pos, cu_seqlens, B, C, W, row_vec);
    SWA_CUDA_TRY(cudaGetLastError());
    return SWA_OK;
}

swa_status_t append_impl(const void *k_new, const void *v_new, void *k_cache, void *v_cache,
                         const int32_t *pos, int B, int T, int Hkv, int D, int W,
                         const swa::RopeTable *rope, cudaStream_t s) {
    if (!k_new || !v_new || !k_cache || !v_cache || !pos) return SWA_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
        (reinterpret_cast<uintptr_t>(pos) & 3u))
        return SWA_ERR_INVALID_ARG;
    if (B < 1 || T < 1 || W < 1 || T > W || Hkv < 1) return SWA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return SWA_ERR_UNSUPPORTED;
    DeviceInfo *dev = nullptr;
    if (swa_status_t e = device_info(&dev)) return e;
    return launch_append(k_new, v_new, k_cache, v_cache, pos, B, T, Hkv, D, W, dev->sms, rope, s);
}

size_t decode_workspace_bytes(int B, int Hq, int Hkv, int D, int W) {
    if (B < 1 || W < 1 || check_heads(Hq, Hkv, D) != SWA_OK) return 0;
    int rep = 1;
    decode_group(Hq, Hkv, &rep);
    if ((long long)Hkv * rep > 65535) return 0;
    const size_t nsm = (size_t)decode_nsplit_max(B, Hkv * rep, W);
    const size_t rows = (size_t)B * Hq * nsm;        // (b, kv head, split, head in group)
    const size_t o_bytes = (rows * D * 4 + 255) & ~size_t(255);
    return o_bytes + rows * 8;
}

swa_status_t decode_checks(const void *q, const void *k_cache, const void *v_cache,
                           const int32_t *pos, const void *out, int B, int Hq, int Hkv, int D,
                           int W, float scale) {
    if (!q || !k_cache || !v_cache || !pos || !out) return SWA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
        (reinterpret_cast<uintptr_t>(pos) & 3u))
        return SWA_ERR_INVALID_ARG;
    if (B < 1 || W < 1 || bad_scale(scale)) return SWA_ERR_INVALID_ARG;
    if (swa_status_t e = check_heads(Hq, Hkv, D)) return e;
    int rep = 1;
    decode_group(Hq, Hkv, &rep);
    if (B > 65535 || (long long)Hkv * rep > 65535) return SWA_ERR_UNSUPPORTED;
    return SWA_OK;
}

swa_status_t decode_launch(const void *q, const void *k_cache, const void *v_cache,
                           const int32_t *pos, void *out, int B, int Hq, int Hkv, int D, int W,
                           float scale, void *workspace, const swa::RopeTable *rope, cudaStream_t s) {
    int rep = 1;
    const int G = decode_group(Hq, Hkv, &rep);
    DeviceInfo *dev = nullptr;
    if (swa_status_t e = device_info(&dev)) return e;
    return D == 128 ? launch_decode_d<128>(G, rep, q, k_cache, v_cache, pos, out, B, Hkv * rep, W, scale, workspace,
                                           rope, s)
                    : launch_decode_d<64>(G, rep, q, k_cache, v_cache, pos, out, B, Hkv * rep, W, scale, workspace,
                                          rope, s);
}

swa_status_t decode_impl(const void *q, const void *k_cache, const void *v_cache,
                         const int32_t *pos, void *out, int B, int Hq, int Hkv, int D, int W,
                         float scale, void *workspace, size_t workspace_bytes,
                         const swa::RopeTable *rope, cudaStream_t s) {
    if (swa_status_t e = decode_checks(q, k_cache, v_cache, pos, out, B, Hq, Hkv, D, W, scale)) return e;
    const size_t need = decode_workspace_bytes(B, Hq, Hkv, D, W);
    int rep = 1;
    decode_group(Hq, Hkv, &rep);
    if (decode_nsplit_max(B, Hkv * rep, W) > 1) {
        if (!workspace || workspace_bytes < need) return SWA_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(workspace) & 255u) return SWA_ERR_INVALID_ARG;
    }
    return decode_launch(q, k_cache, v_cache, pos, out, B, Hq, Hkv, D, W, scale, workspace, rope, s);
}

// ----------------------------------------------------------------- 8-bit rolling cache
bool misaligned(const void *p, uintptr_t by) { return (reinterpret_cast<uintptr_t>(p) & (by - 1)) != 0; }

// Grid of a copy kernel of 256 threads over `vectors` per sequence: about 16
// blocks to an SM in all.
dim3 copy_grid(long long vectors, int B, int sms) {
    long long x = (vectors + 255) / 256;
    const long long most = ((long long)sms * 16 + B - 1) / B;
    if (x > most) x = most;
    return dim3((unsigned)(x < 1 ? 1 : x), B);
}

// Slots per scale: a power of two that the decode kernel's 16-key blocks divide.
bool bad_q8_block(int block) { return block != 16 && block != 32 && block != 64 && block != 128; }

swa_status_t q8_cache_checks(const void *k_cache, const void *v_cache, const float *k_scale, const float *v_scale,
                             const int32_t *pos, int B, int Hkv, int D, int W, int block) {
    if (!k_cache || !v_cache || !k_scale || !v_scale || !pos) return SWA_ERR_INVALID_ARG;
    if (!aligned16(k_cache) || !aligned16(v_cache) || misaligned(k_scale, 4) || misaligned(v_scale, 4) ||
        misaligned(pos, 4))
        return SWA_ERR_INVALID_ARG;
    if (B < 1 || W < 1 || Hkv < 1 || bad_q8_block(block)) return SWA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return SWA_ERR_UNSUPPORTED;
    if (B > 65535) return SWA_ERR_UNSUPPORTED;
    return SWA_OK;
}

template <int BLOCK, int D>
swa_status_t launch_append_q8(const void *k_new, const void *v_new, void *k_cache, void *v_cache, float *k_scale,
                              float *v_scale, const int32_t *pos, int B, int T, int Hkv, int W, cudaStream_t s) {
    const int nblk = (int)(((long long)W + BLOCK - 1) / BLOCK);
    const int ntouch = swa::q8_blocks_touched(T, BLOCK, nblk);
    const long long gx = (long long)ntouch * 2 * Hkv;
    if (gx > 0x7fffffffll) return SWA_ERR_UNSUPPORTED;
    swa::swa_append_q8_kernel<BLOCK, D><<<dim3((unsigned)gx, B), BLOCK * D / 32, 0, s>>>(
        static_cast<const uint4 *>(k_new), static_cast<const uint4 *>(v_new), static_cast<uint2 *>(k_cache),
        static_cast<uint2 *>(v_cache), k_scale, v_scale, pos, T, W, Hkv, nblk, ntouch);
    SWA_CUDA_TRY(cudaGetLastError());
    return SWA_OK;
}

swa_status_t append_q8_impl(const void *k_new, const void *v_new, void *k_cache, void *v_cache, float *k_scale,
                            float *v_scale, const int32_t *pos, int B, int T, int Hkv, int D, int W, int block,
                            cudaStream_t s) {
    if (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new)) return SWA_ERR_INVALID_ARG;
    if (swa_status_t e = q8_cache_checks(k_cache, v_cache, k_scale, v_scale, pos, B, Hkv, D, W, block)) return e;
    if (T < 1 || T > W) return SWA_ERR_INVALID_ARG;
#define SWA_APPEND_Q8(BL)                                                                                          \
    case BL:                                                                                                      \
        return D == 128 ? launch_append_q8<BL, 128>(k_new, v_new, k_cache, v_cache, k_scale, v_scale, pos, B, T,   \
                                                    Hkv, W, s)                                                     \
                        : launch_append_q8<BL, 64>(k_new, v_new, k_cache, v_cache, k_scale, v_scale, pos, B, T,    \
                                                   Hkv, W, s);
    switch (block) {
        SWA_APPEND_Q8(16)
        SWA_APPEND_Q8(32)
        SWA_APPEND_Q8(64)
        SWA_APPEND_Q8(128)
        default: return SWA_ERR_INVALID_ARG;
    }
#undef SWA_APPEND_Q8
}

// Keys per split of an 8-bit decode over L keys by `pairs` (sequence, group of
// heads) pairs: the number of splits with the least estimated time, in the time
// a block takes per key: the rounds of blocks (592 run at once, 4 to an SM) times
// the keys of one and kQ8BlockCost for its start and its merge, and, unless
// there is one split or four (which merge in their cluster), kQ8MergeCost and
// kQ8MergePart per split for the merge kernel.  Splits are multiples of 64 keys,
// at least kDecodeMinSplit.  Against the 16-bit decode's rule (up to 1024 keys):
// B=64, W=4096, 8 KV heads, one split instead of four 88 against 101 us, W=2000
// one instead of two 49 against 58; small batches are cut alike.  With 32 / 8
// heads of 128 and full windows, in us: the rule's number of splits, the best of
// 1 to 18, and one split:
//   W=4096  B=1 10.2 (11 splits), 9.8 (18), 46    B=4 15.8 (11), 14.9 (8), 47
//           B=8 21.1 (8), 20.0 (4), 48            B=16 30.7 (4), the best, 49
//           B=24 41.8 (3), the best, 56           B=32 52.8 (2), the best, 57
//           B=48 75.4 (3), 71.8 (1), 72           B=64 89 (1), the best
//   W=1000  B=1 to 16 7.1 to 13.9 (4), the best, 14 to 16
//           B=24 19.9 (3), 19.0 (1)               B=32 22.6 (2), 19.3 (1)
//           B=48 24.1 (1), the best               B=64 29.5 (1), the best
// A function of the sizes only: the workspace size follows from it, and is asked
// for without a device, so the SM count of the B200 (148, four blocks to each) is
// written into it; on another the results are the same.  The longest split keeps
// the kernels' 32-bit sums of a window and a split in range.
constexpr long long kQ8MaxSplit = 1 << 24;
constexpr int kQ8BlocksAtOnce = 592, kQ8BlockCost = 200, kQ8MergeCost = 60, kQ8MergePart = 37;

int q8_split_keys(int B, int Hkv, int L) {
    const long long pairs = (long long)B * Hkv;
    long long best = 0;
    int split = (int)kQ8MaxSplit;
    for (int n = 1; n <= 128; ++n) {
        const long long s = (((long long)L + n - 1) / n + 63) / 64 * 64;
        if (s > kQ8MaxSplit) continue;
        if (n > 1 && s < swa::kDecodeMinSplit) break;
        const long long rounds = (pairs * n + kQ8BlocksAtOnce - 1) / kQ8BlocksAtOnce;
        const long long cost = rounds * (s + kQ8BlockCost) +
                               (n == 1 || n == swa::kDecodeClusterSplits ? 0 : kQ8MergeCost + n * kQ8MergePart);
        if (best == 0 || cost < best) {
            best = cost;
            split = (int)s;
        }
    }
    return split;
}

int q8_nsplit(int B, int Hkv, int L) {
    const int split = q8_split_keys(B, Hkv, L);
    return (int)(((long long)L + split - 1) / split);
}

// 0 where the window is one split or the splits are merged on chip (or the
// sizes are invalid).
size_t decode_q8_workspace_bytes(int B, int Hq, int Hkv, int D, int W) {
    if (B < 1 || W < 1 || check_heads(Hq, Hkv, D) != SWA_OK) return 0;
    int rep = 1;
    decode_group(Hq, Hkv, &rep);
    if ((long long)Hkv * rep > 65535) return 0;
    const int nsm = q8_nsplit(B, Hkv * rep, W);
    if (nsm == 1 || nsm == swa::kDecodeClusterSplits) return 0;
    const size_t rows = (size_t)B * Hq * nsm;
    return ((rows * D * 4 + 255) & ~size_t(255)) + rows * 8;
}

template <int D, int G>
swa_status_t launch_decode_q8_dg(const void *q, const void *kc, const void *vc, const float *ks, const float *vs,
                                 const int32_t *pos, void *out, int B, int Hkv, int W, int block, float scale,
                                 void *ws, int kv_rep, cudaStream_t s) {
    const int nsm = q8_nsplit(B, Hkv, W);
    const int split = q8_split_keys(B, Hkv, W);
    const bool cluster = nsm == swa::kDecodeClusterSplits;
    const size_t o_elems = (size_t)B * Hkv * nsm * G * D;
    float *ws_o = static_cast<float *>(ws);
    float2 *ws_ml =
        ws ? reinterpret_cast<float2 *>(static_cast<char *>(ws) + ((o_elems * 4 + 255) & ~size_t(255))) : nullptr;
    int block_log2 = 0;
    while ((1 << block_log2) < block) ++block_log2;
    const int nblk = (int)(((long long)W + block - 1) / block);
    CUtensorMap mk, mv;
    if (swa_status_t e = make_codes_map(&mk, kc, D, Hkv / kv_rep, W, B, swa::kQ8Stage)) return e;
    if (swa_status_t e = make_codes_map(&mv, vc, D, Hkv / kv_rep, W, B, swa::kQ8Stage)) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(nsm, Hkv, B);
    cfg.blockDim = dim3(swa::kQ8Warps * 32);
    cfg.dynamicSmemBytes = swa::DecodeQ8Cfg<D, G>::SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = swa::kDecodeClusterSplits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 1 : 0;
    constexpr int smem = swa::DecodeQ8Cfg<D, G>::SMEM_BYTES;
    auto kernel = cluster ? swa::swa_decode_q8_kernel<D, G, swa::kDecodeWindowCluster>
                          : swa::swa_decode_q8_kernel<D, G, swa::kDecodeWindow>;
    if (swa_status_t e = cluster ? allow_smem<swa::swa_decode_q8_kernel<D, G, swa::kDecodeWindowCluster>>(smem)
                                 : allow_smem<swa::swa_decode_q8_kernel<D, G, swa::kDecodeWindow>>(smem))
        return e;
    SWA_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, mk, mv, static_cast<const __nv_bfloat16 *>(q), ks, vs, pos,
                                    static_cast<__nv_bfloat16 *>(out), ws_ml, ws_o, Hkv, W, nsm, scale * kLog2e,
                                    split, kv_rep, block_log2, nblk));
    if (nsm > 1 && !cluster) {
        swa::swa_decode_combine_kernel<D, G><<<dim3(Hkv, B), G * D, 0, s>>>(
            pos, ws_ml, ws_o, static_cast<__nv_bfloat16 *>(out), Hkv, W, nsm, 0, split);
        SWA_CUDA_TRY(cudaGetLastError());
    }
    return SWA_OK;
}

// One call of LAUNCH<D, G>(args) for a run-time D and G (1..8).
#define SWA_DISPATCH_DG(LAUNCH, D, G, ...)                                      \
    switch ((G) + ((D) == 128 ? 8 : 0)) {                                       \
        case 1: return LAUNCH<64, 1>(__VA_ARGS__);                              \
        case 2: return LAUNCH<64, 2>(__VA_ARGS__);                              \
        case 3: return LAUNCH<64, 3>(__VA_ARGS__);                              \
        case 4: return LAUNCH<64, 4>(__VA_ARGS__);                              \
        case 5: return LAUNCH<64, 5>(__VA_ARGS__);                              \
        case 6: return LAUNCH<64, 6>(__VA_ARGS__);                              \
        case 7: return LAUNCH<64, 7>(__VA_ARGS__);                              \
        case 8: return LAUNCH<64, 8>(__VA_ARGS__);                              \
        case 9: return LAUNCH<128, 1>(__VA_ARGS__);                             \
        case 10: return LAUNCH<128, 2>(__VA_ARGS__);                            \
        case 11: return LAUNCH<128, 3>(__VA_ARGS__);                            \
        case 12: return LAUNCH<128, 4>(__VA_ARGS__);                            \
        case 13: return LAUNCH<128, 5>(__VA_ARGS__);                            \
        case 14: return LAUNCH<128, 6>(__VA_ARGS__);                            \
        case 15: return LAUNCH<128, 7>(__VA_ARGS__);                            \
        case 16: return LAUNCH<128, 8>(__VA_ARGS__);                            \
        default: return SWA_ERR_UNSUPPORTED;                                    \
    }

swa_status_t decode_q8_impl(const void *q, const void *k_cache, const void *v_cache, const float *k_scale,
                            const float *v_scale, const int32_t *pos, void *out, int B, int Hq, int Hkv, int D,
                            int W, int block, float scale, void *workspace, size_t workspace_bytes, cudaStream_t s) {
    if (swa_status_t e = decode_checks(q, k_cache, v_cache, pos, out, B, Hq, Hkv, D, W, scale)) return e;
    if (swa_status_t e = q8_cache_checks(k_cache, v_cache, k_scale, v_scale, pos, B, Hkv, D, W, block)) return e;
    int rep = 1;
    const int G = decode_group(Hq, Hkv, &rep);
    const size_t need = decode_q8_workspace_bytes(B, Hq, Hkv, D, W);
    if (need > 0 && (!workspace || workspace_bytes < need || misaligned(workspace, 256))) return SWA_ERR_INVALID_ARG;
    DeviceInfo *dev = nullptr;
    if (swa_status_t e = device_info(&dev)) return e;
    SWA_DISPATCH_DG(launch_decode_q8_dg, D, G, q, k_cache, v_cache, k_scale, v_scale, pos, out, B, Hkv * rep, W, block,
                    scale, workspace, rep, s)
}

// The widened K and V, each [B, W, Hkv, D] bf16.
size_t prefill_chunk_q8_workspace_bytes(int B, int Hkv, int D, int W) {
    if (B < 1 || W < 1 || Hkv < 1 || (D != 64 && D != 128)) return 0;
    return (size_t)B * W * Hkv * D * 2 * 2;
}

swa_status_t prefill_chunk_q8_impl(const void *q, const void *k, const void *v, void *k_cache, void *v_cache,
                                   float *k_scale, float *v_scale, const int32_t *start_pos, void *out, int B, int C,
                                   int Hq, int Hkv, int D, int W, int block, float scale, void *workspace,
                                   size_t workspace_bytes, cudaStream_t s) {
    if (!q || !k || !v || !out || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
        return SWA_ERR_INVALID_ARG;
    if (swa_status_t e = check_heads(Hq, Hkv, D)) return e;
    if (swa_status_t e = q8_cache_checks(k_cache, v_cache, k_scale, v_scale, start_pos, B, Hkv, D, W, block)) return e;
    if (C < 1 || C > W || bad_scale(scale)) return SWA_ERR_INVALID_ARG;
    if (!workspace || misaligned(workspace, 256) ||
        workspace_bytes < prefill_chunk_q8_workspace_bytes(B, Hkv, D, W))
        return SWA_ERR_INVALID_ARG;
    DeviceInfo *dev = nullptr;
    if (swa_status_t e = device_info(&dev)) return e;
    const size_t half = (size_t)B * W * Hkv * D * 2;
    char *kd = static_cast<char *>(workspace), *vd = kd + half;
    const int nblk = (int)(((long long)W + block - 1) / block);
    swa::swa_widen_q8_kernel<<<copy_grid((long long)W * Hkv * (D / 16), B, dev->sms), 256, 0, s>>>(
        static_cast<const uint4 *>(k_cache), static_cast<const uint4 *>(v_cache), k_scale, v_scale, start_pos,
        reinterpret_cast<uint4 *>(kd), reinterpret_cast<uint4 *>(vd), W, Hkv, D / 16, block, nblk);
    SWA_CUDA_TRY(cudaGetLastError());
    if (swa_status_t e = prefill_chunk_impl(q, k, v, kd, vd, start_pos, out, B, C, Hq, Hkv, D, W, scale, nullptr,
                                            nullptr, s, nullptr, nullptr, 0, false))
        return e;
    return append_q8_impl(k, v, k_cache, v_cache, k_scale, v_scale, start_pos, B, C, Hkv, D, W, block, s);
}

// ----------------------------------------------------------------- fixed-size cache with eviction
// Workspace: partial outputs, then {m, l, l} per partial row, then the scores
// [B, Hq, M up to a multiple of 16].
struct ScoresLayout {
    int nsm, split, stride;
    size_t ml_off, scores_off, bytes;
};

ScoresLayout scores_layout(int B, int Hq, int groups, int D, int M) {
    ScoresLayout l;
    l.nsm = decode_nsplit_max(B, groups, M);
    l.split = decode_split_keys(B, groups, M);
    l.stride = (M + 15) & ~15;
    const size_t rows = (size_t)B * Hq * l.nsm;
    l.ml_off = (rows * D * 4 + 255) & ~size_t(255);
    l.scores_off = (l.ml_off + rows * 16 + 255) & ~size_t(255);
    l.bytes = l.scores_off + (size_t)B * Hq * l.stride * 4;
    return l;
}

constexpr int kMaxFinishHeads = 2048;               // 16 bytes of shared memory each

bool scores_supported(int B, int Hq, int Hkv, int M) {
    int rep = 1;
    decode_group(Hq, Hkv, &rep);
    return B <= 65535 && (long long)Hkv * rep <= 65535 && Hq / Hkv <= kMaxFinishHeads && M <= swa::kEvictMaxSlots;
}

// Slots of one block of the cluster form, and whether a call takes that form:
// the group in one piece, at most kDecodeSplit slots to a block, and no more
// blocks than run at once on the B200's 148 SMs (two to an SM where their shared
// memory fits, 115712 bytes each).  As every plan behind a workspace's size it
// depends on the sizes alone.
int scores_cluster_keys(int M) {
    constexpr int k = swa::kDecodeClusterSplits * swa::kDecodeBlk;
    return (int)(((long long)M + k - 1) / k * swa::kDecodeBlk);
}

template <int D, int G>
int scores_cluster_smem(int M) { return swa::DecodeScoresCfg<D, G>::OFF_SCORES + scores_cluster_keys(M) * G * 4; }

bool scores_in_cluster(int B, int Hkv, int G, int rep, int D, int M) {
    if (rep != 1 || scores_cluster_keys(M) > swa::kDecodeSplit) return false;
    const int ring = D == 128 ? swa::DecodeScoresCfg<128, 1>::OFF_SCORES : swa::DecodeScoresCfg<64, 1>::OFF_SCORES;
    const int smem = ring + scores_cluster_keys(M) * G * 4;
    return (long long)B * Hkv * swa::kDecodeClusterSplits <= (smem <= 115712 ? 2 : 1) * 148;
}

// 0 where the merge is on chip (or the sizes are invalid).
size_t decode_weights_workspace_bytes(int B, int Hq, int Hkv, int D, int M) {
    if (B < 1 || M < 1 || check_heads(Hq, Hkv, D) != SWA_OK || !scores_supported(B, Hq, Hkv, M)) return 0;
    int rep = 1;
    const int G = decode_group(Hq, Hkv, &rep);
    if (scores_in_cluster(B, Hkv, G, rep, D, M)) return 0;
    return scores_layout(B, Hq, Hkv * rep, D, M).bytes;
}

template <int D, int G>
swa_status_t launch_decode_weights_dg(const void *q, const void *kc, const void *vc, const int32_t *slot_pos,
                                      const float *weights, float *weights_out, const int32_t *pos, void *out, int B,
                                      int groups, int M, float scale, void *ws, int rep, cudaStream_t s) {
    const __nv_bfloat16 *qb = static_cast<const __nv_bfloat16 *>(q), *kb = static_cast<const __nv_bfloat16 *>(kc),
                        *vb = static_cast<const __nv_bfloat16 *>(vc);
    __nv_bfloat16 *ob = static_cast<__nv_bfloat16 *>(out);
    float4 *ws_ml = nullptr;
    float *ws_o = nullptr, *scores = nullptr;
    if (scores_in_cluster(B, groups, G, rep, D, M)) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(swa::kDecodeClusterSplits, groups, B);
        cfg.blockDim = dim3(swa::kDecodeWarps * 32);
        cfg.dynamicSmemBytes = scores_cluster_smem<D, G>(M);
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = swa::kDecodeClusterSplits;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (swa_status_t e =
                allow_smem<swa::swa_decode_scores_kernel<D, G, true>>(swa::DecodeScoresCfg<D, G>::MAX_SMEM))
            return e;
        SWA_CUDA_TRY(cudaLaunchKernelEx(&cfg, swa::swa_decode_scores_kernel<D, G, true>, qb, kb, vb, slot_pos, pos,
                                        ws_ml, ws_o, scores, scores_cluster_keys(M), groups, M, 1, scale * kLog2e, 0,
                                        rep, weights, weights_out, ob));
        return SWA_OK;
    }
    const ScoresLayout l = scores_layout(B, groups * G, groups, D, M);
    char *base = static_cast<char *>(ws);
    ws_o = reinterpret_cast<float *>(base);
    ws_ml = reinterpret_cast<float4 *>(base + l.ml_off);
    scores = reinterpret_cast<float *>(base + l.scores_off);
    if (swa_status_t e =
            allow_smem<swa::swa_decode_scores_kernel<D, G, false>>(swa::DecodeScoresCfg<D, G>::SMEM_BYTES))
        return e;
    swa::swa_decode_scores_kernel<D, G, false>
        <<<dim3(l.nsm, groups, B), swa::kDecodeWarps * 32, swa::DecodeScoresCfg<D, G>::SMEM_BYTES, s>>>(
            qb, kb, vb, slot_pos, pos, ws_ml, ws_o, scores, l.stride, groups, M, l.nsm, scale * kLog2e, l.split, rep,
            nullptr, nullptr, nullptr);
    SWA_CUDA_TRY(cudaGetLastError());
    const int Hkv = groups / rep, Gall = G * rep;
    swa::swa_weights_finish_kernel<<<dim3((M + swa::kFinishSlots - 1) / swa::kFinishSlots, Hkv, B),
                                     swa::kFinishThreads, Gall * sizeof(float4), s>>>(
        pos, ws_ml, ws_o, scores, l.stride, weights, weights_out, ob, Hkv, Gall, rep, D, M, l.nsm, l.split);
    SWA_CUDA_TRY(cudaGetLastError());
    return SWA_OK;
}

swa_status_t decode_weights_impl(const void *q, const void *k_cache, const void *v_cache, const int32_t *slot_pos,
                                 const float *weights, float *weights_out, const int32_t *pos, void *out, int B,
                                 int Hq, int Hkv, int D, int M, float scale, void *workspace, size_t workspace_bytes,
                                 cudaStream_t s) {
    if (swa_status_t e = decode_checks(q, k_cache, v_cache, pos, out, B, Hq, Hkv, D, M, scale)) return e;
    if (!slot_pos || !weights_out || misaligned(slot_pos, 4) || misaligned(weights, 4) || misaligned(weights_out, 4))
        return SWA_ERR_INVALID_ARG;
    if (!scores_supported(B, Hq, Hkv, M)) return SWA_ERR_UNSUPPORTED;
    const size_t need = decode_weights_workspace_bytes(B, Hq, Hkv, D, M);
    if (need > 0 && (!workspace || misaligned(workspace, 256) || workspace_bytes < need)) return SWA_ERR_INVALID_ARG;
    int rep = 1;
    const int G = decode_group(Hq, Hkv, &rep);
    DeviceInfo *dev = nullptr;
    if (swa_status_t e = device_info(&dev)) return e;
    SWA_DISPATCH_DG(launch_decode_weights_dg, D, G, q, k_cache, v_cache, slot_pos, weights, weights_out, pos, out, B,
                    Hkv * rep, M, scale, workspace, rep, s)
}

// Sizes of a fixed-size cache: M slots of which S sinks and R recent ones
// (the newest among them) are never evicted.
swa_status_t budget_checks(int B, int Hkv, int D, int M, int S, int R) {
    if (B < 1 || Hkv < 1 || M < 1 || S < 0 || R < 1 || (long long)S + R > M) return SWA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return SWA_ERR_UNSUPPORTED;
    if (B > 65535 || M > swa::kEvictMaxSlots) return SWA_ERR_UNSUPPORTED;
    return SWA_OK;
}

swa_status_t evict_append_impl(const void *k_new, const void *v_new, void *k_cache, void *v_cache, int32_t *slot_pos,
                               float *weights, const int32_t *pos, int32_t *slots, int B, int Hkv, int D, int M, int S,
                               int R, cudaStream_t s) {
    if (!k_new || !v_new || !k_cache || !v_cache || !slot_pos || !weights || !pos) return SWA_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
        misaligned(slot_pos, 4) || misaligned(weights, 4) || misaligned(pos, 4) || misaligned(slots, 4))
        return SWA_ERR_INVALID_ARG;
    if (swa_status_t e = budget_checks(B, Hkv, D, M, S, R)) return e;
    const bool vec = M % 4 == 0 && aligned16(slot_pos) && aligned16(weights);
    auto kernel = vec ? swa::swa_evict_append_kernel<true> : swa::swa_evict_append_kernel<false>;
    kernel<<<dim3(Hkv, B), swa::kEvictThreads, 0, s>>>(
        static_cast<const uint4 *>(k_new), static_cast<const uint4 *>(v_new), static_cast<uint4 *>(k_cache),
        static_cast<uint4 *>(v_cache), slot_pos, weights, pos, slots, Hkv, M, D / 8, S, R);
    SWA_CUDA_TRY(cudaGetLastError());
    return SWA_OK;
}

swa_status_t keep_impl(const void *k, const void *v, const float *weights, const int32_t *lens, void *k_cache,
                       void *v_cache, int32_t *slot_pos, float *weights_out, int B, int N, int Hkv, int D, int M,
                       int S, int R, cudaStream_t s) {
    if (!k || !v || !weights || !lens || !k_cache || !v_cache || !slot_pos || !weights_out) return SWA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) || misaligned(weights, 4) ||
        misaligned(lens, 4) || misaligned(slot_pos, 4) || misaligned(weights_out, 4) || N < 1)
        return SWA_ERR_INVALID_ARG;
    if (swa_status_t e = budget_checks(B, Hkv, D, M, S, R)) return e;
    DeviceInfo *dev = nullptr;
    if (swa_status_t e = device_info(&dev)) return e;
    if (swa_status_t e = allow_smem<swa::swa_keep_select_kernel>(swa::kKeepMaxSmem)) return e;
    swa::swa_keep_select_kernel<<<dim3(Hkv, B), swa::kKeepThreads, swa::keep_smem(N), s>>>(
        weights, lens, slot_pos, weights_out, N, Hkv, M, S, R);
    SWA_CUDA_TRY(cudaGetLastError());
    swa::swa_keep_copy_kernel<<<copy_grid((long long)M * Hkv * (D / 8), B, dev->sms), 256, 0, s>>>(
        static_cast<const uint4 *>(k), static_cast<const uint4 *>(v), slot_pos, static_cast<uint4 *>(k_cache),
        static_cast<uint4 *>(v_cache), N, Hkv, M, D / 8);
    SWA_CUDA_TRY(cudaGetLastError());
    return SWA_OK;
}

// ----------------------------------------------------------------- weights of a prompt
// Sizes and workspace of swa_prefill_weights: the lse pass's partial results,
// lse, the weights pass's partial planes.  A function of the sizes only, as the
// workspace size is.
struct WeightsLayout {
    int G, TQ, nqt, nkt, splits1, splits2, planes;
    bool by_query;               // all queries fit in two tiles: they stay in the weights pass too
    long long units1, units2;
    size_t lse_off, part_off, bytes;
};

// Persistent blocks the splits aim at: one per SM of the B200 (a plan behind a
// workspace's size, so it depends on the sizes alone).
constexpr int kWeightsBlocks = 148;

// Splits of a unit's `tiles` streamed tiles.  Units of about the same work fill
// one wave of the persistent blocks; where the work falls off along a triangle,
// six units to a block keep the last ones short.  At least `least` tiles each.
int weights_splits(long long units, long long tiles, bool even, int least) {
    long long s = even ? kWeightsBlocks / units : (6 * kWeightsBlocks + units - 1) / units;
    if (s > tiles / least) s = tiles / least;
    return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

WeightsLayout weights_layout(int B, int T, int N, int Hq, int Hkv, int W) {
    WeightsLayout l;
    l.G = Hq / Hkv;
    l.TQ = 128 / l.G;
    l.nqt = (int)(((long long)T + l.TQ - 1) / l.TQ);
    l.nkt = (int)(((long long)N + 127) / 128);
    l.by_query = l.nqt <= 2;
    const long long weff = W < N ? W : N;
    const long long t1 = (weff + 2 * l.TQ - 2) / 128 + 2, t2 = (weff + 254) / l.TQ + 2;
    const long long bh = (long long)B * Hkv;
    const bool even = T <= N / 4 || W <= N / 4;
    const long long pairs1 = (l.nqt + 1) / 2, pairs2 = (l.nkt + 1) / 2;
    l.splits1 = weights_splits(bh * pairs1, t1 < l.nkt ? t1 : l.nkt, even, 2);
    l.splits2 = l.by_query ? l.splits1 : weights_splits(bh * pairs2, t2 < l.nqt ? t2 : l.nqt, even, 4);
    l.units1 = bh * pairs1 * l.splits1;
    l.units2 = l.by_query ? bh * l.splits2 : bh * pairs2 * l.splits2;
    l.planes = 2 * (l.by_query ? l.nqt : l.splits2);
    const size_t rows = (size_t)bh * l.nqt * 128;
    l.lse_off = rows * 2 * l.splits1 * 8;
    l.part_off = (l.lse_off + rows * 4 + 255) & ~size_t(255);
    l.bytes = l.part_off + (size_t)l.planes * bh * N * 4;
    return l;
}

swa_status_t prefill_weights_sizes(int B, int T, int N, int Hq, int Hkv, int D, int W) {
    if (B < 1 || T < 1 || N < 1 || T > N || W < 1) return SWA_ERR_INVALID_ARG;
    if (swa_status_t e = check_heads(Hq, Hkv, D)) return e;
    if (Hq / Hkv > 128) return SWA_ERR_UNSUPPORTED;          // a query tile holds a position's whole group
    const WeightsLayout l = weights_layout(B, T, N, Hq, Hkv, W);
    if (l.units1 > 0x7fffffffll || l.units2 > 0x7fffffffll || (long long)B * Hkv * l.nqt > 0x7fffffffll)
        return SWA_ERR_UNSUPPORTED;
    return SWA_OK;
}

template <int D, int MODE>
swa_status_t launch_weights_pass(const CUtensorMap &mq, const CUtensorMap &mk, const swa::WeightsParams &p, int sms,
                                 cudaStream_t s) {
    const int grid = p.num_units < sms ? p.num_units : sms;
    if (swa_status_t e = allow_smem<swa::swa_prefill_weights_kernel<D, MODE>>(swa::WeightsCfg<D, MODE>::SMEM_ALLOC))
        return e;
    swa::swa_prefill_weights_kernel<D, MODE>
        <<<grid, swa::WeightsCfg<D, MODE>::THREADS, swa::WeightsCfg<D, MODE>::SMEM_ALLOC, s>>>(mq, mk, p);
    SWA_CUDA_TRY(cudaGetLastError());
    return SWA_OK;
}

swa_status_t launch_weights_pass(int mode, int D, const CUtensorMap &mq, const CUtensorMap &mk,
                                 const swa::WeightsParams &p, int sms, cudaStream_t s) {
    switch (mode + (D == 128 ? 4 : 0)) {
        case swa::kWeightsLse: return launch_weights_pass<64, swa::kWeightsLse>(mq, mk, p, sms, s);
        case swa::kWeightsByKey: return launch_weights_pass<64, swa::kWeightsByKey>(mq, mk, p, sms, s);
        case swa::kWeightsByQuery: return launch_weights_pass<64, swa::kWeightsByQuery>(mq, mk, p, sms, s);
        case swa::kWeightsLse + 4: return launch_weights_pass<128, swa::kWeightsLse>(mq, mk, p, sms, s);
        case swa::kWeightsByKey + 4: return launch_weights_pass<128, swa::kWeightsByKey>(mq, mk, p, sms, s);
        default: return launch_weights_pass<128, swa::kWeightsByQuery>(mq, mk, p, sms, s);
    }
}

swa_status_t prefill_weights_impl(const void *q, const void *k, const int32_t *lens, float *weights, int B, int T,
                                  int N, int Hq, int Hkv, int D, int W, float scale, void *workspace,
                                  size_t workspace_bytes, cudaStream_t s) {
    if (!q || !k || !lens || !weights || !aligned16(q) || !aligned16(k) || misaligned(lens, 4) ||
        misaligned(weights, 4) || bad_scale(scale))
        return SWA_ERR_INVALID_ARG;
    if (swa_status_t e = prefill_weights_sizes(B, T, N, Hq, Hkv, D, W)) return e;
    const WeightsLayout l = weights_layout(B, T, N, Hq, Hkv, W);
    if (!workspace || misaligned(workspace, 256) || workspace_bytes < l.bytes) return SWA_ERR_INVALID_ARG;
    DeviceInfo *dev = nullptr;
    if (swa_status_t e = device_info(&dev)) return e;
    CUtensorMap mq, mk;
    if (swa_status_t e = make_operand_map(&mq, q, D, Hq, T, B, l.G, l.TQ)) return e;
    if (swa_status_t e = make_operand_map(&mk, k, D, Hkv, N, B)) return e;
    char *ws = static_cast<char *>(workspace);
    float *lse = reinterpret_cast<float *>(ws + l.lse_off), *part = reinterpret_cast<float *>(ws + l.part_off);
    swa::WeightsParams p{};
    p.B = B, p.N = N, p.T = T, p.Hkv = Hkv, p.G = l.G, p.TQ = l.TQ;
    p.W = W < N ? W : N;
    p.nqt = l.nqt, p.nkt = l.nkt;
    p.scale_log2 = scale * kLog2e;
    p.lens = lens;
    p.ml = reinterpret_cast<float2 *>(ws);
    p.lse = lse;
    p.part = part;
    p.splits = l.splits1;
    p.num_units = (int)l.units1;
    if (swa_status_t e = launch_weights_pass(swa::kWeightsLse, D, mq, mk, p, dev->sms, s)) return e;
    swa::swa_weights_lse_kernel<<<(unsigned)((long long)B * Hkv * l.nqt), 128, 0, s>>>(
        p.ml, lse, lens, N, T, Hkv, l.G, l.TQ, l.nqt, 2 * l.splits1);
    SWA_CUDA_TRY(cudaGetLastError());
    p.splits = l.splits2;
    p.num_units = (int)l.units2;
    if (swa_status_t e = launch_weights_pass(l.by_query ? swa::kWeightsByQuery : swa::kWeightsByKey, D, mq, mk, p,
                                             dev->sms, s))
        return e;
    const long long n = (long long)B * Hkv * N;
    long long blocks = (n + 255) / 256;
    if (blocks > (long long)dev->sms * 16) blocks = (long long)dev->sms * 16;
    swa::swa_weights_sum_kernel<<<(int)blocks, 256, 0, s>>>(p, weights, l.planes, l.by_query);
    SWA_CUDA_TRY(cudaGetLastError());
    return SWA_OK;
}

}  // namespace

extern "C" {

swa_status_t swa_prefill(const void *q, const void *k, const void *v, void *out, int B, int N,
                         int Hq, int Hkv, int D, int W, int window_mode, float scale,
                         swa_stream_t stream) {
    return prefill_impl(q, k, v, out, B, N, Hq, Hkv, D, W, window_mode, scale, nullptr, nullptr,
                        reinterpret_cast<cudaStream_t>(stream));
}

swa_status_t swa_prefill_chunk(const void *q, const void *k, const void *v, void *k_cache,
                               void *v_cache, const int32_t *start_pos, void *out, int B, int C,
                               int Hq, int Hkv, int D, int W, float scale, swa_stream_t stream) {
    return prefill_chunk_impl(q, k, v, k_cache, v_cache, start_pos, out, B, C, Hq, Hkv, D, W, scale,
                              nullptr, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

swa_status_t swa_cache_append(const void *k_new, const void *v_new, void *k_cache, void *v_cache,
                              const int32_t *pos, int B, int T, int Hkv, int D, int W,
                              swa_stream_t stream) {
    return append_impl(k_new, v_new, k_cache, v_cache, pos, B, T, Hkv, D, W, nullptr,
                       reinterpret_cast<cudaStream_t>(stream));
}

size_t swa_decode_workspace_size(int B, int Hq, int Hkv, int D, int W) {
    return decode_workspace_bytes(B, Hq, Hkv, D, W);
}

swa_status_t swa_decode(const void *q, const void *k_cache, const void *v_cache,
                        const int32_t *pos, void *out, int B, int Hq, int Hkv, int D, int W,
                        float scale, void *workspace, size_t workspace_bytes,
                        swa_stream_t stream) {
    return decode_impl(q, k_cache, v_cache, pos, out, B, Hq, Hkv, D, W, scale, workspace,
                       workspace_bytes, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

swa_status_t swa_decode_noalloc(const void *q, const void *k_cache, const void *v_cache,
                                const int32_t *pos, void *out, int B, int Hq, int Hkv, int D,
                                int W, float scale, swa_stream_t stream) {
    if (swa_status_t e = decode_checks(q, k_cache, v_cache, pos, out, B, Hq, Hkv, D, W, scale)) return e;
    if (decode_workspace_bytes(B, Hq, Hkv, D, W) > kNoallocScratchBytes) return SWA_ERR_UNSUPPORTED;
    void *scratch = nullptr;
    if (swa_status_t e = noalloc_scratch(&scratch)) return e;
    return decode_launch(q, k_cache, v_cache, pos, out, B, Hq, Hkv, D, W, scale, scratch, nullptr,
                         reinterpret_cast<cudaStream_t>(stream));
}

swa_status_t swa_rope(void *x, const int32_t *pos, int B, int T, int H, int D, float theta,
                      swa_stream_t stream) {
    if (!x || !pos || !aligned16(x) || (reinterpret_cast<uintptr_t>(pos) & 3u)) return SWA_ERR_INVALID_ARG;
    if (B < 1 || T < 1 || H < 1 || bad_theta(theta)) return SWA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return SWA_ERR_UNSUPPORTED;
    DeviceInfo *dev = nullptr;
    if (swa_status_t e = device_info(&dev)) return e;
    const swa::RopeTable tab = make_rope_table(theta, D);
    const int row_vec = H * D / 8, head_vec = D / 8;
    const long long total = (long long)B * T * row_vec;
    long long blocks = (total + 255) / 256;
    if (blocks > (long long)dev->sms * 16) blocks = (long long)dev->sms * 16;
    swa::swa_rope_kernel<<<(int)blocks, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        static_cast<uint4 *>(x), pos, B, T, row_vec, head_vec, tab);
    SWA_CUDA_TRY(cudaGetLastError());
    return SWA_OK;
}

swa_status_t swa_cache_append_rope(const void *k_new, const void *v_new, void *k_cache,
                                   void *v_cache, const int32_t *pos, int B, int T, int Hkv,
                                   int D, int W, float theta, swa_stream_t stream) {
    if (bad_theta(theta)) return SWA_ERR_INVALID_ARG;
    const swa::RopeTable tab = make_rope_table(theta, D);
    return append_impl(k_new, v_new, k_cache, v_cache, pos, B, T, Hkv, D, W, &tab,
                       reinterpret_cast<cudaStream_t>(stream));
}

swa_status_t swa_prefill_rope(const void *q, const void *k, const void *v, void *out, int B, int N,
                              int Hq, int Hkv, int D, int W, int window_mode, float scale,
                              float theta, swa_stream_t stream) {
    if (bad_theta(theta)) return SWA_ERR_INVALID_ARG;
    const swa::RopeTable tab = make_rope_table(theta, D);
    return prefill_impl(q, k, v, out, B, N, Hq, Hkv, D, W, window_mode, scale, &tab, nullptr,
                        reinterpret_cast<cudaStream_t>(stream));
}

swa_status_t swa_prefill_chunk_rope(const void *q, const void *k, const void *v, void *k_cache,
                                    void *v_cache, const int32_t *start_pos, void *out, int B,
                                    int C, int Hq, int Hkv, int D, int W, float scale, float theta,
                                    swa_stream_t stream) {
    if (bad_theta(theta)) return SWA_ERR_INVALID_ARG;
    const swa::RopeTable tab = make_rope_table(theta, D);
    return prefill_chunk_impl(q, k, v, k_cache, v_cache, start_pos, out, B, C, Hq, Hkv, D, W, scale,
                              &tab, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

swa_status_t swa_decode_rope(const void *q, const void *k_cache, const void *v_cache,
                             const int32_t *pos, void *out, int B, int Hq, int Hkv, int D, int W,
                             float scale, float theta, void *workspace, size_t workspace_bytes,
                             swa_stream_t stream) {
    if (bad_theta(theta)) return SWA_ERR_INVALID_ARG;
    const swa::RopeTable tab = make_rope_table(theta, D);
    return decode_impl(q, k_cache, v_cache, pos, out, B, Hq, Hkv, D, W, scale, workspace,
                       workspace_bytes, &tab, reinterpret_cast<cudaStream_t>(stream));
}

swa_status_t swa_prefill_varlen(const void *q, const void *k, const void *v, void *out,
                                const int32_t *cu_seqlens, int B, int total, int Hq, int Hkv, int D,
                                int W, int window_mode, float scale, swa_stream_t stream) {
    if (!cu_seqlens) return SWA_ERR_INVALID_ARG;
    return prefill_impl(q, k, v, out, B, total, Hq, Hkv, D, W, window_mode, scale, nullptr, cu_seqlens,
                        reinterpret_cast<cudaStream_t>(stream));
}

swa_status_t swa_prefill_chunk_varlen(const void *q, const void *k, const void *v, void *k_cache,
                                      void *v_cache, const int32_t *start_pos,
                                      const int32_t *cu_seqlens, void *out, int B, int total,
                                      int Hq, int Hkv, int D, int W, float scale,
                                      swa_stream_t stream) {
    if (!cu_seqlens) return SWA_ERR_INVALID_ARG;
    return prefill_chunk_impl(q, k, v, k_cache, v_cache, start_pos, out, B, total, Hq, Hkv, D, W, scale,
                              nullptr, cu_seqlens, reinterpret_cast<cudaStream_t>(stream));
}

swa_status_t swa_prefill_sinks(const void *q, const void *k, const void *v, void *out, int B, int N,
                               int Hq, int Hkv, int D, int W, int S, float scale, swa_stream_t stream) {
    if (S < 0) return SWA_ERR_INVALID_ARG;
    return prefill_impl(q, k, v, out, B, N, Hq, Hkv, D, W, SWA_WINDOW_EXCL_LEFT, scale, nullptr, nullptr,
                        reinterpret_cast<cudaStream_t>(stream), S);
}

swa_status_t swa_prefill_chunk_sinks(const void *q, const void *k, const void *v, void *k_cache,
                                     void *v_cache, void *k_sink, void *v_sink, const int32_t *start_pos,
                                     void *out, int B, int C, int Hq, int Hkv, int D, int W, int S,
                                     float scale, swa_stream_t stream) {
    return prefill_chunk_impl(q, k, v, k_cache, v_cache, start_pos, out, B, C, Hq, Hkv, D, W, scale,
                              nullptr, nullptr, reinterpret_cast<cudaStream_t>(stream), k_sink, v_sink, S);
}

swa_status_t swa_cache_append_sinks(const void *k_new, const void *v_new, void *k_cache, void *v_cache,
                                    void *k_sink, void *v_sink, const int32_t *pos, int B, int T,
                                    int Hkv, int D, int W, int S, swa_stream_t stream) {
    if (S < 0 || (S > 0 && (!k_sink || !v_sink || !aligned16(k_sink) || !aligned16(v_sink))))
        return SWA_ERR_INVALID_ARG;
    if (!k_new || !v_new || !k_cache || !v_cache || !pos) return SWA_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
        (reinterpret_cast<uintptr_t>(pos) & 3u))
        return SWA_ERR_INVALID_ARG;
    if (B < 1 || T < 1 || W < 1 || T > W || Hkv < 1) return SWA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return SWA_ERR_UNSUPPORTED;
    DeviceInfo *dev = nullptr;
    if (swa_status_t e = device_info(&dev)) return e;
    return launch_append(k_new, v_new, k_cache, v_cache, pos, B, T, Hkv, D, W, dev->sms, nullptr,
                         reinterpret_cast<cudaStream_t>(stream), k_sink, v_sink, S);
}

swa_status_t swa_decode_sinks(const void *q, const void *k_cache, const void *v_cache,
                              const void *k_sink, const void *v_sink, const int32_t *pos, void *out,
                              int B, int Hq, int Hkv, int D, int W, int S, float scale,
                              void *workspace, size_t workspace_bytes, swa_stream_t stream) {
    if (S < 0 || (S > 0 && (!k_sink || !v_sink || !aligned16(k_sink) || !aligned16(v_sink))))
        return SWA_ERR_INVALID_ARG;
    if (swa_status_t e = decode_checks(q, k_cache, v_cache, pos, out, B, Hq, Hkv, D, W, scale)) return e;
    if ((long long)W + S > 0x7fffffffll) return SWA_ERR_UNSUPPORTED;
    const size_t need = decode_workspace_bytes(B, Hq, Hkv, D, W + S);
    int rep = 1;
    const int G = decode_group(Hq, Hkv, &rep);
    if (decode_nsplit_max(B, Hkv * rep, W + S) > 1) {
        if (!workspace || workspace_bytes < need) return SWA_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(workspace) & 255u) return SWA_ERR_INVALID_ARG;
    }
    DeviceInfo *dev = nullptr;
    if (swa_status_t e = device_info(&dev)) return e;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return D == 128 ? launch_decode_d<128>(G, rep, q, k_cache, v_cache, pos, out, B, Hkv * rep, W, scale, workspace,
                                           nullptr, s, k_sink, v_sink, S)
                    : launch_decode_d<64>(G, rep, q, k_cache, v_cache, pos, out, B, Hkv * rep, W, scale, workspace,
                                          nullptr, s, k_sink, v_sink, S);
}

swa_status_t swa_cache_append_q8(const void *k_new, const void *v_new, void *k_cache, void *v_cache, float *k_scale,
                                 float *v_scale, const int32_t *pos, int B, int T, int Hkv, int D, int W, int block,
                                 swa_stream_t stream) {
    return append_q8_impl(k_new, v_new, k_cache, v_cache, k_scale, v_scale, pos, B, T, Hkv, D, W, block,
                          reinterpret_cast<cudaStream_t>(stream));
}

swa_status_t swa_decode_q8(const void *q, const void *k_cache, const void *v_cache, const float *k_scale,
                           const float *v_scale, const int32_t *pos, void *out, int B, int Hq, int Hkv, int D, int W,
                           int block, float scale, void *workspace, size_t workspace_bytes, swa_stream_t stream) {
    return decode_q8_impl(q, k_cache, v_cache, k_scale, v_scale, pos, out, B, Hq, Hkv, D, W, block, scale, workspace,
                          workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

size_t swa_decode_q8_workspace_size(int B, int Hq, int Hkv, int D, int W) {
    return decode_q8_workspace_bytes(B, Hq, Hkv, D, W);
}

size_t swa_prefill_chunk_q8_workspace_size(int B, int Hkv, int D, int W) {
    return prefill_chunk_q8_workspace_bytes(B, Hkv, D, W);
}

swa_status_t swa_prefill_chunk_q8(const void *q, const void *k, const void *v, void *k_cache, void *v_cache,
                                  float *k_scale, float *v_scale, const int32_t *start_pos, void *out, int B, int C,
                                  int Hq, int Hkv, int D, int W, int block, float scale, void *workspace,
                                  size_t workspace_bytes, swa_stream_t stream) {
    return prefill_chunk_q8_impl(q, k, v, k_cache, v_cache, k_scale, v_scale, start_pos, out, B, C, Hq, Hkv, D, W,
                                 block, scale, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

size_t swa_decode_weights_workspace_size(int B, int Hq, int Hkv, int D, int M) {
    return decode_weights_workspace_bytes(B, Hq, Hkv, D, M);
}

swa_status_t swa_decode_weights(const void *q, const void *k_cache, const void *v_cache, const int32_t *slot_pos,
                                const float *weights, float *weights_out, const int32_t *pos, void *out, int B, int Hq,
                                int Hkv, int D, int M, float scale, void *workspace, size_t workspace_bytes,
                                swa_stream_t stream) {
    return decode_weights_impl(q, k_cache, v_cache, slot_pos, weights, weights_out, pos, out, B, Hq, Hkv, D, M, scale,
                               workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

swa_status_t swa_cache_evict_append(const void *k_new, const void *v_new, void *k_cache, void *v_cache,
                                    int32_t *slot_pos, float *weights, const int32_t *pos, int32_t *slots, int B,
                                    int Hkv, int D, int M, int S, int R, swa_stream_t stream) {
    return evict_append_impl(k_new, v_new, k_cache, v_cache, slot_pos, weights, pos, slots, B, Hkv, D, M, S, R,
                             reinterpret_cast<cudaStream_t>(stream));
}

swa_status_t swa_cache_keep(const void *k, const void *v, const float *weights, const int32_t *lens, void *k_cache,
                            void *v_cache, int32_t *slot_pos, float *weights_out, int B, int N, int Hkv, int D, int M,
                            int S, int R, swa_stream_t stream) {
    return keep_impl(k, v, weights, lens, k_cache, v_cache, slot_pos, weights_out, B, N, Hkv, D, M, S, R,
                     reinterpret_cast<cudaStream_t>(stream));
}

size_t swa_prefill_weights_workspace_size(int B, int T, int N, int Hq, int Hkv, int D, int W) {
    return prefill_weights_sizes(B, T, N, Hq, Hkv, D, W) == SWA_OK ? weights_layout(B, T, N, Hq, Hkv, W).bytes : 0;
}

swa_status_t swa_prefill_weights(const void *q, const void *k, const int32_t *lens, float *weights, int B, int T,
                                 int N, int Hq, int Hkv, int D, int W, float scale, void *workspace,
                                 size_t workspace_bytes, swa_stream_t stream) {
    return prefill_weights_impl(q, k, lens, weights, B, T, N, Hq, Hkv, D, W, scale, workspace, workspace_bytes,
                                reinterpret_cast<cudaStream_t>(stream));
}

swa_status_t swa_get_device_status(swa_stream_t stream) {
    SWA_CUDA_TRY(cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)));
    int v = 0;
    SWA_CUDA_TRY(cudaMemcpyFromSymbol(&v, swa::g_status, sizeof(int)));
    const int zero = 0;
    SWA_CUDA_TRY(cudaMemcpyToSymbol(swa::g_status, &zero, sizeof(int)));
    return static_cast<swa_status_t>(v);
}

swa_status_t swa_set_wait_limit_ns(unsigned long long limit_ns) {
    SWA_CUDA_TRY(cudaMemcpyToSymbol(swa::g_wait_limit_ns, &limit_ns, sizeof(limit_ns)));
    return SWA_OK;
}

swa_status_t swa_selftest_wait_timeout(swa_stream_t stream) {
    swa_selftest_wait_kernel<<<1, 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>();
    SWA_CUDA_TRY(cudaGetLastError());
    return SWA_OK;
}

swa_status_t swa_selftest_exp2(const float *x, float *y, int n, swa_stream_t stream) {
    if (!x || !y || n < 1) return SWA_ERR_INVALID_ARG;
    const int pairs = (n + 1) / 2;
    swa_selftest_exp2_kernel<false><<<(pairs + 255) / 256, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(x, y, n);
    SWA_CUDA_TRY(cudaGetLastError());
    return SWA_OK;
}

swa_status_t swa_selftest_exp2_fine(const float *x, float *y, int n, swa_stream_t stream) {
    if (!x || !y || n < 1) return SWA_ERR_INVALID_ARG;
    const int pairs = (n + 1) / 2;
    swa_selftest_exp2_kernel<true><<<(pairs + 255) / 256, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(x, y, n);
    SWA_CUDA_TRY(cudaGetLastError());
    return SWA_OK;
}

const char *swa_status_string(swa_status_t status) {
    switch (status) {
        case SWA_OK: return "SWA_OK";
        case SWA_ERR_INVALID_ARG: return "SWA_ERR_INVALID_ARG";
        case SWA_ERR_UNSUPPORTED: return "SWA_ERR_UNSUPPORTED";
        case SWA_ERR_CUDA: return "SWA_ERR_CUDA";
        case SWA_ERR_TIMEOUT: return "SWA_ERR_TIMEOUT";
        default: return "SWA_ERR_UNKNOWN";
    }
}

int swa_last_cuda_error(void) { return t_last_cuda_error; }

}  // extern "C"
