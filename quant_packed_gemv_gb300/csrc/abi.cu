// The C ABI of libplm: argument checks on the host, then one or more kernel
// launches on the caller's stream.  Nothing is allocated and nothing waits.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/plm.h"
#include "plm_device.cuh"
#include "plm_internal.h"

namespace plm {

// Set (bitwise or) by kernels whose bounded wait on an asynchronous copy ran
// out; read and cleared by plm_device_fault.  One word per device, in the
// module's static device memory (nothing is allocated).
__device__ unsigned g_plm_fault = 0;

unsigned* fault_word() {
    // the symbol's address is fixed per device while the device's primary
    // context lives (the library must not be used across a cudaDeviceReset);
    // remember it for the first 64 devices.  Threads that race here store
    // the same address.
    static std::atomic<void*> cache[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
    if (dev >= 0 && dev < 64) {
        void* c = cache[dev].load(std::memory_order_acquire);
        if (c) return static_cast<unsigned*>(c);
    }
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_plm_fault) != cudaSuccess) return nullptr;
    if (dev >= 0 && dev < 64) cache[dev].store(p, std::memory_order_release);
    return static_cast<unsigned*>(p);
}

namespace {
std::atomic<int> g_overlap{1};
}
int overlap_mode() { return g_overlap.load(std::memory_order_relaxed); }

int num_sms() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
    return n;
}

}  // namespace plm

namespace {

thread_local int g_last_cuda_error = 0;

constexpr int64_t kMaxIndex = 0x7FFFFFFFLL;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

plm_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return PLM_OK;
    g_last_cuda_error = (int)e;
    return PLM_ERR_CUDA;
}

// Shape checks shared by the matmul entry points.
plm_status check_matmul(const void* w, const void* xq, const void* y, int64_t m, int64_t n,
                        int64_t k, int64_t max_m) {
    if (!w || !xq || !y) return PLM_ERR_INVALID_ARG;
    if (m <= 0 || n <= 0 || k <= 0 || k % plm::QK != 0) return PLM_ERR_INVALID_ARG;
    if (m > max_m || n > kMaxIndex || k > kMaxIndex) return PLM_ERR_INVALID_ARG;
    if (m * (k / plm::QK) > kMaxIndex || n * (k / plm::QK) > kMaxIndex) return PLM_ERR_INVALID_ARG;
    if (!aligned(w, 16) || !aligned(xq, 4) || !aligned(y, 4)) return PLM_ERR_MISALIGNED;
    return PLM_OK;
}

plm_status gemv_common(int fmt, const void* w, const void* xq, float* y, int64_t m, int64_t n,
                       int64_t k, cudaStream_t stream) {
    plm_status s = check_matmul(w, xq, y, m, n, k, plm::GEMV_MAX_M);
    if (s != PLM_OK) return s;
    if (!plm::gemv_supported(fmt, (int)k)) return PLM_ERR_UNSUPPORTED;
    return cuda_status(plm::launch_gemv(fmt, (const uint8_t*)w, (const uint8_t*)xq, y, (int)m,
                                        (int)n, (int)k, stream));
}

plm_status grouped_common(int fmt, const plm_gemv_problem* problems, int64_t count, int64_t m,
                          cudaStream_t stream) {
    if (!problems || count <= 0 || count > kMaxIndex) return PLM_ERR_INVALID_ARG;
    if (m <= 0 || m > plm::GEMV_MAX_M) return PLM_ERR_INVALID_ARG;
    constexpr int kChunk = 256;
    plm::GroupItem items[kChunk];
    // argument checks for every problem first, then size support
    for (int64_t j = 0; j < count; ++j) {
        const plm_gemv_problem& p = problems[j];
        plm_status s = check_matmul(p.w, p.xq, p.y, m, p.n, p.k, plm::GEMV_MAX_M);
        if (s != PLM_OK) return s;
    }
    for (int64_t j = 0; j < count; ++j)
        if (!plm::gemv_supported(fmt, (int)problems[j].k)) return PLM_ERR_UNSUPPORTED;
    for (int64_t p0 = 0; p0 < count; p0 += kChunk) {
        const int cnt = (int)(count - p0 < kChunk ? count - p0 : kChunk);
        for (int j = 0; j < cnt; ++j) {
            const plm_gemv_problem& p = problems[p0 + j];
            items[j] = plm::GroupItem{(const uint8_t*)p.w, (const uint8_t*)p.xq, p.y, (int)p.n, (int)p.k};
        }
        plm_status s = cuda_status(plm::launch_gemv_grouped(fmt, items, cnt, (int)m, stream));
        if (s != PLM_OK) return s;
    }
    return PLM_OK;
}

// Fused quantize + GEMV: f32 activations, 16-byte aligned for vector loads.
plm_status qgemv_common(const plm_qgemv_problem* problems, int64_t count, int64_t m, cudaStream_t stream) {
    if (!problems || count <= 0 || count > kMaxIndex) return PLM_ERR_INVALID_ARG;
    if (m <= 0 || m > plm::GEMV_MAX_M) return PLM_ERR_INVALID_ARG;
    for (int64_t j = 0; j < count; ++j) {
        const plm_qgemv_problem& p = problems[j];
        plm_status s = check_matmul(p.w, p.x, p.y, m, p.n, p.k, plm::GEMV_MAX_M);
        if (s != PLM_OK) return s;
        if (!aligned(p.x, 16)) return PLM_ERR_MISALIGNED;
    }
    for (int64_t j = 0; j < count; ++j)
        if (!plm::gemv_supported(4, (int)problems[j].k)) return PLM_ERR_UNSUPPORTED;
    constexpr int kChunk = 256;
    plm::GroupItem items[kChunk];
    for (int64_t p0 = 0; p0 < count; p0 += kChunk) {
        const int cnt = (int)(count - p0 < kChunk ? count - p0 : kChunk);
        for (int j = 0; j < cnt; ++j) {
            const plm_qgemv_problem& p = problems[p0 + j];
            items[j] = plm::GroupItem{(const uint8_t*)p.w, (const uint8_t*)p.x, p.y, (int)p.n, (int)p.k};
        }
        plm_status s = cuda_status(plm::launch_quantize_gemv_q4K(items, cnt, (int)m, stream));
        if (s != PLM_OK) return s;
    }
    return PLM_OK;
}

// Gate/up pairs: both matrices checked like a GEMV's weights.
plm_status swiglu_common(const plm_swiglu_problem* problems, int64_t count, int64_t m, cudaStream_t stream) {
    if (!problems || count <= 0 || count > kMaxIndex) return PLM_ERR_INVALID_ARG;
    if (m <= 0 || m > plm::GEMV_MAX_M) return PLM_ERR_INVALID_ARG;
    for (int64_t j = 0; j < count; ++j) {
        const plm_swiglu_problem& p = problems[j];
        plm_status s = check_matmul(p.w_gate, p.xq, p.h, m, p.n, p.k, plm::GEMV_MAX_M);
        if (s != PLM_OK) return s;
        s = check_matmul(p.w_up, p.xq, p.h, m, p.n, p.k, plm::GEMV_MAX_M);
        if (s != PLM_OK) return s;
    }
    for (int64_t j = 0; j < count; ++j)
        if (!plm::gemv_supported(4, (int)problems[j].k)) return PLM_ERR_UNSUPPORTED;
    constexpr int kChunk = 256;
    plm::GroupItem items[kChunk];
    for (int64_t p0 = 0; p0 < count; p0 += kChunk) {
        const int cnt = (int)(count - p0 < kChunk ? count - p0 : kChunk);
        for (int j = 0; j < cnt; ++j) {
            const plm_swiglu_problem& p = problems[p0 + j];
            items[j] = plm::GroupItem{(const uint8_t*)p.w_gate, (const uint8_t*)p.xq, p.h, (int)p.n, (int)p.k,
                                      (const uint8_t*)p.w_up};
        }
        plm_status s = cuda_status(plm::launch_gemv_q4K_swiglu(items, cnt, (int)m, stream));
        if (s != PLM_OK) return s;
    }
    return PLM_OK;
}

plm_status gemm_common(int fmt, const void* w, const void* xq, float* y, int64_t m, int64_t n,
                       int64_t k, cudaStream_t stream) {
    plm_status s = check_matmul(w, xq, y, m, n, k, kMaxIndex);
    if (s != PLM_OK) return s;
    if (m * n > (int64_t)1 << 40) return PLM_ERR_INVALID_ARG;
    if (!plm::gemv_supported(fmt, (int)k)) return PLM_ERR_UNSUPPORTED;
    return cuda_status(plm::launch_gemm(fmt, (const uint8_t*)w, (const uint8_t*)xq, y, m, (int)n,
                                        (int)k, stream));
}

plm_status gemm_ws_common(int fmt, const void* w, const void* xq, float* y, int64_t m, int64_t n,
                          int64_t k, void* ws, size_t ws_bytes, cudaStream_t stream) {
    plm_status s = check_matmul(w, xq, y, m, n, k, kMaxIndex);
    if (s != PLM_OK) return s;
    if (m * n > (int64_t)1 << 40) return PLM_ERR_INVALID_ARG;
    const size_t need = plm::gemm_workspace_need(fmt, m, (int)k);
    if (need > 0 && (!ws || ws_bytes < need)) return PLM_ERR_INVALID_ARG;
    if (ws && !aligned(ws, 256)) return PLM_ERR_MISALIGNED;
    if (!plm::gemv_supported(fmt, (int)k)) return PLM_ERR_UNSUPPORTED;
    return cuda_status(plm::launch_gemm_ws(fmt, (const uint8_t*)w, (const uint8_t*)xq, y, m, (int)n, (int)k,
                                           ws, ws_bytes, stream));
}

plm_status gemm_swiglu_common(const void* wg, const void* wu, const void* xq, float* h, int64_t m, int64_t n,
                              int64_t k, bool caller_ws, void* ws, size_t ws_bytes, cudaStream_t stream) {
    plm_status s = check_matmul(wg, xq, h, m, n, k, kMaxIndex);
    if (s != PLM_OK) return s;
    s = check_matmul(wu, xq, h, m, n, k, kMaxIndex);
    if (s != PLM_OK) return s;
    if (m * n > (int64_t)1 << 40) return PLM_ERR_INVALID_ARG;
    if (caller_ws) {
        const size_t need = plm::gemm_swiglu_workspace_min(m, (int)n, (int)k);
        if (need > 0 && (!ws || ws_bytes < need)) return PLM_ERR_INVALID_ARG;
        if (ws && !aligned(ws, 256)) return PLM_ERR_MISALIGNED;
    }
    if (!plm::gemv_supported(4, (int)k)) return PLM_ERR_UNSUPPORTED;
    const uint8_t *g8 = (const uint8_t*)wg, *u8 = (const uint8_t*)wu, *x8 = (const uint8_t*)xq;
    return cuda_status(caller_ws ? plm::launch_gemm_q4K_swiglu_ws(g8, u8, x8, h, m, (int)n, (int)k, ws, ws_bytes, stream)
                                 : plm::launch_gemm_q4K_swiglu(g8, u8, x8, h, m, (int)n, (int)k, stream));
}

plm_status subdots_common(int fmt, const void* w, const void* xq, int32_t* out, int64_t m,
                          int64_t n, int64_t k, cudaStream_t stream) {
    plm_status s = check_matmul(w, xq, out, m, n, k, plm::GEMV_MAX_M);
    if (s != PLM_OK) return s;
    if (!plm::gemv_supported(fmt, (int)k)) return PLM_ERR_UNSUPPORTED;
    return cuda_status(plm::launch_subdots(fmt, (const uint8_t*)w, (const uint8_t*)xq, out, (int)m,
                                           (int)n, (int)k, stream));
}

size_t x16_size(int fmt, int64_t n, int64_t k) {
    if (n <= 0 || k <= 0 || k % plm::QK != 0 || n > kMaxIndex || k > kMaxIndex) return 0;
    if (((n + 15) / 16) * (k / plm::QK) > kMaxIndex) return 0;
    return plm::x16_bytes(fmt, n, (int)k);
}

plm_status x16_repack(int fmt, const void* w, void* w_x16, int64_t n, int64_t k, cudaStream_t stream) {
    if (!w || !w_x16) return PLM_ERR_INVALID_ARG;
    if (x16_size(fmt, n, k) == 0) return PLM_ERR_INVALID_ARG;
    if (!aligned(w, 16) || !aligned(w_x16, 16)) return PLM_ERR_MISALIGNED;
    return cuda_status(plm::launch_repack_x16(fmt, (const uint8_t*)w, (uint8_t*)w_x16, (int)n, (int)k, stream));
}

plm_status x16_gemv(int fmt, const void* w_x16, const void* xq, float* y, int64_t m, int64_t n, int64_t k,
                    cudaStream_t stream) {
    plm_status s = check_matmul(w_x16, xq, y, m, n, k, plm::GEMV_MAX_M);
    if (s != PLM_OK) return s;
    if (x16_size(fmt, n, k) == 0) return PLM_ERR_INVALID_ARG;
    return cuda_status(plm::launch_gemv_x16(fmt, (const uint8_t*)w_x16, (const uint8_t*)xq, y, (int)m, (int)n,
                                            (int)k, stream));
}

}  // namespace

extern "C" {

int plm_abi_version(void) { return PLM_ABI_VERSION; }

int plm_set_overlap(int mode) {
    if (mode < PLM_OVERLAP_OFF || mode > PLM_OVERLAP_PREFETCH) return -PLM_ERR_INVALID_ARG;
    return plm::g_overlap.exchange(mode);
}

const char* plm_status_string(int status) {
    switch (status) {
        case PLM_OK: return "ok";
        case PLM_ERR_INVALID_ARG: return "invalid argument";
        case PLM_ERR_MISALIGNED: return "misaligned pointer";
        case PLM_ERR_UNSUPPORTED: return "unsupported size";
        case PLM_ERR_CUDA: return "CUDA launch error";
        default: return "unknown status";
    }
}

int plm_last_cuda_error(void) { return g_last_cuda_error; }

plm_status plm_device_fault(uint32_t* code, int clear) {
    if (!code) return PLM_ERR_INVALID_ARG;
    unsigned v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, plm::g_plm_fault, sizeof v);
    if (e != cudaSuccess) return cuda_status(e);
    *code = v;
    if (clear && v) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(plm::g_plm_fault, &zero, sizeof zero);
        if (e != cudaSuccess) return cuda_status(e);
    }
    return PLM_OK;
}

plm_status plm_quantize_q8K(const float* x, void* xq, int64_t m, int64_t k, cudaStream_t stream) {
    if (!x || !xq) return PLM_ERR_INVALID_ARG;
    if (m <= 0 || k <= 0 || k % plm::QK != 0) return PLM_ERR_INVALID_ARG;
    if (m > kMaxIndex || k > kMaxIndex || m * (k / plm::QK) > kMaxIndex) return PLM_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(xq, 4)) return PLM_ERR_MISALIGNED;
    return cuda_status(plm::launch_quantize_q8K(x, (uint8_t*)xq, m, k, stream));
}

plm_status plm_gemv_q4K(const void* w, const void* xq, float* y, int64_t m, int64_t n, int64_t k,
                        cudaStream_t stream) {
    return gemv_common(4, w, xq, y, m, n, k, stream);
}

plm_status plm_gemv_q6K(const void* w, const void* xq, float* y, int64_t m, int64_t n, int64_t k,
                        cudaStream_t stream) {
    return gemv_common(6, w, xq, y, m, n, k, stream);
}

plm_status plm_gemv_q4K_grouped(const plm_gemv_problem* problems, int64_t count, int64_t m,
                                cudaStream_t stream) {
    return grouped_common(4, problems, count, m, stream);
}

plm_status plm_gemv_q6K_grouped(const plm_gemv_problem* problems, int64_t count, int64_t m,
                                cudaStream_t stream) {
    return grouped_common(6, problems, count, m, stream);
}

plm_status plm_gemv_q2K(const void* w, const void* xq, float* y, int64_t m, int64_t n, int64_t k,
                        cudaStream_t stream) {
    return gemv_common(2, w, xq, y, m, n, k, stream);
}

plm_status plm_gemv_q2K_grouped(const plm_gemv_problem* problems, int64_t count, int64_t m,
                                cudaStream_t stream) {
    return grouped_common(2, problems, count, m, stream);
}

plm_status plm_gemm_q2K(const void* w, const void* xq, float* y, int64_t m, int64_t n, int64_t k,
                        cudaStream_t stream) {
    return gemm_common(2, w, xq, y, m, n, k, stream);
}

plm_status plm_gemm_q2K_ws(const void* w, const void* xq, float* y, int64_t m, int64_t n, int64_t k,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    return gemm_ws_common(2, w, xq, y, m, n, k, workspace, workspace_bytes, stream);
}

plm_status plm_subdots_q2K(const void* w, const void* xq, int32_t* out, int64_t m, int64_t n, int64_t k,
                           cudaStream_t stream) {
    return subdots_common(2, w, xq, out, m, n, k, stream);
}

plm_status plm_gemv_q3K(const void* w, const void* xq, float* y, int64_t m, int64_t n, int64_t k,
                        cudaStream_t stream) {
    return gemv_common(3, w, xq, y, m, n, k, stream);
}

plm_status plm_gemv_q3K_grouped(const plm_gemv_problem* problems, int64_t count, int64_t m,
                                cudaStream_t stream) {
    return grouped_common(3, problems, count, m, stream);
}

plm_status plm_gemm_q3K(const void* w, const void* xq, float* y, int64_t m, int64_t n, int64_t k,
                        cudaStream_t stream) {
    return gemm_common(3, w, xq, y, m, n, k, stream);
}

plm_status plm_gemm_q3K_ws(const void* w, const void* xq, float* y, int64_t m, int64_t n, int64_t k,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    return gemm_ws_common(3, w, xq, y, m, n, k, workspace, workspace_bytes, stream);
}

plm_status plm_subdots_q3K(const void* w, const void* xq, int32_t* out, int64_t m, int64_t n, int64_t k,
                           cudaStream_t stream) {
    return subdots_common(3, w, xq, out, m, n, k, stream);
}

plm_status plm_gemv_q5K(const void* w, const void* xq, float* y, int64_t m, int64_t n, int64_t k,
                        cudaStream_t stream) {
    return gemv_common(5, w, xq, y, m, n, k, stream);
}

plm_status plm_gemv_q5K_grouped(const plm_gemv_problem* problems, int64_t count, int64_t m,
                                cudaStream_t stream) {
    return grouped_common(5, problems, count, m, stream);
}

plm_status plm_gemm_q5K(const void* w, const void* xq, float* y, int64_t m, int64_t n, int64_t k,
                        cudaStream_t stream) {
    return gemm_common(5, w, xq, y, m, n, k, stream);
}

plm_status plm_gemm_q5K_ws(const void* w, const void* xq, float* y, int64_t m, int64_t n, int64_t k,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    return gemm_ws_common(5, w, xq, y, m, n, k, workspace, workspace_bytes, stream);
}

plm_status plm_subdots_q5K(const void* w, const void* xq, int32_t* out, int64_t m, int64_t n, int64_t k,
                           cudaStream_t stream) {
    return subdots_common(5, w, xq, out, m, n, k, stream);
}

plm_status plm_gemm_q4K(const void* w, const void* xq, float* y, int64_t m, int64_t n, int64_t k,
                        cudaStream_t stream) {
    return gemm_common(4, w, xq, y, m, n, k, stream);
}

plm_status plm_gemm_q6K(const void* w, const void* xq, float* y, int64_t m, int64_t n, int64_t k,
                        cudaStream_t stream) {
    return gemm_common(6, w, xq, y, m, n, k, stream);
}

size_t plm_gemm_workspace_size_split(int fmt, int64_t m, int64_t n, int64_t k) {
    if (fmt < 2 || fmt > 6 || m <= 0 || n <= 0 || k <= 0 || k % plm::QK != 0 || k > kMaxIndex || n > kMaxIndex ||
        m * n > (int64_t)1 << 40)
        return 0;
    return plm::gemm_workspace_need_split(fmt, m, (int)n, (int)k);
}

size_t plm_gemm_swiglu_workspace_size(int64_t m, int64_t n, int64_t k) {
    if (m <= 0 || n <= 0 || k <= 0 || k % plm::QK != 0 || k > kMaxIndex || n > kMaxIndex || m * n > (int64_t)1 << 40)
        return 0;
    return plm::gemm_swiglu_workspace_need(m, (int)n, (int)k);
}

size_t plm_gemm_workspace_size(int fmt, int64_t m, int64_t k) {
    if (fmt < 2 || fmt > 6 || m <= 0 || k <= 0 || k % plm::QK != 0 || k > kMaxIndex) return 0;
    return plm::gemm_workspace_need(fmt, m, (int)k);
}

plm_status plm_gemm_q4K_ws(const void* w, const void* xq, float* y, int64_t m, int64_t n, int64_t k,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    return gemm_ws_common(4, w, xq, y, m, n, k, workspace, workspace_bytes, stream);
}

plm_status plm_gemm_q6K_ws(const void* w, const void* xq, float* y, int64_t m, int64_t n, int64_t k,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    return gemm_ws_common(6, w, xq, y, m, n, k, workspace, workspace_bytes, stream);
}

plm_status plm_gemm_q4K_noalloc(const void* w, const void* xq, float* y, int64_t m, int64_t n, int64_t k,
                                cudaStream_t stream) {
    plm_status s = check_matmul(w, xq, y, m, n, k, kMaxIndex);
    if (s != PLM_OK) return s;
    if (m * n > (int64_t)1 << 40) return PLM_ERR_INVALID_ARG;
    if (!plm::gemm_noalloc_fits(m, (int)k)) return PLM_ERR_UNSUPPORTED;   // beyond the fixed array
    if (!plm::gemv_supported(4, (int)k)) return PLM_ERR_UNSUPPORTED;
    return cuda_status(plm::launch_gemm_q4K_noalloc((const uint8_t*)w, (const uint8_t*)xq, y, m, (int)n, (int)k,
                                                    stream));
}

size_t plm_q4K_x16_size(int64_t n, int64_t k) { return x16_size(4, n, k); }
size_t plm_q6K_x16_size(int64_t n, int64_t k) { return x16_size(6, n, k); }

plm_status plm_q4K_to_x16(const void* w, void* w_x16, int64_t n, int64_t k, cudaStream_t stream) {
    return x16_repack(4, w, w_x16, n, k, stream);
}
plm_status plm_q6K_to_x16(const void* w, void* w_x16, int64_t n, int64_t k, cudaStream_t stream) {
    return x16_repack(6, w, w_x16, n, k, stream);
}

plm_status plm_gemv_q4K_x16(const void* w_x16, const void* xq, float* y, int64_t m, int64_t n, int64_t k,
                            cudaStream_t stream) {
    return x16_gemv(4, w_x16, xq, y, m, n, k, stream);
}
plm_status plm_gemv_q6K_x16(const void* w_x16, const void* xq, float* y, int64_t m, int64_t n, int64_t k,
                            cudaStream_t stream) {
    return x16_gemv(6, w_x16, xq, y, m, n, k, stream);
}

plm_status plm_quantize_gemv_q4K(const void* w, const float* x, float* y, int64_t m, int64_t n, int64_t k,
                                 cudaStream_t stream) {
    const plm_qgemv_problem p{w, x, y, n, k};
    return qgemv_common(&p, 1, m, stream);
}

plm_status plm_quantize_gemv_q4K_grouped(const plm_qgemv_problem* problems, int64_t count, int64_t m,
                                         cudaStream_t stream) {
    return qgemv_common(problems, count, m, stream);
}

plm_status plm_gemv_q4K_swiglu(const void* w_gate, const void* w_up, const void* xq, float* h, int64_t m,
                               int64_t n, int64_t k, cudaStream_t stream) {
    const plm_swiglu_problem p{w_gate, w_up, xq, h, n, k};
    return swiglu_common(&p, 1, m, stream);
}

plm_status plm_gemm_q4K_swiglu(const void* w_gate, const void* w_up, const void* xq, float* h, int64_t m,
                               int64_t n, int64_t k, cudaStream_t stream) {
    return gemm_swiglu_common(w_gate, w_up, xq, h, m, n, k, false, nullptr, 0, stream);
}

plm_status plm_gemm_q4K_swiglu_ws(const void* w_gate, const void* w_up, const void* xq, float* h, int64_t m,
                                  int64_t n, int64_t k, void* workspace, size_t workspace_bytes,
                                  cudaStream_t stream) {
    return gemm_swiglu_common(w_gate, w_up, xq, h, m, n, k, true, workspace, workspace_bytes, stream);
}

plm_status plm_gemv_q4K_swiglu_grouped(const plm_swiglu_problem* problems, int64_t count, int64_t m,
                                       cudaStream_t stream) {
    return swiglu_common(problems, count, m, stream);
}

plm_status plm_subdots_q4K(const void* w, const void* xq, int32_t* out, int64_t m, int64_t n,
                           int64_t k, cudaStream_t stream) {
    return subdots_common(4, w, xq, out, m, n, k, stream);
}

plm_status plm_subdots_q6K(const void* w, const void* xq, int32_t* out, int64_t m, int64_t n,
                           int64_t k, cudaStream_t stream) {
    return subdots_common(6, w, xq, out, m, n, k, stream);
}

}  // extern "C"

namespace {

// ---------------------------------------------------------------------------
// Rotary positions, cache pages, attention
// ---------------------------------------------------------------------------
int64_t type_size(int type) { return type == PLM_F32 ? 4 : type == PLM_F16 || type == PLM_BF16 ? 2 : 0; }

bool in_range(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }

plm_status check_kv(const plm_kv_state* kv) {
    if (!kv || !kv->table || !kv->lens || !kv->refs) return PLM_ERR_INVALID_ARG;
    if (!in_range(kv->pages, 1, kMaxIndex) || !in_range(kv->max_seqs, 1, kMaxIndex) ||
        !in_range(kv->max_pages, 1, kMaxIndex) || !in_range(kv->page_tokens, 1, kMaxIndex))
        return PLM_ERR_INVALID_ARG;
    if (kv->max_seqs > (INT64_MAX >> 8) / kv->max_pages) return PLM_ERR_INVALID_ARG;
    if (!aligned(kv->table, 4) || !aligned(kv->lens, 4) || !aligned(kv->refs, 4) || !aligned(kv->status, 4))
        return PLM_ERR_MISALIGNED;
    return PLM_OK;
}

// The pool, for the calls that move pages.
plm_status check_pool(const plm_kv_state* kv) {
    if (!kv->pool || kv->page_bytes < 16 || kv->page_bytes % 16 != 0) return PLM_ERR_INVALID_ARG;
    if (kv->page_bytes > (INT64_MAX >> 8) / kv->pages) return PLM_ERR_INVALID_ARG;
    return aligned(kv->pool, 16) ? PLM_OK : PLM_ERR_MISALIGNED;
}

plm_status check_kv_workspace(const plm_kv_state* kv, int64_t n, const void* ws, size_t bytes) {
    if (!ws || bytes < plm::kv_workspace_bytes(kv->pages, n)) return PLM_ERR_INVALID_ARG;
    return aligned(ws, 256) ? PLM_OK : PLM_ERR_MISALIGNED;
}

}  // namespace

extern "C" {

plm_status plm_rope_freqs(uint64_t* freqs, int64_t rotary_dim, double base, const plm_rope_scaling* scaling,
                          float* scale) {
    if (!freqs || !in_range(rotary_dim, 2, 65536) || rotary_dim % 2 || !(base > 1.0) || !std::isfinite(base))
        return PLM_ERR_INVALID_ARG;
    const int kind = scaling ? scaling->kind : PLM_ROPE_SCALING_NONE;
    if (!in_range(kind, PLM_ROPE_SCALING_NONE, PLM_ROPE_SCALING_RAMP)) return PLM_ERR_INVALID_ARG;
    const bool blend = kind == PLM_ROPE_SCALING_BANDS || kind == PLM_ROPE_SCALING_RAMP;
    const double factor = kind == PLM_ROPE_SCALING_NONE ? 1.0 : scaling->factor;
    if (!(factor >= 1.0) || !std::isfinite(factor)) return PLM_ERR_INVALID_ARG;
    if (blend && !(scaling->trained >= 1.0 && scaling->low > 0.0 && scaling->high > scaling->low &&
                   std::isfinite(scaling->trained) && std::isfinite(scaling->high)))
        return PLM_ERR_INVALID_ARG;
    if (kind == PLM_ROPE_SCALING_BASE && rotary_dim == 2) return PLM_ERR_INVALID_ARG;
    const double kTwoPi = 6.283185307179586476925286766559;
    const double R = (double)rotary_dim;
    const double b = kind == PLM_ROPE_SCALING_BASE ? base * std::pow(factor, R / (R - 2.0)) : base;
    double first = 0.0, last = 0.0;   // RAMP: the pairs between which r falls from 1 to 0
    if (kind == PLM_ROPE_SCALING_RAMP) {
        // pair i makes trained / (2 pi) base^(-2i/R) turns
        auto pair_of = [&](double turns) { return R * std::log(scaling->trained / (turns * kTwoPi)) / (2.0 * std::log(base)); };
        first = std::fmax(std::floor(pair_of(scaling->high)), 0.0);
        last = std::fmin(std::ceil(pair_of(scaling->low)), R - 1.0);
        if (last <= first) last = first + 0.001;
    }
    for (int64_t i = 0; i < rotary_dim / 2; ++i) {
        double w = std::pow(b, -2.0 * (double)i / R);
        if (kind == PLM_ROPE_SCALING_LINEAR) w /= factor;
        if (blend) {
            const double r = kind == PLM_ROPE_SCALING_BANDS
                                 ? (scaling->trained * w / kTwoPi - scaling->low) / (scaling->high - scaling->low)
                                 : 1.0 - ((double)i - first) / (last - first);
            const double keep = std::fmin(1.0, std::fmax(0.0, r));
            w = w * (keep + (1.0 - keep) / factor);
        }
        // w <= 1 radian: below a sixth of a turn, so the product is below 2^62
        freqs[i] = (uint64_t)std::llround(w / kTwoPi * 18446744073709551616.0);
    }
    if (scale) *scale = kind == PLM_ROPE_SCALING_RAMP ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return PLM_OK;
}

plm_status plm_rope(const plm_rope_tensor* tensors, int64_t count, const int32_t* positions, const uint64_t* freqs,
                    int64_t tokens, int64_t head_dim, int64_t rotary_dim, int layout, float scale, int inverse,
                    cudaStream_t stream) {
    if (!tensors || !in_range(count, 1, PLM_ROPE_MAX_TENSORS) || !positions || !freqs) return PLM_ERR_INVALID_ARG;
    if (!in_range(tokens, 0, kMaxIndex) || !in_range(head_dim, 2, 1024) || head_dim % 2) return PLM_ERR_INVALID_ARG;
    if (!in_range(rotary_dim, 2, head_dim) || rotary_dim % 2) return PLM_ERR_INVALID_ARG;
    if (layout != PLM_ROPE_HALF && layout != PLM_ROPE_INTERLEAVED) return PLM_ERR_INVALID_ARG;
    int64_t heads = 0;
    for (int64_t j = 0; j < count; ++j) {
        const plm_rope_tensor& t = tensors[j];
        if (!t.x || !t.y || !type_size(t.x_type) || !type_size(t.y_type) || !in_range(t.heads, 1, 65536))
            return PLM_ERR_INVALID_ARG;
        if (t.slots && (!in_range(t.page_tokens, 1, kMaxIndex) || !in_range(t.pages, 1, kMaxIndex)))
            return PLM_ERR_INVALID_ARG;
        if (t.x == t.y && (t.slots || t.x_type != t.y_type || t.x_token_stride != t.y_token_stride ||
                           t.x_head_stride != t.y_head_stride))
            return PLM_ERR_INVALID_ARG;
        heads += t.heads;
    }
    if (heads > 65536) return PLM_ERR_INVALID_ARG;
    if (!aligned(positions, 4) || !aligned(freqs, 8)) return PLM_ERR_MISALIGNED;
    for (int64_t j = 0; j < count; ++j) {
        const plm_rope_tensor& t = tensors[j];
        if (!aligned(t.x, type_size(t.x_type)) || !aligned(t.y, type_size(t.y_type)) || !aligned(t.slots, 8))
            return PLM_ERR_MISALIGNED;
    }
    if (tokens == 0) return PLM_OK;
    return cuda_status(plm::launch_rope(tensors, (int)count, positions, freqs, tokens, (int)head_dim, (int)rotary_dim,
                                        layout, scale, inverse != 0, stream));
}

size_t plm_kv_workspace_size(int64_t pages, int64_t n) {
    if (!in_range(pages, 1, kMaxIndex) || !in_range(n, 0, kMaxIndex)) return 0;
    return plm::kv_workspace_bytes(pages, n);
}

plm_status plm_kv_reserve(const plm_kv_state* kv, const int32_t* seqs, const int32_t* add, int64_t n, int64_t* slots,
                          int64_t slots_stride, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    plm_status s = check_kv(kv);
    if (s != PLM_OK) return s;
    if ((n != 0 && (!seqs || !add)) || !in_range(n, 0, kMaxIndex)) return PLM_ERR_INVALID_ARG;
    if (slots && !in_range(slots_stride, 1, kMaxIndex)) return PLM_ERR_INVALID_ARG;
    s = check_kv_workspace(kv, n, workspace, workspace_bytes);
    if (s != PLM_OK) return s;
    if (!aligned(seqs, 4) || !aligned(add, 4) || !aligned(slots, 8)) return PLM_ERR_MISALIGNED;
    if (n == 0) return PLM_OK;
    return cuda_status(plm::launch_kv_reserve(*kv, seqs, add, n, reinterpret_cast<long long*>(slots),
                                              slots ? slots_stride : 0, workspace, stream));
}

plm_status plm_kv_fork(const plm_kv_state* kv, const int32_t* parents, const int32_t* children, const int32_t* keep,
                       int64_t n, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    plm_status s = check_kv(kv);
    if (s == PLM_OK) s = check_pool(kv);
    if (s != PLM_OK) return s;
    if ((n != 0 && (!parents || !children)) || !in_range(n, 0, kMaxIndex)) return PLM_ERR_INVALID_ARG;
    s = check_kv_workspace(kv, n, workspace, workspace_bytes);
    if (s != PLM_OK) return s;
    if (!aligned(parents, 4) || !aligned(children, 4) || !aligned(keep, 4)) return PLM_ERR_MISALIGNED;
    if (n == 0) return PLM_OK;
    return cuda_status(plm::launch_kv_fork(*kv, parents, children, keep, n, workspace, stream));
}

plm_status plm_kv_free(const plm_kv_state* kv, const int32_t* seqs, int64_t n, cudaStream_t stream) {
    plm_status s = check_kv(kv);
    if (s != PLM_OK) return s;
    if ((n != 0 && !seqs) || !in_range(n, 0, kMaxIndex)) return PLM_ERR_INVALID_ARG;
    if (!aligned(seqs, 4)) return PLM_ERR_MISALIGNED;
    if (n == 0) return PLM_OK;
    return cuda_status(plm::launch_kv_free(*kv, seqs, n, stream));
}

plm_status plm_kv_compact(const plm_kv_state* kv, int32_t* live, void* workspace, size_t workspace_bytes,
                          cudaStream_t stream) {
    plm_status s = check_kv(kv);
    if (s == PLM_OK) s = check_pool(kv);
    if (s == PLM_OK) s = check_kv_workspace(kv, 0, workspace, workspace_bytes);
    if (s != PLM_OK) return s;
    if (!aligned(live, 4)) return PLM_ERR_MISALIGNED;
    return cuda_status(plm::launch_kv_compact(*kv, live, workspace, stream));
}

plm_status plm_kv_copy_pages(const plm_kv_state* kv, const int32_t* src, const int32_t* dst, int64_t n,
                             cudaStream_t stream) {
    plm_status s = check_kv(kv);
    if (s == PLM_OK) s = check_pool(kv);
    if (s != PLM_OK) return s;
    if ((n != 0 && (!src || !dst)) || !in_range(n, 0, kMaxIndex)) return PLM_ERR_INVALID_ARG;
    if (!aligned(src, 4) || !aligned(dst, 4)) return PLM_ERR_MISALIGNED;
    if (n == 0) return PLM_OK;
    return cuda_status(plm::launch_kv_copy_pages(*kv, src, dst, n, stream));
}

size_t plm_attn_workspace_size(int64_t batch, int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim,
                               int64_t prefix_len, int64_t max_len) {
    if (!in_range(batch, 1, kMaxIndex) || !in_range(tokens, 1, kMaxIndex) || !in_range(heads, 1, kMaxIndex) ||
        !in_range(kv_heads, 1, heads) || heads % kv_heads || (head_dim != 64 && head_dim != 128) ||
        !in_range(max_len, 1, kMaxIndex) || !in_range(prefix_len, 0, max_len))
        return 0;
    if (batch * tokens > kMaxIndex / heads) return 0;
    const size_t need = plm::attn_workspace_bytes(batch, tokens, heads, kv_heads, head_dim, prefix_len, max_len);
    return need == SIZE_MAX ? 0 : need;
}

plm_status plm_attn_shared_prefix(const plm_attn_problem* p, void* workspace, size_t workspace_bytes,
                                  cudaStream_t stream) {
    if (!p || !p->q || !p->o || !p->k || !p->v || !p->table || !p->lens) return PLM_ERR_INVALID_ARG;
    if (!in_range(p->batch, 0, kMaxIndex) || !in_range(p->tokens, 1, kMaxIndex) || !in_range(p->heads, 1, kMaxIndex) ||
        !in_range(p->kv_heads, 1, p->heads) || p->heads % p->kv_heads || p->head_dim < 1)
        return PLM_ERR_INVALID_ARG;
    if (p->batch * p->tokens > kMaxIndex / p->heads) return PLM_ERR_INVALID_ARG;
    if ((p->type != PLM_F16 && p->type != PLM_BF16) || (p->o_type != p->type && p->o_type != PLM_F32))
        return PLM_ERR_INVALID_ARG;
    if (!in_range(p->pages, 1, kMaxIndex) || !in_range(p->rows, 1, kMaxIndex) || p->page_tokens < 1 ||
        !in_range(p->table_stride, 1, kMaxIndex) || !in_range(p->max_len, 1, kMaxIndex) ||
        !in_range(p->prefix_len, 0, p->max_len) || p->prefix_len % p->page_tokens)
        return PLM_ERR_INVALID_ARG;
    if (p->page_stride < 0 || p->kv_head_stride < 0 || p->kv_token_stride < 0) return PLM_ERR_INVALID_ARG;
    if ((p->head_dim != 64 && p->head_dim != 128) || !in_range(p->page_tokens, 16, 1 << 30) ||
        (p->page_tokens & (p->page_tokens - 1)))
        return PLM_ERR_UNSUPPORTED;
    if (p->batch == 0) return PLM_OK;
    const size_t need = plm::attn_workspace_bytes(p->batch, p->tokens, p->heads, p->kv_heads, p->head_dim,
                                                  p->prefix_len, p->max_len);
    if (need == SIZE_MAX) return PLM_ERR_UNSUPPORTED;
    if (need && (!workspace || workspace_bytes < need)) return PLM_ERR_INVALID_ARG;
    const int64_t oe = p->o_type == PLM_F32 ? 4 : 8;   // elements of 16 bytes
    if (!aligned(p->q, 16) || !aligned(p->o, 16) || !aligned(p->k, 16) || !aligned(p->v, 16) || !aligned(p->lse, 4) ||
        !aligned(p->table, 4) || !aligned(p->lens, 4) || !aligned(p->seqs, 4) || !aligned(workspace, 256))
        return PLM_ERR_MISALIGNED;
    if (p->q_token_stride % 8 || p->q_head_stride % 8 || p->o_token_stride % oe || p->o_head_stride % oe ||
        p->page_stride % 8 || p->kv_head_stride % 8 || p->kv_token_stride % 8)
        return PLM_ERR_MISALIGNED;
    return cuda_status(plm::launch_attn(*p, workspace, stream));
}

plm_status plm_call(int entry, const void* args) {
    if (!args) return PLM_ERR_INVALID_ARG;
    const int64_t* a = static_cast<const int64_t*>(args);
    auto ptr = [&](int i) { return reinterpret_cast<void*>(a[i]); };
    auto ints = [&](int i) { return static_cast<const int32_t*>(ptr(i)); };
    auto stream = [&](int i) { return static_cast<cudaStream_t>(ptr(i)); };
    auto kv = [&](int i) { return reinterpret_cast<const plm_kv_state*>(a + i); };
    switch (entry) {
        case 0: {
            double scale;
            std::memcpy(&scale, a + 7, sizeof scale);
            return plm_rope(reinterpret_cast<const plm_rope_tensor*>(a + 10), a[0], ints(1),
                            static_cast<const uint64_t*>(ptr(2)), a[3], a[4], a[5], (int)a[6], (float)scale, (int)a[8],
                            stream(9));
        }
        case 1:
            return plm_kv_reserve(kv(8), ints(0), ints(1), a[2], static_cast<int64_t*>(ptr(3)), a[4], ptr(5), (size_t)a[6],
                                  stream(7));
        case 2: return plm_kv_fork(kv(7), ints(0), ints(1), ints(2), a[3], ptr(4), (size_t)a[5], stream(6));
        case 3: return plm_kv_free(kv(3), ints(0), a[1], stream(2));
        case 4: return plm_kv_compact(kv(4), static_cast<int32_t*>(ptr(0)), ptr(1), (size_t)a[2], stream(3));
        case 5: return plm_kv_copy_pages(kv(4), ints(0), ints(1), a[2], stream(3));
        case 6:
            return plm_attn_shared_prefix(reinterpret_cast<const plm_attn_problem*>(a + 3), ptr(0), (size_t)a[1], stream(2));
        default: return PLM_ERR_INVALID_ARG;
    }
}

}  // extern "C"
