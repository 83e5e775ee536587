// api.cpp -- the C ABI of libfp8mi.so: argument validation, device check and
// dispatch to the gfx950 kernels.  Every invalid combination is rejected
// before anything is launched, with a message naming the argument (the
// up-front rejection convention of [Soup, lbrq.cn], list of configuration
// errors caught at load time, including the explicit "needs hardware X").
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>

#include "fp8mi.h"
#include "launch.hpp"

namespace {

thread_local std::string g_last_error;

fp8_status fail(fp8_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return st;
}

fp8_status ok() {
    g_last_error.clear();
    return FP8_OK;
}

struct DeviceInfo {
    std::atomic<int> state{0};   // 0 unknown, 1 gfx950, 2 other
    int num_cus = 0;
    char arch[64] = {0};
};

constexpr int kMaxDevices = 64;
DeviceInfo g_devices[kMaxDevices];
std::mutex g_dev_mutex;

// Current device must be gfx950; returns its CU count through *cus.
fp8_status check_device(int* cus) {
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return fail(FP8_ERR_HIP, "hipGetDevice failed: %s", hipGetErrorString(e));
    if (dev < 0 || dev >= kMaxDevices) return fail(FP8_ERR_UNSUPPORTED_DEVICE, "device index %d out of range", dev);
    DeviceInfo& d = g_devices[dev];
    if (d.state.load(std::memory_order_acquire) == 0) {
        std::lock_guard<std::mutex> lock(g_dev_mutex);
        if (d.state.load(std::memory_order_relaxed) == 0) {
            hipDeviceProp_t prop;
            e = hipGetDeviceProperties(&prop, dev);
            if (e != hipSuccess)
                return fail(FP8_ERR_HIP, "hipGetDeviceProperties failed: %s", hipGetErrorString(e));
            std::strncpy(d.arch, prop.gcnArchName, sizeof(d.arch) - 1);
            d.num_cus = prop.multiProcessorCount;
            const bool is950 = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
            d.state.store(is950 ? 1 : 2, std::memory_order_release);
        }
    }
    if (d.state.load(std::memory_order_acquire) != 1)
        return fail(FP8_ERR_UNSUPPORTED_DEVICE,
                    "device %d is %s; this library needs gfx950 (MI355X / MI350X): FP8 MFMA and OCP FP8 conversion",
                    dev, d.arch);
    *cus = d.num_cus;
    return FP8_OK;
}

// The caller's workspace: needed by the per-tensor reductions and the grouped
// GEMM's tile table, optional elsewhere.
fp8_status check_workspace(bool needed, void* ws, int64_t bytes, uint32_t** out) {
    *out = static_cast<uint32_t*>(ws);
    if (!needed) return FP8_OK;
    if (ws == nullptr) return fail(FP8_ERR_INVALID_ARG, "workspace is NULL (this call needs fp8_workspace_size() bytes)");
    if (bytes < FP8_WORKSPACE_BYTES)
        return fail(FP8_ERR_INVALID_ARG, "workspace_bytes=%lld is below fp8_workspace_size()=%d", (long long)bytes,
                    FP8_WORKSPACE_BYTES);
    if ((uintptr_t)ws % 16 != 0) return fail(FP8_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    return FP8_OK;
}

fp8_status launch_result(hipError_t e, const char* what) {
    if (e != hipSuccess) return fail(FP8_ERR_HIP, "%s: launch failed: %s", what, hipGetErrorString(e));
    return ok();
}

bool is_aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

fp8_status check_matrix_in(const void* x, int in_dtype, int64_t rows, int64_t cols, int64_t ld) {
    if (x == nullptr && rows > 0 && cols > 0) return fail(FP8_ERR_INVALID_ARG, "x is NULL");
    if (in_dtype != FP8_IN_F32 && in_dtype != FP8_IN_BF16)
        return fail(FP8_ERR_INVALID_ARG, "in_dtype %d is not FP8_IN_F32 or FP8_IN_BF16", in_dtype);
    if (rows < 0 || cols < 0) return fail(FP8_ERR_INVALID_ARG, "negative size rows=%lld cols=%lld",
                                          (long long)rows, (long long)cols);
    if (ld < cols || ld < 1) return fail(FP8_ERR_INVALID_ARG, "ld=%lld must be >= max(cols, 1)=%lld",
                                         (long long)ld, (long long)(cols > 1 ? cols : 1));
    const int esz = in_dtype == FP8_IN_F32 ? 4 : 2;
    if (!is_aligned(x, esz)) return fail(FP8_ERR_MISALIGNED, "x is not aligned to its %d-byte element", esz);
    if (rows > (int64_t(1) << 31) || cols > (int64_t(1) << 31))
        return fail(FP8_ERR_UNSUPPORTED_SHAPE, "rows and cols must each be <= 2^31");
    if ((rows * ((cols + 7) / 8)) > fp8mi::kMaxUnits)
        return fail(FP8_ERR_UNSUPPORTED_SHAPE, "tensor too large: more than 2^34 elements");
    return FP8_OK;
}

bool valid_gran(int g) {
    return g == FP8_GRAN_TENSOR || g == FP8_GRAN_ROW || g == FP8_GRAN_BLOCK_1x128 ||
           g == FP8_GRAN_BLOCK_128x128;
}

int64_t num_groups(int gran, int64_t rows, int64_t cols) {
    switch (gran) {
    case FP8_GRAN_TENSOR: return 1;
    case FP8_GRAN_ROW: return rows;
    case FP8_GRAN_BLOCK_1x128: return rows * ((cols + 127) / 128);
    default: return ((rows + 127) / 128) * ((cols + 127) / 128);
    }
}

}  // namespace

extern "C" {

int fp8_abi_version(void) { return FP8MI_ABI_VERSION; }

const char* fp8_status_string(fp8_status s) {
    switch (s) {
    case FP8_OK: return "FP8_OK";
    case FP8_ERR_INVALID_ARG: return "FP8_ERR_INVALID_ARG";
    case FP8_ERR_UNSUPPORTED_SHAPE: return "FP8_ERR_UNSUPPORTED_SHAPE";
    case FP8_ERR_MISALIGNED: return "FP8_ERR_MISALIGNED";
    case FP8_ERR_UNSUPPORTED_DEVICE: return "FP8_ERR_UNSUPPORTED_DEVICE";
    case FP8_ERR_HIP: return "FP8_ERR_HIP";
    }
    return "FP8_ERR_UNKNOWN";
}

const char* fp8_last_error(void) { return g_last_error.c_str(); }

int64_t fp8_workspace_size(void) { return FP8_WORKSPACE_BYTES; }

fp8_status fp8_history_init(fp8_amax_history* hist, int32_t len, void* stream) {
    if (hist == nullptr) return fail(FP8_ERR_INVALID_ARG, "hist is NULL");
    if (len < 1 || len > 16) return fail(FP8_ERR_INVALID_ARG, "history length %d not in 1..16", len);
    if (!is_aligned(hist, 16)) return fail(FP8_ERR_MISALIGNED, "hist must be 16-byte aligned");
    int cus = 0;
    fp8_status st = check_device(&cus);
    if (st != FP8_OK) return st;
    return launch_result(fp8mi::launch_history_init(hist, len, (hipStream_t)stream), "fp8_history_init");
}

fp8_status fp8_history_set_guard(fp8_amax_history* hist, float threshold, void* stream) {
    if (hist == nullptr) return fail(FP8_ERR_INVALID_ARG, "hist is NULL");
    if (!is_aligned(hist, 16)) return fail(FP8_ERR_MISALIGNED, "hist must be 16-byte aligned");
    int cus = 0;
    fp8_status st = check_device(&cus);
    if (st != FP8_OK) return st;
    return launch_result(fp8mi::launch_history_set_guard(hist, threshold, (hipStream_t)stream),
                         "fp8_history_set_guard");
}

fp8_status fp8_amax(const void* x, fp8_in_dtype in_dtype, int64_t rows, int64_t cols, int64_t ld,
                    fp8_granularity gran, float* amax_out, void* workspace, int64_t workspace_bytes,
                    void* stream) {
    fp8_status st = check_matrix_in(x, in_dtype, rows, cols, ld);
    if (st != FP8_OK) return st;
    if (!valid_gran(gran)) return fail(FP8_ERR_INVALID_ARG, "granularity %d is not a fp8_granularity", (int)gran);
    if (amax_out == nullptr && num_groups(gran, rows, cols) > 0)
        return fail(FP8_ERR_INVALID_ARG, "amax_out is NULL");
    if (!is_aligned(amax_out, 4)) return fail(FP8_ERR_MISALIGNED, "amax_out is not 4-byte aligned");
    uint32_t* scratch = nullptr;
    st = check_workspace(gran == FP8_GRAN_TENSOR, workspace, workspace_bytes, &scratch);
    if (st != FP8_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != FP8_OK) return st;
    if (num_groups(gran, rows, cols) == 0) return ok();
    fp8mi::QuantArgs a;
    a.x = x; a.in_bf16 = in_dtype == FP8_IN_BF16; a.rows = rows; a.cols = cols; a.ld = ld;
    a.gran = gran; a.write_q = false; a.amax = amax_out; a.ldq = cols; a.scratch = scratch;
    a.stream = (hipStream_t)stream; a.num_cus = cus;
    return launch_result(fp8mi::launch_quantize(a), "fp8_amax");
}

// fp8_quantize and fp8_quantize_dual (qt != nullptr: q untransposed plus qt
// transposed, per tensor).
static fp8_status quantize_impl(const char* what, const void* x, fp8_in_dtype in_dtype, int64_t rows, int64_t cols,
                                int64_t ld, fp8_format fmt, fp8_granularity gran, uint32_t flags,
                                fp8_amax_history* hist, uint8_t* q, int64_t ldq, uint8_t* qt, int64_t ldqt,
                                bool dual, float* scale_inv_out, float* amax_out, fp8_diag* diag,
                                void* workspace, int64_t workspace_bytes, void* stream) {
    fp8_status st = check_matrix_in(x, in_dtype, rows, cols, ld);
    if (st != FP8_OK) return st;
    if (fmt != FP8_E4M3 && fmt != FP8_E5M2)
        return fail(FP8_ERR_INVALID_ARG, "format %d is not FP8_E4M3 or FP8_E5M2", (int)fmt);
    if (!valid_gran(gran)) return fail(FP8_ERR_INVALID_ARG, "granularity %d is not a fp8_granularity", (int)gran);
    const uint32_t known = FP8_SCALE_POW2 | FP8_SPIKE_GUARD | (dual ? 0u : FP8_TRANSPOSE_OUT);
    if (flags & ~known) return fail(FP8_ERR_INVALID_ARG, "unknown flag bits 0x%x", flags & ~known);
    if ((flags & FP8_SPIKE_GUARD) && hist == nullptr)
        return fail(FP8_ERR_INVALID_ARG, "FP8_SPIKE_GUARD needs delayed scaling (hist != NULL)");
    const bool transpose = dual || (flags & FP8_TRANSPOSE_OUT) != 0;
    if (transpose && !dual && gran != FP8_GRAN_TENSOR)
        return fail(FP8_ERR_INVALID_ARG, "FP8_TRANSPOSE_OUT needs FP8_GRAN_TENSOR");
    if (hist != nullptr && gran != FP8_GRAN_TENSOR)
        return fail(FP8_ERR_INVALID_ARG, "delayed scaling (hist != NULL) needs FP8_GRAN_TENSOR");
    if (hist != nullptr && !is_aligned(hist, 16)) return fail(FP8_ERR_MISALIGNED, "hist must be 16-byte aligned");
    if (q == nullptr && rows > 0 && cols > 0) return fail(FP8_ERR_INVALID_ARG, "q is NULL");
    if (dual) {
        if (qt == nullptr && rows > 0 && cols > 0) return fail(FP8_ERR_INVALID_ARG, "qt is NULL");
        if (ldq < cols || ldq < 1)
            return fail(FP8_ERR_INVALID_ARG, "ldq=%lld must be >= cols=%lld", (long long)ldq, (long long)cols);
        if (ldqt < rows || ldqt < 1)
            return fail(FP8_ERR_INVALID_ARG, "ldqt=%lld must be >= rows=%lld", (long long)ldqt, (long long)rows);
    } else {
        const int64_t qcols = transpose ? rows : cols;
        if (ldq < qcols || ldq < 1)
            return fail(FP8_ERR_INVALID_ARG, "ldq=%lld must be >= %s=%lld", (long long)ldq,
                        transpose ? "rows (transposed output)" : "cols", (long long)qcols);
    }
    const int64_t ng = num_groups(gran, rows, cols);
    if (scale_inv_out == nullptr && ng > 0) return fail(FP8_ERR_INVALID_ARG, "scale_inv_out is NULL");
    if (amax_out == nullptr && ng > 0) return fail(FP8_ERR_INVALID_ARG, "amax_out is NULL");
    if (!is_aligned(scale_inv_out, 4) || !is_aligned(amax_out, 4))
        return fail(FP8_ERR_MISALIGNED, "scale_inv_out and amax_out must be 4-byte aligned");
    if (diag != nullptr && !is_aligned(diag, 4)) return fail(FP8_ERR_MISALIGNED, "diag must be 4-byte aligned");
    uint32_t* scratch = nullptr;
    st = check_workspace(gran == FP8_GRAN_TENSOR, workspace, workspace_bytes, &scratch);
    if (st != FP8_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != FP8_OK) return st;
    if (num_groups(gran, rows, cols) == 0) return ok();
    fp8mi::QuantArgs a;
    a.scratch = scratch;
    a.x = x; a.in_bf16 = in_dtype == FP8_IN_BF16; a.rows = rows; a.cols = cols; a.ld = ld;
    a.fmt = fmt; a.gran = gran; a.pow2 = (flags & FP8_SCALE_POW2) != 0; a.transpose = transpose;
    a.write_q = true; a.hist = hist; a.guard = (flags & FP8_SPIKE_GUARD) != 0;
    if (dual) {   // the kernel's main output is the transposed one
        a.q = qt; a.ldq = ldqt; a.q2 = q; a.ldq2 = ldq;
    } else {
        a.q = q; a.ldq = ldq;
    }
    a.scale_inv = scale_inv_out;
    a.amax = amax_out; a.diag = diag; a.stream = (hipStream_t)stream; a.num_cus = cus;
    return launch_result(fp8mi::launch_quantize(a), what);
}

fp8_status fp8_quantize(const void* x, fp8_in_dtype in_dtype, int64_t rows, int64_t cols, int64_t ld,
                        fp8_format fmt, fp8_granularity gran, uint32_t flags, fp8_amax_history* hist,
                        uint8_t* q, int64_t ldq, float* scale_inv_out, float* amax_out, fp8_diag* diag,
                        void* workspace, int64_t workspace_bytes, void* stream) {
    return quantize_impl("fp8_quantize", x, in_dtype, rows, cols, ld, fmt, gran, flags, hist, q, ldq, nullptr, 0,
                         false, scale_inv_out, amax_out, diag, workspace, workspace_bytes, stream);
}

fp8_status fp8_quantize_noalloc(const void* x, fp8_in_dtype in_dtype, int64_t rows, int64_t cols, int64_t ld,
                                fp8_format fmt, fp8_granularity gran, uint32_t flags, fp8_amax_history* hist,
                                uint8_t* q, int64_t ldq, float* scale_inv_out, float* amax_out, fp8_diag* diag,
                                void* stream) {
    int cus = 0;
    fp8_status st = check_device(&cus);
    if (st != FP8_OK) return st;
    uint32_t* ws = nullptr;
    const hipError_t e = fp8mi::static_workspace(&ws);
    if (e != hipSuccess)
        return fail(FP8_ERR_HIP, "fp8_quantize_noalloc: the device workspace's address: %s", hipGetErrorString(e));
    return quantize_impl("fp8_quantize_noalloc", x, in_dtype, rows, cols, ld, fmt, gran, flags, hist, q, ldq,
                         nullptr, 0, false, scale_inv_out, amax_out, diag, ws, FP8_WORKSPACE_BYTES, stream);
}

fp8_status fp8_quantize_dual(const void* x, fp8_in_dtype in_dtype, int64_t rows, int64_t cols, int64_t ld,
                             fp8_format fmt, uint32_t flags, fp8_amax_history* hist, uint8_t* q, int64_t ldq,
                             uint8_t* qt, int64_t ldqt, float* scale_inv_out, float* amax_out, fp8_diag* diag,
                             void* workspace, int64_t workspace_bytes, void* stream) {
    return quantize_impl("fp8_quantize_dual", x, in_dtype, rows, cols, ld, fmt, FP8_GRAN_TENSOR, flags, hist, q,
                         ldq, qt, ldqt, true, scale_inv_out, amax_out, diag, workspace, workspace_bytes, stream);
}

fp8_status fp8_quantize_tensors(const fp8_tensor* tensors, int32_t count, fp8_in_dtype in_dtype, fp8_format fmt,
                                uint32_t flags, void* workspace, int64_t workspace_bytes, void* stream) {
    if (tensors == nullptr) return fail(FP8_ERR_INVALID_ARG, "tensors is NULL");
    if (count < 1 || count > FP8_MAX_TENSORS)
        return fail(FP8_ERR_INVALID_ARG, "count=%d not in 1..%d", (int)count, FP8_MAX_TENSORS);
    if (in_dtype != FP8_IN_F32 && in_dtype != FP8_IN_BF16)
        return fail(FP8_ERR_INVALID_ARG, "in_dtype %d is not FP8_IN_F32 or FP8_IN_BF16", (int)in_dtype);
    if (fmt != FP8_E4M3 && fmt != FP8_E5M2)
        return fail(FP8_ERR_INVALID_ARG, "format %d is not FP8_E4M3 or FP8_E5M2", (int)fmt);
    if (flags & ~FP8_SCALE_POW2)
        return fail(FP8_ERR_INVALID_ARG, "unknown flag bits 0x%x (only FP8_SCALE_POW2 applies)",
                    flags & ~FP8_SCALE_POW2);
    fp8mi::MultiQuantArgs a;
    for (int t = 0; t < count; ++t) {
        const fp8_tensor& d = tensors[t];
        if (d.rows < 0 || d.cols < 0)
            return fail(FP8_ERR_INVALID_ARG, "tensor %d: negative size rows=%lld cols=%lld", t, (long long)d.rows,
                        (long long)d.cols);
        if (d.rows > (int64_t(1) << 31) || d.cols > (int64_t(1) << 31))
            return fail(FP8_ERR_UNSUPPORTED_SHAPE, "tensor %d: rows and cols must each be <= 2^31", t);
        const int64_t elems = d.rows * d.cols;
        if (elems / 8 > fp8mi::kMaxUnits)
            return fail(FP8_ERR_UNSUPPORTED_SHAPE, "tensor %d too large: more than 2^34 elements", t);
        if (elems > 0 && d.x == nullptr) return fail(FP8_ERR_INVALID_ARG, "tensor %d: x is NULL", t);
        if (elems > 0 && d.q == nullptr) return fail(FP8_ERR_INVALID_ARG, "tensor %d: q is NULL", t);
        if (d.scale_inv == nullptr) return fail(FP8_ERR_INVALID_ARG, "tensor %d: scale_inv is NULL", t);
        if (d.amax == nullptr) return fail(FP8_ERR_INVALID_ARG, "tensor %d: amax is NULL", t);
        if (!is_aligned(d.x, 16)) return fail(FP8_ERR_MISALIGNED, "tensor %d: x must be 16-byte aligned", t);
        if (!is_aligned(d.q, 8)) return fail(FP8_ERR_MISALIGNED, "tensor %d: q must be 8-byte aligned", t);
        if (!is_aligned(d.scale_inv, 4) || !is_aligned(d.amax, 4))
            return fail(FP8_ERR_MISALIGNED, "tensor %d: scale_inv and amax must be 4-byte aligned", t);
        if (d.diag != nullptr && !is_aligned(d.diag, 4))
            return fail(FP8_ERR_MISALIGNED, "tensor %d: diag must be 4-byte aligned", t);
        a.x[t] = d.x; a.elems[t] = elems; a.q[t] = d.q;
        a.scale_inv[t] = d.scale_inv; a.amax[t] = d.amax; a.diag[t] = d.diag;
    }
    uint32_t* scratch = nullptr;
    fp8_status st = check_workspace(true, workspace, workspace_bytes, &scratch);
    if (st != FP8_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != FP8_OK) return st;
    a.n = count; a.in_bf16 = in_dtype == FP8_IN_BF16; a.fmt = fmt; a.pow2 = (flags & FP8_SCALE_POW2) != 0;
    a.scratch = scratch; a.stream = (hipStream_t)stream; a.num_cus = cus;
    return launch_result(fp8mi::launch_quantize_multi(a), "fp8_quantize_tensors");
}

static fp8_status check_gemm_common(const uint8_t* A, int64_t lda, const uint8_t* B, int64_t ldb, int64_t M,
                                    int64_t N, int64_t K, const float* sa, const float* sb, void* C,
                                    int out_dtype, int64_t ldc) {
    if ((A == nullptr && M > 0 && K > 0) || (B == nullptr && N > 0 && K > 0))
        return fail(FP8_ERR_INVALID_ARG, "A or B is NULL");
    if (C == nullptr && M > 0 && N > 0) return fail(FP8_ERR_INVALID_ARG, "C is NULL");
    if ((sa == nullptr || sb == nullptr) && M > 0 && N > 0)
        return fail(FP8_ERR_INVALID_ARG, "a_scale_inv or b_scale_inv is NULL");
    if (out_dtype != FP8_OUT_F32 && out_dtype != FP8_OUT_BF16)
        return fail(FP8_ERR_INVALID_ARG, "out_dtype %d is not FP8_OUT_F32 or FP8_OUT_BF16", out_dtype);
    if (M < 0 || N < 0 || K < 0)
        return fail(FP8_ERR_INVALID_ARG, "negative size M=%lld N=%lld K=%lld", (long long)M, (long long)N,
                    (long long)K);
    if (M >= (int64_t(1) << 31) || N >= (int64_t(1) << 31) || K >= (int64_t(1) << 31))
        return fail(FP8_ERR_UNSUPPORTED_SHAPE, "M, N and K must each be < 2^31");
    if (K % 16 != 0) return fail(FP8_ERR_UNSUPPORTED_SHAPE, "K=%lld must be a multiple of 16", (long long)K);
    if (K > 0) {
        if (lda < K || ldb < K) return fail(FP8_ERR_INVALID_ARG, "lda and ldb must be >= K");
        if (!is_aligned(A, 16) || !is_aligned(B, 16))
            return fail(FP8_ERR_MISALIGNED, "A and B must be 16-byte aligned");
        if (lda % 16 != 0 || ldb % 16 != 0) return fail(FP8_ERR_MISALIGNED, "lda and ldb must be multiples of 16");
        // the loads address one 256-row tile through a 32-bit byte offset
        if (lda > (int64_t(1) << 23) || ldb > (int64_t(1) << 23))
            return fail(FP8_ERR_UNSUPPORTED_SHAPE, "lda and ldb must be <= 2^23 bytes");
    }
    if (ldc < N || ldc < 1) return fail(FP8_ERR_INVALID_ARG, "ldc=%lld must be >= N", (long long)ldc);
    if (!is_aligned(C, out_dtype == FP8_OUT_F32 ? 4 : 2))
        return fail(FP8_ERR_MISALIGNED, "C is not aligned to its element size");
    if (!is_aligned(sa, 4) || !is_aligned(sb, 4)) return fail(FP8_ERR_MISALIGNED, "scale arrays must be 4-byte aligned");
    const int64_t tiles = ((M + 255) / 256) * ((N + 127) / 128);
    if (tiles >= (int64_t(1) << 31)) return fail(FP8_ERR_UNSUPPORTED_SHAPE, "too many output tiles");
    return FP8_OK;
}

fp8_status fp8_scaled_gemm(const uint8_t* A, fp8_format fa, int64_t lda, const uint8_t* B, fp8_format fb,
                           int64_t ldb, int64_t M, int64_t N, int64_t K, const float* a_scale_inv,
                           int a_per_row, const float* b_scale_inv, int b_per_row, void* C,
                           fp8_out_dtype out_dtype, int64_t ldc, void* stream) {
    if ((fa != FP8_E4M3 && fa != FP8_E5M2) || (fb != FP8_E4M3 && fb != FP8_E5M2))
        return fail(FP8_ERR_INVALID_ARG, "formats fa=%d fb=%d must be FP8_E4M3 or FP8_E5M2", (int)fa, (int)fb);
    if ((a_per_row != 0 && a_per_row != 1) || (b_per_row != 0 && b_per_row != 1))
        return fail(FP8_ERR_INVALID_ARG, "a_per_row and b_per_row must be 0 or 1");
    fp8_status st = check_gemm_common(A, lda, B, ldb, M, N, K, a_scale_inv, b_scale_inv, C, out_dtype, ldc);
    if (st != FP8_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != FP8_OK) return st;
    if (M == 0 || N == 0) return ok();
    fp8mi::GemmArgs g;
    g.A = A; g.B = B; g.fa = fa; g.fb = fb; g.lda = lda; g.ldb = ldb; g.M = M; g.N = N; g.K = K;
    g.sa = a_scale_inv; g.sb = b_scale_inv; g.sa_per_row = a_per_row; g.sb_per_row = b_per_row;
    g.C = C; g.out_bf16 = out_dtype == FP8_OUT_BF16; g.ldc = ldc; g.stream = (hipStream_t)stream;
    g.num_cus = cus;
    return launch_result(fp8mi::launch_scaled_gemm(g), "fp8_scaled_gemm");
}

fp8_status fp8_blockscaled_gemm(const uint8_t* A, int64_t lda, const uint8_t* B, int64_t ldb, int64_t M, int64_t N,
                                int64_t K, const float* a_scale_inv, const float* b_scale_inv, void* C,
                                fp8_out_dtype out_dtype, int64_t ldc, void* stream) {
    fp8_status st = check_gemm_common(A, lda, B, ldb, M, N, K, a_scale_inv, b_scale_inv, C, out_dtype, ldc);
    if (st != FP8_OK) return st;
    if (K == 0 || K % 128 != 0 || N % 128 != 0)
        return fail(FP8_ERR_UNSUPPORTED_SHAPE, "block-scaled GEMM needs K > 0, K %% 128 == 0 and N %% 128 == 0 (K=%lld N=%lld)",
                    (long long)K, (long long)N);
    int cus = 0;
    st = check_device(&cus);
    if (st != FP8_OK) return st;
    if (M == 0 || N == 0) return ok();
    fp8mi::GemmArgs g;
    g.A = A; g.B = B; g.fa = FP8_E4M3; g.fb = FP8_E4M3; g.lda = lda; g.ldb = ldb; g.M = M; g.N = N; g.K = K;
    g.sa = a_scale_inv; g.sb = b_scale_inv; g.sa_per_row = true; g.sb_per_row = true;
    g.C = C; g.out_bf16 = out_dtype == FP8_OUT_BF16; g.ldc = ldc; g.stream = (hipStream_t)stream;
    g.num_cus = cus;
    return launch_result(fp8mi::launch_blockscaled_gemm(g), "fp8_blockscaled_gemm");
}

static_assert(FP8_GROUPED_MAX_TILES == fp8mi::kGroupTableTiles, "grouped GEMM table size");
static_assert(FP8_WORKSPACE_BYTES == 4 * fp8mi::kScratchWords, "workspace size");

fp8_status fp8_grouped_gemm(const uint8_t* A, fp8_format fa, int64_t lda, const uint8_t* B, fp8_format fb,
                            int64_t ldb, int64_t b_group_stride, int64_t M, int64_t N, int64_t K, int32_t groups,
                            const int32_t* group_offsets, const float* a_scale_inv, int a_per_row,
                            const float* b_scale_inv, int b_per_row, void* C, fp8_out_dtype out_dtype, int64_t ldc,
                            void* workspace, int64_t workspace_bytes, void* stream) {
    if ((fa != FP8_E4M3 && fa != FP8_E5M2) || (fb != FP8_E4M3 && fb != FP8_E5M2))
        return fail(FP8_ERR_INVALID_ARG, "formats fa=%d fb=%d must be FP8_E4M3 or FP8_E5M2", (int)fa, (int)fb);
    if ((a_per_row != 0 && a_per_row != 1) || (b_per_row != 0 && b_per_row != 1))
        return fail(FP8_ERR_INVALID_ARG, "a_per_row and b_per_row must be 0 or 1");
    fp8_status st = check_gemm_common(A, lda, B, ldb, M, N, K, a_scale_inv, b_scale_inv, C, out_dtype, ldc);
    if (st != FP8_OK) return st;
    if (groups < 1) return fail(FP8_ERR_INVALID_ARG, "groups=%d must be >= 1", (int)groups);
    if (group_offsets == nullptr) return fail(FP8_ERR_INVALID_ARG, "group_offsets is NULL");
    if (!is_aligned(group_offsets, 4)) return fail(FP8_ERR_MISALIGNED, "group_offsets must be 4-byte aligned");
    if (K > 0 && N > 0) {
        if (b_group_stride < (N - 1) * ldb + K)
            return fail(FP8_ERR_INVALID_ARG, "b_group_stride=%lld must be >= (N-1)*ldb + K = %lld",
                        (long long)b_group_stride, (long long)((N - 1) * ldb + K));
        if (b_group_stride % 16 != 0)
            return fail(FP8_ERR_MISALIGNED, "b_group_stride=%lld must be a multiple of 16", (long long)b_group_stride);
    }
    if ((M + 255) / 256 + groups > FP8_GROUPED_MAX_TILES)
        return fail(FP8_ERR_UNSUPPORTED_SHAPE, "ceil(M/256) + groups = %lld exceeds FP8_GROUPED_MAX_TILES (%d)",
                    (long long)((M + 255) / 256 + groups), FP8_GROUPED_MAX_TILES);
    uint32_t* scratch = nullptr;
    st = check_workspace(true, workspace, workspace_bytes, &scratch);
    if (st != FP8_OK) return st;
    int cus = 0;
    st = check_device(&cus);
    if (st != FP8_OK) return st;
    if (M == 0 || N == 0) return ok();
    fp8mi::GemmArgs g;
    g.A = A; g.B = B; g.fa = fa; g.fb = fb; g.lda = lda; g.ldb = ldb; g.M = M; g.N = N; g.K = K;
    g.sa = a_scale_inv; g.sb = b_scale_inv; g.sa_per_row = a_per_row; g.sb_per_row = b_per_row;
    g.C = C; g.out_bf16 = out_dtype == FP8_OUT_BF16; g.ldc = ldc; g.stream = (hipStream_t)stream;
    g.num_cus = cus; g.groups = groups; g.group_offsets = group_offsets; g.b_group_stride = b_group_stride;
    g.scratch = scratch;
    return launch_result(fp8mi::launch_grouped_gemm(g), "fp8_grouped_gemm");
}

// Shape and alignment rules shared by fp8_kv_store and fp8_kv_load.
static fp8_status check_kv_common(const void* cache, int storage, int scaling, const void* scale_inv,
                                  int64_t capacity, int32_t heads, int32_t head_dim, int64_t n_tokens) {
    if (storage != FP8_KV_E4M3 && storage != FP8_KV_E5M2 && storage != FP8_KV_BF16)
        return fail(FP8_ERR_INVALID_ARG, "storage %d is not FP8_KV_E4M3, FP8_KV_E5M2 or FP8_KV_BF16", storage);
    if (scaling != FP8_KV_PER_TOKEN_HEAD && scaling != FP8_KV_PER_HEAD)
        return fail(FP8_ERR_INVALID_ARG, "scaling %d is not FP8_KV_PER_TOKEN_HEAD or FP8_KV_PER_HEAD", scaling);
    if (n_tokens < 0 || capacity < 0 || heads < 0)
        return fail(FP8_ERR_INVALID_ARG, "negative size n_tokens=%lld capacity=%lld heads=%d",
                    (long long)n_tokens, (long long)capacity, (int)heads);
    if (head_dim < 8 || head_dim > 2048 || head_dim % 8 != 0)
        return fail(FP8_ERR_UNSUPPORTED_SHAPE, "head_dim=%d must be a multiple of 8 in 8..2048", (int)head_dim);
    if (heads > 0 && n_tokens >= (int64_t(1) << 31) / heads)
        return fail(FP8_ERR_UNSUPPORTED_SHAPE, "n_tokens * heads must be < 2^31");
    if (cache == nullptr && capacity > 0 && heads > 0) return fail(FP8_ERR_INVALID_ARG, "cache is NULL");
    if (!is_aligned(cache, 16)) return fail(FP8_ERR_MISALIGNED, "cache must be 16-byte aligned");
    if (storage != FP8_KV_BF16) {
        if (scale_inv == nullptr && heads > 0) return fail(FP8_ERR_INVALID_ARG, "scale_inv is NULL");
        if (!is_aligned(scale_inv, 4)) return fail(FP8_ERR_MISALIGNED, "scale_inv must be 4-byte aligned");
    }
    return FP8_OK;
}

fp8_status fp8_kv_store(const void* x, fp8_in_dtype in_dtype, int64_t n_tokens, int64_t ld, int32_t heads,
                        int32_t head_dim, const int64_t* slots, fp8_kv_storage storage, fp8_kv_scaling scaling,
                        uint32_t flags, void* cache, float* scale_inv, int64_t capacity, fp8_diag* diag,
                        void* stream) {
    fp8_status st = check_kv_common(cache, storage, scaling, scale_inv, capacity, heads, head_dim, n_tokens);
    if (st != FP8_OK) return st;
    if (in_dtype != FP8_IN_F32 && in_dtype != FP8_IN_BF16)
        return fail(FP8_ERR_INVALID_ARG, "in_dtype %d is not FP8_IN_F32 or FP8_IN_BF16", (int)in_dtype);
    if (flags & ~FP8_SCALE_POW2) return fail(FP8_ERR_INVALID_ARG, "unknown flag bits 0x%x", flags & ~FP8_SCALE_POW2);
    const int64_t width = (int64_t)heads * head_dim;
    if (ld < width || ld < 1)
        return fail(FP8_ERR_INVALID_ARG, "ld=%lld must be >= heads*head_dim=%lld", (long long)ld, (long long)width);
    if (ld % 8 != 0) return fail(FP8_ERR_MISALIGNED, "ld=%lld must be a multiple of 8", (long long)ld);
    if (x == nullptr && n_tokens > 0 && heads > 0) return fail(FP8_ERR_INVALID_ARG, "x is NULL");
    if (!is_aligned(x, 16)) return fail(FP8_ERR_MISALIGNED, "x must be 16-byte aligned");
    if (!is_aligned(slots, 8)) return fail(FP8_ERR_MISALIGNED, "slots must be 8-byte aligned");
    if (diag != nullptr && !is_aligned(diag, 4)) return fail(FP8_ERR_MISALIGNED, "diag must be 4-byte aligned");
    int cus = 0;
    st = check_device(&cus);
    if (st != FP8_OK) return st;
    if (n_tokens == 0 || heads == 0 || capacity == 0) return ok();
    fp8mi::KvStoreArgs a;
    a.x = x; a.in_bf16 = in_dtype == FP8_IN_BF16; a.n_tokens = n_tokens; a.ld = ld; a.heads = heads;
    a.head_dim = head_dim; a.slots = slots; a.capacity = capacity; a.storage = storage;
    a.per_head = scaling == FP8_KV_PER_HEAD; a.pow2 = (flags & FP8_SCALE_POW2) != 0; a.cache = cache;
    a.scale_inv = scale_inv; a.diag = storage == FP8_KV_BF16 ? nullptr : diag; a.stream = (hipStream_t)stream;
    return launch_result(fp8mi::launch_kv_store(a), "fp8_kv_store");
}

fp8_status fp8_kv_load(const void* cache, fp8_kv_storage storage, fp8_kv_scaling scaling, const float* scale_inv,
                       int64_t capacity, int32_t heads, int32_t head_dim, const int64_t* slots, int64_t n_tokens,
                       fp8_out_dtype out_dtype, void* out, int64_t ld_out, void* stream) {
    fp8_status st = check_kv_common(cache, storage, scaling, scale_inv, capacity, heads, head_dim, n_tokens);
    if (st != FP8_OK) return st;
    if (out_dtype != FP8_OUT_F32 && out_dtype != FP8_OUT_BF16)
        return fail(FP8_ERR_INVALID_ARG, "out_dtype %d is not FP8_OUT_F32 or FP8_OUT_BF16", (int)out_dtype);
    const int64_t width = (int64_t)heads * head_dim;
    if (ld_out < width || ld_out < 1)
        return fail(FP8_ERR_INVALID_ARG, "ld_out=%lld must be >= heads*head_dim=%lld", (long long)ld_out,
                    (long long)width);
    if (ld_out % 8 != 0) return fail(FP8_ERR_MISALIGNED, "ld_out=%lld must be a multiple of 8", (long long)ld_out);
    if (out == nullptr && n_tokens > 0 && heads > 0) return fail(FP8_ERR_INVALID_ARG, "out is NULL");
    if (!is_aligned(out, 16)) return fail(FP8_ERR_MISALIGNED, "out must be 16-byte aligned");
    if (!is_aligned(slots, 8)) return fail(FP8_ERR_MISALIGNED, "slots must be 8-byte aligned");
    int cus = 0;
    st = check_device(&cus);
    if (st != FP8_OK) return st;
    if (n_tokens == 0 || heads == 0 || capacity == 0) return ok();
    fp8mi::KvLoadArgs a;
    a.cache = cache; a.storage = storage; a.per_head = scaling == FP8_KV_PER_HEAD; a.scale_inv = scale_inv;
    a.capacity = capacity; a.heads = heads; a.head_dim = head_dim; a.slots = slots; a.n_tokens = n_tokens;
    a.out_bf16 = out_dtype == FP8_OUT_BF16; a.out = out; a.ld_out = ld_out; a.stream = (hipStream_t)stream;
    return launch_result(fp8mi::launch_kv_load(a), "fp8_kv_load");
}

// Shape and alignment rules of fp8_kv_attention and fp8_kv_evict.  `sizes`:
// sizes only (the workspace query reads no pointer).
static_assert(sizeof(fp8_kv_pair) == 104, "fp8_kv_pair layout");

static fp8_status check_kv_pair(const fp8_kv_pair* c, bool sizes, fp8mi::KvView* out) {
    if (c == nullptr) return fail(FP8_ERR_INVALID_ARG, "cache is NULL");
    if (c->reserved != 0) return fail(FP8_ERR_INVALID_ARG, "reserved=%d must be 0", (int)c->reserved);
    if (c->head_dim % 16 != 0 || c->head_dim < 16 || c->head_dim > 256)
        return fail(FP8_ERR_UNSUPPORTED_SHAPE, "head_dim=%d must be a multiple of 16 in 16..256", (int)c->head_dim);
    if (c->heads < 1 || c->heads > 65535)
        return fail(FP8_ERR_INVALID_ARG, "heads=%d must be in 1..65535", (int)c->heads);
    if (c->batch < 0 || c->max_len < 0)
        return fail(FP8_ERR_INVALID_ARG, "negative size batch=%d max_len=%lld", (int)c->batch, (long long)c->max_len);
    if (c->batch > 65535) return fail(FP8_ERR_UNSUPPORTED_SHAPE, "batch=%d must be <= 65535", (int)c->batch);
    if (c->max_len >= (int64_t(1) << 30) || c->capacity >= (int64_t(1) << 31))
        return fail(FP8_ERR_UNSUPPORTED_SHAPE, "max_len must be < 2^30 and capacity < 2^31");
    const int32_t ps = c->page_size;
    if (ps < 1 || ps > (1 << 20) || (ps & (ps - 1)) != 0)
        return fail(FP8_ERR_UNSUPPORTED_SHAPE, "page_size=%d must be a power of two <= 2^20", (int)ps);
    const int64_t pages = (c->max_len + ps - 1) / ps;
    if (c->page_ld < pages)
        return fail(FP8_ERR_INVALID_ARG, "page_ld=%lld must be >= max_len / page_size = %lld", (long long)c->page_ld,
                    (long long)pages);
    if (!sizes) {
        // a cache without rows has no per-(token, head) scales
        static const float none = 0.0f;
        const float* least = c->capacity == 0 && c->scaling == FP8_KV_PER_TOKEN_HEAD ? &none : nullptr;
        fp8_status st = check_kv_common(c->k, c->k_storage, c->scaling, c->k_scale_inv ? c->k_scale_inv : least,
                                        c->capacity, c->heads, c->head_dim, 0);
        if (st != FP8_OK) return st;
        st = check_kv_common(c->v, c->v_storage, c->scaling, c->v_scale_inv ? c->v_scale_inv : least, c->capacity,
                             c->heads, c->head_dim, 0);
        if (st != FP8_OK) return st;
        if (c->batch > 0 && c->lens == nullptr) return fail(FP8_ERR_INVALID_ARG, "lens is NULL");
        if (c->batch > 0 && pages > 0 && c->page_table == nullptr)
            return fail(FP8_ERR_INVALID_ARG, "page_table is NULL");
        if (!is_aligned(c->lens, 4) || !is_aligned(c->page_table, 4))
            return fail(FP8_ERR_MISALIGNED, "lens and page_table must be 4-byte aligned");
    }
    out->k = c->k; out->v = c->v;
    out->k_scale = c->k_storage == FP8_KV_BF16 ? nullptr : c->k_scale_inv;
    out->v_scale = c->v_storage == FP8_KV_BF16 ? nullptr : c->v_scale_inv;
    out->k_st = c->k_storage; out->v_st = c->v_storage; out->per_head = c->scaling == FP8_KV_PER_HEAD;
    out->heads = c->heads; out->head_dim = c->head_dim; out->capacity = c->capacity;
    out->table = c->page_table; out->table_ld = c->page_ld; out->page_shift = __builtin_ctz((unsigned)ps);
    out->lens = c->lens; out->batch = c->batch; out->max_len = c->max_len;
    return FP8_OK;
}

fp8_status fp8_kv_append(const fp8_kv_pair* cache, const void* k, int64_t ldk, const void* v, int64_t ldv,
                         const void* q, int64_t ldq, int32_t q_heads, void* q_out, int64_t ldqo,
                         fp8_in_dtype in_dtype, int64_t n_tokens, const int64_t* slots, const int64_t* positions,
                         int64_t pos_ld, const int32_t* sections, int32_t axes, const float* inv_freq,
                         int32_t rotary_dim, uint32_t flags, fp8_diag* diag, void* stream) {
    if (cache == nullptr) return fail(FP8_ERR_INVALID_ARG, "cache is NULL");
    fp8_kv_pair caches = *cache;
    caches.page_table = nullptr; caches.page_ld = 0; caches.lens = nullptr; caches.max_len = 0;
    caches.page_size = 1; caches.batch = 0; caches.reserved = 0;
    fp8mi::KvAppendArgs a;
    fp8_status st = check_kv_pair(&caches, false, &a.kv);
    if (st != FP8_OK) return st;
    if (in_dtype != FP8_IN_F32 && in_dtype != FP8_IN_BF16)
        return fail(FP8_ERR_INVALID_ARG, "in_dtype %d is not FP8_IN_F32 or FP8_IN_BF16", (int)in_dtype);
    if (flags & ~(FP8_SCALE_POW2 | FP8_ROTARY_INTERLEAVED))
        return fail(FP8_ERR_INVALID_ARG, "unknown flag bits 0x%x", flags & ~(FP8_SCALE_POW2 | FP8_ROTARY_INTERLEAVED));
    if (n_tokens < 0 || q_heads < 0)
        return fail(FP8_ERR_INVALID_ARG, "negative size n_tokens=%lld q_heads=%d", (long long)n_tokens, (int)q_heads);
    if (q_heads > 65535) return fail(FP8_ERR_UNSUPPORTED_SHAPE, "q_heads=%d must be <= 65535", (int)q_heads);
    const int64_t heads = cache->heads, D = cache->head_dim;
    // a block has 16 rows or more: a launch stays below 2^32 threads
    if (n_tokens >= (int64_t(1) << 27) / (q_heads + 2 * heads))
        return fail(FP8_ERR_UNSUPPORTED_SHAPE, "n_tokens * (q_heads + 2 * heads) must be < 2^27");
    if (ldk < heads * D || ldv < heads * D || (q_heads > 0 && (ldq < q_heads * D || ldqo < q_heads * D)))
        return fail(FP8_ERR_INVALID_ARG,
                    "ldk=%lld and ldv=%lld must be >= heads*head_dim=%lld, ldq=%lld and ldqo=%lld >= q_heads*head_dim=%lld",
                    (long long)ldk, (long long)ldv, (long long)(heads * D), (long long)ldq, (long long)ldqo,
                    (long long)(q_heads * D));
    if (ldk % 8 != 0 || ldv % 8 != 0 || (q_heads > 0 && (ldq % 8 != 0 || ldqo % 8 != 0)))
        return fail(FP8_ERR_MISALIGNED, "ldk=%lld, ldv=%lld, ldq=%lld and ldqo=%lld must be multiples of 8",
                    (long long)ldk, (long long)ldv, (long long)ldq, (long long)ldqo);
    if (n_tokens > 0 && (k == nullptr || v == nullptr)) return fail(FP8_ERR_INVALID_ARG, "k or v is NULL");
    if (q_heads == 0 && (q != nullptr || q_out != nullptr))
        return fail(FP8_ERR_INVALID_ARG, "q or q_out is given with q_heads=0");
    if (n_tokens > 0 && q_heads > 0 && (q == nullptr || q_out == nullptr))
        return fail(FP8_ERR_INVALID_ARG, "q or q_out is NULL");
    if (q_out != nullptr && q_out == q && (in_dtype != FP8_IN_BF16 || ldqo != ldq))
        return fail(FP8_ERR_INVALID_ARG, "q_out is q, which needs bf16 and ldqo=%lld equal to ldq=%lld",
                    (long long)ldqo, (long long)ldq);
    if (!is_aligned(k, 16) || !is_aligned(v, 16) || !is_aligned(q, 16) || !is_aligned(q_out, 16))
        return fail(FP8_ERR_MISALIGNED, "q, k, v and q_out must be 16-byte aligned");
    if (cache->k == cache->v && cache->capacity > 0)
        return fail(FP8_ERR_INVALID_ARG, "the K and V caches are one array");
    if (!is_aligned(slots, 8) || !is_aligned(positions, 8))
        return fail(FP8_ERR_MISALIGNED, "slots and positions must be 8-byte aligned");
    if (!is_aligned(inv_freq, 4) || !is_aligned(diag, 4))
        return fail(FP8_ERR_MISALIGNED, "inv_freq and diag must be 4-byte aligned");
    if (rotary_dim < 0 || rotary_dim > D || rotary_dim % 16 != 0)
        return fail(FP8_ERR_UNSUPPORTED_SHAPE, "rotary_dim=%d must be a multiple of 16 in 0..head_dim=%lld",
                    (int)rotary_dim, (long long)D);
    if (rotary_dim > 0) {
        if (axes < 1 || axes > 4) return fail(FP8_ERR_UNSUPPORTED_SHAPE, "axes=%d must be in 1..4", (int)axes);
        if (inv_freq == nullptr) return fail(FP8_ERR_INVALID_ARG, "inv_freq is NULL");
        if (n_tokens > 0 && positions == nullptr) return fail(FP8_ERR_INVALID_ARG, "positions is NULL");
        if (axes > 1 && pos_ld != 0 && pos_ld < n_tokens)
            return fail(FP8_ERR_INVALID_ARG, "pos_ld=%lld must be 0 or >= n_tokens=%lld", (long long)pos_ld,
                        (long long)n_tokens);
        if (sections == nullptr && axes > 1) return fail(FP8_ERR_INVALID_ARG, "sections is NULL with axes=%d", (int)axes);
        int64_t pairs = 0;
        for (int i = 0; i < axes; ++i) {
            a.sections[i] = sections ? sections[i] : rotary_dim / 2;
            if (a.sections[i] < 0) return fail(FP8_ERR_INVALID_ARG, "sections[%d]=%d must be >= 0", i, a.sections[i]);
            pairs += a.sections[i];
        }
        if (pairs != rotary_dim / 2)
            return fail(FP8_ERR_INVALID_ARG, "sections hold %lld pairs, rotary_dim/2 is %d", (long long)pairs,
                        (int)(rotary_dim / 2));
        a.axes = axes;
    }
    int cus = 0;
    st = check_device(&cus);
    if (st != FP8_OK) return st;
    if (n_tokens == 0) return ok();
    a.q = q; a.k = k; a.v = v; a.in_bf16 = in_dtype == FP8_IN_BF16; a.ldq = ldq; a.ldk = ldk; a.ldv = ldv;
    a.q_heads = q_heads; a.q_out = static_cast<uint16_t*>(q_out); a.ldqo = ldqo; a.n_tokens = n_tokens;
    a.slots = slots; a.positions = positions; a.pos_ld = pos_ld; a.inv_freq = inv_freq; a.rotary = rotary_dim;
    a.interleaved = (flags & FP8_ROTARY_INTERLEAVED) != 0; a.pow2 = (flags & FP8_SCALE_POW2) != 0;
    a.diag = diag; a.stream = (hipStream_t)stream; a.num_cus = cus;
    return launch_result(fp8mi::launch_kv_append(a), "fp8_kv_append");
}

static bool one_each(const fp8mi::AttnArgs& a, bool ragged) { return !ragged && a.total_q == a.kv.batch; }

static fp8_status attention_args(const fp8_kv_pair* cache, bool sizes, int64_t total_q, int32_t q_heads, bool ragged,
                                 int32_t window, int32_t sinks, bool weighted, int64_t shared, fp8mi::AttnArgs* a) {
    fp8_status st = check_kv_pair(cache, sizes, &a->kv);
    if (st != FP8_OK) return st;
    if (total_q < 0) return fail(FP8_ERR_INVALID_ARG, "negative size total_q=%lld", (long long)total_q);
    if (q_heads < 1 || q_heads % cache->heads != 0)
        return fail(FP8_ERR_INVALID_ARG, "q_heads=%d must be a multiple of heads=%d", (int)q_heads,
                    (int)cache->heads);
    // rows are counted in 32 bits, rounded up to a tile of 128 and one more
    if (total_q >= (int64_t(1) << 30) || total_q > ((int64_t(1) << 31) - 256) / q_heads || q_heads > 65535)
        return fail(FP8_ERR_UNSUPPORTED_SHAPE,
                    "total_q must be < 2^30, total_q * q_heads <= 2^31 - 256 and q_heads <= 65535");
    // blocks of the launches
    if ((int64_t)cache->batch * cache->heads >= (int64_t(1) << 30) ||
        (cache->max_len / 128 + 1) * cache->heads >= (int64_t(1) << 31))
        return fail(FP8_ERR_UNSUPPORTED_SHAPE, "batch * heads must be < 2^30 and max_len / 128 * heads < 2^31");
    if (total_q > 0 && cache->batch == 0) return fail(FP8_ERR_INVALID_ARG, "total_q=%lld with batch=0", (long long)total_q);
    if (!ragged && cache->batch > 0 && total_q % cache->batch != 0)
        return fail(FP8_ERR_INVALID_ARG, "total_q=%lld must be a multiple of batch=%d without q_offsets",
                    (long long)total_q, (int)cache->batch);
    if (window < 0 || sinks < 0)
        return fail(FP8_ERR_INVALID_ARG, "window=%d and sinks=%d must be >= 0", (int)window, (int)sinks);
    if (cache->batch * cache->max_len >= (int64_t(1) << 35))
        return fail(FP8_ERR_UNSUPPORTED_SHAPE, "batch * max_len must be < 2^35");
    if (shared < 0 || shared > cache->max_len)
        return fail(FP8_ERR_INVALID_ARG, "shared=%lld must be in 0..max_len=%lld", (long long)shared,
                    (long long)cache->max_len);
    a->total_q = total_q; a->q_heads = q_heads; a->weighted = weighted;
    if (cache->capacity == 0) a->kv.max_len = 0;    // a cache without rows holds no token
    // a window that reaches every token is none; sinks past the end are all
    a->window = window >= cache->max_len ? 0 : window;
    a->sinks = sinks > cache->max_len ? (int)cache->max_len : sinks;
    // the prefix in whole steps, the rest of it with the sequences' own tokens; a
    // window sees little of it, and one sequence has nobody to share it with
    if (a->window == 0 && cache->batch > 1 && a->kv.max_len > 0) a->from = (int)(shared / 64 * 64);
    if (total_q > 0) {
        const int64_t blocks = a->from > 0           ? fp8mi::shared_blocks(*a, ragged)
                               : one_each(*a, ragged) ? fp8mi::decode_blocks(*a)
                                                      : fp8mi::extend_blocks(*a, ragged);
        if (blocks > fp8mi::kMaxAttnBlocks)
            return fail(FP8_ERR_UNSUPPORTED_SHAPE,
                        "%lld blocks (row tiles * heads, with weights also max_len / 128 * heads) must be < 2^24",
                        (long long)blocks);
    }
    return FP8_OK;
}


static int64_t attention_bytes(const fp8mi::AttnArgs& a, bool ragged) {
    if (a.total_q == 0) return 0;
    if (a.from > 0) return fp8mi::shared_workspace(a, ragged);
    return one_each(a, ragged) ? fp8mi::decode_workspace(a) : fp8mi::extend_workspace(a, ragged);
}

int64_t fp8_kv_attention_shared_workspace(const fp8_kv_pair* cache, int64_t total_q, int32_t q_heads, int32_t ragged,
                                          int32_t window, int32_t sinks, int32_t weighted, int64_t shared) {
    fp8mi::AttnArgs a;
    if (attention_args(cache, true, total_q, q_heads, ragged != 0, window, sinks, weighted != 0, shared, &a) != FP8_OK)
        return -1;
    ok();
    return attention_bytes(a, ragged != 0);
}

int64_t fp8_kv_attention_workspace(const fp8_kv_pair* cache, int64_t total_q, int32_t q_heads, int32_t ragged,
                                   int32_t window, int32_t sinks, int32_t weighted) {
    return fp8_kv_attention_shared_workspace(cache, total_q, q_heads, ragged, window, sinks, weighted, 0);
}

static fp8_status attention(const fp8_kv_pair* cache, const void* q, int64_t ldq, int64_t total_q, int32_t q_heads,
                            const int32_t* q_offsets, float scale, int32_t window, int32_t sinks, int64_t shared,
                            void* out, int64_t ldo, float* lse, float* weights, int64_t ldw, void* workspace,
                            int64_t workspace_bytes, void* stream, const char* what) {
    fp8mi::AttnArgs a;
    const bool ragged = q_offsets != nullptr;
    fp8_status st =
        attention_args(cache, false, total_q, q_heads, ragged, window, sinks, weights != nullptr, shared, &a);
    if (st != FP8_OK) return st;
    const int64_t width = (int64_t)q_heads * cache->head_dim;
    if (ldq < width || ldo < width)
        return fail(FP8_ERR_INVALID_ARG, "ldq=%lld and ldo=%lld must be >= q_heads*head_dim=%lld", (long long)ldq,
                    (long long)ldo, (long long)width);
    if (ldq % 8 != 0 || ldo % 8 != 0)
        return fail(FP8_ERR_MISALIGNED, "ldq=%lld and ldo=%lld must be multiples of 8", (long long)ldq,
                    (long long)ldo);
    if (total_q > 0 && q == nullptr) return fail(FP8_ERR_INVALID_ARG, "q is NULL");
    if (total_q > 0 && out == nullptr) return fail(FP8_ERR_INVALID_ARG, "out is NULL");
    if (!is_aligned(q, 16) || !is_aligned(out, 16))
        return fail(FP8_ERR_MISALIGNED, "q and out must be 16-byte aligned");
    if (!is_aligned(q_offsets, 4) || !is_aligned(lse, 4) || !is_aligned(weights, 4))
        return fail(FP8_ERR_MISALIGNED, "q_offsets, lse and weights must be 4-byte aligned");
    if (!(scale > -3.4e38f && scale < 3.4e38f)) return fail(FP8_ERR_INVALID_ARG, "scale must be finite");
    if (weights != nullptr && lse == nullptr) return fail(FP8_ERR_INVALID_ARG, "lse is NULL (weights need it)");
    if (weights != nullptr && ldw < cache->max_len)
        return fail(FP8_ERR_INVALID_ARG, "ldw=%lld must be >= max_len=%lld", (long long)ldw,
                    (long long)cache->max_len);
    const int64_t need = attention_bytes(a, ragged);
    if (need > 0) {
        if (workspace == nullptr)
            return fail(FP8_ERR_INVALID_ARG, "workspace is NULL (this call needs %lld bytes)", (long long)need);
        if (workspace_bytes < need)
            return fail(FP8_ERR_INVALID_ARG, "workspace_bytes=%lld is below the %lld this call needs",
                        (long long)workspace_bytes, (long long)need);
        if (!is_aligned(workspace, 16)) return fail(FP8_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    }
    int cus = 0;
    st = check_device(&cus);
    if (st != FP8_OK) return st;
    if (total_q == 0) return ok();
    a.q = static_cast<const uint16_t*>(q); a.ldq = ldq; a.q_offsets = q_offsets; a.scale = scale;
    a.out = static_cast<uint16_t*>(out); a.ldo = ldo; a.lse = lse; a.weights = weights; a.ldw = ldw;
    a.workspace = static_cast<uint8_t*>(workspace); a.stream = (hipStream_t)stream;
    return launch_result(a.from > 0           ? fp8mi::launch_shared(a)
                         : one_each(a, ragged) ? fp8mi::launch_decode(a)
                                               : fp8mi::launch_extend(a),
                         what);
}

fp8_status fp8_kv_attention(const fp8_kv_pair* cache, const void* q, int64_t ldq, int64_t total_q, int32_t q_heads,
                            const int32_t* q_offsets, float scale, int32_t window, int32_t sinks, void* out,
                            int64_t ldo, float* lse, float* weights, int64_t ldw, void* workspace,
                            int64_t workspace_bytes, void* stream) {
    return attention(cache, q, ldq, total_q, q_heads, q_offsets, scale, window, sinks, 0, out, ldo, lse, weights, ldw,
                     workspace, workspace_bytes, stream, "fp8_kv_attention");
}

fp8_status fp8_kv_attention_shared(const fp8_kv_pair* cache, const void* q, int64_t ldq, int64_t total_q,
                                   int32_t q_heads, const int32_t* q_offsets, float scale, int32_t window,
                                   int32_t sinks, int64_t shared, void* out, int64_t ldo, float* lse, float* weights,
                                   int64_t ldw, void* workspace, int64_t workspace_bytes, void* stream) {
    return attention(cache, q, ldq, total_q, q_heads, q_offsets, scale, window, sinks, shared, out, ldo, lse, weights,
                     ldw, workspace, workspace_bytes, stream, "fp8_kv_attention_shared");
}

fp8_status fp8_kv_evict(const fp8_kv_pair* cache, float* weights, int64_t ldw, int32_t budget, int32_t sinks,
                        int32_t recent, const int32_t* dst_page_table, int64_t dst_page_ld, float* weights_out,
                        int64_t ldwo, int32_t* kept, int32_t* new_lens, void* stream) {
    fp8mi::EvictArgs a;
    fp8_status st = check_kv_pair(cache, false, &a.kv);
    if (st != FP8_OK) return st;
    if (budget < 1) return fail(FP8_ERR_INVALID_ARG, "budget=%d must be >= 1", (int)budget);
    // positions advance by whole blocks and grids past the budget in 32 bits
    if (budget >= 1 << 30) return fail(FP8_ERR_UNSUPPORTED_SHAPE, "budget=%d must be < 2^30", (int)budget);
    if (sinks < 0 || recent < 0 || (int64_t)sinks + recent > budget)
        return fail(FP8_ERR_INVALID_ARG, "sinks=%d and recent=%d must be >= 0 and together <= budget=%d", (int)sinks,
                    (int)recent, (int)budget);
    if (cache->batch > 0 && weights == nullptr) return fail(FP8_ERR_INVALID_ARG, "weights is NULL");
    if (ldw < cache->max_len || ldw < 1)
        return fail(FP8_ERR_INVALID_ARG, "ldw=%lld must be >= max(max_len, 1)=%lld", (long long)ldw,
                    (long long)cache->max_len);
    if (weights_out != nullptr && weights_out != weights && ldwo < budget)
        return fail(FP8_ERR_INVALID_ARG, "ldwo=%lld must be >= budget=%d", (long long)ldwo, (int)budget);
    if (weights_out == weights && weights_out != nullptr && ldwo != ldw)
        return fail(FP8_ERR_INVALID_ARG, "ldwo=%lld must be ldw=%lld when weights_out is weights", (long long)ldwo,
                    (long long)ldw);
    if (dst_page_table != nullptr) {
        if (dst_page_ld < 1 || dst_page_ld < ((int64_t)budget + cache->page_size - 1) / cache->page_size)
            return fail(FP8_ERR_INVALID_ARG, "dst_page_ld=%lld holds fewer than budget=%d tokens",
                        (long long)dst_page_ld, (int)budget);
        if (dst_page_table == cache->page_table)
            return fail(FP8_ERR_INVALID_ARG, "dst_page_table is page_table (NULL moves in place)");
    }
    if (cache->batch > 0 && kept == nullptr) return fail(FP8_ERR_INVALID_ARG, "kept is NULL");
    if (cache->batch > 0 && new_lens == nullptr) return fail(FP8_ERR_INVALID_ARG, "new_lens is NULL");
    if (new_lens != nullptr && new_lens == cache->lens)
        return fail(FP8_ERR_INVALID_ARG, "new_lens is lens (which the call still reads)");
    if (!is_aligned(weights, 4) || !is_aligned(weights_out, 4) || !is_aligned(kept, 4) || !is_aligned(new_lens, 4) ||
        !is_aligned(dst_page_table, 4))
        return fail(FP8_ERR_MISALIGNED, "weights, weights_out, kept, new_lens and dst_page_table must be 4-byte aligned");
    int cus = 0;
    st = check_device(&cus);
    if (st != FP8_OK) return st;
    if (cache->batch == 0) return ok();
    a.weights = weights; a.ldw = ldw;
    a.weights_out = weights_out ? weights_out : weights; a.ldwo = weights_out ? ldwo : ldw;
    a.budget = budget; a.sinks = sinks; a.recent = recent; a.dst_table = dst_page_table; a.dst_ld = dst_page_ld;
    a.kept = kept; a.new_lens = new_lens; a.stream = (hipStream_t)stream;
    return launch_result(fp8mi::launch_evict(a), "fp8_kv_evict");
}

static fp8_status lora_args(int64_t rows, int64_t columns, int64_t inner, int32_t rank, int32_t adapters, int32_t slices,
                            fp8mi::LoraArgs* a) {
    if (rows < 0 || columns < 0 || inner < 0)
        return fail(FP8_ERR_INVALID_ARG, "negative size rows=%lld columns=%lld inner=%lld", (long long)rows,
                    (long long)columns, (long long)inner);
    if (rank < 8 || rank > 128 || rank % 8 != 0)
        return fail(FP8_ERR_UNSUPPORTED_SHAPE, "rank=%d must be a multiple of 8 in 8..128", (int)rank);
    if (slices < 1 || slices > 4) return fail(FP8_ERR_UNSUPPORTED_SHAPE, "slices=%d must be in 1..4", (int)slices);
    if (adapters < 1 || adapters > (1 << 20))
        return fail(FP8_ERR_UNSUPPORTED_SHAPE, "adapters=%d must be in 1..2^20", (int)adapters);
    if (inner % 8 != 0 || columns % 8 != 0)
        return fail(FP8_ERR_UNSUPPORTED_SHAPE, "inner=%lld and columns=%lld must be multiples of 8", (long long)inner,
                    (long long)columns);
    if (inner >= (1 << 24) || columns >= (1 << 24) || rows >= (1 << 30))
        return fail(FP8_ERR_UNSUPPORTED_SHAPE, "inner and columns must be < 2^24 and rows < 2^30");
    a->rows = rows; a->columns = columns; a->inner = inner; a->rank = rank; a->adapters = adapters; a->slices = slices;
    if (rows > 0 && fp8mi::lora_blocks(*a) >= (1 << 24))
        return fail(FP8_ERR_UNSUPPORTED_SHAPE, "rows=%lld times columns=%lld need 2^24 blocks or more", (long long)rows,
                    (long long)columns);
    return FP8_OK;
}

int64_t fp8_lora_workspace(int64_t rows, int64_t columns, int64_t inner, int32_t rank, int32_t adapters,
                           int32_t slices) {
    fp8mi::LoraArgs a;
    if (lora_args(rows, columns, inner, rank, adapters, slices, &a) != FP8_OK) return -1;
    ok();
    return fp8mi::lora_workspace(a);
}

fp8_status fp8_lora_add(const void* y, int64_t ldy, const void* x, int64_t ldx, const void* a_, const void* b,
                        const int32_t* ids, const float* gain, void* out, int64_t ldo, fp8_out_dtype dtype,
                        int64_t rows, int64_t columns, int64_t inner, int32_t rank, int32_t adapters,
                        const int32_t* slice_columns, int32_t slices, void* workspace, int64_t workspace_bytes,
                        void* stream) {
    fp8mi::LoraArgs a;
    fp8_status st = lora_args(rows, columns, inner, rank, adapters, slices, &a);
    if (st != FP8_OK) return st;
    if (dtype != FP8_OUT_F32 && dtype != FP8_OUT_BF16)
        return fail(FP8_ERR_INVALID_ARG, "dtype %d is not FP8_OUT_F32 or FP8_OUT_BF16", (int)dtype);
    if (slice_columns == nullptr && slices > 1)
        return fail(FP8_ERR_INVALID_ARG, "slice_columns is NULL with slices=%d", (int)slices);
    int64_t sum = 0;
    for (int i = 0; i < slices; ++i) {
        a.columns_of[i] = slice_columns ? slice_columns[i] : (int)columns;
        if (a.columns_of[i] < 0 || a.columns_of[i] % 8 != 0)
            return fail(FP8_ERR_UNSUPPORTED_SHAPE, "slice_columns[%d]=%d must be a multiple of 8, >= 0", i, a.columns_of[i]);
        sum += a.columns_of[i];
    }
    if (sum != columns)
        return fail(FP8_ERR_INVALID_ARG, "slice_columns add up to %lld, columns is %lld", (long long)sum,
                    (long long)columns);
    if (ldx < inner || ldy < columns || ldo < columns)
        return fail(FP8_ERR_INVALID_ARG, "ldx=%lld must be >= inner=%lld, ldy=%lld and ldo=%lld >= columns=%lld",
                    (long long)ldx, (long long)inner, (long long)ldy, (long long)ldo, (long long)columns);
    if (ldx % 8 != 0 || ldy % 8 != 0 || ldo % 8 != 0)
        return fail(FP8_ERR_MISALIGNED, "ldx=%lld, ldy=%lld and ldo=%lld must be multiples of 8", (long long)ldx,
                    (long long)ldy, (long long)ldo);
    if (rows > 0 && columns > 0) {
        if (y == nullptr || out == nullptr) return fail(FP8_ERR_INVALID_ARG, "y or out is NULL");
        if (inner > 0 && x == nullptr) return fail(FP8_ERR_INVALID_ARG, "x is NULL");
        if (inner > 0 && a_ == nullptr) return fail(FP8_ERR_INVALID_ARG, "a is NULL");
        if (b == nullptr) return fail(FP8_ERR_INVALID_ARG, "b is NULL");
        if (ids == nullptr) return fail(FP8_ERR_INVALID_ARG, "ids is NULL");
    }
    if (out == y && ldo != ldy)
        return fail(FP8_ERR_INVALID_ARG, "out is y, which needs ldo=%lld equal to ldy=%lld", (long long)ldo,
                    (long long)ldy);
    if (!is_aligned(x, 16) || !is_aligned(a_, 16) || !is_aligned(b, 16) || !is_aligned(y, 16) || !is_aligned(out, 16))
        return fail(FP8_ERR_MISALIGNED, "x, a, b, y and out must be 16-byte aligned");
    if (!is_aligned(ids, 4) || !is_aligned(gain, 4))
        return fail(FP8_ERR_MISALIGNED, "ids and gain must be 4-byte aligned");
    const int64_t need = fp8mi::lora_workspace(a);
    if (need > 0) {
        if (workspace == nullptr)
            return fail(FP8_ERR_INVALID_ARG, "workspace is NULL (this call needs %lld bytes)", (long long)need);
        if (workspace_bytes < need)
            return fail(FP8_ERR_INVALID_ARG, "workspace_bytes=%lld is below the %lld this call needs",
                        (long long)workspace_bytes, (long long)need);
        if (!is_aligned(workspace, 16)) return fail(FP8_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    }
    int cus = 0;
    st = check_device(&cus);
    if (st != FP8_OK) return st;
    if (rows == 0 || columns == 0) return ok();
    a.x = static_cast<const uint16_t*>(x); a.ldx = ldx; a.a = static_cast<const uint16_t*>(a_);
    a.b = static_cast<const uint16_t*>(b); a.ids = ids; a.gain = gain; a.y = y; a.ldy = ldy; a.out = out; a.ldo = ldo;
    a.out_bf16 = dtype == FP8_OUT_BF16; a.workspace = static_cast<uint8_t*>(workspace); a.stream = (hipStream_t)stream;
    return launch_result(fp8mi::launch_lora(a), "fp8_lora_add");
}

}  // extern "C"
