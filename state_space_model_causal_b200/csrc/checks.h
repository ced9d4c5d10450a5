// checks.h -- what every entry point of the C ABI does before it launches
// anything: checks of tensor descriptors (rank, strides, extents, overlap),
// device queries that are made once, and the launch report.
#pragma once

#include "../../include/ssm_causal.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstdlib>
#include <initializer_list>

#include "problem.h"

namespace ssm {

constexpr int kDefaultSms = 148;  // B200
// ------------------------------------------------------------ tensor checks --
inline bool present(const ssm_tensor& t) { return t.data != nullptr; }

inline int esize(int dt) {
    switch (dt) {
        case SSM_F32: return 4;
        case SSM_F16: return 2;
        case SSM_BF16: return 2;
        case SSM_I32: return 4;
        default: return 0;
    }
}

inline bool is_float(int dt) { return dt == SSM_F32 || dt == SSM_F16 || dt == SSM_BF16; }

// Largest element count and byte span a tensor may describe: far above any
// device memory, low enough that no size, offset or extent computed from the
// tensor overflows int64.
constexpr int64_t kMaxSpan = (int64_t)1 << 56;

// rank, non-negative sizes and strides, element-aligned pointer, element
// count and byte span within kMaxSpan
inline ssm_status basic(const ssm_tensor& t) {
    if (!t.data) return SSM_ERR_NULL;
    if (t.ndim < 1 || t.ndim > SSM_MAX_DIMS) return SSM_ERR_SHAPE;
    if (esize(t.dtype) == 0) return SSM_ERR_DTYPE;
    for (int i = 0; i < t.ndim; ++i) {
        if (t.shape[i] < 0) return SSM_ERR_SHAPE;
        if (t.stride[i] < 0) return SSM_ERR_STRIDE;
    }
    if (reinterpret_cast<uintptr_t>(t.data) % esize(t.dtype) != 0) return SSM_ERR_STRIDE;
    for (int i = 0; i < t.ndim; ++i)
        if (t.shape[i] == 0) return SSM_OK;  // empty: touches no memory
    int64_t count = 1, last = 0;
    for (int i = 0; i < t.ndim; ++i)
        if (__builtin_mul_overflow(count, t.shape[i], &count) || count > kMaxSpan)
            return SSM_ERR_UNSUPPORTED;
    for (int i = 0; i < t.ndim; ++i) {
        int64_t step = 0;
        if (__builtin_mul_overflow(t.shape[i] - 1, t.stride[i], &step) ||
            __builtin_add_overflow(last, step, &last) || last > kMaxSpan)
            return SSM_ERR_UNSUPPORTED;
    }
    if ((last + 1) * esize(t.dtype) > kMaxSpan) return SSM_ERR_UNSUPPORTED;
    return SSM_OK;
}

inline ssm_status want_shape(const ssm_tensor& t, int nd, const int64_t* dims) {
    if (t.ndim != nd) return SSM_ERR_SHAPE;
    for (int i = 0; i < nd; ++i)
        if (t.shape[i] != dims[i]) return SSM_ERR_SHAPE;
    return SSM_OK;
}

inline ssm_status want(const ssm_tensor& t, std::initializer_list<int64_t> dims) {
    return want_shape(t, (int)dims.size(), dims.begin());
}

inline int64_t numel(const ssm_tensor& t) {
    int64_t n = 1;
    for (int i = 0; i < t.ndim; ++i) n *= t.shape[i];
    return n;
}

// Byte range [lo, hi) the tensor touches (empty tensors touch nothing).
inline void extent(const ssm_tensor& t, uintptr_t* lo, uintptr_t* hi) {
    const uintptr_t base = reinterpret_cast<uintptr_t>(t.data);
    if (!t.data || numel(t) == 0) {
        *lo = *hi = base;
        return;
    }
    int64_t last = 0;
    for (int i = 0; i < t.ndim; ++i) last += (t.shape[i] - 1) * t.stride[i];
    *lo = base;
    *hi = base + (uintptr_t)((last + 1) * esize(t.dtype));
}

inline bool overlap(const ssm_tensor& a, const ssm_tensor& b) {
    uintptr_t al, ah, bl, bh;
    extent(a, &al, &ah);
    extent(b, &bl, &bh);
    if (al == ah || bl == bh) return false;
    return al < bh && bl < ah;
}

// An output must not write one address twice: sort the non-trivial dims by
// stride and require each stride to clear the span of the smaller ones.
inline bool non_overlapping(const ssm_tensor& t) {
    if (numel(t) == 0) return true;  // writes nothing
    int64_t st[SSM_MAX_DIMS], sh[SSM_MAX_DIMS];
    int n = 0;
    for (int i = 0; i < t.ndim; ++i) {
        if (t.shape[i] <= 1) continue;
        st[n] = t.stride[i];
        sh[n] = t.shape[i];
        ++n;
    }
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < n; ++j)
            if (st[j] < st[i]) {
                std::swap(st[i], st[j]);
                std::swap(sh[i], sh[j]);
            }
    int64_t span = 1;
    for (int i = 0; i < n; ++i) {
        if (st[i] < span) return false;
        span = st[i] * (sh[i] - 1) + span;
    }
    return true;
}

// stride of dim i, with size-1 dims reading as 0 (never stepped)
inline int64_t sd(const ssm_tensor& t, int i) { return t.shape[i] == 1 ? 0 : t.stride[i]; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// An integer environment switch: only a whole decimal number counts; anything
// else (unset, empty, trailing characters) leaves the caller's default.
inline bool env_int(const char* name, long long* v) {
    const char* e = std::getenv(name);
    if (!e || !*e) return false;
    char* end = nullptr;
    const long long x = std::strtoll(e, &end, 10);
    if (!end || *end != '\0') return false;
    *v = x;
    return true;
}

constexpr long long kWaitBudget = 4000000000LL;  // cycles (~2 s) before a bounded wait gives up
constexpr long long kMinTestBudget = 10000000LL; // shortest wait a failure test may ask for

// A failure test's wait budget, never below kMinTestBudget.
inline long long clamp_test_budget(long long v) { return v < kMinTestBudget ? kMinTestBudget : v; }

// The current device (0 in dry-run mode, which makes no CUDA call).
inline int current_device(bool dry_run) {
    int dev = 0;
    if (!dry_run && cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    return dev;
}

// SM count of a device, queried once per device (dry-run mode assumes a B200).
inline int sm_count(bool dry_run, int dev) {
    if (dry_run) return kDefaultSms;
    static std::atomic<int> cache[kMaxDevices];
    if (dev < 0 || dev >= kMaxDevices) return kDefaultSms;
    int n = cache[dev].load(std::memory_order_acquire);
    if (n > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        return kDefaultSms;
    cache[dev].store(n, std::memory_order_release);
    return n;
}
inline int sm_count(bool dry_run) { return sm_count(dry_run, current_device(dry_run)); }

inline void fill_info(ssm_launch_info* info, int kernel, int grid, int block, int smem, int64_t rows,
               int64_t items) {
    if (!info) return;
    info->kernel = kernel;
    info->grid = grid;
    info->block = block;
    info->smem_bytes = smem;
    info->rows_per_item = (int32_t)rows;
    info->work_items = items;
}

inline ssm_status info_ok(const ssm_launch_info* info) {
    if (info && info->struct_size != sizeof(ssm_launch_info)) return SSM_ERR_VERSION;
    return SSM_OK;
}

#define SSM_TRY(expr)                  \
    do {                               \
        ssm_status _s = (expr);        \
        if (_s != SSM_OK) return _s;   \
    } while (0)

}  // namespace ssm
