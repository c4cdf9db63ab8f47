// views.h -- the argument checks shared by the C ABI's translation units
// (mbx_api.cu, train_api.cu): views in one form, extents without overflow,
// overlap, alignment, and the device checks.  Internal; not part of the ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "mbx.h"

namespace {

constexpr int64_t kMaxHidden = 8192;  // MAX_HIDDEN_SIZE of the pages' guard

struct V {  // a view in one form, for the checks
    const void* data;
    int64_t rows, cols, stride;
    int32_t dtype;
};

inline V of(const mbx_cview* v) { return V{v->data, v->rows, v->cols, v->row_stride, v->dtype}; }
inline V of(const mbx_view* v) { return V{v->data, v->rows, v->cols, v->row_stride, v->dtype}; }

inline int64_t esize(int32_t dtype) {
    switch (dtype) {
        case MBX_F64: return 8;
        case MBX_F32:
        case MBX_I32: return 4;
        case MBX_E4M3:
        case MBX_E2M1X2: return 1;
        default: return 2;
    }
}

// Bytes from a view's first element to one past its last.  Only called on
// views that extent_ok() accepted, so nothing here can overflow.
inline int64_t extent_bytes(const V& v) {
    return ((v.rows > 1 ? (v.rows - 1) * v.stride : 0) + v.cols) * esize(v.dtype);
}

// A view whose extent does not fit in 63 bits, or whose end address would
// wrap around, cannot lie inside any allocation: refused as out of bounds
// before any other check does arithmetic on it.  rows, cols > 0 and
// stride >= cols (for rows > 1) are checked first.
inline int extent_ok(const V& v) {
    int64_t span = 0, elems = 0, bytes = 0;
    uintptr_t end = 0;
    if (v.rows > 1 && __builtin_mul_overflow(v.rows - 1, v.stride, &span)) return MBX_E_BOUNDS;
    if (__builtin_add_overflow(span, v.cols, &elems)) return MBX_E_BOUNDS;
    if (__builtin_mul_overflow(elems, esize(v.dtype), &bytes)) return MBX_E_BOUNDS;
    if (__builtin_add_overflow(reinterpret_cast<uintptr_t>(v.data), (uintptr_t)bytes, &end))
        return MBX_E_BOUNDS;
    return MBX_OK;
}

// Whether the rows lie in order.  A single row has no stride, but a negative one
// says that the caller's row is not contiguous.
inline bool stride_ok(const V& v) { return v.rows > 1 ? v.stride >= v.cols : v.stride >= 0; }

// Step 1 of a view: dtype, non-empty, stride, alignment, extent.
inline int basic(const V& v) {
    if (v.data == nullptr) return MBX_E_NULL;
    if (v.dtype != MBX_BF16) return MBX_E_DTYPE;
    if (v.rows <= 0 || v.cols <= 0) return MBX_E_EMPTY;
    if (!stride_ok(v)) return MBX_E_STRIDE;
    if (reinterpret_cast<uintptr_t>(v.data) % 2) return MBX_E_ALIGN;
    return extent_ok(v);
}

inline bool overlaps(const V& a, const V& b) {
    uintptr_t a0 = reinterpret_cast<uintptr_t>(a.data), b0 = reinterpret_cast<uintptr_t>(b.data);
    uintptr_t a1 = a0 + (uintptr_t)extent_bytes(a), b1 = b0 + (uintptr_t)extent_bytes(b);
    return a0 < b1 && b0 < a1;
}

inline bool same_view(const V& a, const V& b) {
    return a.data == b.data && a.rows == b.rows && a.cols == b.cols &&
           (a.rows == 1 || a.stride == b.stride);
}

inline bool aligned16(const V& v) {
    return reinterpret_cast<uintptr_t>(v.data) % 16 == 0 && (v.rows == 1 || (v.stride * esize(v.dtype)) % 16 == 0);
}

// basic() for an operand that may be bfloat16 or binary32.
inline int basic_any(const V& v) {
    if (v.data == nullptr) return MBX_E_NULL;
    if (v.dtype != MBX_BF16 && v.dtype != MBX_F32) return MBX_E_DTYPE;
    if (v.rows <= 0 || v.cols <= 0) return MBX_E_EMPTY;
    if (!stride_ok(v)) return MBX_E_STRIDE;
    if (reinterpret_cast<uintptr_t>(v.data) % esize(v.dtype)) return MBX_E_ALIGN;
    return extent_ok(v);
}

inline int check_variant_eps(int variant, float eps) {
    if (variant != MBX_LOSSLESS && variant != MBX_HIGH) return MBX_E_VARIANT;
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return MBX_E_ARG;
    return MBX_OK;
}

// ---------------------------------------------------------------- device checks

typedef CUresult (*AddrRangeFn)(CUdeviceptr*, size_t*, CUdeviceptr);

inline AddrRangeFn addr_range_fn() {
    static AddrRangeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuMemGetAddressRange", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<AddrRangeFn>(p);
        cudaGetLastError();
    });
    return fn;
}

// The device checks of one call.  The allocation found last is kept for the
// call's other views: tensors of a framework's allocator often share one, and
// a query costs more than the rest of a view's checks.
struct DeviceCheck {
    int dev = -1;
    uintptr_t lo = 0, hi = 0;  // an allocation of this device

    int ok(const void* ptr, int64_t bytes) {
        const uintptr_t p0 = reinterpret_cast<uintptr_t>(ptr);
        if (bytes >= 0 && p0 >= lo && p0 < hi && (uintptr_t)bytes <= hi - p0) return MBX_OK;
        if (dev < 0 && cudaGetDevice(&dev) != cudaSuccess) {
            cudaGetLastError();
            dev = -1;
            return MBX_E_DEVICE;
        }
        cudaPointerAttributes a;
        if (cudaPointerGetAttributes(&a, ptr) != cudaSuccess) {
            cudaGetLastError();
            return MBX_E_DEVICE;
        }
        if (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged) return MBX_E_DEVICE;
        if (a.type == cudaMemoryTypeDevice && a.device != dev) return MBX_E_DEVICE;
        AddrRangeFn fn = addr_range_fn();
        if (fn == nullptr) return MBX_E_DEVICE;
        CUdeviceptr base = 0;
        size_t size = 0;
        if (fn(&base, &size, reinterpret_cast<CUdeviceptr>(ptr)) != CUDA_SUCCESS) {
            return a.type == cudaMemoryTypeManaged ? MBX_OK : MBX_E_BOUNDS;
        }
        // base <= ptr < base + size; compare the remaining room, never a sum
        const uintptr_t b0 = (uintptr_t)base;
        if (p0 < b0 || bytes < 0 || (uintptr_t)bytes > b0 + size - p0) return MBX_E_BOUNDS;
        lo = b0;
        hi = b0 + size;
        return MBX_OK;
    }
};

inline int views_on_device(const V* vs, int n) {
    DeviceCheck c;
    for (int i = 0; i < n; ++i)
        if (int st = c.ok(vs[i].data, extent_bytes(vs[i]))) return st;
    return MBX_OK;
}

inline int raw_on_device(const void* p, int64_t bytes) {
    DeviceCheck c;
    return c.ok(p, bytes);
}

#define MBX_TRY(expr)                   \
    do {                                \
        int _st = (expr);               \
        if (_st != MBX_OK) return _st;  \
    } while (0)

// Modulation view m against x: same width, rows of x a multiple of its rows.
inline int check_mod(const V& m, const V& x) {
    if (m.cols != x.cols) return MBX_E_SHAPE;
    if (x.rows % m.rows != 0) return MBX_E_SHAPE;
    return MBX_OK;
}

inline int check_weight(const V& w, const V& x) {
    if (w.rows != 1 || w.cols != x.cols) return MBX_E_SHAPE;
    return MBX_OK;
}

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? MBX_OK : MBX_E_CUDA; }

}  // namespace
