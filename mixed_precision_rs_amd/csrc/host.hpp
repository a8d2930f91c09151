// Host helpers shared by the files that implement the C ABI: the thread's
// error detail, the device of a stream, and checks of row-strided matrices.
// Not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <new>

#include "tide.h"

namespace tide {

// Set the thread's error detail (tide_last_error_detail) and return `st`.
__attribute__((format(printf, 2, 3))) tide_status fail(tide_status st, const char* fmt, ...);
tide_status hip_fail(hipError_t e, const char* what);

#define TIDE_HIP_TRY(expr)                                      \
    do {                                                        \
        hipError_t e_ = (expr);                                 \
        if (e_ != hipSuccess) return hip_fail(e_, #expr);       \
    } while (0)

#define TIDE_TRY(expr)                        \
    do {                                      \
        tide_status s_ = (expr);              \
        if (s_ != TIDE_OK) return s_;         \
    } while (0)

// Makes `dev` the current device for the guard's lifetime. Allocations,
// events and kernel attributes belong to the current device, and a caller's
// stream may sit on another one.
class DeviceGuard {
  public:
    explicit DeviceGuard(int dev) {
        if (hipGetDevice(&prev_) != hipSuccess) prev_ = -1;
        if (prev_ != dev) {
            status_ = hipSetDevice(dev);
            changed_ = status_ == hipSuccess && prev_ >= 0;
        }
    }
    ~DeviceGuard() {
        if (changed_) (void)hipSetDevice(prev_);
    }
    DeviceGuard(const DeviceGuard&) = delete;
    DeviceGuard& operator=(const DeviceGuard&) = delete;
    hipError_t status() const { return status_; }

  private:
    int prev_ = -1;
    bool changed_ = false;
    hipError_t status_ = hipSuccess;
};

tide_status stream_device(hipStream_t stream, int* dev);

// A matrix argument: `rows` rows of `width` bytes, `stride` bytes apart (a
// plain array is one row).
struct Mat {
    const char* name;
    uintptr_t base;
    int64_t rows, width, stride;
};

// Fills *out from a pointer, sizes in elements of `size` bytes and the
// alignment its elements need. Errors: INVALID_ARG (NULL with work to do,
// negative sizes, stride < cols), ALIGNMENT, OVERFLOW (extent past int64).
tide_status matrix(const char* name, const void* p, int64_t rows, int64_t cols, int64_t stride,
                   int32_t size, Mat* out);

// INVALID_ARG when one of the nw matrices written shares memory with one of
// the nr read or with another one written. Rows of one stride that interleave
// (column windows of a wider matrix) do not share memory.
tide_status no_overlap(const Mat* written, int nw, const Mat* read, int nr);

// Runs the body of a C entry point; no exception leaves it.
template <class F>
tide_status guarded(F&& body) {
    try {
        return body();
    } catch (const std::bad_alloc&) {
        return fail(TIDE_ERR_NO_MEMORY, "host allocation failed");
    } catch (...) {
        return fail(TIDE_ERR_INVALID_ARG, "unexpected exception");
    }
}

// Launches a kernel and returns this launch's own error: hipGetLastError would
// also report, and take away, one that the caller's earlier calls left behind.
template <class... P, class... A>
hipError_t enqueue(void (*kernel)(P...), dim3 grid, uint32_t threads, size_t lds, hipStream_t stream,
                   A... values) {
    return [&](P... v) {
        void* args[] = {(void*)&v...};
        return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(threads), args, lds, stream);
    }(values...);
}

// Runs launch(stream), which returns a hipError_t, with the stream's device
// current.
template <class F>
tide_status on_stream(void* stream_v, F&& launch) {
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_v);
    int dev = 0;
    TIDE_TRY(stream_device(stream, &dev));
    DeviceGuard guard(dev);
    if (guard.status() != hipSuccess) return hip_fail(guard.status(), "hipSetDevice");
    const hipError_t e = launch(stream);
    return e == hipSuccess ? TIDE_OK : hip_fail(e, "kernel launch");
}

}  // namespace tide
