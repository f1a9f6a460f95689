// Host-side helpers shared by the files that implement the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>
#include <stddef.h>

#include <mutex>

namespace stepq {

// Sets the thread's stepq_last_error() message and returns `code`.
int fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int cuda_fail(cudaError_t e, const char *what);
int check_ptr(const void *p, size_t align, const char *name);

// Strides of `rows` token rows of `width` elements of `dtype` starting at p (include/stepq.h, stepq_tokens).
int check_dtype(int dtype, const char *what);
int check_rows(const void *p, int dtype, long long stride, long long width, const char *name);

struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};

// A device error word: kernels set bits of it, the host takes them.  Both are atomic, so that no bit is lost whatever
// streams the kernels run on, and nothing waits for a stream that is not named.
class ErrorWord {
   public:
    // Allocates the word on the current device; zero when this returns.
    cudaError_t create();
    void destroy();
    // The word after all that `st` holds, and 0 in its place.
    cudaError_t take(cudaStream_t st, int &word);
    int *device() const { return mem_; }

   private:
    int *mem_ = nullptr;  // the word, and where a take puts it
    std::mutex mu_;       // from a take's exchange to its copy
};

// Makes `device` current for a scope and puts the caller's device back.
class DeviceScope {
   public:
    explicit DeviceScope(int device) {
        err_ = cudaGetDevice(&before_);
        if (err_ == cudaSuccess && before_ != device) {
            err_ = cudaSetDevice(device);
            moved_ = err_ == cudaSuccess;
        }
    }
    ~DeviceScope() {
        if (moved_) cudaSetDevice(before_);
    }
    DeviceScope(const DeviceScope &) = delete;
    DeviceScope &operator=(const DeviceScope &) = delete;
    cudaError_t error() const { return err_; }

   private:
    int before_ = 0;
    bool moved_ = false;
    cudaError_t err_;
};

}  // namespace stepq
