// What every C entry point needs around its kernels: error reporting, the
// engine's device and its stream-ordered scratch.  Shared by the files that
// implement entry points (not installed).
#pragma once

#include <string>

#include "bi_internal.h"

namespace bi {

// Record an error on the engine (or on the calling thread) and return `st`.
bi_status fail(bi_engine eng, bi_status st, const std::string& msg);
bi_status cuda_fail(bi_engine eng, cudaError_t e, const char* where);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int64_t dsize(bi_dtype dt) { return dt == BI_F32 ? 4 : 2; }
inline int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }

// Makes the engine's device current for the duration of a call, then restores.
struct DeviceGuard {
    int prev = -1;
    bool ok = true;
    explicit DeviceGuard(int dev) {
        if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
        if (prev != dev) ok = cudaSetDevice(dev) == cudaSuccess;
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

// Stream-ordered scratch from the engine's pool, released in stream order.
struct Scratch {
    bi_engine eng;
    cudaStream_t stream;
    void* ptr = nullptr;
    cudaError_t err = cudaSuccess;
    Scratch(bi_engine e, cudaStream_t s, size_t bytes) : eng(e), stream(s) {
        if (!bytes) return;
        if (take_injected_failure(e)) {  // bi_engine_fail_allocations: fail as an exhausted pool would
            err = cudaErrorMemoryAllocation;
            return;
        }
        err = cudaMallocFromPoolAsync(&ptr, bytes, e->pool, s);
    }
    static bool take_injected_failure(bi_engine e) {
        int64_t v = e->failing_allocs.load();
        while (v != 0) {
            if (v < 0) return true;
            if (e->failing_allocs.compare_exchange_weak(v, v - 1)) return true;
        }
        return false;
    }
    ~Scratch() {
        if (ptr) cudaFreeAsync(ptr, stream);
    }
};

inline LaunchCtx ctx(bi_engine eng, void* stream) {
    return LaunchCtx{eng, static_cast<cudaStream_t>(stream), eng->sm_count, eng->d_status, eng->wait_limit_ns};
}

}  // namespace bi
