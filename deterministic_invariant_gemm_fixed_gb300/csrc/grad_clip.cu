// Global norm of a set of tensors, and the set scaled to a maximum norm.  See
// include/bi.h (bi_grad_norm, bi_grad_clip).
//
// The set is cut into chunks of GC_CHUNK consecutive elements of one tensor.  A
// chunk's sum of squares is taken by one block: f32 FMAs per thread (8 running
// sums), an f32 tree per warp, the 16 warps in f64; a chunk whose f32 sum leaves
// f32's range (an overflow, or squares below its normal numbers) is summed again
// in f64, so every finite input has its norm.  A finishing block adds the chunk
// sums in f64 in a fixed order.  Cuts and orders depend on the sizes alone: the
// norm is the same bit for bit from run to run.
//
// Both passes are bound by memory.  The scaling pass walks the chunks from the
// last to the first, so what the norm pass read last is still in L2, and stores
// past L2's keep-list (st.cs): of a set that fits L2 nothing is read twice from
// memory, of a larger one about 100 MB less.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "abi_util.h"

namespace bi {
namespace {

constexpr int64_t GC_CHUNK = 32768;  // elements
constexpr int GC_THREADS = 512;
constexpr int GC_WARPS = GC_THREADS / 32;
constexpr int GC_TENSORS = 128;      // per launch: their table travels in the kernel's parameters

struct Tensor {
    void* dst;
    const void* src;
    int64_t count;
};
struct Table {
    Tensor t[GC_TENSORS];
    int first[GC_TENSORS + 1];  // first chunk of each tensor, counted within the launch; [n] = all
    uint8_t dtype[GC_TENSORS];
    uint8_t vec[GC_TENSORS];    // 16-byte aligned: 16-byte loads and stores
    int n;
};

// One chunk: its tensor, first element and length.
struct Piece {
    int i;
    int64_t e0;
    int len;
};
__device__ __forceinline__ Piece piece_of(const Table& t, int chunk) {
    int lo = 0, hi = t.n - 1;  // the last tensor whose first chunk is <= chunk (empty tensors share their successor's)
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= chunk) lo = mid; else hi = mid - 1;
    }
    const int64_t e0 = static_cast<int64_t>(chunk - t.first[lo]) * GC_CHUNK;
    return {lo, e0, static_cast<int>(lmin(GC_CHUNK, t.t[lo].count - e0))};
}

template <typename T> __device__ __forceinline__ float up(T v);
template <> __device__ __forceinline__ float up<float>(float v) { return v; }
template <> __device__ __forceinline__ float up<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float up<__half>(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T down(float v);
template <> __device__ __forceinline__ float down<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 down<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half down<__half>(float v) { return __float2half_rn(v); }

constexpr float GC_TINY = 0x1p-90f;  // a chunk sum below this may have lost squares to underflow

// The block's sum over its threads' f32 values, in f64, in every thread.
__device__ __forceinline__ double block_sum(float v, double* s_w) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();  // s_w free again
    if ((threadIdx.x & 31) == 0) s_w[threadIdx.x >> 5] = v;
    __syncthreads();
    double d = 0.0;
#pragma unroll
    for (int w = 0; w < GC_WARPS; ++w) d += s_w[w];
    return d;
}

template <typename T>
__device__ double chunk_square_sum(const T* src, int len, bool vec, double* s_w) {
    constexpr int PER = 16 / sizeof(T);
    const int tid = threadIdx.x;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    bool nz = false;
    int done = 0;
    if (vec) {
        const int nv = len / PER;
        const uint4* v = reinterpret_cast<const uint4*>(src);
        constexpr int U = 8;  // 16-byte loads in flight per thread
        for (int b = tid; b < nv; b += U * GC_THREADS) {
            uint4 raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                raw[u] = b + u * GC_THREADS < nv ? v[b + u * GC_THREADS] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const T* e = reinterpret_cast<const T*>(&raw[u]);
                constexpr uint32_t MAG = sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu;
                nz = nz || ((raw[u].x | raw[u].y | raw[u].z | raw[u].w) & MAG) != 0;
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const float f = up<T>(e[j]);
                    acc[(u * PER + j) & 7] = fmaf(f, f, acc[(u * PER + j) & 7]);
                }
            }
        }
        done = nv * PER;
    }
    for (int i = done + tid; i < len; i += GC_THREADS) {
        const float f = up<T>(src[i]);
        nz = nz || f != 0.0f;
        acc[0] = fmaf(f, f, acc[0]);
    }
    const float s = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
    double d = block_sum(s, s_w);
    const bool any = __syncthreads_or(nz) != 0;
    // out of f32's range (or NaN): again in f64, the warps' f64 sums in the same tree
    if (any && !(d >= static_cast<double>(GC_TINY) && d <= 3.0e38)) {
        double a = 0.0;
        for (int i = tid; i < len; i += GC_THREADS) {
            const double f = up<T>(src[i]);
            a += f * f;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        if ((tid & 31) == 0) s_w[tid >> 5] = a;
        __syncthreads();
        d = 0.0;
        for (int w = 0; w < GC_WARPS; ++w) d += s_w[w];
    }
    return d;
}

__global__ void __launch_bounds__(GC_THREADS, 2) square_sum_kernel(const __grid_constant__ Table t, double* partials) {
    __shared__ double s_w[GC_WARPS];
    grid_dep_wait();
    grid_dep_launch();
    const int chunks = t.first[t.n];
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const Piece p = piece_of(t, c);
        const bool vec = t.vec[p.i] != 0;
        double d;
        if (t.dtype[p.i] == BI_F32) d = chunk_square_sum(static_cast<const float*>(t.t[p.i].src) + p.e0, p.len, vec, s_w);
        else if (t.dtype[p.i] == BI_BF16)
            d = chunk_square_sum(static_cast<const __nv_bfloat16*>(t.t[p.i].src) + p.e0, p.len, vec, s_w);
        else d = chunk_square_sum(static_cast<const __half*>(t.t[p.i].src) + p.e0, p.len, vec, s_w);
        if (threadIdx.x == 0) partials[c] = d;
    }
}

// norm = sqrt of the chunk sums, added thread-strided in order, then by a tree.
__global__ void __launch_bounds__(1024) norm_finish_kernel(const double* partials, int64_t n, float* norm) {
    __shared__ double s_w[32];
    grid_dep_wait();
    grid_dep_launch();
    double a = 0.0;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < n; i += 1024) a += partials[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if ((threadIdx.x & 31) == 0) s_w[threadIdx.x >> 5] = a;
    __syncthreads();
    if (threadIdx.x < 32) {
        a = s_w[threadIdx.x];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(a));
    }
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const Tensor& t, int64_t e0, int len, bool vec, float coef, bool exact) {
    constexpr int PER = 16 / sizeof(T);
    const T* src = static_cast<const T*>(t.src) + e0;
    T* dst = static_cast<T*>(t.dst) + e0;
    int done = 0;
    if (vec) {
        const int nv = len / PER;
        const uint4* v = reinterpret_cast<const uint4*>(src);
        uint4* o = reinterpret_cast<uint4*>(dst);
        constexpr int U = 4;
        for (int b = threadIdx.x; b < nv; b += U * GC_THREADS) {
            uint4 raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (b + u * GC_THREADS < nv) raw[u] = __ldcs(v + b + u * GC_THREADS);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (b + u * GC_THREADS >= nv) continue;
                if (!exact) {
                    T* e = reinterpret_cast<T*>(&raw[u]);
#pragma unroll
                    for (int j = 0; j < PER; ++j) e[j] = down<T>(up<T>(e[j]) * coef);
                }
                __stcs(o + b + u * GC_THREADS, raw[u]);
            }
        }
        done = nv * PER;
    }
    for (int i = done + threadIdx.x; i < len; i += GC_THREADS) dst[i] = exact ? src[i] : down<T>(up<T>(src[i]) * coef);
}

// dst = round(src * coef), coef = norm > max_norm ? max_norm / norm : 1 (NaN for
// a NaN norm).  coef = 1 copies the bits, and leaves a tensor in place alone.
__global__ void __launch_bounds__(GC_THREADS, 2)
    scale_kernel(const __grid_constant__ Table t, const float* norm, float max_norm) {
    grid_dep_wait();
    grid_dep_launch();
    const float n = __ldg(norm);
    const float coef = n > max_norm ? max_norm / n : (n == n ? 1.0f : n);
    const bool exact = coef == 1.0f;
    const int chunks = t.first[t.n];
    for (int c = chunks - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x) {
        const Piece p = piece_of(t, c);
        const Tensor& x = t.t[p.i];
        if (exact && x.dst == x.src) continue;
        const bool vec = t.vec[p.i] != 0;
        if (t.dtype[p.i] == BI_F32) scale_chunk<float>(x, p.e0, p.len, vec, coef, exact);
        else if (t.dtype[p.i] == BI_BF16) scale_chunk<__nv_bfloat16>(x, p.e0, p.len, vec, coef, exact);
        else scale_chunk<__half>(x, p.e0, p.len, vec, coef, exact);
    }
}

constexpr int64_t GC_MAX_CHUNKS = (int64_t(1) << 31) - 1;

bi_status check_set(bi_engine eng, const void* const* src, void* const* dst, bool need_dst, const int64_t* counts,
                    const int* dtypes, int64_t n, int64_t* chunks) {
    if (!eng) return fail(nullptr, BI_ERR_INVALID_ARG, "engine is NULL");
    if (n < 0) return fail(eng, BI_ERR_INVALID_ARG, "n must be >= 0");
    if (n > 0 && (!src || !counts || !dtypes || (need_dst && !dst)))
        return fail(eng, BI_ERR_INVALID_ARG, "the tensor tables must not be NULL");
    *chunks = 0;
    for (int64_t i = 0; i < n; ++i) {
        if (dtypes[i] != BI_F32 && dtypes[i] != BI_BF16 && dtypes[i] != BI_F16)
            return fail(eng, BI_ERR_INVALID_ARG, "dtype must be BI_F32, BI_BF16 or BI_F16");
        if (counts[i] < 0) return fail(eng, BI_ERR_INVALID_ARG, "counts must be >= 0");
        if (counts[i] > 0 && (!src[i] || (need_dst && !dst[i])))
            return fail(eng, BI_ERR_INVALID_ARG, "a tensor with elements has a NULL pointer");
        const uintptr_t es = static_cast<uintptr_t>(dsize(static_cast<bi_dtype>(dtypes[i])));
        if (counts[i] > 0 && (reinterpret_cast<uintptr_t>(src[i]) % es != 0 ||
                              (need_dst && reinterpret_cast<uintptr_t>(dst[i]) % es != 0)))
            return fail(eng, BI_ERR_MISALIGNED, "a tensor is not aligned to its element size");
        const int64_t c = (counts[i] - 1) / GC_CHUNK + (counts[i] > 0);
        if (c > GC_MAX_CHUNKS - *chunks) return fail(eng, BI_ERR_UNSUPPORTED, "the set is beyond 2^31 - 1 chunks of 32768 elements");
        *chunks += c;
    }
    return BI_OK;
}

// Runs `launch(table, first chunk of the launch)` over the set, GC_TENSORS
// tensors at a time; `reverse` starts with the last ones.
template <typename F>
cudaError_t over_set(const void* const* src, void* const* dst, const int64_t* counts, const int* dtypes, int64_t n,
                     bool reverse, int64_t chunks, F&& launch) {
    Table t;
    const int64_t groups = (n + GC_TENSORS - 1) / GC_TENSORS;
    int64_t before = reverse ? chunks : 0;
    for (int64_t q = 0; q < groups; ++q) {
        const int64_t i0 = (reverse ? groups - 1 - q : q) * GC_TENSORS;
        t.n = static_cast<int>(lmin(GC_TENSORS, n - i0));
        int64_t at = 0;
        for (int j = 0; j < t.n; ++j) {
            const int64_t i = i0 + j;
            t.t[j] = {dst ? dst[i] : nullptr, src[i], counts[i]};
            t.first[j] = static_cast<int>(at);
            t.dtype[j] = static_cast<uint8_t>(dtypes[i]);
            t.vec[j] = aligned16(src[i]) && (!dst || aligned16(dst[i]));
            at += (counts[i] + GC_CHUNK - 1) / GC_CHUNK;
        }
        t.first[t.n] = static_cast<int>(at);
        if (reverse) before -= at;
        if (at > 0) {
            const cudaError_t e = launch(t, before, at);
            if (e != cudaSuccess) return e;
        }
        if (!reverse) before += at;
    }
    return cudaSuccess;
}

}  // namespace
}  // namespace bi

using namespace bi;

extern "C" {

bi_status bi_grad_norm(bi_engine eng, float* norm, const void* const* tensors, const int64_t* counts,
                       const int* dtypes, int64_t n, void* stream) {
    int64_t chunks = 0;
    bi_status st = check_set(eng, tensors, nullptr, false, counts, dtypes, n, &chunks);
    if (st != BI_OK) return st;
    if (!norm) return fail(eng, BI_ERR_INVALID_ARG, "norm must not be NULL");
    DeviceGuard g(eng->device);
    if (!g.ok) return fail(eng, BI_ERR_CUDA, "cudaSetDevice failed");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (chunks == 0) {
        const cudaError_t e = cudaMemsetAsync(norm, 0, 4, s);
        return e == cudaSuccess ? BI_OK : cuda_fail(eng, e, "bi_grad_norm");
    }
    const LaunchCtx c = ctx(eng, stream);
    Scratch sc(eng, s, static_cast<size_t>(chunks * 8));
    if (sc.err != cudaSuccess) return cuda_fail(eng, sc.err, "norm scratch");
    double* partials = static_cast<double*>(sc.ptr);
    cudaError_t e = over_set(tensors, nullptr, counts, dtypes, n, false, chunks,
                             [&](const Table& t, int64_t first, int64_t count) {
        const dim3 grid(static_cast<unsigned>(lmin(count, 2 * int64_t(c.sm_count))));
        const cudaError_t r = launch_pdl(square_sum_kernel, grid, dim3(GC_THREADS), 0, c.stream, t, partials + first);
        if (r == cudaSuccess) c.count();
        return r;
    });
    if (e == cudaSuccess) {
        e = launch_pdl(norm_finish_kernel, dim3(1), dim3(1024), 0, c.stream, partials, chunks, norm);
        if (e == cudaSuccess) c.count();
    }
    return e == cudaSuccess ? BI_OK : cuda_fail(eng, e, "bi_grad_norm");
}

bi_status bi_grad_clip(bi_engine eng, void* const* dst, const void* const* src, const int64_t* counts,
                       const int* dtypes, int64_t n, const float* norm, float max_norm, void* stream) {
    int64_t chunks = 0;
    bi_status st = check_set(eng, src, dst, true, counts, dtypes, n, &chunks);
    if (st != BI_OK) return st;
    if (!norm) return fail(eng, BI_ERR_INVALID_ARG, "norm must not be NULL");
    if (!(max_norm >= 0.0f)) return fail(eng, BI_ERR_INVALID_ARG, "max_norm must be >= 0");
    if (chunks == 0) return BI_OK;
    DeviceGuard g(eng->device);
    if (!g.ok) return fail(eng, BI_ERR_CUDA, "cudaSetDevice failed");
    const LaunchCtx c = ctx(eng, stream);
    const cudaError_t e = over_set(src, dst, counts, dtypes, n, true, chunks,
                                   [&](const Table& t, int64_t, int64_t count) {
        const dim3 grid(static_cast<unsigned>(lmin(count, 2 * int64_t(c.sm_count))));
        const cudaError_t r = launch_pdl(scale_kernel, grid, dim3(GC_THREADS), 0, c.stream, t, norm, max_norm);
        if (r == cudaSuccess) c.count();
        return r;
    });
    return e == cudaSuccess ? BI_OK : cuda_fail(eng, e, "bi_grad_clip");
}

}  // extern "C"
