// Global norm of a set of tensors, and the set scaled to a maximum norm.  See
// include/bi.h (bi_grad_norm, bi_grad_clip).
//
// The set is cut into units of `unit` consecutive elements of one tensor (2048 to
// 16384, by the set's size), dealt out in turn to GC_BLOCKS x 8 warps.  A lane sums the squares of 4
// 16-byte vectors (16 or 32 elements) in f32, in 8 running sums, and adds that to
// its f64 sum; a batch whose f32 sum leaves f32's range (an overflow, or squares
// below its normal numbers) is summed again in f64 from the registers, so every
// finite input has its norm.  A lane keeps its sum over all of its warp's units; the lanes'
// sums are added by a tree, the warps' by a finishing block, in f64 in a fixed
// order.  Cuts, dealing and orders depend on the sizes alone (a tensor off 16-byte
// alignment has the same vectors, loaded element by element): the norm is the same
// bit for bit from run to run and wherever in memory the tensors lie.
//
// Both passes are bound by memory (a set beyond the caches: 5.3 and 5.5 TB/s of the
// copy rate's 6.7).  No barrier stands between a warp's loads and
// the next ones (512-thread blocks that reduced every 64 KB read 3.1 TB/s of the
// copy rate's 6.7).  The scaling pass walks the units from the last to the first,
// so what the norm pass read last is still in L2, and stores past L2's keep-list
// (st.cs): of a set that fits L2 nothing is read twice from memory, of a larger one
// about 100 MB less.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <type_traits>

#include "abi_util.h"

namespace bi {
namespace {

constexpr int64_t GC_UNIT_MIN = 2048, GC_UNIT_MAX = 16384;  // elements
constexpr int GC_THREADS = 256, GC_WARPS = GC_THREADS / 32;
constexpr int GC_BLOCKS = 608;       // at most, whatever the GPU: four on each of 152 SMs
constexpr int GC_VECS = 4;           // 16-byte loads in flight per lane: 64 KB per SM at 32 warps
constexpr int GC_TENSORS = 128;      // per launch: their table travels in the kernel's parameters

struct Tensor {
    void* dst;
    const void* src;
    int64_t count;
};
struct Table {
    Tensor t[GC_TENSORS];
    int first[GC_TENSORS + 1];  // first unit of each tensor, counted within the launch; [n] = all
    uint8_t dtype[GC_TENSORS];
    uint8_t vec[GC_TENSORS];    // 16-byte aligned: 16-byte loads and stores
    int n, unit;
};

// One unit: its tensor, first element and length.
struct Piece {
    int i;
    int64_t e0;
    int len;
};
__device__ __forceinline__ Piece piece_of(const Table& t, int at) {
    int lo = 0, hi = t.n - 1;  // the last tensor whose first unit is <= at (empty tensors share their successor's)
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= at) lo = mid; else hi = mid - 1;
    }
    const int64_t e0 = static_cast<int64_t>(at - t.first[lo]) * t.unit;
    return {lo, e0, static_cast<int>(lmin(t.unit, t.t[lo].count - e0))};
}

template <typename T> __device__ __forceinline__ float up(T v);
template <> __device__ __forceinline__ float up<float>(float v) { return v; }
template <> __device__ __forceinline__ float up<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float up<__half>(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T down(float v);
template <> __device__ __forceinline__ float down<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 down<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half down<__half>(float v) { return __float2half_rn(v); }

constexpr float GC_TINY = 0x1p-90f, GC_BIG = 3.0e38f;  // a batch sum outside may have lost squares

// 16 bytes of elements, in one load where they are aligned.
template <typename T, bool VEC>
__device__ __forceinline__ uint4 load16(const T* src) {
    if (VEC) return *reinterpret_cast<const uint4*>(src);
    uint4 raw;
    T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int j = 0; j < static_cast<int>(16 / sizeof(T)); ++j) e[j] = src[j];
    return raw;
}

// Adds one lane's part of a unit's sum of squares to `total`.
template <typename T, bool VEC>
__device__ __forceinline__ void lane_square_sum(const T* src, int len, int lane, double& total) {
    constexpr int PER = 16 / sizeof(T);
    const int nv = len / PER;
    for (int b = lane; b < nv; b += 32 * GC_VECS) {
        uint4 raw[GC_VECS];
#pragma unroll
        for (int u = 0; u < GC_VECS; ++u)
            raw[u] = b + 32 * u < nv ? load16<T, VEC>(src + static_cast<int64_t>(b + 32 * u) * PER) : make_uint4(0, 0, 0, 0);
        float acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
#pragma unroll
        for (int u = 0; u < GC_VECS; ++u) {
            const T* e = reinterpret_cast<const T*>(&raw[u]);
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const float f = up<T>(e[j]);
                acc[(u * PER + j) & 7] = fmaf(f, f, acc[(u * PER + j) & 7]);
            }
        }
        const float s = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
        if (s >= GC_TINY && s <= GC_BIG) {
            total += static_cast<double>(s);
        } else {  // zeros, or squares (or their sum) that f32 does not hold, or not finite
            constexpr uint32_t MAG = sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu;
            uint32_t bits = 0;
#pragma unroll
            for (int u = 0; u < GC_VECS; ++u) bits |= raw[u].x | raw[u].y | raw[u].z | raw[u].w;
            if ((bits & MAG) != 0) {
#pragma unroll
                for (int u = 0; u < GC_VECS; ++u) {
                    const T* e = reinterpret_cast<const T*>(&raw[u]);
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        const double f = up<T>(e[j]);
                        total = fma(f, f, total);
                    }
                }
            }
        }
    }
    for (int i = nv * PER + lane; i < len; i += 32) {  // the last elements
        const double f = up<T>(src[i]);
        total = fma(f, f, total);
    }
}

__global__ void __launch_bounds__(GC_THREADS, 4) square_sum_kernel(const __grid_constant__ Table t, double* partials) {
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31, units = t.first[t.n];
    const int warp = blockIdx.x * GC_WARPS + (threadIdx.x >> 5), warps = gridDim.x * GC_WARPS;
    double d = 0.0;
    for (int c = warp; c < units; c += warps) {
        const Piece p = piece_of(t, c);
        const void* src = t.t[p.i].src;
        auto add = [&](auto* e) {
            using T = std::remove_const_t<std::remove_pointer_t<decltype(e)>>;
            if (t.vec[p.i] != 0) lane_square_sum<T, true>(e + p.e0, p.len, lane, d);
            else lane_square_sum<T, false>(e + p.e0, p.len, lane, d);
        };
        if (t.dtype[p.i] == BI_F32) add(static_cast<const float*>(src));
        else if (t.dtype[p.i] == BI_BF16) add(static_cast<const __nv_bfloat16*>(src));
        else add(static_cast<const __half*>(src));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) partials[warp] = d;
}

// sqrt of the warps' sums, in every thread of a block of GC_THREADS: each thread
// adds every GC_THREADS-th sum in order, then a tree.
__device__ __forceinline__ float norm_of(const double* partials, int64_t n, double* s_w) {
    double a = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 8 * GC_THREADS) {  // eight loads in flight
        double t[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) t[u] = i + u * GC_THREADS < n ? partials[i + u * GC_THREADS] : 0.0;
#pragma unroll
        for (int u = 0; u < 8; ++u) a += t[u];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if ((threadIdx.x & 31) == 0) s_w[threadIdx.x >> 5] = a;
    __syncthreads();
    a = 0.0;
#pragma unroll
    for (int w = 0; w < GC_WARPS; ++w) a += s_w[w];
    return static_cast<float>(sqrt(a));
}

__global__ void __launch_bounds__(GC_THREADS) norm_finish_kernel(const double* partials, int64_t n, float* norm) {
    __shared__ double s_w[GC_WARPS];
    grid_dep_wait();
    grid_dep_launch();
    const float v = norm_of(partials, n, s_w);
    if (threadIdx.x == 0) *norm = v;
}

template <typename T>
__device__ __forceinline__ void scale_unit(const Tensor& t, int64_t e0, int len, bool vec, int lane, float coef, bool exact) {
    constexpr int PER = 16 / sizeof(T);
    const T* src = static_cast<const T*>(t.src) + e0;
    T* dst = static_cast<T*>(t.dst) + e0;
    int done = 0;
    if (vec) {
        const int nv = len / PER;
        const uint4* v = reinterpret_cast<const uint4*>(src);
        uint4* o = reinterpret_cast<uint4*>(dst);
        for (int b = lane; b < nv; b += 32 * GC_VECS) {
            uint4 raw[GC_VECS];
#pragma unroll
            for (int u = 0; u < GC_VECS; ++u)
                if (b + 32 * u < nv) raw[u] = __ldcs(v + b + 32 * u);
#pragma unroll
            for (int u = 0; u < GC_VECS; ++u) {
                if (b + 32 * u >= nv) continue;
                if (!exact) {
                    T* e = reinterpret_cast<T*>(&raw[u]);
#pragma unroll
                    for (int j = 0; j < PER; ++j) e[j] = down<T>(up<T>(e[j]) * coef);
                }
                __stcs(o + b + 32 * u, raw[u]);
            }
        }
        done = nv * PER;
    }
    for (int i = done + lane; i < len; i += 32) dst[i] = exact ? src[i] : down<T>(up<T>(src[i]) * coef);
}

// dst = round(src * coef), coef = norm > max_norm ? max_norm / norm : 1 (NaN for
// a NaN norm).  coef = 1 copies the bits, and leaves a tensor in place alone.
// With `partials` every block adds up the norm itself, and block 0 of the launch
// that has `norm_out` writes it.
__global__ void __launch_bounds__(GC_THREADS, 4)
    scale_kernel(const __grid_constant__ Table t, const float* norm, float max_norm, const double* partials, int64_t sums,
                 float* norm_out) {
    __shared__ double s_w[GC_WARPS];
    grid_dep_wait();
    grid_dep_launch();
    float n;
    if (partials != nullptr) {
        n = norm_of(partials, sums, s_w);
        if (norm_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = n;
    } else {
        n = __ldg(norm);
    }
    const float coef = n > max_norm ? max_norm / n : (n == n ? 1.0f : n);
    const bool exact = coef == 1.0f;
    const int lane = threadIdx.x & 31, units = t.first[t.n];
    const int warps = gridDim.x * GC_WARPS;
    for (int c = units - 1 - static_cast<int>(blockIdx.x * GC_WARPS + (threadIdx.x >> 5)); c >= 0; c -= warps) {
        const Piece p = piece_of(t, c);
        const Tensor& x = t.t[p.i];
        if (exact && x.dst == x.src) continue;
        const bool vec = t.vec[p.i] != 0;
        if (t.dtype[p.i] == BI_F32) scale_unit<float>(x, p.e0, p.len, vec, lane, coef, exact);
        else if (t.dtype[p.i] == BI_BF16) scale_unit<__nv_bfloat16>(x, p.e0, p.len, vec, lane, coef, exact);
        else scale_unit<__half>(x, p.e0, p.len, vec, lane, coef, exact);
    }
}

constexpr int64_t GC_MAX_UNITS = (int64_t(1) << 31) - 1;

// A set's unit: about eight for each warp, so the warps' loads even out and a small
// set's few loads run side by side.
int64_t unit_of(int64_t elements) {
    int64_t u = GC_UNIT_MIN;
    while (u < GC_UNIT_MAX && 2 * u * (8 * GC_BLOCKS * GC_WARPS) <= elements) u *= 2;
    return u;
}
int64_t blocks_of(int64_t units) { return lmin((units + GC_WARPS - 1) / GC_WARPS, GC_BLOCKS); }
struct Cuts {
    int64_t unit, units;
};

bi_status check_set(bi_engine eng, const void* const* src, void* const* dst, bool need_dst, const int64_t* counts,
                    const int* dtypes, int64_t n, Cuts* cuts) {
    if (!eng) return fail(nullptr, BI_ERR_INVALID_ARG, "engine is NULL");
    if (n < 0) return fail(eng, BI_ERR_INVALID_ARG, "n must be >= 0");
    if (n > 0 && (!src || !counts || !dtypes || (need_dst && !dst)))
        return fail(eng, BI_ERR_INVALID_ARG, "the tensor tables must not be NULL");
    *cuts = {GC_UNIT_MIN, 0};
    int64_t elements = 0;
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
        if (counts[i] > GC_MAX_UNITS * GC_UNIT_MAX - elements)
            return fail(eng, BI_ERR_UNSUPPORTED, "the set is beyond 2^31 - 1 units of 16384 elements");
        elements += counts[i];
    }
    cuts->unit = unit_of(elements);
    for (int64_t i = 0; i < n; ++i) {
        const int64_t c = counts[i] / cuts->unit + (counts[i] % cuts->unit != 0);
        if (c > GC_MAX_UNITS - cuts->units)
            return fail(eng, BI_ERR_UNSUPPORTED, "the set is beyond 2^31 - 1 units of 16384 elements");
        cuts->units += c;
    }
    return BI_OK;
}

// Runs `launch(table, units of the launch)` over the set, GC_TENSORS tensors at a
// time; `reverse` starts with the last ones.
template <typename F>
cudaError_t over_set(const void* const* src, void* const* dst, const int64_t* counts, const int* dtypes, int64_t n,
                     bool reverse, const Cuts& cuts, F&& launch) {
    Table t;
    t.unit = static_cast<int>(cuts.unit);
    const int64_t groups = (n + GC_TENSORS - 1) / GC_TENSORS;
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
            at += counts[i] / cuts.unit + (counts[i] % cuts.unit != 0);
        }
        t.first[t.n] = static_cast<int>(at);
        if (at > 0) {
            const cudaError_t e = launch(t, at);
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

// The warps' sums of the set into partials; their number in *sums.
cudaError_t launch_sums(const LaunchCtx& c, const void* const* tensors, const int64_t* counts, const int* dtypes, int64_t n,
                        const Cuts& cuts, double* partials, int64_t* sums) {
    *sums = 0;
    return over_set(tensors, nullptr, counts, dtypes, n, false, cuts, [&](const Table& t, int64_t count) {
        const cudaError_t r = launch_pdl(square_sum_kernel, dim3(static_cast<unsigned>(blocks_of(count))), dim3(GC_THREADS), 0,
                                         c.stream, t, partials + *sums);
        *sums += blocks_of(count) * GC_WARPS;
        if (r == cudaSuccess) c.count();
        return r;
    });
}

cudaError_t launch_scale(const LaunchCtx& c, void* const* dst, const void* const* src, const int64_t* counts,
                         const int* dtypes, int64_t n, const Cuts& cuts, const float* norm, float max_norm,
                         const double* partials, int64_t sums, float* norm_out) {
    return over_set(src, dst, counts, dtypes, n, true, cuts, [&](const Table& t, int64_t count) {
        const cudaError_t r = launch_pdl(scale_kernel, dim3(static_cast<unsigned>(blocks_of(count))), dim3(GC_THREADS), 0,
                                         c.stream, t, norm, max_norm, partials, sums, norm_out);
        norm_out = nullptr;  // written by the first launch
        if (r == cudaSuccess) c.count();
        return r;
    });
}

// One sum per warp of every launch over the set.
int64_t sums_bytes(int64_t n, const Cuts& cuts) {
    const int64_t groups = (n + GC_TENSORS - 1) / GC_TENSORS;
    return lmin(cuts.units + groups * GC_WARPS, groups * GC_BLOCKS * GC_WARPS) * 8;
}
// Up to this many warps' sums are added up by every block of the scaling pass (a
// small set, 24 tensors of 1.5 million f32: 14.7 us with a finishing kernel, 12.6
// without); more would queue for the f64 units (4864 sums, 40 million f32: 80 us
// against 87).
constexpr int64_t GC_FUSE = 1024;

}  // namespace
}  // namespace bi

using namespace bi;

extern "C" {

bi_status bi_grad_norm(bi_engine eng, float* norm, const void* const* tensors, const int64_t* counts,
                       const int* dtypes, int64_t n, void* stream) {
    Cuts cuts;
    bi_status st = check_set(eng, tensors, nullptr, false, counts, dtypes, n, &cuts);
    if (st != BI_OK) return st;
    if (!norm) return fail(eng, BI_ERR_INVALID_ARG, "norm must not be NULL");
    DeviceGuard g(eng->device);
    if (!g.ok) return fail(eng, BI_ERR_CUDA, "cudaSetDevice failed");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cuts.units == 0) {
        const cudaError_t e = cudaMemsetAsync(norm, 0, 4, s);
        return e == cudaSuccess ? BI_OK : cuda_fail(eng, e, "bi_grad_norm");
    }
    const LaunchCtx c = ctx(eng, stream);
    Scratch sc(eng, s, static_cast<size_t>(sums_bytes(n, cuts)));
    if (sc.err != cudaSuccess) return cuda_fail(eng, sc.err, "norm scratch");
    double* partials = static_cast<double*>(sc.ptr);
    int64_t sums = 0;
    cudaError_t e = launch_sums(c, tensors, counts, dtypes, n, cuts, partials, &sums);
    if (e == cudaSuccess) {
        e = launch_pdl(norm_finish_kernel, dim3(1), dim3(GC_THREADS), 0, c.stream, partials, sums, norm);
        if (e == cudaSuccess) c.count();
    }
    return e == cudaSuccess ? BI_OK : cuda_fail(eng, e, "bi_grad_norm");
}

bi_status bi_grad_clip(bi_engine eng, void* const* dst, const void* const* src, const int64_t* counts,
                       const int* dtypes, int64_t n, const float* norm, float max_norm, void* stream) {
    Cuts cuts;
    bi_status st = check_set(eng, src, dst, true, counts, dtypes, n, &cuts);
    if (st != BI_OK) return st;
    if (!norm) return fail(eng, BI_ERR_INVALID_ARG, "norm must not be NULL");
    if (!(max_norm >= 0.0f)) return fail(eng, BI_ERR_INVALID_ARG, "max_norm must be >= 0");
    if (cuts.units == 0) return BI_OK;
    DeviceGuard g(eng->device);
    if (!g.ok) return fail(eng, BI_ERR_CUDA, "cudaSetDevice failed");
    const cudaError_t e =
        launch_scale(ctx(eng, stream), dst, src, counts, dtypes, n, cuts, norm, max_norm, nullptr, 0, nullptr);
    return e == cudaSuccess ? BI_OK : cuda_fail(eng, e, "bi_grad_clip");
}

bi_status bi_grad_norm_clip(bi_engine eng, void* const* dst, const void* const* src, const int64_t* counts,
                            const int* dtypes, int64_t n, float* norm, float max_norm, void* stream) {
    Cuts cuts;
    bi_status st = check_set(eng, src, dst, true, counts, dtypes, n, &cuts);
    if (st != BI_OK) return st;
    if (!norm) return fail(eng, BI_ERR_INVALID_ARG, "norm must not be NULL");
    if (!(max_norm >= 0.0f)) return fail(eng, BI_ERR_INVALID_ARG, "max_norm must be >= 0");
    if (cuts.units == 0 || sums_bytes(n, cuts) / 8 > GC_FUSE) {
        st = bi_grad_norm(eng, norm, src, counts, dtypes, n, stream);
        return st == BI_OK ? bi_grad_clip(eng, dst, src, counts, dtypes, n, norm, max_norm, stream) : st;
    }
    DeviceGuard g(eng->device);
    if (!g.ok) return fail(eng, BI_ERR_CUDA, "cudaSetDevice failed");
    const LaunchCtx c = ctx(eng, stream);
    Scratch sc(eng, static_cast<cudaStream_t>(stream), static_cast<size_t>(sums_bytes(n, cuts)));
    if (sc.err != cudaSuccess) return cuda_fail(eng, sc.err, "norm scratch");
    double* partials = static_cast<double*>(sc.ptr);
    int64_t sums = 0;
    cudaError_t e = launch_sums(c, src, counts, dtypes, n, cuts, partials, &sums);
    if (e == cudaSuccess) e = launch_scale(c, dst, src, counts, dtypes, n, cuts, nullptr, max_norm, partials, sums, norm);
    return e == cudaSuccess ? BI_OK : cuda_fail(eng, e, "bi_grad_norm_clip");
}

}  // extern "C"
