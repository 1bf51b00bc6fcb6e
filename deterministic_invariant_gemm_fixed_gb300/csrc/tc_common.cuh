// What the tensor-core kernels share: mbarriers with bounded waits, shared-memory
// matrix descriptors, tensor-memory loads, output types, tensor maps.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bi_internal.h"

namespace bi {

// ---------------------------------------------------------------- PTX helpers

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ unsigned long long globaltimer() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Bounded wait.  Returns false if this CTA is aborting or the limit ran out
// (then the status word is written and the CTA-wide abort flag raised).
static __device__ __noinline__ bool mbar_wait_impl(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                            int* status, unsigned long long limit, int code) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = globaltimer();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 15u) == 0) {
            if (*abort_flag) return false;
            if (globaltimer() - t0 > limit) {
                *abort_flag = 1;
                if (status) *reinterpret_cast<volatile int*>(status) = code;
                return false;
            }
        }
    }
}
#define mbar_wait(bar, parity, abort_flag, p, code) \
    mbar_wait_impl((bar), (parity), (abort_flag), (p).status, (p).wait_limit, (code))
// The same with the first try inline: a barrier that is complete costs no call.
#define mbar_wait_fast(bar, parity, abort_flag, p, code) \
    (mbar_try_wait((bar), (parity)) || mbar_wait((bar), (parity), (abort_flag), p, (code)))

// A wait for what is in flight, by a CTA that gives up: nothing but the time ends it
// early (the abort flag is up already, and the limit of the ordinary waits may have
// been set to nearly nothing).
constexpr unsigned long long DRAIN_LIMIT_NS = 2000000000ull;
static __device__ __noinline__ void mbar_drain(uint32_t bar, uint32_t parity) {
    const unsigned long long t0 = globaltimer();
    while (!mbar_try_wait(bar, parity) && globaltimer() - t0 <= DRAIN_LIMIT_NS) {}
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void fence_proxy_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Shared-memory matrix descriptor (tcgen05 format): start address, leading and
// stride byte offsets (>> 4), version 1 at bit 46, 128-byte swizzle (2) at bit 61.
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32;
    d |= 1ull << 46;
    d |= 2ull << 61;
    return d;
}

// Low and high word of a tile's descriptor (128-byte swizzle, 8-row groups 1024
// bytes apart): K-major, or MN-major with 8192 bytes from one 64-column atom to
// the next.  One MMA's step along K: 32 bytes, or 16 rows of 128.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, bool mn) { return ((saddr & 0x3FFFFu) >> 4) | ((mn ? 512u : 1u) << 16); }
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t K_STEP = 32 >> 4, MN_STEP_16 = 2048 >> 4;

// 1 in one lane of the warp, always the same.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
    return r;
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
          "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ---------------------------------------------------------------- output types

template <int FMT> struct OutT;
template <> struct OutT<0> {
    using T = __half;
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&h);
    }
    static __device__ __forceinline__ float load(const void* p, int64_t i) {
        return __half2float(reinterpret_cast<const __half*>(p)[i]);
    }
    static __device__ __forceinline__ void store1(void* p, int64_t i, float v) {
        reinterpret_cast<__half*>(p)[i] = __float2half_rn(v);
    }
};
template <> struct OutT<1> {
    using T = __nv_bfloat16;
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&h);
    }
    static __device__ __forceinline__ float load(const void* p, int64_t i) {
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
    }
    static __device__ __forceinline__ void store1(void* p, int64_t i, float v) {
        reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    }
};

// ---------------------------------------------------------------- tensor maps

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// 16-bit row-major tensor [outer][inner] (optionally [depth][outer][inner]),
// box {64, box_outer(, 1)}, 128-byte swizzle, zero fill out of bounds.
inline cudaError_t make_map(CUtensorMap* m, bi_dtype dt, const void* ptr, uint64_t inner, uint64_t outer,
                     uint64_t depth, uint32_t box_outer, bool rank3 = false) {
    auto enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const CUtensorMapDataType t =
        dt == BI_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    cuuint64_t dims[3] = {inner, outer, depth};
    cuuint64_t strides[2] = {inner * 2, inner * outer * 2};
    cuuint32_t box[3] = {64, box_outer, 1};
    cuuint32_t es[3] = {1, 1, 1};
    const cuuint32_t rank = rank3 ? 3 : 2;
    CUresult r = enc(m, t, rank, const_cast<void*>(ptr), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Output [depth][outer][inner] (row stride ld elements; out_fmt 0 f16, 1 bf16,
// 2 f32) for the TMA-store epilogue: box {128 bytes of columns, 32 rows (, 1)},
// 128-byte swizzle; stores past the extents are clipped.
inline cudaError_t make_out_map(CUtensorMap* m, int out_fmt, const void* ptr, uint64_t inner, uint64_t outer, uint64_t ld,
                         uint64_t depth = 1, bool rank3 = false) {
    auto enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const CUtensorMapDataType t = out_fmt == 2 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                : out_fmt == 1 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                               : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const uint64_t es = out_fmt == 2 ? 4 : 2;
    cuuint64_t dims[3] = {inner, outer, depth};
    cuuint64_t strides[2] = {ld * es, ld * outer * es};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / es), 32, 1};
    cuuint32_t el[3] = {1, 1, 1};
    CUresult r = enc(m, t, rank3 ? 3 : 2, const_cast<void*>(ptr), dims, strides, box, el,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// 32-bit K-major tensor [outer][inner] with row stride ld elements (ld >= inner,
// a multiple of 4), box {32, box_outer}, 128-byte swizzle.
inline cudaError_t make_map32(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer, uint64_t ld, uint32_t box_outer) {
    auto enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    cuuint64_t dims[2] = {inner, outer};
    cuuint64_t strides[1] = {ld * 4};
    cuuint32_t box[2] = {32, box_outer};
    cuuint32_t es[2] = {1, 1};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(ptr), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace bi
