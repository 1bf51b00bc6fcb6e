// MXFP4: 4-bit floating point in blocks of 32 with a power-of-two scale each
// (OCP Microscaling Formats v1.0), quantization, dequantization and the entry
// points of the product.  See include/bi.h (bi_fp4_*); the product is fp4_tc.cu.
//
// A block of 32 consecutive values along the contraction has the scale 2^s,
//   s = max(floor(log2 max|v|) - 2, -127),   kept as the byte s + 127,
// and the codes e2m1(v / 2^s): round to nearest even on {0, .5, 1, 1.5, 2, 3, 4, 6},
// larger ones to 6.  2^s is a power of two, so v / 2^s is exact in f32 (what
// underflows there is far below the smallest code's border), and the code is the
// one rounding.  A block with an infinity or NaN has the scale byte 255 (NaN) and
// codes 0.
//
// Layout of an operand [R][C], contraction along C: codes [R][Cp/2] bytes with
// Cp = C rounded up to 256 (128 bytes, one swizzle row of the product's tiles;
// code 2i in the low half of byte i), and scales in pieces of 128 rows x 4 blocks
// (512 bytes, row r at byte 16 (r % 32) + 4 (r / 32)), pieces [ceil(R/128)][Cp/128]:
// the order in which the tensor cores take scales from shared memory, so the product
// copies them as they are.  Padding has code 0 and scale byte 0.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>

#include "abi_util.h"
#include "fp4.h"

namespace bi {
namespace {

template <typename T> __device__ __forceinline__ float up(T v);
template <> __device__ __forceinline__ float up<float>(float v) { return v; }
template <> __device__ __forceinline__ float up<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float up<__half>(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T down(float v);
template <> __device__ __forceinline__ float down<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 down<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half down<__half>(float v) { return __float2half_rn(v); }

// The scale's byte from the largest magnitude's bits: its exponent field less 2.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    const uint32_t e = amax_bits >> 23;
    return e == 255u ? 255u : (e < 2u ? 0u : e - 2u);
}
// 2^-s of a scale byte <= 252: exponent field 254 - byte, at least 2.
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
    return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}
// Two codes, the first in the low half.
__device__ __forceinline__ uint32_t codes2(float a, float b) {
    return static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(a, b), __NV_E2M1, cudaRoundNearest));
}
// The code of a value of a block without scale is 0: an infinity or NaN times the
// zero inverse is NaN, which the conversion would make the largest code.
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], uint32_t byte) {
    if (byte == 255u) return 0u;
    const float inv = inverse_scale(byte);
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) r |= codes2(v[2 * i] * inv, v[2 * i + 1] * inv) << (8 * i);
    return r;
}
// Largest magnitude as bits: infinities and NaN compare above every number.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// One 128 x 128 tile of src per block: its codes and scales along the columns (q, s)
// and along the rows (qt, st: the operand's transpose), either of them absent.  The
// tile is read once; the rows' direction works on the values as loaded, four
// lanes to a block of 32, the columns' direction on the tile in shared memory, a
// thread to a column's block.  Bound by memory: src read once, a quarter (bf16) of
// it written per direction.
constexpr int QT = 128;            // tile edge
constexpr int Q_THREADS = 256;
template <typename T> constexpr int q_pitch() { return QT + 8 / static_cast<int>(sizeof(T)); }  // elements
template <typename T> constexpr int q_smem(bool cols) { return cols ? QT * q_pitch<T>() * static_cast<int>(sizeof(T)) + QT * 80 : 0; }

template <typename T>
__global__ void __launch_bounds__(Q_THREADS) fp4_quantize_kernel(const T* __restrict__ src, uint8_t* q, uint8_t* s, uint8_t* qt,
                                                                uint8_t* st, int64_t R, int64_t C, int tiles_c, int vec) {
    grid_dep_wait();
    grid_dep_launch();
    extern __shared__ __align__(16) uint8_t smem_raw[];
    T* tile = reinterpret_cast<T*>(smem_raw);
    uint8_t* tcode = smem_raw + QT * q_pitch<T>() * sizeof(T);  // [128 columns][80]: 64 bytes of codes
    __shared__ __align__(16) uint8_t sc[2][512];
    const int tc = static_cast<int>(blockIdx.x % static_cast<unsigned>(tiles_c));
    const int tr = static_cast<int>(blockIdx.x / static_cast<unsigned>(tiles_c));
    const int64_t r0 = static_cast<int64_t>(tr) * QT, c0 = static_cast<int64_t>(tc) * QT;
    const int64_t Cp = fp4_padded(C), Rp = fp4_padded(R);
    const int tid = threadIdx.x;

    // 16 lanes to a row of the tile, 8 values each
    const int row_in = tid >> 4, part = tid & 15;
    const int64_t c = c0 + part * 8;
#pragma unroll 4
    for (int i = 0; i < QT / 16; ++i) {
        const int lr = i * 16 + row_in;
        const int64_t r = r0 + lr;
        float v[8];
        const bool in = r < R && c < C;
        if (in && vec && c + 8 <= C) {
            const uint4* p = reinterpret_cast<const uint4*>(src + r * C + c);
            if constexpr (sizeof(T) == 4) {
                const uint4 a = __ldcs(p), b = __ldcs(p + 1);
                v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
                v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
            } else {
                const uint4 a = __ldcs(p);
                const T* e = reinterpret_cast<const T*>(&a);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = up<T>(e[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = in && c + j < C ? up<T>(src[r * C + c + j]) : 0.0f;
        }
        if (q != nullptr) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, mag(v[j]));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const uint32_t byte = scale_byte(m);
            const uint32_t code = codes8(v, byte);
            if (r < R && c < Cp) *reinterpret_cast<uint32_t*>(q + r * (Cp / 2) + c / 2) = code;
            if ((part & 3) == 0) sc[0][(lr & 31) * 16 + (lr >> 5) * 4 + (part >> 2)] = static_cast<uint8_t>(r < R ? byte : 0u);
        }
        if (qt != nullptr) {
            T* d = tile + lr * q_pitch<T>() + part * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = down<T>(v[j]);  // exact: the value came from T
        }
    }
    __syncthreads();
    if (q != nullptr && tr < (R + QT - 1) / QT && tid < 32)
        reinterpret_cast<uint4*>(s + (static_cast<int64_t>(tr) * (Cp / QT) + tc) * 512)[tid] = reinterpret_cast<const uint4*>(sc[0])[tid];
    if (qt == nullptr || c0 >= C) return;
    // a column's block of 32 rows per thread, two of them
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int lc = tid & 127, b = (tid >> 7) + 2 * i;
        const T* colp = tile + b * 32 * q_pitch<T>() + lc;
        float v[4][8];
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            v[j >> 3][j & 7] = up<T>(colp[j * q_pitch<T>()]);
            m = max(m, mag(v[j >> 3][j & 7]));
        }
        const uint32_t byte = scale_byte(m);
        uint4 o;
        o.x = codes8(v[0], byte);
        o.y = codes8(v[1], byte);
        o.z = codes8(v[2], byte);
        o.w = codes8(v[3], byte);
        *reinterpret_cast<uint4*>(tcode + lc * 80 + b * 16) = o;
        sc[1][(lc & 31) * 16 + (lc >> 5) * 4 + b] = static_cast<uint8_t>(byte);  // columns past C are zeros: byte 0
    }
    __syncthreads();
    if (r0 < Rp) {
        for (int i = tid; i < QT * 4; i += Q_THREADS) {
            const int lc = i >> 2, part4 = i & 3;
            if (c0 + lc < C)
                *reinterpret_cast<uint4*>(qt + (c0 + lc) * (Rp / 2) + r0 / 2 + part4 * 16) =
                    *reinterpret_cast<const uint4*>(tcode + lc * 80 + part4 * 16);
        }
        if (tid < 32)
            reinterpret_cast<uint4*>(st + (static_cast<int64_t>(tc) * (Rp / QT) + tr) * 512)[tid] =
                reinterpret_cast<const uint4*>(sc[1])[tid];
    }
}

// dst[r][c] = code * 2^s, rounded to T (exact where T's range holds it).  Eight
// values per thread and step.
template <typename T>
__global__ void __launch_bounds__(256) fp4_dequantize_kernel(T* dst, const uint8_t* __restrict__ q, const uint8_t* __restrict__ s,
                                                             int64_t R, int64_t C, int vec) {
    grid_dep_wait();
    grid_dep_launch();
    const int64_t per = (C + 7) / 8, n = R * per, Cp = fp4_padded(C);
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        const int64_t r = i / per, c = (i - r * per) * 8;
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(q + r * (Cp / 2) + c / 2));
        const uint32_t byte = __ldg(s + fp4_scale_at(r, c / 32, Cp));
        const float scale = fp4_scale_value(byte);
        T o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = down<T>(fp4_code_value((w >> (4 * j)) & 15u) * scale);
        T* d = dst + r * C + c;
        if (vec && c + 8 <= C) {
#pragma unroll
            for (int j = 0; j < static_cast<int>(sizeof(T)) / 2; ++j) reinterpret_cast<uint4*>(d)[j] = reinterpret_cast<const uint4*>(o)[j];
        } else {
            for (int j = 0; j < 8 && c + j < C; ++j) d[j] = o[j];
        }
    }
}

template <typename T>
cudaError_t quantize_t(const LaunchCtx& c, uint8_t* q, uint8_t* s, uint8_t* qt, uint8_t* st, const void* src, int64_t R, int64_t C) {
    // tiles of the padded operands: along the columns to a multiple of 256, along the
    // rows too where the transpose is asked for
    const int64_t tiles_c = q ? fp4_padded(C) / QT : (C + QT - 1) / QT;
    const int64_t tiles_r = qt ? fp4_padded(R) / QT : (R + QT - 1) / QT;
    if (tiles_c * tiles_r > 0x7fffffffll) return cudaErrorInvalidValue;
    const int smem = q_smem<T>(qt != nullptr);
    auto kern = fp4_quantize_kernel<T>;
    static PerDeviceOnce setup;
    const cudaError_t e = setup.run(c.eng->device, [&](int&) {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, q_smem<T>(true));
    });
    if (e != cudaSuccess) return e;
    const int vec = C % (16 / static_cast<int64_t>(sizeof(T))) == 0 && aligned16(src);
    const cudaError_t l = launch_pdl(kern, dim3(static_cast<unsigned>(tiles_c * tiles_r)), dim3(Q_THREADS), smem, c.stream,
                                     static_cast<const T*>(src), q, s, qt, st, R, C, static_cast<int>(tiles_c), vec);
    if (l != cudaSuccess) return l;
    c.count();
    return cudaGetLastError();
}

template <typename T>
cudaError_t dequantize_t(const LaunchCtx& c, void* dst, const uint8_t* q, const uint8_t* s, int64_t R, int64_t C) {
    const int64_t n = R * ((C + 7) / 8);
    const int64_t blocks = lmin((n + 255) / 256, static_cast<int64_t>(c.sm_count) * 16);
    const int vec = C % 8 == 0 && aligned16(dst);
    const cudaError_t l = launch_pdl(fp4_dequantize_kernel<T>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, c.stream,
                                     static_cast<T*>(dst), q, s, R, C, vec);
    if (l != cudaSuccess) return l;
    c.count();
    return cudaGetLastError();
}

constexpr int64_t FP4_MAX_DIM = 0x7fffff00ll;

bi_status check_matrix(bi_engine eng, bi_dtype dt, int64_t rows, int64_t cols) {
    if (!eng) return fail(nullptr, BI_ERR_INVALID_ARG, "engine is NULL");
    if (dt != BI_F32 && dt != BI_BF16 && dt != BI_F16) return fail(eng, BI_ERR_INVALID_ARG, "dtype must be BI_F32, BI_BF16 or BI_F16");
    if (rows < 0 || cols <= 0) return fail(eng, BI_ERR_INVALID_ARG, "rows must be >= 0 and cols > 0");
    if (rows > FP4_MAX_DIM || cols > FP4_MAX_DIM || fp4_padded(rows) / QT * (fp4_padded(cols) / QT) > 0x7fffffffll)
        return fail(eng, BI_ERR_UNSUPPORTED, "rows and cols are limited to 2^31 - 256, and to 2^31 - 1 tiles of 128 x 128");
    return BI_OK;
}

}  // namespace
}  // namespace bi

using bi::aligned16;
using bi::ctx;
using bi::cuda_fail;
using bi::DeviceGuard;
using bi::fail;

extern "C" {

int64_t bi_fp4_code_bytes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0 || rows > bi::FP4_MAX_DIM || cols > bi::FP4_MAX_DIM) return -1;
    return rows * (bi::fp4_padded(cols) / 2);
}

int64_t bi_fp4_scale_bytes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0 || rows > bi::FP4_MAX_DIM || cols > bi::FP4_MAX_DIM) return -1;
    return (rows + 127) / 128 * (bi::fp4_padded(cols) / 128) * 512;
}

bi_status bi_fp4_quantize(bi_engine eng, uint8_t* q, uint8_t* s, uint8_t* qt, uint8_t* st, const void* src, int64_t rows,
                          int64_t cols, bi_dtype dtype, void* stream) {
    const bi_status stt = bi::check_matrix(eng, dtype, rows, cols);
    if (stt != BI_OK) return stt;
    if ((q == nullptr) != (s == nullptr) || (qt == nullptr) != (st == nullptr))
        return fail(eng, BI_ERR_INVALID_ARG, "codes and scales go together: q with s, qt with st");
    if (rows == 0) return BI_OK;
    if (!src || (!q && !qt)) return fail(eng, BI_ERR_INVALID_ARG, "src, and q with s or qt with st, must not be NULL");
    if (!aligned16(q) || !aligned16(s) || !aligned16(qt) || !aligned16(st))
        return fail(eng, BI_ERR_MISALIGNED, "codes and scales need 16-byte alignment");
    DeviceGuard g(eng->device);
    if (!g.ok) return fail(eng, BI_ERR_CUDA, "cudaSetDevice failed");
    const bi::LaunchCtx c = ctx(eng, stream);
    const cudaError_t e = dtype == BI_F32    ? bi::quantize_t<float>(c, q, s, qt, st, src, rows, cols)
                          : dtype == BI_BF16 ? bi::quantize_t<__nv_bfloat16>(c, q, s, qt, st, src, rows, cols)
                                             : bi::quantize_t<__half>(c, q, s, qt, st, src, rows, cols);
    return e == cudaSuccess ? BI_OK : cuda_fail(eng, e, "bi_fp4_quantize");
}

bi_status bi_fp4_dequantize(bi_engine eng, void* dst, const uint8_t* q, const uint8_t* s, int64_t rows, int64_t cols,
                            bi_dtype dtype, void* stream) {
    const bi_status stt = bi::check_matrix(eng, dtype, rows, cols);
    if (stt != BI_OK) return stt;
    if (rows == 0) return BI_OK;
    if (!dst || !q || !s) return fail(eng, BI_ERR_INVALID_ARG, "dst, q and s must not be NULL");
    if (!aligned16(q) || !aligned16(s)) return fail(eng, BI_ERR_MISALIGNED, "codes and scales need 16-byte alignment");
    DeviceGuard g(eng->device);
    if (!g.ok) return fail(eng, BI_ERR_CUDA, "cudaSetDevice failed");
    const bi::LaunchCtx c = ctx(eng, stream);
    const cudaError_t e = dtype == BI_F32    ? bi::dequantize_t<float>(c, dst, q, s, rows, cols)
                          : dtype == BI_BF16 ? bi::dequantize_t<__nv_bfloat16>(c, dst, q, s, rows, cols)
                                             : bi::dequantize_t<__half>(c, dst, q, s, rows, cols);
    return e == cudaSuccess ? BI_OK : cuda_fail(eng, e, "bi_fp4_dequantize");
}

}  // extern "C"

namespace {

// out [rows][cols] = a [rows][depth] b [cols][depth]^T (+ bias), both operands in MXFP4.
bi_status fp4_product(bi_engine eng, void* out, const uint8_t* a, const uint8_t* as, const uint8_t* b, const uint8_t* bs,
                      const void* bias, int64_t rows, int64_t cols, int64_t depth, bool zero_depth, bi_dtype out_dtype, void* stream,
                      const char* name) {
    if (!out || (!zero_depth && (!a || !as || !b || !bs)))
        return fail(eng, BI_ERR_INVALID_ARG, "outputs, codes and scales must not be NULL");
    if (!aligned16(a) || !aligned16(as) || !aligned16(b) || !aligned16(bs))
        return fail(eng, BI_ERR_MISALIGNED, "codes and scales need 16-byte alignment");
    if (reinterpret_cast<uintptr_t>(out) % bi::dsize(out_dtype) != 0 || reinterpret_cast<uintptr_t>(bias) % bi::dsize(out_dtype) != 0)
        return fail(eng, BI_ERR_MISALIGNED, "outputs and bias need the alignment of their type");
    DeviceGuard g(eng->device);
    if (!g.ok) return fail(eng, BI_ERR_CUDA, "cudaSetDevice failed");
    cudaError_t e;
    if (zero_depth)
        e = cudaMemsetAsync(out, 0, static_cast<size_t>(rows * cols * bi::dsize(out_dtype)), static_cast<cudaStream_t>(stream));
    else
        e = bi::tc_fp4_product(ctx(eng, stream), out_dtype, out, a, as, b, bs, bias, rows, cols, depth);
    return e == cudaSuccess ? BI_OK : cuda_fail(eng, e, name);
}

bi_status check_product(bi_engine eng, bi_dtype dt, int64_t m, int64_t k, int64_t n) {
    if (!eng) return fail(nullptr, BI_ERR_INVALID_ARG, "engine is NULL");
    const char* why = "";
    const bi_status st = bi::check_sizes(dt, m, k, n, -1, &why);
    if (st != BI_OK) return fail(eng, st, why);
    // 256 x 256 output tiles are counted in 32 bits
    const int64_t tm = (m + 255) / 256, tn = (n + 255) / 256, tk = (k + 255) / 256;
    if (m > bi::FP4_MAX_DIM || tm * tn > 0x3fffffffll || tm * tk > 0x3fffffffll || tk * tn > 0x3fffffffll)
        return fail(eng, BI_ERR_UNSUPPORTED, "more than 2^30 - 1 output tiles of 256 x 256");
    return BI_OK;
}

}  // namespace

extern "C" {

bi_status bi_fp4_forward(bi_engine eng, void* y, const uint8_t* xq, const uint8_t* xs, const uint8_t* wq, const uint8_t* ws,
                         const void* bias, int64_t m, int64_t k, int64_t n, bi_dtype out_dtype, void* stream) {
    const bi_status st = check_product(eng, out_dtype, m, k, n);
    if (st != BI_OK || m == 0) return st;
    return fp4_product(eng, y, xq, xs, wq, ws, bias, m, n, k, false, out_dtype, stream, "bi_fp4_forward");
}

bi_status bi_fp4_backward_dx(bi_engine eng, void* dx, const uint8_t* gq, const uint8_t* gs, const uint8_t* wq, const uint8_t* ws,
                             int64_t m, int64_t k, int64_t n, bi_dtype out_dtype, void* stream) {
    const bi_status st = check_product(eng, out_dtype, m, k, n);
    if (st != BI_OK || m == 0) return st;
    return fp4_product(eng, dx, gq, gs, wq, ws, nullptr, m, k, n, false, out_dtype, stream, "bi_fp4_backward_dx");
}

bi_status bi_fp4_backward_dw(bi_engine eng, void* dw, const uint8_t* xq, const uint8_t* xs, const uint8_t* gq, const uint8_t* gs,
                             int64_t m, int64_t k, int64_t n, bi_dtype out_dtype, void* stream) {
    const bi_status st = check_product(eng, out_dtype, m, k, n);
    if (st != BI_OK) return st;
    return fp4_product(eng, dw, xq, xs, gq, gs, nullptr, k, n, m, m == 0, out_dtype, stream, "bi_fp4_backward_dw");
}

}  // extern "C"
