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

#include <type_traits>

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
// Eight codes, the first in the lowest half byte.
__device__ __forceinline__ uint32_t codes_of(float a, float b, float c, float d, float e, float f, float g, float h) {
    uint32_t r;
    asm("{\n\t.reg .b8 w, x, y, z;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 w, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 x, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 y, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 z, %8, %7;\n\t"
        "mov.b32 %0, {w, x, y, z};\n\t}" : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d), "f"(e), "f"(f), "f"(g), "f"(h));
    return r;
}
// The code of a value of a block without scale is 0: an infinity or NaN times the
// zero inverse is NaN, which the conversion would make the largest code.
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], uint32_t byte) {
    if (byte == 255u) return 0u;
    const float inv = inverse_scale(byte);
    return codes_of(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv, v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
}
// The same of two columns of bf16, in the halves of eight words, with a block each: the
// products of a pair at once (exact, but for values far below the smallest code's border).
__device__ __forceinline__ void codes8x2_bf16(const uint32_t* w, uint32_t byte0, uint32_t byte1, uint32_t& c0, uint32_t& c1) {
    const uint32_t inv = (byte0 == 255u ? 0u : (254u - byte0) << 7) | (byte1 == 255u ? 0u : (254u - byte1) << 23);
    uint32_t p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(p[i]) : "r"(w[i]), "r"(inv));
    auto lo = [&](int i) { return __uint_as_float(p[i] << 16); };
    auto hi = [&](int i) { return __uint_as_float(p[i] & 0xffff0000u); };
    c0 = codes_of(lo(0), lo(1), lo(2), lo(3), lo(4), lo(5), lo(6), lo(7));
    c1 = codes_of(hi(0), hi(1), hi(2), hi(3), hi(4), hi(5), hi(6), hi(7));
    if (byte0 == 255u) c0 = 0;
    if (byte1 == 255u) c1 = 0;
}
// Largest magnitude as bits: infinities and NaN compare above every number.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// One tile of src per block, TR rows (32 or 128) by 128 columns: its codes and scales
// along the columns (q, s) and along the rows (qt, st: the operand's transpose), either of
// them absent.  The tile is read once, all of a thread's loads in flight together; the
// rows' direction works on the values as loaded, four lanes to a block of 32, the
// columns' direction on the tile in shared memory, a thread to a block of one column (two
// columns of 16-bit values, whose magnitudes are compared in pairs).
//
// Issue, beside memory, is what is busiest where there are many tiles (8192 x 4096 in bf16, both
// directions: 103 MB in 25 us, issue 70 %); the rows' direction scales bf16 a value at a time,
// where the columns' scales pairs.  A small matrix waits for one tile's chain of steps instead, and
// takes the tiles of 32 rows, whose chain is a third as long; their column direction
// writes 16 bytes at a time where the others write 64.
constexpr int QT = 128;            // tile columns
constexpr int Q_THREADS = 256;
template <typename T> constexpr int q_pitch() { return QT + 16 / static_cast<int>(sizeof(T)); }  // elements: rows stay on 16 bytes
template <typename T, int TR> constexpr int q_smem(bool cols) { return cols ? TR * q_pitch<T>() * static_cast<int>(sizeof(T)) + QT * (TR / 2 + 16) : 0; }

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// The f32 bits of a 16-bit magnitude.
template <typename T> __device__ __forceinline__ uint32_t mag16(uint32_t h) {
    if constexpr (sizeof(T) == 4) return h;
    else return __float_as_uint(up<T>(*reinterpret_cast<const T*>(&h)));
}

template <typename T, int TR>
__global__ void __launch_bounds__(Q_THREADS) fp4_quantize_kernel(const T* __restrict__ src, uint8_t* q, uint8_t* s, uint8_t* qt,
                                                                uint8_t* st, int64_t R, int64_t C, int tiles_c, int vec) {
    grid_dep_wait();
    grid_dep_launch();
    constexpr int WORDS = 2 * static_cast<int>(sizeof(T));  // 32-bit words of eight values
    constexpr int ROUNDS = TR / 16, PITCH = q_pitch<T>(), CPITCH = TR / 2 + 16;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    T* tile = reinterpret_cast<T*>(smem_raw);
    uint8_t* tcode = smem_raw + TR * PITCH * sizeof(T);  // [128 columns][CPITCH]: TR / 2 bytes of codes
    __shared__ __align__(16) uint8_t row_scale[TR][4];
    __shared__ __align__(16) uint8_t col_scale[QT][4];
    const int tc = static_cast<int>(blockIdx.x % static_cast<unsigned>(tiles_c));
    const int64_t tr = blockIdx.x / static_cast<unsigned>(tiles_c);
    const int64_t r0 = tr * TR, c0 = static_cast<int64_t>(tc) * QT;
    const int64_t Cp = fp4_padded(C), Rp = fp4_padded(R);
    const int tid = threadIdx.x;

    // 16 lanes to a row of the tile, 8 values each
    const int row_in = tid >> 4, part = tid & 15;
    const int64_t c = c0 + part * 8;
    constexpr int GROUP = sizeof(T) == 4 && ROUNDS > 4 ? 4 : ROUNDS;  // rows in flight
#pragma unroll
    for (int g = 0; g < ROUNDS; g += GROUP) {
        uint32_t w[GROUP][WORDS];
#pragma unroll
        for (int i = 0; i < GROUP; ++i) {
            const int64_t r = r0 + (g + i) * 16 + row_in;
            const bool in = r < R && c < C;
            if (in && vec && c + 8 <= C) {
                const uint4* p = reinterpret_cast<const uint4*>(src + r * C + c);
#pragma unroll
                for (int x = 0; x < WORDS; x += 4) {
                    const uint4 a = __ldcs(p + x / 4);
                    w[i][x] = a.x; w[i][x + 1] = a.y; w[i][x + 2] = a.z; w[i][x + 3] = a.w;
                }
            } else {
                T* e = reinterpret_cast<T*>(w[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) e[j] = in && c + j < C ? src[r * C + c + j] : down<T>(0.0f);
            }
        }
#pragma unroll
        for (int i = 0; i < GROUP; ++i) {
            const int lr = (g + i) * 16 + row_in;
            if (q != nullptr) {
                uint32_t m = 0;
                if constexpr (WORDS == 4) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) m = max_u16x2(m, w[i][x] & 0x7fff7fffu);
                    m = max(m >> 16, m & 0xffffu);
                } else {
#pragma unroll
                    for (int x = 0; x < WORDS; ++x) m = max(m, w[i][x] & 0x7fffffffu);
                }
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const uint32_t byte = scale_byte(mag16<T>(m));
                float v[8];
                const T* e = reinterpret_cast<const T*>(w[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = up<T>(e[j]);
                const uint32_t code = codes8(v, byte);
                const int64_t r = r0 + lr;
                if (r < R) *reinterpret_cast<uint32_t*>(q + r * (Cp / 2) + c / 2) = code;
                if ((part & 3) == 0) row_scale[lr][part >> 2] = static_cast<uint8_t>(r < R ? byte : 0u);
            }
            if (qt != nullptr) {
                uint4* d = reinterpret_cast<uint4*>(tile + lr * PITCH + part * 8);
#pragma unroll
                for (int x = 0; x < WORDS; x += 4) d[x / 4] = make_uint4(w[i][x], w[i][x + 1], w[i][x + 2], w[i][x + 3]);
            }
        }
    }
    __syncthreads();
    if (q != nullptr && tid < TR && r0 + tid < (R + 127) / 128 * 128)
        *reinterpret_cast<uint32_t*>(s + fp4_scale_at(r0 + tid, c0 / 32, Cp)) = *reinterpret_cast<const uint32_t*>(row_scale[tid]);
    if (qt == nullptr || c0 >= C) return;
    if constexpr (WORDS == 4) {  // two columns' blocks of 32 rows per thread
        if (tid < 64 * (TR / 32)) {
            const int lc = (tid & 63) * 2, b = tid >> 6;
            const uint32_t* colp = reinterpret_cast<const uint32_t*>(tile + b * 32 * PITCH + lc);
            uint32_t w[32], m = 0;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                w[j] = colp[j * PITCH / 2];
                m = max_u16x2(m, w[j] & 0x7fff7fffu);
            }
            if constexpr (!std::is_same<T, __half>::value) {
                const uint32_t b0 = scale_byte(m << 16), b1 = scale_byte(m & 0xffff0000u);
                uint32_t o[2][4];
#pragma unroll
                for (int x = 0; x < 4; ++x) codes8x2_bf16(w + 8 * x, b0, b1, o[0][x], o[1][x]);
#pragma unroll
                for (int h = 0; h < 2; ++h) *reinterpret_cast<uint4*>(tcode + (lc + h) * CPITCH + b * 16) = make_uint4(o[h][0], o[h][1], o[h][2], o[h][3]);
                col_scale[lc][b] = static_cast<uint8_t>(b0);  // columns past C are zeros: byte 0
                col_scale[lc + 1][b] = static_cast<uint8_t>(b1);
            } else
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t byte = scale_byte(mag16<T>(h ? m >> 16 : m & 0xffffu));
                uint32_t o[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = up<T>(reinterpret_cast<const T*>(&w[8 * x + j])[h]);
                    o[x] = codes8(v, byte);
                }
                *reinterpret_cast<uint4*>(tcode + (lc + h) * CPITCH + b * 16) = make_uint4(o[0], o[1], o[2], o[3]);
                col_scale[lc + h][b] = static_cast<uint8_t>(byte);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < (TR == 128 ? 2 : 1); ++i) {
            const int lc = tid & 127, b = (tid >> 7) + 2 * i;
            if (b >= TR / 32) break;
            const T* colp = tile + b * 32 * PITCH + lc;
            float v[4][8];
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                v[j >> 3][j & 7] = up<T>(colp[j * PITCH]);
                m = max(m, mag(v[j >> 3][j & 7]));
            }
            const uint32_t byte = scale_byte(m);
            *reinterpret_cast<uint4*>(tcode + lc * CPITCH + b * 16) =
                make_uint4(codes8(v[0], byte), codes8(v[1], byte), codes8(v[2], byte), codes8(v[3], byte));
            col_scale[lc][b] = static_cast<uint8_t>(byte);
        }
    }
    __syncthreads();
    constexpr int PIECES = TR / 32;  // of 16 bytes in a column's codes
    for (int i = tid; i < QT * PIECES; i += Q_THREADS) {
        const int lc = i / PIECES, piece = i % PIECES;
        if (c0 + lc < C)
            *reinterpret_cast<uint4*>(qt + (c0 + lc) * (Rp / 2) + r0 / 2 + piece * 16) =
                *reinterpret_cast<const uint4*>(tcode + lc * CPITCH + piece * 16);
    }
    if (tid < QT) {
        uint8_t* to = st + fp4_scale_at(c0 + tid, r0 / 32, Rp);
        if constexpr (TR == 128) *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(col_scale[tid]);
        else *to = col_scale[tid][0];
    }
}

// dst[r][c] = code * 2^s, rounded to T (exact where T's range holds it).  Eight values
// per thread and row, threads along the columns, several rows in flight (16 values of
// 16 bits: 24 against 22 us for 8192 x 4096, half of each store's sector at a time).
template <typename T>
__global__ void __launch_bounds__(256) fp4_dequantize_kernel(T* dst, const uint8_t* __restrict__ q, const uint8_t* __restrict__ s,
                                                             int64_t R, int64_t C, int vec) {
    grid_dep_wait();
    grid_dep_launch();
    constexpr int ROWS = 4, V = 8;
    const int64_t c = (blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x) * V, Cp = fp4_padded(C);
    if (c >= C) return;
    const int64_t step = static_cast<int64_t>(gridDim.y) * blockDim.y;
    for (int64_t ra = blockIdx.y * static_cast<int64_t>(blockDim.y) + threadIdx.y; ra < R; ra += ROWS * step) {
        uint32_t w[ROWS], byte[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int64_t r = lmin(ra + i * step, R - 1);
            w[i] = __ldg(reinterpret_cast<const uint32_t*>(q + r * (Cp / 2) + c / 2));
            byte[i] = __ldg(s + fp4_scale_at(r, c / 32, Cp));
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int64_t r = ra + i * step;
            if (r >= R) break;
            // a code's bits as an f32's (or bf16's) are the value * 2^-126; 2^126 2^s as one
            // factor where it is in range
            const bool one = byte[i] <= 128u;
            if constexpr (sizeof(T) == 2 && !std::is_same<T, __half>::value) {
                // bf16: codes j and j + 4 in the halves of a register, one product for both
                if (one && vec) {
                    const uint32_t f = (byte[i] + 126u) * 0x00800080u;
                    uint32_t p[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t u = w[i] << (12 - 4 * j);
                        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(p[j]) : "r"((u & 0x80008000u) | ((u >> 6) & 0x01c001c0u)), "r"(f));
                    }
                    __stcs(reinterpret_cast<uint4*>(dst + r * C + c),
                           make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410), __byte_perm(p[0], p[1], 0x7632),
                                      __byte_perm(p[2], p[3], 0x7632)));
                    continue;
                }
            }
            const float scale = one ? __uint_as_float((byte[i] + 126u) << 23) : fp4_scale_value(byte[i]);
            __align__(16) T o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const uint32_t code = w[i] >> (4 * j);
                float v = __uint_as_float(((code & 8u) << 28) | ((code & 7u) << 22));
                if (!one) v *= 8.507059173023462e37f;
                o[j] = down<T>(v * scale);
            }
            T* d = dst + r * C + c;
            if (vec && c + V <= C) {
#pragma unroll
                for (int j = 0; j < V * static_cast<int>(sizeof(T)) / 16; ++j) __stcs(reinterpret_cast<uint4*>(d) + j, reinterpret_cast<const uint4*>(o)[j]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (c + j < C) d[j] = o[j];
            }
        }
    }
}

template <typename T, int TR>
cudaError_t quantize_tiles(const LaunchCtx& c, uint8_t* q, uint8_t* s, uint8_t* qt, uint8_t* st, const void* src, int64_t R, int64_t C) {
    // tiles of the padded operands: along the columns to a multiple of 256, along the
    // rows too where the transpose is asked for, to whole pieces of scales where not
    const int64_t tiles_c = q ? fp4_padded(C) / QT : (C + QT - 1) / QT;
    const int64_t tiles_r = (qt ? fp4_padded(R) : (R + 127) / 128 * 128) / TR;
    auto kern = fp4_quantize_kernel<T, TR>;
    static PerDeviceOnce setup;
    const cudaError_t e = setup.run(c.eng->device, [&](int&) {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, q_smem<T, TR>(true));
    });
    if (e != cudaSuccess) return e;
    const int vec = C % (16 / static_cast<int64_t>(sizeof(T))) == 0 && aligned16(src);
    const cudaError_t l = launch_pdl(kern, dim3(static_cast<unsigned>(tiles_c * tiles_r)), dim3(Q_THREADS), q_smem<T, TR>(qt != nullptr),
                                     c.stream, static_cast<const T*>(src), q, s, qt, st, R, C, static_cast<int>(tiles_c), vec);
    if (l != cudaSuccess) return l;
    c.count();
    return cudaGetLastError();
}

template <typename T>
cudaError_t quantize_t(const LaunchCtx& c, uint8_t* q, uint8_t* s, uint8_t* qt, uint8_t* st, const void* src, int64_t R, int64_t C) {
    // tiles of 32 rows until four of them per SM: then the SMs are busy with either
    const int64_t small = fp4_padded(C) / QT * ((R + 31) / 32);
    return small <= 4 * c.sm_count ? quantize_tiles<T, 32>(c, q, s, qt, st, src, R, C) : quantize_tiles<T, 128>(c, q, s, qt, st, src, R, C);
}

template <typename T>
cudaError_t dequantize_t(const LaunchCtx& c, void* dst, const uint8_t* q, const uint8_t* s, int64_t R, int64_t C) {
    const int64_t per = (C + 7) / 8;
    unsigned bx = 8;
    while (bx < 256 && bx < per) bx *= 2;
    const unsigned by = 256 / bx;
    const int64_t gx = (per + bx - 1) / bx;
    int64_t gy = (R + by - 1) / by;
    const int64_t most = lmax(1, c.sm_count * 32ll / gx);  // blocks enough for the whole GPU
    if (gy > most) gy = most;
    if (gy > 65535) gy = 65535;
    const int vec = C % (16 / static_cast<int64_t>(sizeof(T))) == 0 && aligned16(dst);
    const cudaError_t l = launch_pdl(fp4_dequantize_kernel<T>, dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), dim3(bx, by), 0,
                                     c.stream, static_cast<T*>(dst), q, s, R, C, vec);
    if (l != cudaSuccess) return l;
    c.count();
    return cudaGetLastError();
}

constexpr int64_t FP4_MAX_DIM = 0x7fffff00ll;

bi_status check_matrix(bi_engine eng, bi_dtype dt, int64_t rows, int64_t cols) {
    if (!eng) return fail(nullptr, BI_ERR_INVALID_ARG, "engine is NULL");
    if (dt != BI_F32 && dt != BI_BF16 && dt != BI_F16) return fail(eng, BI_ERR_INVALID_ARG, "dtype must be BI_F32, BI_BF16 or BI_F16");
    if (rows < 0 || cols <= 0) return fail(eng, BI_ERR_INVALID_ARG, "rows must be >= 0 and cols > 0");
    if (rows > FP4_MAX_DIM || cols > FP4_MAX_DIM || fp4_padded(rows) / QT * (fp4_padded(cols) / QT) > 0x1fffffffll)
        return fail(eng, BI_ERR_UNSUPPORTED, "rows and cols are limited to 2^31 - 256, and to 2^29 - 1 tiles of 128 x 128");
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
    if (reinterpret_cast<uintptr_t>(src) % bi::dsize(dtype) != 0) return fail(eng, BI_ERR_MISALIGNED, "src needs the alignment of its type");
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
    if (reinterpret_cast<uintptr_t>(dst) % bi::dsize(dtype) != 0) return fail(eng, BI_ERR_MISALIGNED, "dst needs the alignment of its type");
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
