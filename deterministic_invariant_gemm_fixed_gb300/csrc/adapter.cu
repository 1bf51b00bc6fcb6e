// Low-rank adapters of many requests beside a shared projection: entry points,
// and the kernels that every tier shares or that run in plain f32 FMAs.  See
// include/bi.h (bi_adapter_forward, bi_adapter_backward).
//
//   h[m,:] = X[m,:] A[g]^T          g = row_adapters[m]
//   Y[m,:] = round( X[m,:] W + bias + (s_g h[m,:]) B[g] )
//   u[m,:] = s_g dY[m,:] B[g]^T,    dX[m,:] = round( dY[m,:] W^T + u[m,:] A[g] )
//   dA[g]  = sum_m u[m,:]^T X[m,:], dB[g]  = sum_m (s_g h[m,:])^T dY[m,:]
//
// With A stored [G, R, K] and B stored [G, R, N] the two directions are the same
// two products: a narrow one that contracts a row of length L against P[g]
// [R, L] (h and u), and a wide one that adds R terms of Q[g] [R, C] (to Y and
// dX); dA and dB are one product too, [R, C] summed over an adapter's rows.
//
// A row's h, u, Y and dX read only its own operands and its own adapter, in an
// order fixed by K, N and R: they do not depend on the other rows of the batch,
// on their number, or on other requests' adapters (an infinity or NaN in one
// adapter stays in its rows).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <mutex>
#include <type_traits>

#include "abi_util.h"
#include "adapter.h"
#include "adapter_parts.cuh"

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

// ---------------------------------------------------------------- chunk tables

// Chunk tables of the sorted rows (AdapterChunks), one block.
__global__ void __launch_bounds__(1024) adapter_chunks_kernel(const uint32_t* off, uint32_t G, AdapterChunks ch) {
    __shared__ uint32_t s_a[32], s_b[32];
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t base_a = 0, base_b = 0;
    for (uint32_t g0 = 0; g0 < G; g0 += 1024) {
        const uint32_t g = g0 + tid;
        const uint32_t n = g < G ? (off[g + 1] - off[g] + ADAPTER_CHUNK - 1) / ADAPTER_CHUNK : 0;
        uint32_t a = n, b = n > 1 ? n : 0;
        const uint32_t own_a = a, own_b = b;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t ya = __shfl_up_sync(0xffffffffu, a, o), yb = __shfl_up_sync(0xffffffffu, b, o);
            if (lane >= o) { a += ya; b += yb; }
        }
        __syncthreads();
        if (lane == 31) { s_a[warp] = a; s_b[warp] = b; }
        __syncthreads();
        uint32_t pa = base_a, pb = base_b;
        for (int w = 0; w < 32; ++w) {
            if (w < warp) { pa += s_a[w]; pb += s_b[w]; }
            base_a += s_a[w];
            base_b += s_b[w];
        }
        if (g < G) {
            ch.first[g] = pa + a - own_a;
            ch.part[g] = pb + b - own_b;
        }
    }
    if (tid == 0) {
        ch.first[G] = base_a;
        ch.part[G] = base_b;
    }
}

// ---------------------------------------------------------------- narrow product, scalar

// partial[piece][m][r] = sum over the piece's l of X[m,l] P[g][r,l].  A warp has
// ROWS rows (four; one where that leaves SMs without warps) and one piece, the
// rows' 512 values in registers (lane j holds l = 128 i + 4 j + 0..3), and for each
// of up to 16 ranks reads P's 512 values once, for all of its rows if they have
// one adapter: lane sums (16 FMAs, l ascending) and a shuffle tree, the same order
// for a row alone or among others.  Rows of other warps find P in L1.  (One result
// per thread, operands staged in shared memory per adapter among 16 rows, took 81
// us where this takes 7: 999 x 1000, rank 5, seven adapters in no order.)
constexpr int NS_RANKS = 16, NS_WARPS = 4;
template <typename T>
__device__ __forceinline__ void load_lane(const T* p, int64_t l0, int64_t L, bool vec, int lane, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t l = l0 + 128 * i + 4 * lane;
        if (vec && l + 4 <= L) {  // L % 4 == 0 and aligned rows
            if constexpr (sizeof(T) == 4) {
                const float4 q = *reinterpret_cast<const float4*>(p + l);
                v[4 * i] = q.x; v[4 * i + 1] = q.y; v[4 * i + 2] = q.z; v[4 * i + 3] = q.w;
            } else {
                const uint2 q = *reinterpret_cast<const uint2*>(p + l);
                const T* e = reinterpret_cast<const T*>(&q);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[4 * i + j] = up<T>(e[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * i + j] = l + j < L ? up<T>(p[l + j]) : 0.0f;
        }
    }
}
template <typename T, int ROWS>
__global__ void __launch_bounds__(32 * NS_WARPS)
    narrow_scalar_kernel(const T* x, const T* p, const uint32_t* ids, float* partial, int64_t M, int64_t L, int R, uint32_t G,
                         int vec) {
    grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t m0 = (static_cast<int64_t>(blockIdx.x) * NS_WARPS + warp) * ROWS;
    if (m0 >= M) return;
    const int r0 = blockIdx.z * NS_RANKS, r1 = min(R, r0 + NS_RANKS);
    const int64_t l0 = static_cast<int64_t>(blockIdx.y) * ADAPTER_PIECE, l1 = lmin(L, l0 + ADAPTER_PIECE);
    uint32_t g[ROWS];
    float v[ROWS][16];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        g[i] = m0 + i < M ? ids[m0 + i] : G;
        if (g[i] < G) load_lane(x + (m0 + i) * L, l0, l1, vec != 0, lane, v[i]);
    }
    // values past l1 are 0 in v and in P: they add +0 products
    auto row_sum = [&](const float (&a)[16], const float (&b)[16]) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) s = fmaf(a[k], b[k], s);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        return s;
    };
    float* out = partial + (static_cast<int64_t>(blockIdx.y) * M + m0) * R;
    bool one = g[0] < G;
#pragma unroll
    for (int i = 1; i < ROWS; ++i) one = one && g[i] == g[0];
    if (one) {
        const T* pg = p + static_cast<int64_t>(g[0]) * R * L;
#pragma unroll 2
        for (int r = r0; r < r1; ++r) {
            float b[16];
            load_lane(pg + static_cast<int64_t>(r) * L, l0, l1, vec != 0, lane, b);
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const float s = row_sum(v[i], b);
                if (lane == i) out[static_cast<int64_t>(i) * R + r] = s;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            if (g[i] >= G) continue;
            const T* pg = p + static_cast<int64_t>(g[i]) * R * L;
#pragma unroll 2
            for (int r = r0; r < r1; ++r) {
                float b[16];
                load_lane(pg + static_cast<int64_t>(r) * L, l0, l1, vec != 0, lane, b);
                const float s = row_sum(v[i], b);
                if (lane == 0) out[static_cast<int64_t>(i) * R + r] = s;
            }
        }
    }
}

// v = the pieces' sums added in order (+0 for a row without adapter); h = v,
// hs = s_g v (either nullable).
__global__ void __launch_bounds__(256)
    narrow_finish_kernel(const float* partial, const uint32_t* ids, const float* scales, float* h, float* hs,
                         int64_t M, int R, uint32_t G, int pieces) {
    grid_dep_wait();
    grid_dep_launch();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= M * R) return;
    const uint32_t g = ids[i / R];
    float v = 0.0f, s = 0.0f;
    if (g < G) {
        v = partial[i];
        for (int q = 1; q < pieces; ++q) v += partial[static_cast<int64_t>(q) * M * R + i];
        s = scales != nullptr ? v * scales[g] : v;
    }
    if (h != nullptr) h[i] = v;
    if (hs != nullptr) hs[i] = s;
}

// The same for the tensor cores: v = the pieces' sums (row stride rp), or h_in;
// h = v; then s_g v in two parts (hh, for the wide product; `over` gets a bit for a
// row that they cannot carry) and in four (v4, for dA and dB), any of them nullable.
// A part that would be an infinity's remainder is 0, so an infinity stays one.  One
// thread per row and 8 ranks
// (16-byte stores) up to the formats' padded width (zeros past R); block row y
// does job y.
struct FinishJob {
    const float* partial;
    const float* h_in;
    float* h;
    void* hh;
    void* v4;
};
struct FinishJobs {
    FinishJob job[2];
};
template <typename T>
__device__ __forceinline__ float part_rest(float v, T hi, float scale) {
    const float h = up<T>(hi) * scale;
    return isinf(h) ? 0.0f : v - h;
}
template <typename T>
__device__ __forceinline__ void four_parts(float s, T (&part)[4]) {
    part[0] = down<T>(0.0f);
    if (std::is_same<T, __half>::value) {  // see adapter.h
        float rest = s, scale = 0x1p11f;
#pragma unroll
        for (int i = 0; i < 4; ++i, scale *= 0x1p-11f) {
            const float x = rest * (1.0f / scale);
            const bool none = i == 0 ? !(fabsf(s) > 65504.0f) : (i < 3 && fabsf(x) < 0x1p-14f);
            part[i] = down<T>(none ? 0.0f : x);
            rest = none ? rest : part_rest<T>(rest, part[i], scale);
        }
    } else {
        part[1] = down<T>(s);
        const float r1 = part_rest<T>(s, part[1], 1.0f);
        part[2] = down<T>(r1);
        part[3] = down<T>(part_rest<T>(r1, part[2], 1.0f));
    }
}
template <typename T>
__global__ void __launch_bounds__(256)
    narrow_finish_tc_kernel(const __grid_constant__ FinishJobs jobs, const uint32_t* ids, const float* scales, uint32_t* over,
                            int64_t M, int R, int rp, uint32_t G, int pieces, int per_row) {
    grid_dep_wait();
    grid_dep_launch();
    const FinishJob& jb = jobs.job[blockIdx.y];
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= M * per_row) return;
    const int64_t m = M * per_row <= 0x7fffffff ? static_cast<int64_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(per_row))
                                                : i / per_row;
    const int r0 = static_cast<int>(i - m * per_row) * 8;
    const uint32_t g = ids[m];
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = 0.0f;
    if (g < G && r0 < R) {
        if (jb.partial != nullptr) {  // rp - r0 is a multiple of 8: whole vectors
            sum_pieces8(jb.partial + m * rp + r0, M * rp, pieces, v);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (r0 + u >= R) v[u] = 0.0f;
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (r0 + u < R) v[u] = jb.h_in[m * R + r0 + u];
        }
    }
    if (jb.h != nullptr) {
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (r0 + u < R) jb.h[m * R + r0 + u] = v[u];
    }
    const float scale = g < G && scales != nullptr ? scales[g] : 1.0f;
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = r0 + u < R ? v[u] * scale : 0.0f;  // (0 times an infinite scale is no padding)
    __align__(16) T out[4][8];
    if (jb.hh != nullptr && r0 < (R + 31) / 32 * 32) {
        uint32_t hi[4], lo[4];
        if (two_parts8<std::is_same<T, __half>::value ? 0 : 1>(v, hi, lo)) atomicOr(over + (m >> 5), 1u << (m & 31));
        T* o = static_cast<T*>(jb.hh) + m * ((R + 31) / 32 * 64) + (r0 / 32) * 64 + r0 % 32;
        *reinterpret_cast<uint4*>(o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(o + 32) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    const int run = adapter_rank_run(R);
    if (jb.v4 != nullptr && r0 < (R + 63) / 64 * run) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            T part[4];
            four_parts<T>(v[u], part);
#pragma unroll
            for (int q = 0; q < 4; ++q) out[q][u] = part[q];
        }
        T* o = static_cast<T*>(jb.v4) + m * adapter_grad_cols(R) + (r0 / 64) * 256 + r0 % 64;
#pragma unroll
        for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(o + q * run) = *reinterpret_cast<const uint4*>(out[q]);
    }
}

// hs = s_g h, 0 for a row without adapter.
__global__ void __launch_bounds__(256) scale_rows_kernel(const float* h, const uint32_t* ids, const float* scales, float* hs, int64_t M,
                                                         int R, uint32_t G) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= M * R) return;
    const uint32_t g = ids[i / R];
    hs[i] = g < G ? (scales != nullptr ? h[i] * scales[g] : h[i]) : 0.0f;
}

// ---------------------------------------------------------------- wide product, scalar

// out[m,c] = round( base[m,c] + sum over r ascending of hs[m,r] Q[g][r,c] ), base
// in f32 (for f32 it is out itself).  ROWS rows by 256 columns per block (16; 4
// where that leaves SMs without blocks), a column per thread: an element of Q is read once for all of the block's rows with
// that adapter.
//
// hs comes from the finish kernel, or (hs null) from the pieces themselves, added
// and scaled here in the same order; then the first column of blocks writes h.
struct WideSource {
    const float* hs;
    const float* partial;  // [pieces][M][R]
    const float* scales;
    float* h;
    int pieces;
};
template <typename T, int ROWS>
__global__ void __launch_bounds__(256) wide_scalar_kernel(T* out, const float* base, const WideSource src, const T* q,
                                                          const uint32_t* ids, int64_t M, int64_t C, int R, uint32_t G) {
    extern __shared__ float s_h[];  // [R rounded up to 8][ROWS], zeros past R
    __shared__ uint32_t s_id[ROWS], s_mask[ROWS];  // row i's adapter; the rows with it, at the first of them (else 0)
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x;
    const int64_t m0 = static_cast<int64_t>(blockIdx.x) * ROWS;
    const int64_t c = static_cast<int64_t>(blockIdx.y) * 256 + tid;
    if (tid < 32) {
        const uint32_t id = tid < ROWS && m0 + tid < M ? ids[m0 + tid] : G;
        const uint32_t same = __match_any_sync(0xffffffffu, id);
        if (tid < ROWS) {
            s_id[tid] = id;
            s_mask[tid] = id < G && (same & ((1u << tid) - 1)) == 0 ? same : 0;
        }
    }
    const int R8 = (R + 7) / 8 * 8;
    for (int i = tid; i < ROWS * R8; i += 256) {
        const int row = i / R8, r = i % R8;
        const int64_t at = (m0 + row) * R + r;
        float v = 0.0f;
        if (m0 + row < M && r < R) {
            if (src.hs != nullptr) {
                v = src.hs[at];
            } else {
                const uint32_t g = ids[m0 + row];
                if (g < G) {
                    v = src.partial[at];
                    for (int p = 1; p < src.pieces; ++p) v += src.partial[static_cast<int64_t>(p) * M * R + at];
                }
                if (src.h != nullptr && blockIdx.y == 0) src.h[at] = v;
                if (g < G && src.scales != nullptr) v *= src.scales[g];
            }
        }
        s_h[r * ROWS + row] = v;
    }
    float b[ROWS];
    if (c < C) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) b[i] = m0 + i < M ? base[(m0 + i) * C + c] : 0.0f;
    }
    __syncthreads();
    if (c >= C) return;
    const bool in_place = reinterpret_cast<const void*>(base) == reinterpret_cast<const void*>(out);
    if constexpr (ROWS == 4) {  // few blocks: each row reads its own adapter, all loads in flight at once
        float acc[ROWS] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int r = 0; r < R; r += 8) {
            float v[ROWS][8];
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const T* qg = q + (static_cast<int64_t>(s_id[i]) * R + r) * C + c;
#pragma unroll
                for (int u = 0; u < 8; ++u) v[i][u] = s_id[i] < G && r + u < R ? up<T>(qg[static_cast<int64_t>(u) * C]) : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int i = 0; i < ROWS; ++i) acc[i] = fmaf(s_h[(r + u) * ROWS + i], v[i][u], acc[i]);
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            if (s_id[i] < G) out[(m0 + i) * C + c] = down<T>(b[i] + acc[i]);
            else if (!in_place && m0 + i < M) out[(m0 + i) * C + c] = down<T>(b[i]);
        }
        return;
    }
    uint32_t any = 0;
    for (int e = 0; e < ROWS; ++e) {
        const uint32_t mask = s_mask[e];
        if (mask == 0) continue;
        any |= mask;
        const T* qg = q + static_cast<int64_t>(s_id[e]) * R * C + c;
        float acc[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) acc[i] = 0.0f;
        for (int r = 0; r < R; r += 8) {  // eight loads in flight; past R both factors are 0
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = r + u < R ? up<T>(qg[static_cast<int64_t>(r + u) * C]) : 0.0f;
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int i = 0; i < ROWS; ++i) acc[i] = fmaf(s_h[(r + u) * ROWS + i], v[u], acc[i]);
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if ((mask >> i) & 1u) out[(m0 + i) * C + c] = down<T>(b[i] + acc[i]);
    }
    if (in_place) return;
#pragma unroll
    for (int i = 0; i < ROWS; ++i)  // rows without adapter
        if (!((any >> i) & 1u) && m0 + i < M) out[(m0 + i) * C + c] = down<T>(b[i]);
}

// ---------------------------------------------------------------- dA, dB, scalar

// One block: one chunk of one adapter's sorted rows, 128 columns, 16 ranks;
// a column per thread, out[r][c] = the chain over the chunk's rows ascending of
// hs[m,r] Z[m,c].  Adapters of one chunk write out, others their partial slot.
constexpr int GR_ROWS = 32;
template <typename T>
__global__ void __launch_bounds__(128)
    grad_scalar_kernel(float* out, float* parts, const float* hs, const T* z, const uint32_t* off, const uint32_t* perm,
                       AdapterChunks ch, int64_t C, int R, uint32_t G) {
    __shared__ float s_h[GR_ROWS][16];
    __shared__ uint32_t s_row[GR_ROWS];
    const uint32_t chunk = blockIdx.x;
    if (chunk >= ch.first[G]) return;
    uint32_t lo = 0, hi = G - 1;  // the last g with first[g] <= chunk
    while (lo < hi) {
        const uint32_t mid = (lo + hi + 1) >> 1;
        if (ch.first[mid] <= chunk) lo = mid; else hi = mid - 1;
    }
    const uint32_t j = chunk - ch.first[lo], nchunks = ch.first[lo + 1] - ch.first[lo];
    const uint32_t s0 = off[lo] + j * static_cast<uint32_t>(ADAPTER_CHUNK);
    const uint32_t s1 = min(off[lo + 1], s0 + static_cast<uint32_t>(ADAPTER_CHUNK));
    const int64_t c = static_cast<int64_t>(blockIdx.y) * 128 + threadIdx.x;
    const int r0 = blockIdx.z * 16;
    float acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
    for (uint32_t s = s0; s < s1; s += GR_ROWS) {
        const int n = static_cast<int>(min(s1 - s, static_cast<uint32_t>(GR_ROWS)));
        __syncthreads();
        for (int i = threadIdx.x; i < GR_ROWS * 16; i += 128) {
            const int a = i >> 4, b = i & 15;
            s_h[a][b] = a < n && r0 + b < R ? hs[static_cast<int64_t>(perm[s + a]) * R + r0 + b] : 0.0f;
        }
        if (threadIdx.x < GR_ROWS) s_row[threadIdx.x] = static_cast<int>(threadIdx.x) < n ? perm[s + threadIdx.x] : 0;
        __syncthreads();
        if (c < C) {
#pragma unroll 4
            for (int a = 0; a < n; ++a) {
                const float v = up<T>(z[static_cast<int64_t>(s_row[a]) * C + c]);
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[i] = fmaf(s_h[a][i], v, acc[i]);
            }
        }
    }
    if (c >= C) return;
    float* dst = nchunks > 1 ? parts + static_cast<int64_t>(ch.part[lo] + j) * R * C : out + static_cast<int64_t>(lo) * R * C;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (r0 + i < R) dst[static_cast<int64_t>(r0 + i) * C + c] = acc[i];
}

// out[g] = the chunks' sums added in order; +0 for an adapter without rows.  An
// adapter of one chunk has its result already.  Block row z does job z.
__global__ void __launch_bounds__(256)
    grad_sum_kernel(const __grid_constant__ AdapterGradJobs jobs, AdapterChunks ch, int R) {
    grid_dep_wait();
    grid_dep_launch();
    const uint32_t g = blockIdx.x;
    const uint32_t n = ch.first[g + 1] - ch.first[g];
    if (n == 1) return;
    const AdapterGradJob& jb = jobs.job[blockIdx.z];
    const int64_t RC = R * jb.C;
    float* o = jb.out + static_cast<int64_t>(g) * RC;
    const float* p = jb.parts + static_cast<int64_t>(ch.part[g]) * RC;
    for (int64_t i = static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x; i < RC; i += static_cast<int64_t>(gridDim.y) * 256) {
        float v = 0.0f;
        for (uint32_t j0 = 0; j0 < n; j0 += 4) {  // four chunks' loads in flight
            float t[4];
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) t[j] = j0 + j < n ? p[static_cast<int64_t>(j0 + j) * RC + i] : 0.0f;
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
                if (j0 + j < n) v = j0 + j == 0 ? t[j] : v + t[j];
        }
        o[i] = v;
    }
}

// ---------------------------------------------------------------- launchers

cudaError_t launched(const LaunchCtx& c) {
    c.count();
    return cudaGetLastError();
}

unsigned grid1(int64_t n) { return static_cast<unsigned>((n + 255) / 256); }
int pieces_of(int64_t L) { return static_cast<int>((L + ADAPTER_PIECE - 1) / ADAPTER_PIECE); }

template <typename T>
cudaError_t narrow_scalar(const LaunchCtx& c, const T* x, const T* p, const uint32_t* ids, float* partial, int64_t M,
                          int64_t L, int R, int64_t G) {
    const bool few = (M + 3) / 4 * pieces_of(L) < 16 * int64_t(c.sm_count);  // too few warps of four rows
    const int64_t rows = (few ? 1 : 4) * NS_WARPS;
    const dim3 grid(static_cast<unsigned>((M + rows - 1) / rows), static_cast<unsigned>(pieces_of(L)),
                    static_cast<unsigned>((R + NS_RANKS - 1) / NS_RANKS));
    const int vec = L % 4 == 0 && reinterpret_cast<uintptr_t>(x) % (4 * sizeof(T)) == 0 &&
                    reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0;
    const cudaError_t e = launch_pdl(few ? narrow_scalar_kernel<T, 1> : narrow_scalar_kernel<T, 4>, grid, dim3(32 * NS_WARPS), 0, c.stream, x, p, ids, partial, M, L, R,
                                     static_cast<uint32_t>(G), vec);
    if (e == cudaSuccess) c.count();
    return e;
}

cudaError_t narrow_finish(const LaunchCtx& c, const float* partial, const uint32_t* ids, const float* scales, float* h, float* hs,
                          int64_t M, int R, int64_t G, int pieces) {
    const cudaError_t e = launch_pdl(narrow_finish_kernel, dim3(grid1(M * R)), dim3(256), 0, c.stream, partial, ids, scales, h, hs,
                                     M, R, static_cast<uint32_t>(G), pieces);
    if (e == cudaSuccess) c.count();
    return e;
}

template <typename T>
cudaError_t wide_scalar(const LaunchCtx& c, T* out, const float* base, const WideSource& src, const T* q, const uint32_t* ids,
                        int64_t M, int64_t C, int R, int64_t G) {
    const bool few = (M + 15) / 16 * ((C + 255) / 256) < 4 * int64_t(c.sm_count);
    const int rows = few ? 4 : 16;
    const dim3 grid(static_cast<unsigned>((M + rows - 1) / rows), static_cast<unsigned>((C + 255) / 256));
    const cudaError_t e = launch_pdl(few ? wide_scalar_kernel<T, 4> : wide_scalar_kernel<T, 16>, grid, dim3(256),
                                     static_cast<size_t>(rows * ((R + 7) / 8 * 8) * 4), c.stream, out, base, src, q, ids, M, C,
                                     R, static_cast<uint32_t>(G));
    if (e == cudaSuccess) c.count();
    return e;
}

// A row's sums of pieces that the wide kernel's blocks take on themselves, each
// for its own columns (then no finish kernel runs): few enough to be noise there.
constexpr int64_t WIDE_FUSE = 512;

template <typename T>
cudaError_t grad_scalar(const LaunchCtx& c, float* out, float* parts, const float* hs, const T* z, const uint32_t* seg,
                        const uint32_t* perm, const AdapterChunks& ch, int64_t M, int64_t C, int R, int64_t G) {
    const dim3 grid(static_cast<unsigned>(AdapterChunks::max_chunks(M, G)), static_cast<unsigned>((C + 127) / 128),
                    static_cast<unsigned>((R + 15) / 16));
    grad_scalar_kernel<T><<<grid, 128, 0, c.stream>>>(out, parts, hs, z, seg, perm, ch, C, R, static_cast<uint32_t>(G));
    return launched(c);
}

cudaError_t grad_sum(const LaunchCtx& c, const AdapterGradJob* jobs, int count, const AdapterChunks& ch, int R, int64_t M,
                     int64_t G) {
    AdapterGradJobs js{};
    int64_t most = 0;
    for (int i = 0; i < count; ++i) {
        js.job[i] = jobs[i];
        most = lmax(most, R * jobs[i].C);
    }
    // about eight blocks per SM in all: most adapters have one chunk and nothing to add
    const int64_t y = lmax(1, lmin((most + 255) / 256, 8 * int64_t(c.sm_count) / (G * count)));
    const dim3 grid(static_cast<unsigned>(G), static_cast<unsigned>(y), static_cast<unsigned>(count));
    const cudaError_t e = launch_plain(grad_sum_kernel, grid, dim3(256), 0, c.stream, js, ch, R);
    if (e == cudaSuccess) c.count();
    return e;
}

// One or two jobs over the same rows: the second's partial is null.
cudaError_t narrow_finish_tc(const LaunchCtx& c, bi_dtype dt, const FinishJob& a, const FinishJob* b, const uint32_t* ids,
                             const float* scales, uint32_t* over, int64_t M, int R, int64_t G, int pieces) {
    const FinishJobs jobs{{a, b ? *b : FinishJob{}}};
    const int rp = (R + 15) / 16 * 16;
    const bool hh = a.hh || (b && b->hh), v4 = a.v4 || (b && b->v4);
    const int per_row = static_cast<int>(lmax(hh ? (R + 31) / 32 * 32 : rp, v4 ? (R + 63) / 64 * adapter_rank_run(R) : rp)) / 8;
    const dim3 grid(static_cast<unsigned>((M * per_row + 255) / 256), b ? 2 : 1);
    const cudaError_t e =
        dt == BI_BF16 ? launch_pdl(narrow_finish_tc_kernel<__nv_bfloat16>, grid, dim3(256), 0, c.stream, jobs, ids, scales, over, M,
                                   R, rp, static_cast<uint32_t>(G), pieces, per_row)
                      : launch_pdl(narrow_finish_tc_kernel<__half>, grid, dim3(256), 0, c.stream, jobs, ids, scales, over, M, R, rp,
                                   static_cast<uint32_t>(G), pieces, per_row);
    if (e == cudaSuccess) c.count();
    return e;
}

// Calls f with a null pointer of dt's element type.
template <typename F>
cudaError_t with_type(bi_dtype dt, F&& f) {
    return dt == BI_F32 ? f(static_cast<float*>(nullptr))
         : dt == BI_BF16 ? f(static_cast<__nv_bfloat16*>(nullptr)) : f(static_cast<__half*>(nullptr));
}

bi_status check_adapter(bi_engine eng, bi_dtype dt, int64_t m, int64_t k, int64_t n, int64_t r, int64_t g) {
    if (!eng) return fail(nullptr, BI_ERR_INVALID_ARG, "engine is NULL");
    const char* why = "";
    const bi_status st = check_sizes(dt, m, k, n, -1, &why);
    if (st != BI_OK) return fail(eng, st, why);
    if (r <= 0 || g <= 0) return fail(eng, BI_ERR_INVALID_ARG, "r and g must be > 0");
    if (r > ADAPTER_MAX_RANK) return fail(eng, BI_ERR_UNSUPPORTED, "adapters are limited to rank 256");
    if (g > 65535) return fail(eng, BI_ERR_UNSUPPORTED, "g is limited to 65535 adapters");
    return BI_OK;
}

// The f32-FMA kernels count pieces (512 elements), the wide product's columns (256) and
// the gradients' (128) in a grid's second dimension.
bool too_long(int64_t length, int64_t per_block) { return (length + per_block - 1) / per_block > 65535; }
bi_status fail_too_long(bi_engine eng) {
    return fail(eng, BI_ERR_UNSUPPORTED,
                "adapters in plain f32: a contraction is limited to 33553920 elements, y's and dx's columns to 16776960, da's and "
                "db's to 8388480");
}

// One adapter call on a device at a time: a call on another stream than the one before
// waits for it on the device.  (With three streams' calls under way at once one of
// them never ended, within some 250 turns, on a GPU that had nothing else left to do
// and answered again once the process was gone.  No bounded wait had run out; which of
// the hardware's own it was is not known.  Two streams ran 300 thousand turns.)  A
// single stream pays a comparison.  The first call on a second stream waits for the
// device on the host, as nothing marks where the first one's last call ends; from then
// on an event does.  Calls that are being captured are left out: a graph's replays are
// not seen here.
struct TurnState {
    std::mutex mu;
    bool begun = false, many = false;
    cudaStream_t stream = nullptr;  // of the last call; compared only, it may be gone
    cudaEvent_t event = nullptr;    // behind that call, once there were two streams
};
struct AdapterTurn {
    TurnState& state;
    cudaStream_t stream;
    std::lock_guard<std::mutex> lock;
    cudaError_t err = cudaSuccess;
    bool capturing = false;
    static TurnState& of(int device) {
        static TurnState states[MAX_DEVICES];
        return states[device >= 0 && device < MAX_DEVICES ? device : 0];
    }
    AdapterTurn(bi_engine eng, cudaStream_t s) : state(of(eng->device)), stream(s), lock(state.mu) {
        if (state.begun && !state.many && s == state.stream) return;
        cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
        if (cudaStreamIsCapturing(s, &st) != cudaSuccess) cudaGetLastError();
        capturing = st != cudaStreamCaptureStatusNone;
        if (capturing) return;
        if (state.begun && !state.many) {
            if (state.event == nullptr) err = cudaEventCreateWithFlags(&state.event, cudaEventDisableTiming);
            if (err != cudaSuccess) return;
            cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;  // another thread may be capturing
            cudaThreadExchangeStreamCaptureMode(&mode);
            err = cudaDeviceSynchronize();
            cudaThreadExchangeStreamCaptureMode(&mode);
            if (err != cudaSuccess) return;
            state.many = true;
        } else if (state.many && (s != state.stream || s == cudaStreamPerThread)) {
            err = cudaStreamWaitEvent(s, state.event, 0);
            if (err != cudaSuccess) return;
        }
        state.begun = true;
        state.stream = s;
    }
    ~AdapterTurn() {
        if (state.many && !capturing && err == cudaSuccess) cudaEventRecord(state.event, stream);
    }
};

// Cuts of one scratch allocation.
struct Cut {
    int64_t at = 0;
    int64_t take(int64_t bytes) {
        const int64_t r = at;
        at += round256(bytes);
        return r;
    }
};

}  // namespace
}  // namespace bi

using namespace bi;

extern "C" {

bi_status bi_adapter_forward(bi_engine eng, void* y, float* h, const void* x, const void* w, const void* bias,
                             const void* a, const void* b, const float* scales, const uint32_t* row_adapters,
                             int64_t m, int64_t k, int64_t n, int64_t r, int64_t g, bi_dtype dtype, void* stream,
                             int tensor_cores) {
    bi_status st = check_adapter(eng, dtype, m, k, n, r, g);
    if (st != BI_OK) return st;
    if (m == 0) return BI_OK;
    if (!y || !x || !w || !a || !b || !row_adapters)
        return fail(eng, BI_ERR_INVALID_ARG, "y, x, w, a, b and row_adapters must not be NULL");
    // (f32 takes its tier in the shared product; the adapters' terms are f32 FMAs)
    const int tier = dtype != BI_F32 && bi_dispatch_tier(BI_PASS_FORWARD, dtype, tensor_cores, k, n);
    if (tier && (!aligned16(y) || !aligned16(x) || !aligned16(w) || !aligned16(a) || !aligned16(b)))
        return fail(eng, BI_ERR_MISALIGNED, "tensor-core tier needs 16-byte aligned y, x, w, a, b");
    DeviceGuard guard(eng->device);
    if (!guard.ok) return fail(eng, BI_ERR_CUDA, "cudaSetDevice failed");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const AdapterTurn turn(eng, s);
    if (turn.err != cudaSuccess) return cuda_fail(eng, turn.err, "adapter turn");
    const LaunchCtx c = ctx(eng, stream);
    const int R = static_cast<int>(r), pieces = pieces_of(k);
    if (tier) {
        // scratch: plan | pieces of h | s h in two parts
        Cut cut;
        const int64_t o_plan = cut.take(AdapterPlan::words(m) * 4), o_part = cut.take(pieces * m * ((r + 15) / 16 * 16) * 4),
                      o_hh = cut.take(m * adapter_part_cols(r) * 2);
        Scratch sc(eng, s, static_cast<size_t>(cut.at));
        if (sc.err != cudaSuccess) return cuda_fail(eng, sc.err, "adapter scratch");
        uint8_t* p = static_cast<uint8_t*>(sc.ptr);
        const AdapterPlan plan = AdapterPlan::at(p + o_plan, m);
        float* part = reinterpret_cast<float*>(p + o_part);
        cudaError_t e = tc_adapter_narrow(c, dtype, part, x, a, row_adapters, plan, m, k, R, g);
        const AdapterPieces src{part, row_adapters, scales, h, pieces};
        if (adapter_small_fuses(c, m, n, k, R)) {
            if (e == cudaSuccess)
                e = tc_adapter_rows_small(c, dtype, 0, y, x, w, bias, nullptr, b, plan, src, m, k, n, R, g, true);
            return e == cudaSuccess ? BI_OK : cuda_fail(eng, e, "bi_adapter_forward");
        }
        if (e == cudaSuccess)
            e = narrow_finish_tc(c, dtype, {part, nullptr, h, p + o_hh, nullptr}, nullptr, row_adapters, scales, plan.over, m, R,
                                 g, pieces);
        if (e == cudaSuccess) e = tc_adapter_rows(c, dtype, 0, y, x, w, bias, p + o_hh, b, plan, src, m, k, n, R, g);
        return e == cudaSuccess ? BI_OK : cuda_fail(eng, e, "bi_adapter_forward");
    }
    if (too_long(k, ADAPTER_PIECE) || too_long(n, 256)) return fail_too_long(eng);
    // scratch: pieces of h | s h | the shared product in f32 (16-bit types)
    Cut cut;
    const int64_t o_part = cut.take(pieces * m * r * 4), o_hs = cut.take(m * r * 4),
                  o_base = cut.take(dtype == BI_F32 ? 0 : m * n * 4);
    Scratch sc(eng, s, static_cast<size_t>(cut.at));
    if (sc.err != cudaSuccess) return cuda_fail(eng, sc.err, "adapter scratch");
    uint8_t* p = static_cast<uint8_t*>(sc.ptr);
    float* part = reinterpret_cast<float*>(p + o_part);
    float* hs = reinterpret_cast<float*>(p + o_hs);
    float* base = dtype == BI_F32 ? static_cast<float*>(y) : reinterpret_cast<float*>(p + o_base);
    // the shared product first: it may need scratch of its own, and a call that
    // gets none must leave nothing enqueued
    cudaError_t e = cudaSuccess;
    if (dtype == BI_F32) {
        st = adapter_projection_f32(eng, c, 0, y, x, w, bias, m, k, n, tensor_cores);
        if (st != BI_OK) return st;
    } else {
        e = scalar_rows(c, dtype, base, x, w, bias, m, k, n, 0, 1);
    }
    if (e == cudaSuccess)
        e = with_type(dtype, [&](auto* t) {
            using T = std::remove_pointer_t<decltype(t)>;
            return narrow_scalar<T>(c, static_cast<const T*>(x), static_cast<const T*>(a), row_adapters, part, m, k, R, g);
        });
    const bool fuse = pieces * r <= WIDE_FUSE;
    if (e == cudaSuccess && !fuse) e = narrow_finish(c, part, row_adapters, scales, h, hs, m, R, g, pieces);
    if (e == cudaSuccess)
        e = with_type(dtype, [&](auto* t) {
            using T = std::remove_pointer_t<decltype(t)>;
            return wide_scalar<T>(c, static_cast<T*>(y), base, WideSource{fuse ? nullptr : hs, part, scales, h, pieces},
                                  static_cast<const T*>(b), row_adapters, m, n, R, g);
        });
    return e == cudaSuccess ? BI_OK : cuda_fail(eng, e, "bi_adapter_forward");
}

bi_status bi_adapter_backward(bi_engine eng, void* dx, float* da, float* db, const void* x, const float* h,
                              const void* w, const void* dy, const void* a, const void* b, const float* scales,
                              const uint32_t* row_adapters, int64_t m, int64_t k, int64_t n, int64_t r, int64_t g,
                              bi_dtype dtype, void* stream, int tensor_cores) {
    bi_status st = check_adapter(eng, dtype, m, k, n, r, g);
    if (st != BI_OK) return st;
    DeviceGuard guard(eng->device);
    if (!guard.ok) return fail(eng, BI_ERR_CUDA, "cudaSetDevice failed");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (m == 0) {  // empty sums
        cudaError_t e = da ? cudaMemsetAsync(da, 0, static_cast<size_t>(g * r * k * 4), s) : cudaSuccess;
        if (e == cudaSuccess && db) e = cudaMemsetAsync(db, 0, static_cast<size_t>(g * r * n * 4), s);
        return e == cudaSuccess ? BI_OK : cuda_fail(eng, e, "bi_adapter_backward");
    }
    if (!dx && !da && !db) return BI_OK;
    if (!dy || !row_adapters || ((dx || da) && !b) || (dx && (!w || !a)) || (da && !x) || (db && !h))
        return fail(eng, BI_ERR_INVALID_ARG, "an operand that a requested gradient needs is NULL");
    const AdapterTurn turn(eng, s);
    if (turn.err != cudaSuccess) return cuda_fail(eng, turn.err, "adapter turn");
    const LaunchCtx c = ctx(eng, stream);
    const int R = static_cast<int>(r), pieces = pieces_of(n);
    const bool need_u = dx || da;
    const int tier = dtype != BI_F32 && bi_dispatch_tier(BI_PASS_DX, dtype, tensor_cores, k, n);
    if (tier) {
        if (!aligned16(dy) || (need_u && !aligned16(b)) || (da && !aligned16(x)) ||
            (dx && (!aligned16(dx) || !aligned16(w) || !aligned16(a))))
            return fail(eng, BI_ERR_MISALIGNED, "tensor-core tier needs 16-byte aligned dx, x, w, dy, a, b");
        // scratch: plan | pieces of u | u in two parts | u, s h in four parts |
        // sorted rows | chunk tables | chunk sums
        const bool grads = da || db;
        Cut cut;
        const int64_t o_plan = cut.take(need_u ? AdapterPlan::words(m) * 4 : 0),
                      o_part = cut.take(need_u ? pieces * m * ((r + 15) / 16 * 16) * 4 : 0),
                      o_uu = cut.take(dx ? m * adapter_part_cols(r) * 2 : 0),
                      o_u3 = cut.take(da ? m * adapter_grad_cols(R) * 2 : 0), o_h3 = cut.take(db ? m * adapter_grad_cols(R) * 2 : 0),
                      o_seg = cut.take(grads ? seg_table_len(g) * 4 : 0), o_perm = cut.take(grads ? m * 4 : 0),
                      o_hist = cut.take(grads ? segment_scratch_bytes(m, g) : 0),
                      o_ch = cut.take(grads ? AdapterChunks::words(g) * 4 : 0),
                      o_sum = cut.take(grads ? AdapterChunks::max_parts(m) * r * ((da ? k : 0) + (db ? n : 0)) * 4 : 0);
        Scratch sc(eng, s, static_cast<size_t>(cut.at));
        if (sc.err != cudaSuccess) return cuda_fail(eng, sc.err, "adapter scratch");
        uint8_t* p = static_cast<uint8_t*>(sc.ptr);
        const AdapterPlan plan = AdapterPlan::at(p + o_plan, m);
        float* part = reinterpret_cast<float*>(p + o_part);
        uint32_t* seg = reinterpret_cast<uint32_t*>(p + o_seg);
        uint32_t* perm = reinterpret_cast<uint32_t*>(p + o_perm);
        const AdapterChunks ch = AdapterChunks::at(p + o_ch, g);
        float* sums = reinterpret_cast<float*>(p + o_sum);
        cudaError_t e = cudaSuccess;
        if (grads) {  // the rows sorted by adapter, for dA and dB
            e = segment(c, row_adapters, m, g, seg, perm, p + o_hist);
            if (e == cudaSuccess) {
                e = launch_plain(adapter_chunks_kernel, dim3(1), dim3(1024), 0, s, seg, static_cast<uint32_t>(g), ch);
                if (e == cudaSuccess) c.count();
            }
        }
        if (e == cudaSuccess && need_u) {
            e = tc_adapter_narrow(c, dtype, part, dy, b, row_adapters, plan, m, n, R, g);
            const FinishJob u{part, nullptr, nullptr, dx ? p + o_uu : nullptr, da ? p + o_u3 : nullptr};
            const FinishJob hs{nullptr, h, nullptr, nullptr, p + o_h3};
            if (e == cudaSuccess) e = narrow_finish_tc(c, dtype, u, db ? &hs : nullptr, row_adapters, scales, plan.over, m, R, g,
                                                      pieces);
        }
        if (e == cudaSuccess && dx)
            e = tc_adapter_rows(c, dtype, 1, dx, dy, w, nullptr, p + o_uu, a, plan, {part, row_adapters, scales, nullptr, pieces}, m,
                                k, n, R, g);
        if (e == cudaSuccess && db && !need_u) {
            const FinishJob hs{nullptr, h, nullptr, nullptr, p + o_h3};
            e = narrow_finish_tc(c, dtype, hs, nullptr, row_adapters, scales, nullptr, m, R, g, 0);
        }
        if (e == cudaSuccess && grads) {
            AdapterGradJob jobs[2];
            int count = 0;
            float* db_sums = sums + (da ? AdapterChunks::max_parts(m) * r * k : 0);
            if (da) jobs[count++] = {da, sums, p + o_u3, x, k};
            if (db) jobs[count++] = {db, db_sums, p + o_h3, dy, n};
            e = tc_adapter_grad(c, dtype, jobs, count, seg, perm, ch, m, R, g);
            if (e == cudaSuccess) e = grad_sum(c, jobs, count, ch, R, m, g);
        }
        return e == cudaSuccess ? BI_OK : cuda_fail(eng, e, "bi_adapter_backward");
    }
    if ((need_u && too_long(n, ADAPTER_PIECE)) || (dx && too_long(k, 256)) || (da && too_long(k, 128)) || (db && too_long(n, 128)))
        return fail_too_long(eng);
    // scratch: pieces of u | u | s h | sorted rows | chunk tables | chunk
    // sums (of dA, then of dB) | the shared product in f32 (16-bit types)
    Cut cut;
    const int64_t o_part = cut.take(need_u ? pieces * m * r * 4 : 0),
                  o_u = cut.take(need_u ? m * r * 4 : 0), o_hs = cut.take(db ? m * r * 4 : 0);
    const bool grads = da || db;
    const int64_t o_seg = cut.take(grads ? seg_table_len(g) * 4 : 0), o_perm = cut.take(grads ? m * 4 : 0),
                  o_hist = cut.take(grads ? segment_scratch_bytes(m, g) : 0),
                  o_ch = cut.take(grads ? AdapterChunks::words(g) * 4 : 0),
                  o_sum = cut.take(grads ? AdapterChunks::max_parts(m) * r * lmax(da ? k : 0, db ? n : 0) * 4 : 0),
                  o_base = cut.take(dx && dtype != BI_F32 ? m * k * 4 : 0);
    Scratch sc(eng, s, static_cast<size_t>(cut.at));
    if (sc.err != cudaSuccess) return cuda_fail(eng, sc.err, "adapter scratch");
    uint8_t* p = static_cast<uint8_t*>(sc.ptr);
    float* part = reinterpret_cast<float*>(p + o_part);
    float* u = reinterpret_cast<float*>(p + o_u);
    float* hs = reinterpret_cast<float*>(p + o_hs);
    uint32_t* seg = reinterpret_cast<uint32_t*>(p + o_seg);
    uint32_t* perm = reinterpret_cast<uint32_t*>(p + o_perm);
    const AdapterChunks ch = AdapterChunks::at(p + o_ch, g);
    float* sums = reinterpret_cast<float*>(p + o_sum);
    float* base = dtype == BI_F32 ? static_cast<float*>(dx) : reinterpret_cast<float*>(p + o_base);
    const uint32_t G = static_cast<uint32_t>(g);
    cudaError_t e = cudaSuccess;
    if (dx && dtype == BI_F32) {  // first, as in the forward
        st = adapter_projection_f32(eng, c, 1, dx, dy, w, nullptr, m, k, n, tensor_cores);
        if (st != BI_OK) return st;
    } else if (dx) {
        e = scalar_rows(c, dtype, base, dy, w, nullptr, m, n, k, 1, 1);
    }
    if (e == cudaSuccess && need_u) {
        e = with_type(dtype, [&](auto* t) {
            using T = std::remove_pointer_t<decltype(t)>;
            return narrow_scalar<T>(c, static_cast<const T*>(dy), static_cast<const T*>(b), row_adapters, part, m, n, R, g);
        });
        if (e == cudaSuccess) e = narrow_finish(c, part, row_adapters, scales, nullptr, u, m, R, g, pieces);
    }
    if (e == cudaSuccess && grads) {
        e = segment(c, row_adapters, m, g, seg, perm, p + o_hist);
        if (e == cudaSuccess) {
            e = launch_plain(adapter_chunks_kernel, dim3(1), dim3(1024), 0, s, seg, G, ch);
            if (e == cudaSuccess) c.count();
        }
    }
    if (e == cudaSuccess && dx) {
        e = with_type(dtype, [&](auto* t) {
            using T = std::remove_pointer_t<decltype(t)>;
            return wide_scalar<T>(c, static_cast<T*>(dx), base, WideSource{u, nullptr, nullptr, nullptr, 0},
                                  static_cast<const T*>(a), row_adapters, m, k, R, g);
        });
    }
    if (e == cudaSuccess && grads) {
        auto one = [&](float* out, const float* f, const void* z, int64_t C) {
            cudaError_t err = with_type(dtype, [&](auto* t) {
                using T = std::remove_pointer_t<decltype(t)>;
                return grad_scalar<T>(c, out, sums, f, static_cast<const T*>(z), seg, perm, ch, m, C, R, g);
            });
            const AdapterGradJob job{out, sums, nullptr, z, C};
            if (err == cudaSuccess) err = grad_sum(c, &job, 1, ch, R, m, g);
            return err;
        };
        if (e == cudaSuccess && da) e = one(da, u, x, k);
        if (e == cudaSuccess && db) {
            scale_rows_kernel<<<grid1(m * r), 256, 0, s>>>(h, row_adapters, scales, hs, m, R, G);
            e = launched(c);
            if (e == cudaSuccess) e = one(db, hs, dy, n);
        }
    }
    return e == cudaSuccess ? BI_OK : cuda_fail(eng, e, "bi_adapter_backward");
}

}  // extern "C"
