// A mixture-of-experts layer for the few tokens of a decoding step, two kernels.
// See include/bi.h (bi_moe_forward).
//
//   h[t,j]  = act(x[t] Wg[e]^T) * (x[t] Wu[e]^T),  e = ids[t,j]     (hidden kernel)
//   y[t]    = round( sum_j weights[t,j] * (h[t,j] Wd[e]^T) )        (output kernel)
//
// A decoding step is bound by reading the weights of the experts that its tokens
// chose, each once: a block of either kernel takes some weight rows of an expert and
// multiplies them with all the tokens that chose it.  Every inner product is summed in
// f32 in an order that the contraction length alone decides, and a token's choices are
// added in the order j = 0, 1, ..: a row of y does not depend on the tokens beside it.
//
// Two forms of both kernels.  f32 operands (and 16-bit weights whose rows do not start
// on 16 bytes) run in f32 FMAs, a warp to two weight rows, h in f32.  The others run on
// the tensor cores' warp-level MMAs, m16n8k16: 16 weight rows by eight tokens, the
// weights going from memory to the registers that the MMA reads them from.  (tcgen05
// would want them in shared memory, and the 4-bit ones expanded there; at a few
// tokens a weight the MMA rate is not what bounds.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "abi_util.h"
#include "fp4.h"

namespace bi {
namespace {

constexpr int64_t MOE_MAX_PAIRS = 2048;  // token choices of a call: their sums stay in shared memory
constexpr int64_t MOE_MAX_E = 1024;
constexpr int M_WARPS = 8, M_THREADS = 32 * M_WARPS;
constexpr int M_ROWS = 2;                // weight rows of a warp
constexpr int M_BLOCK = M_WARPS * M_ROWS;

template <typename T> __device__ __forceinline__ float up(T v);
template <> __device__ __forceinline__ float up<float>(float v) { return v; }
template <> __device__ __forceinline__ float up<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float up<__half>(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T down(float v);
template <> __device__ __forceinline__ float down<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 down<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half down<__half>(float v) { return __float2half_rn(v); }

// Eight consecutive elements of a row of length L from k on, zeros past its end;
// vec: rows start on 16 bytes and L is a multiple of 8.
template <typename T>
__device__ __forceinline__ void load8(const T* __restrict__ row, int64_t k, int64_t L, bool vec, float (&v)[8]) {
    if (vec && k < L) {
        if constexpr (sizeof(T) == 4) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(row + k)), b = __ldg(reinterpret_cast<const float4*>(row + k) + 1);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const uint4 a = __ldg(reinterpret_cast<const uint4*>(row + k));
            const T* e = reinterpret_cast<const T*>(&a);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = up<T>(e[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = k + i < L ? up<T>(__ldg(row + k + i)) : 0.0f;
    }
}

// Weight rows [rows][L]: of type T, or MXFP4 codes and scales (T = uint8_t).
template <typename T>
struct Weights {
    const T* w;
    const uint8_t* s;
    int64_t L;
    int vec;
    __device__ __forceinline__ void load(int64_t row, int64_t k, float (&v)[8]) const {
        if constexpr (sizeof(T) == 1) {
            const int64_t Lp = fp4_padded(L);
            if (k >= L) {  // (codes past L are 0)
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = 0.0f;
                return;
            }
            const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(w + row * (Lp / 2) + k / 2));
            const float scale = fp4_scale_value(__ldg(s + fp4_scale_at(row, k >> 5, Lp)));
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fp4_code_value((c >> (4 * i)) & 15u) * scale;
        } else {
            load8<T>(w + row * L, k, L, vec != 0, v);
        }
    }
};

// acc[r][c] += rows row0 + r of W times columns c of the operand (colp[c], of length L).
template <typename WT, typename XT, int NC>
__device__ __forceinline__ void dot_rows(const Weights<WT>& W, int64_t row0, int nrows, const XT* const (&colp)[NC], bool xvec,
                                         float (&acc)[M_ROWS][NC]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int r = 0; r < M_ROWS; ++r)
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[r][c] = 0.0f;
#pragma unroll 2
    for (int64_t k = lane * 8; k < W.L; k += 256) {
        float w[M_ROWS][8];
#pragma unroll
        for (int r = 0; r < M_ROWS; ++r) W.load(row0 + min(r, nrows - 1), k, w[r]);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float x[8];
            load8<XT>(colp[c], k, W.L, xvec, x);
#pragma unroll
            for (int r = 0; r < M_ROWS; ++r)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[r][c] = fmaf(w[r][i], x[i], acc[r][c]);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < M_ROWS; ++r)
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[r][c] += __shfl_xor_sync(0xffffffffu, acc[r][c], o);
}

// The choices of a call by expert, built by every block in its shared memory:
// cnt[e] choices of expert e, first[e] the first of them in list.
struct Plan {
    uint32_t* cnt;     // [E]
    uint32_t* first;   // [E]
    uint16_t* list;    // [P]
    uint16_t* active;  // [E] experts with choices, ascending
    int n;             // how many
};
// (a multiple of 16, the last four bytes n)
__host__ __device__ constexpr int64_t plan_bytes(int64_t E, int64_t P) { return (10 * E + 2 * P + 4 + 15) / 16 * 16; }

__device__ __forceinline__ Plan build_plan(uint8_t* smem, const uint32_t* __restrict__ ids, int P, int E) {
    Plan p;
    p.cnt = reinterpret_cast<uint32_t*>(smem);
    p.first = p.cnt + E;
    p.list = reinterpret_cast<uint16_t*>(p.first + E);
    p.active = p.list + P;
    uint32_t* n = reinterpret_cast<uint32_t*>(smem + plan_bytes(E, P)) - 1;
    for (int e = threadIdx.x; e < E; e += blockDim.x) p.cnt[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < P; i += blockDim.x) {
        const uint32_t e = __ldg(ids + i);
        if (e < static_cast<uint32_t>(E)) atomicAdd(p.cnt + e, 1u);
    }
    __syncthreads();
    if (threadIdx.x < 32) {  // prefix sums over the experts
        uint32_t run = 0, act = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + threadIdx.x;
            const uint32_t c = e < E ? p.cnt[e] : 0u;
            uint32_t s = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, s, o);
                if (static_cast<int>(threadIdx.x) >= o) s += v;
            }
            const uint32_t has = __ballot_sync(0xffffffffu, c != 0);
            if (e < E) p.first[e] = run + s - c;
            if (c) p.active[act + __popc(has & ((1u << threadIdx.x) - 1u))] = static_cast<uint16_t>(e);
            run += __shfl_sync(0xffffffffu, s, 31);
            act += __popc(has);
        }
        if (threadIdx.x == 0) *n = act;
    }
    __syncthreads();
    // the lists, in any order: no result depends on it
    for (int i = threadIdx.x; i < P; i += blockDim.x) {
        const uint32_t e = __ldg(ids + i);
        if (e < static_cast<uint32_t>(E)) p.list[p.first[e] + atomicSub(p.cnt + e, 1u) - 1] = static_cast<uint16_t>(i);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < P; i += blockDim.x) {  // the counts again
        const uint32_t e = __ldg(ids + i);
        if (e < static_cast<uint32_t>(E)) atomicAdd(p.cnt + e, 1u);
    }
    __syncthreads();
    p.n = static_cast<int>(*n);
    return p;
}

template <typename WT>
struct MoeArgs {
    Weights<WT> gate, up, down;  // gate.w null: no gate
    const void* x;
    const uint32_t* ids;
    const float* weights;
    float* h;                    // [P][F]
    void* y;
    int T, C, E, act, xvec, hvec;
    int64_t K, F, N;
};

__device__ __forceinline__ float activate(float v, int act) {
    if (act == BI_ACT_SILU) return v / (1.0f + expf(-v));
    if (act == BI_ACT_GELU) return 0.5f * v * (1.0f + tanhf(0.79788456f * (v + 0.044715f * v * v * v)));
    return fmaxf(v, 0.0f) + (v != v ? v : 0.0f);  // relu; NaN stays
}

template <typename WT, typename XT, int NC>
__device__ __forceinline__ void hidden_tokens(const MoeArgs<WT>& a, const Plan& p, int e, int c0, int cn, int64_t f0, int nrows) {
    const XT* colp[NC];
    int pair[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        pair[c] = p.list[p.first[e] + c0 + min(c, cn - 1)];
        colp[c] = static_cast<const XT*>(a.x) + static_cast<int64_t>(pair[c] / a.C) * a.K;
    }
    float u[M_ROWS][NC], g[M_ROWS][NC];
    dot_rows<WT, XT, NC>(a.up, e * a.F + f0, nrows, colp, a.xvec != 0, u);
    if (a.gate.w != nullptr) dot_rows<WT, XT, NC>(a.gate, e * a.F + f0, nrows, colp, a.xvec != 0, g);
    if ((threadIdx.x & 31) != 0) return;
    for (int c = 0; c < NC && c < cn; ++c)
        for (int r = 0; r < nrows; ++r)
            a.h[pair[c] * a.F + f0 + r] = a.gate.w != nullptr ? activate(g[r][c], a.act) * u[r][c] : activate(u[r][c], a.act);
}

template <typename WT, typename XT>
__global__ void __launch_bounds__(M_THREADS) moe_hidden_kernel(const MoeArgs<WT> a) {
    extern __shared__ __align__(16) uint8_t smem[];
    grid_dep_wait();
    grid_dep_launch();
    const Plan p = build_plan(smem, a.ids, a.T * a.C, a.E);
    const int64_t f0 = static_cast<int64_t>(blockIdx.x) * M_BLOCK + (threadIdx.x >> 5) * M_ROWS;
    if (static_cast<int>(blockIdx.y) >= p.n || f0 >= a.F) return;
    const int e = p.active[blockIdx.y], n = static_cast<int>(p.cnt[e]);
    const int nrows = static_cast<int>(lmin(M_ROWS, a.F - f0));
    for (int c0 = 0; c0 < n; c0 += 4) {
        const int cn = min(4, n - c0);
        if (cn == 1) hidden_tokens<WT, XT, 1>(a, p, e, c0, cn, f0, nrows);
        else hidden_tokens<WT, XT, 4>(a, p, e, c0, cn, f0, nrows);
    }
}

template <typename WT, int NC>
__device__ __forceinline__ void output_tokens(const MoeArgs<WT>& a, const Plan& p, float* part, int e, int c0, int cn, int64_t n0,
                                              int nrows) {
    const float* colp[NC];
    int pair[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        pair[c] = p.list[p.first[e] + c0 + min(c, cn - 1)];
        colp[c] = a.h + pair[c] * a.F;
    }
    float o[M_ROWS][NC];
    dot_rows<WT, float, NC>(a.down, e * a.N + n0, nrows, colp, a.hvec != 0, o);
    if ((threadIdx.x & 31) == 0)
        for (int c = 0; c < NC && c < cn; ++c)
            for (int r = 0; r < M_ROWS; ++r) part[pair[c] * M_BLOCK + r] = o[r][c];
}

template <typename WT, typename XT>
__global__ void __launch_bounds__(M_THREADS) moe_output_kernel(const MoeArgs<WT> a) {
    extern __shared__ __align__(16) uint8_t smem[];
    grid_dep_wait();
    grid_dep_launch();
    const int P = a.T * a.C;
    const Plan p = build_plan(smem, a.ids, P, a.E);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * M_BLOCK + warp * M_ROWS;
    if (n0 >= a.N) return;
    const int nrows = static_cast<int>(lmin(M_ROWS, a.N - n0));
    float* part = reinterpret_cast<float*>(smem + plan_bytes(a.E, P)) + warp * M_ROWS;  // [P][M_BLOCK], this warp's rows
    for (int i = 0; i < p.n; ++i) {
        const int e = p.active[i], n = static_cast<int>(p.cnt[e]);
        for (int c0 = 0; c0 < n; c0 += 4) {
            const int cn = min(4, n - c0);
            if (cn == 1) output_tokens<WT, 1>(a, p, part, e, c0, cn, n0, nrows);
            else output_tokens<WT, 4>(a, p, part, e, c0, cn, n0, nrows);
        }
    }
    __syncwarp();
    for (int t = lane; t < a.T; t += 32)
        for (int r = 0; r < nrows; ++r) {
            float s = 0.0f;
            for (int j = 0; j < a.C; ++j)
                if (__ldg(a.ids + t * a.C + j) < static_cast<uint32_t>(a.E))
                    s = fmaf(__ldg(a.weights + t * a.C + j), part[(t * a.C + j) * M_BLOCK + r], s);
            static_cast<XT*>(a.y)[t * a.N + n0 + r] = down<XT>(s);
        }
}

template <typename WT, typename XT>
cudaError_t moe_t(const LaunchCtx& c, const MoeArgs<WT>& a) {
    const int64_t P = static_cast<int64_t>(a.T) * a.C;
    const int64_t plan = plan_bytes(a.E, P), out_smem = plan + P * M_BLOCK * 4;
    auto kh = moe_hidden_kernel<WT, XT>;
    auto ko = moe_output_kernel<WT, XT>;
    static PerDeviceOnce setup;
    cudaError_t e = setup.run(c.eng->device, [&](int&) {
        return cudaFuncSetAttribute(ko, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(plan_bytes(MOE_MAX_E, MOE_MAX_PAIRS) + MOE_MAX_PAIRS * M_BLOCK * 4));
    });
    if (e != cudaSuccess) return e;
    const dim3 gh(static_cast<unsigned>((a.F + M_BLOCK - 1) / M_BLOCK), static_cast<unsigned>(lmin(a.E, P)));
    if ((e = launch_pdl(kh, gh, dim3(M_THREADS), plan, c.stream, a)) != cudaSuccess) return e;
    c.count();
    const dim3 go(static_cast<unsigned>((a.N + M_BLOCK - 1) / M_BLOCK));
    if ((e = launch_pdl(ko, go, dim3(M_THREADS), out_smem, c.stream, a)) != cudaSuccess) return e;
    c.count();
    return cudaGetLastError();
}

// ---------------------------------------------------------------- tensor-core form
//
// A contraction is cut into RUNS equal runs of chunks; a run is one chain of MMAs and
// the runs' sums are added in order, whichever warps take them.
//
// A lane loads 16 bytes of a weight row at a time (the MMA's row g = lane / 4 and the
// row 8 below), four lanes 64 consecutive bytes, and its elements become the MMA's
// contraction slots as they come: the order of the contraction within a chunk is free
// as long as the tokens' operand has the same one.  Weights of 16 bits: chunks of 64.
// MXFP4: chunks of 128, a lane's 16 bytes are one block of 32 with its scale; the
// codes are taken in pairs (i, i + 4) of eight, which one shift brings to the two
// halves of a register, and become bf16: the code's bits at bf16's exponent are the
// value * 2^-126 (its subnormal being e2m1's), and one multiplication by 2^126 2^s makes
// it the value, exactly.
//
// x enters as it is where it has the MMA's type; h, and f16 x beside MXFP4 weights,
// as two bf16 parts, high part and remainder (to 2^-17 of the value, and f16's 11 bits
// exactly), two MMAs into the same sum.  f16 weights in the output kernel are split
// into two bf16 parts too, exactly, since h may be beyond f16's range.

constexpr int RUNS = 8;
enum WeightKind { W_BF16 = 0, W_F16 = 1, W_FP4 = 2 };

__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1, bool half) {
    if (half)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// Two f32 values as bf16 parts: v = hi + lo to 2^-17 of v.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = pack_bf16(a, b);
    lo = pack_bf16(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
}
__device__ __forceinline__ void split_f16x2(uint32_t w, uint32_t& hi, uint32_t& lo) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    split2(f.x, f.y, hi, lo);
}
// The factor 2^126 2^s of a scale byte s + 127, as two bf16 factors whose product it
// is (the second is 1 for s <= 1, as weights have); byte 255 gives NaN.
__device__ __forceinline__ uint32_t scale_factor(uint32_t byte, uint32_t& second) {
    const uint32_t e = byte + 126;  // exponent field of 2^(byte - 1) = 2^126 2^(byte - 127), bias 127
    const uint32_t first = min(e, 254u);
    second = byte == 255u ? 0x7fc07fc0u : (127u + e - first) * 0x00800080u;
    return first * 0x00800080u;
}

constexpr int t_chunk(int wk) { return wk == W_FP4 ? 128 : 64; }

// The weights' way: a lane copies its 16 bytes of a row to its own slot of shared
// memory (cp.async, DEPTH chunks ahead) and reads them back itself, so a warp's copies
// run ahead of its MMAs without holding registers and without waiting for anyone.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {  // the rest of the 16: zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 slot_read(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

template <int WK, int NM>
struct Feed {
    static constexpr int V = WK == W_FP4 ? 1 : 2;                        // 16-byte pieces per row and chunk
    static constexpr int SLOTS = NM * 2 * V + (WK == W_FP4 ? 1 : 0);     // ... per lane and chunk, the scales' words in one
    static constexpr int STAGE = SLOTS * 512;                            // bytes of a warp's chunk
    const uint8_t* row[NM][2];    // the lane's first piece of chunk 0 of its rows (g and g + 8 of each matrix)
    const uint8_t* scale[NM][2];  // MXFP4: the word of the row's four scale bytes of chunk 0
    const uint8_t* any;           // an address of the weights, for copies of nothing
    int64_t L;                    // contraction length, in elements
    uint32_t slot;                // the lane's first slot
    __device__ __forceinline__ void set(int m, int i, const void* w, const uint8_t* s, int64_t r) {
        const int t = threadIdx.x & 3;
        any = static_cast<const uint8_t*>(w);
        if constexpr (WK == W_FP4) {
            const int64_t Lp = fp4_padded(L);
            row[m][i] = static_cast<const uint8_t*>(w) + r * (Lp / 2) + t * 16;
            scale[m][i] = s + fp4_scale_at(r, 0, Lp);
        } else {
            row[m][i] = static_cast<const uint8_t*>(w) + (r * L + t * 8) * 2;
        }
    }
    __device__ __forceinline__ void copy(int stage, int chunk) const {
        const uint32_t to = slot + stage * STAGE;
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if constexpr (WK == W_FP4) {  // codes and scales are padded to 256 elements
                    copy16(to + (m * 2 + i) * 512, row[m][i] + static_cast<int64_t>(chunk) * 64, 16);
                    copy4(to + NM * 2 * 512 + (m * 2 + i) * 4, scale[m][i] + static_cast<int64_t>(chunk) * 512);
                } else {
                    const int64_t k = static_cast<int64_t>(chunk) * 64 + (threadIdx.x & 3) * 8;
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const bool in = k + v * 32 < L;  // (whole pieces: L is a multiple of 8)
                        copy16(to + ((m * 2 + i) * 2 + v) * 512, in ? row[m][i] + static_cast<int64_t>(chunk) * 128 + v * 64 : any,
                               in ? 16 : 0);
                    }
                }
            }
    }
};

// The tokens' operand: NT tiles of 8 columns, a lane's own column of each.
//   PLANES  two bf16 planes [2][L] per column, L a multiple of 128, zeros past the
//           contraction; for MXFP4 weights eight elements lie in the order 0 4 1 5 2 6 3 7
//   else    rows of length L (a multiple of 8) of the MMA's type
template <int WK, int NT, bool PLANES>
struct Columns {
    static constexpr int PARTS = PLANES ? 2 : 1;
    const uint16_t* col[NT];
    int64_t L;
    // the eight elements from k on, in the order in which the weights' are used
    __device__ __forceinline__ void load(uint4 (&b)[PARTS], int nt, int64_t k) const {
        if constexpr (PLANES) {
            b[0] = __ldg(reinterpret_cast<const uint4*>(col[nt] + k));
            b[PARTS - 1] = __ldg(reinterpret_cast<const uint4*>(col[nt] + L + k));
        } else {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (k < L) x = __ldg(reinterpret_cast<const uint4*>(col[nt] + k));
            b[0] = x;
        }
    }
    static __device__ __forceinline__ void order(uint4 (&b)[PARTS]) {
        if constexpr (WK == W_FP4 && !PLANES)
            b[0] = make_uint4(__byte_perm(b[0].x, b[0].z, 0x5410), __byte_perm(b[0].x, b[0].z, 0x7632),
                              __byte_perm(b[0].y, b[0].w, 0x5410), __byte_perm(b[0].y, b[0].w, 0x7632));
    }
};

// acc += one chunk, its weights in the lane's slots from `at` on.
template <int WK, int NM, int NT, bool PLANES>
__device__ __forceinline__ void chunk_mma(float (&acc)[NM][NT][4], uint32_t at, const Columns<WK, NT, PLANES>& cols, int chunk) {
    constexpr int PARTS = Columns<WK, NT, PLANES>::PARTS;
    const int t = threadIdx.x & 3;
    if constexpr (WK == W_FP4) {
        uint32_t f[NM][2], f2[NM][2];
        const uint4 sw = slot_read(at + NM * 2 * 512);
        bool large = false;
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t word = m == 0 ? (i == 0 ? sw.x : sw.y) : (i == 0 ? sw.z : sw.w), byte = (word >> (8 * t)) & 255u;
                f[m][i] = scale_factor(byte, f2[m][i]);
                large |= byte > 128u;
            }
        large = __any_sync(0xffffffffu, large);
        uint4 w[NM][2];
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) w[m][i] = slot_read(at + (m * 2 + i) * 512);
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // eight codes of the lane's 32
            uint32_t a[NM][2][4];
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t c = q == 0 ? w[m][i].x : q == 1 ? w[m][i].y : q == 2 ? w[m][i].z : w[m][i].w;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t u = c << (12 - 4 * j);
                        a[m][i][j] = mul_bf16x2((u & 0x80008000u) | ((u >> 6) & 0x01c001c0u), f[m][i]);
                        if (large) a[m][i][j] = mul_bf16x2(a[m][i][j], f2[m][i]);
                    }
                }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint4 b[PARTS];
                cols.load(b, nt, static_cast<int64_t>(chunk) * 128 + t * 32 + q * 8);
                cols.order(b);
#pragma unroll
                for (int p = 0; p < PARTS; ++p)
#pragma unroll
                    for (int m = 0; m < NM; ++m) {
                        mma16(acc[m][nt], a[m][0][0], a[m][1][0], a[m][0][1], a[m][1][1], b[p].x, b[p].y, false);
                        mma16(acc[m][nt], a[m][0][2], a[m][1][2], a[m][0][3], a[m][1][3], b[p].z, b[p].w, false);
                    }
            }
        }
    } else {
        constexpr bool SPLIT = WK == W_F16 && PLANES, HALF = WK == W_F16 && !PLANES;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            uint4 w[NM][2], lo[NM][2];
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 r = slot_read(at + ((m * 2 + i) * 2 + v) * 512);
                    w[m][i] = r;
                    if constexpr (SPLIT) {
                        split_f16x2(r.x, w[m][i].x, lo[m][i].x);
                        split_f16x2(r.y, w[m][i].y, lo[m][i].y);
                        split_f16x2(r.z, w[m][i].z, lo[m][i].z);
                        split_f16x2(r.w, w[m][i].w, lo[m][i].w);
                    }
                }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                uint4 b[PARTS];
                cols.load(b, nt, static_cast<int64_t>(chunk) * 64 + v * 32 + t * 8);
#pragma unroll
                for (int p = 0; p < PARTS; ++p)
#pragma unroll
                    for (int m = 0; m < NM; ++m) {
                        const uint4 *u = w[m], &x = b[p];
                        mma16(acc[m][nt], u[0].x, u[1].x, u[0].y, u[1].y, x.x, x.y, HALF);
                        mma16(acc[m][nt], u[0].z, u[1].z, u[0].w, u[1].w, x.z, x.w, HALF);
                        if constexpr (SPLIT) {
                            mma16(acc[m][nt], lo[m][0].x, lo[m][1].x, lo[m][0].y, lo[m][1].y, x.x, x.y, false);
                            mma16(acc[m][nt], lo[m][0].z, lo[m][1].z, lo[m][0].w, lo[m][1].w, x.z, x.w, false);
                        }
                    }
            }
        }
    }
}

// Run r of a contraction of so many chunks begins at:
__host__ __device__ __forceinline__ int run_begin(int r, int chunks) { return static_cast<int>(static_cast<int64_t>(r) * chunks / RUNS); }

template <int NM, int NT>
__device__ __forceinline__ void zero(float (&acc)[NM][NT][4]) {
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][nt][i] = 0.0f;
}

struct MoeTcArgs {
    const void *gate, *up, *down;
    const uint8_t *gate_s, *up_s, *down_s;
    const uint16_t* x;     // [T][xL], or planes [T][2][xL]
    const uint32_t* ids;
    const float* weights;
    uint16_t* h;           // planes [P][2][Fp]
    void* y;
    int T, C, E, act;
    int64_t K, F, N, xL, Fp;
};
__host__ __device__ __forceinline__ int64_t plane_length(int64_t l) { return (l + 127) / 128 * 128; }

constexpr int TH_WARPS = RUNS, TH_THREADS = 32 * TH_WARPS;  // hidden kernel: a warp to a run
constexpr int TO_WARPS = 16, TO_THREADS = 32 * TO_WARPS;
constexpr int red_pitch(int nt) { return nt * 8 + 2; }      // floats of a row of partial sums
// Chunks a warp's copies run ahead: 12 KB a warp with two hidden blocks of 8 warps on an
// SM; an output block of 16 warps has an SM alone, and 8 KB a warp (MXFP4 9) beside 64 KB of
// choices' sums, 4 KB (4.5) beside 128 KB.
constexpr int th_depth(int wk, int nm) { return 12 * 1024 / (wk == W_FP4 ? (nm * 2 + 1) * 512 : nm * 2048); }
constexpr int to_depth(int wk, bool deep) { return wk == W_FP4 ? (deep ? 6 : 3) : (deep ? 4 : 2); }

// Position of element f of a plane.
template <int WK>
__device__ __forceinline__ int64_t plane_at(int64_t f) {
    const int64_t k = f & 7;
    return WK == W_FP4 ? (f & ~7ll) + (k < 4 ? 2 * k : 2 * k - 7) : f;
}

template <int WK, bool XPLANES, int NM, int NT>
__device__ __forceinline__ void hidden_pass(const MoeTcArgs& a, const Plan& p, const Feed<WK, NM>& feed, float* red, int e, int c0, int cn,
                                            int64_t f0) {
    constexpr int DEPTH = th_depth(WK, NM);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    Columns<WK, NT, XPLANES> cols;
    cols.L = a.xL;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int64_t tok = p.list[p.first[e] + c0 + min(nt * 8 + g, cn - 1)] / a.C;
        cols.col[nt] = a.x + tok * (XPLANES ? 2 * a.xL : a.xL);
    }
    float acc[NM][NT][4];
    zero<NM, NT>(acc);
    const int chunks = static_cast<int>((a.K + t_chunk(WK) - 1) / t_chunk(WK));
    const int begin = run_begin(warp, chunks), end = run_begin(warp + 1, chunks);
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
        if (begin + d < end) feed.copy(d, begin + d);
        copies_commit();
    }
    int st = 0;
    for (int c = begin; c < end; ++c) {
        copies_wait<DEPTH - 1>();
        chunk_mma<WK, NM, NT, XPLANES>(acc, feed.slot + st * Feed<WK, NM>::STAGE, cols, c);
        if (c + DEPTH < end) feed.copy(st, c + DEPTH);
        copies_commit();
        if (++st == DEPTH) st = 0;
    }
    constexpr int PITCH = red_pitch(NT);
    __syncthreads();  // the warps' slots become the sums' place
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<float2*>(red + ((warp * NM + m) * 16 + g + 8 * i) * PITCH + nt * 8 + 2 * t) =
                    make_float2(acc[m][nt][2 * i], acc[m][nt][2 * i + 1]);
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * cn; i += TH_THREADS) {
        const int r = i & 15, c = i >> 4;
        float v[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            v[m] = 0.0f;
#pragma unroll
            for (int s = 0; s < RUNS; ++s) v[m] = __fadd_rn(v[m], red[((s * NM + m) * 16 + r) * PITCH + c]);
        }
        if (f0 + r < a.F) {
            const float h = NM == 2 ? activate(v[NM - 1], a.act) * v[0] : activate(v[0], a.act);
            uint16_t* o = a.h + static_cast<int64_t>(p.list[p.first[e] + c0 + c]) * 2 * a.Fp + plane_at<WK>(f0 + r);
            uint32_t hi, lo;
            split2(h, 0.0f, hi, lo);
            o[0] = static_cast<uint16_t>(hi);
            o[a.Fp] = static_cast<uint16_t>(lo);
        }
    }
    if (blockIdx.x == gridDim.x - 1) {  // the planes' ends
        const int n = static_cast<int>(a.Fp - a.F);
        for (int i = threadIdx.x; i < n * cn; i += TH_THREADS) {
            uint16_t* o = a.h + static_cast<int64_t>(p.list[p.first[e] + c0 + i / n]) * 2 * a.Fp + plane_at<WK>(a.F + i % n);
            o[0] = 0;
            o[a.Fp] = 0;
        }
    }
    __syncthreads();
}

// A block: 16 rows of the hidden layer (of the gate's weights and of up's) of one
// expert, a warp to each of the contraction's runs.
template <int WK, bool XPLANES, int NM>
__global__ void __launch_bounds__(TH_THREADS, 2) moe_hidden_tc_kernel(const MoeTcArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    grid_dep_wait();
    grid_dep_launch();
    const int P = a.T * a.C;
    const Plan p = build_plan(smem, a.ids, P, a.E);
    if (static_cast<int>(blockIdx.y) >= p.n) return;
    float* red = reinterpret_cast<float*>(smem + plan_bytes(a.E, P));  // the slots of the weights, then the runs' sums
    const int e = p.active[blockIdx.y], n = static_cast<int>(p.cnt[e]);
    const int64_t f0 = static_cast<int64_t>(blockIdx.x) * 16;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Feed<WK, NM> feed;
    feed.L = a.K;
    feed.slot = static_cast<uint32_t>(__cvta_generic_to_shared(red)) + warp * th_depth(WK, NM) * Feed<WK, NM>::STAGE + lane * 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t r = e * a.F + lmin(f0 + (lane >> 2) + 8 * i, a.F - 1);
        feed.set(0, i, a.up, a.up_s, r);
        if constexpr (NM == 2) feed.set(1, i, a.gate, a.gate_s, r);
    }
    for (int c0 = 0; c0 < n; c0 += 32) {
        const int cn = min(32, n - c0);
        if (cn <= 8) hidden_pass<WK, XPLANES, NM, 1>(a, p, feed, red, e, c0, cn, f0);
        else if (cn <= 16) hidden_pass<WK, XPLANES, NM, 2>(a, p, feed, red, e, c0, cn, f0);
        else hidden_pass<WK, XPLANES, NM, 4>(a, p, feed, red, e, c0, cn, f0);
    }
}

// The work of one warp of an output block, item after item: an expert, a stretch of the
// contraction and up to 32 of the expert's choices.
//   SPLIT: one run at a time, so that the runs of few experts are spread over the warps
//   else:  the whole contraction
template <bool SPLIT>
struct Items {
    int j, width;        // item number over all warps (SPLIT: without the columns); columns per item
    int i, e, n, c0, run;
    __device__ __forceinline__ void first(const Plan& p, int warp, int w) {
        width = w;
        j = SPLIT ? warp : -1;
        i = -1;
        n = c0 = run = 0;
        if (SPLIT) open(p);
        else next(p, warp);
    }
    __device__ __forceinline__ void open(const Plan& p) {
        i = j / RUNS;
        run = j % RUNS;
        c0 = 0;
        if (i < p.n) { e = p.active[i]; n = static_cast<int>(p.cnt[e]); }
    }
    __device__ __forceinline__ bool more(const Plan& p) const { return i < p.n; }
    __device__ __forceinline__ void next(const Plan& p, int warp) {
        c0 += width;
        if (SPLIT) {
            if (c0 < n) return;
            j += TO_WARPS;
            open(p);
            return;
        }
        for (;;) {
            if (i < 0 || c0 >= n) {
                c0 = 0;
                if (++i >= p.n) return;
                e = p.active[i];
                n = static_cast<int>(p.cnt[e]);
            }
            if (++j % TO_WARPS == warp) return;
            c0 += width;
        }
    }
    __device__ __forceinline__ int begin(int chunks) const { return SPLIT ? run_begin(run, chunks) : 0; }
    __device__ __forceinline__ int end(int chunks) const { return SPLIT ? run_begin(run + 1, chunks) : chunks; }
};

// The stream of chunks that a warp's copies bring in: its items' chunks, one after the
// other, DEPTH ahead of the item that is computed.
template <int WK, bool SPLIT, int DEPTH>
struct Stream {
    Feed<WK, 1> feed;
    Items<SPLIT> it;
    int c, in, out;  // next chunk of the item; stages to fill and to read
    __device__ __forceinline__ void rows(const MoeTcArgs& a, const Plan& p, int64_t n0, int chunks, int warp) {
        while (it.more(p) && it.begin(chunks) == it.end(chunks)) it.next(p, warp);  // runs without chunks
        if (!it.more(p)) return;
        c = it.begin(chunks);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            feed.set(0, i, a.down, a.down_s, it.e * a.N + lmin(n0 + ((threadIdx.x & 31) >> 2) + 8 * i, a.N - 1));
    }
    __device__ __forceinline__ void push(const MoeTcArgs& a, const Plan& p, int64_t n0, int chunks, int warp) {
        if (it.more(p)) {
            feed.copy(in, c);
            if (++in == DEPTH) in = 0;
            if (++c == it.end(chunks)) {
                it.next(p, warp);
                rows(a, p, n0, chunks, warp);
            }
        }
        copies_commit();
    }
};

template <int WK, int NT, bool SPLIT, int DEPTH>
__device__ __forceinline__ void output_item(const MoeTcArgs& a, const Plan& p, float* part, Stream<WK, SPLIT, DEPTH>& s, const Items<SPLIT>& it,
                                            int cn, int64_t n0, int chunks, int warp) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    Columns<WK, NT, true> cols;
    cols.L = a.Fp;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        cols.col[nt] = a.h + static_cast<int64_t>(p.list[p.first[it.e] + it.c0 + min(nt * 8 + g, cn - 1)]) * 2 * a.Fp;
    float acc[1][NT][4], sum[1][NT][4];
    zero<1, NT>(acc);
    zero<1, NT>(sum);
    auto close = [&] {  // a run's sum joins the ones before
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[0][nt][i] = __fadd_rn(sum[0][nt][i], acc[0][nt][i]);
        zero<1, NT>(acc);
    };
    int run = 0;
    for (int c = it.begin(chunks); c < it.end(chunks); ++c) {
        if (!SPLIT)
            for (; c == run_begin(run + 1, chunks); ++run) close();
        copies_wait<DEPTH - 1>();
        chunk_mma<WK, 1, NT, true>(acc, s.feed.slot + s.out * Feed<WK, 1>::STAGE, cols, c);
        if (++s.out == DEPTH) s.out = 0;
        s.push(a, p, n0, chunks, warp);
    }
    if (!SPLIT) close();
    const int P = a.T * a.C;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = nt * 8 + 2 * t + i;
            if (c >= cn) continue;
            float* o = part + (it.run * P + p.list[p.first[it.e] + it.c0 + c]) * 16;
            o[g] = SPLIT ? acc[0][nt][i] : sum[0][nt][i];
            o[g + 8] = SPLIT ? acc[0][nt][2 + i] : sum[0][nt][2 + i];
        }
}

// A block: 16 rows of the output for all tokens.  Its warps leave the choices' sums in
// shared memory and the block adds them, weighted: no partial sum leaves the SM.
template <int WK, typename XT, bool SPLIT, bool DEEP>
__global__ void __launch_bounds__(TO_THREADS, 1) moe_output_tc_kernel(const MoeTcArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    grid_dep_wait();
    grid_dep_launch();
    const int P = a.T * a.C, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Plan p = build_plan(smem, a.ids, P, a.E);
    float* part = reinterpret_cast<float*>(smem + plan_bytes(a.E, P));  // [RUNS or 1][P][16]
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
    const int chunks = static_cast<int>((a.F + t_chunk(WK) - 1) / t_chunk(WK));
    // columns per item: all warps have some
    const int width = SPLIT || P <= 16 * TO_WARPS ? 16 : 32;
    Items<SPLIT> it;
    it.first(p, warp, width);
    constexpr int DEPTH = to_depth(WK, DEEP);
    Stream<WK, SPLIT, DEPTH> s;
    s.feed.L = a.F;
    s.feed.slot = static_cast<uint32_t>(__cvta_generic_to_shared(part + static_cast<int64_t>(SPLIT ? RUNS : 1) * P * 16)) +
                  warp * DEPTH * Feed<WK, 1>::STAGE + lane * 16;
    s.it = it;
    s.in = s.out = 0;
    s.rows(a, p, n0, chunks, warp);
    for (int d = 0; d < DEPTH; ++d) s.push(a, p, n0, chunks, warp);
    for (; it.more(p); it.next(p, warp)) {
        const int cn = min(width, it.n - it.c0);
        if (cn <= 8) output_item<WK, 1, SPLIT, DEPTH>(a, p, part, s, it, cn, n0, chunks, warp);
        else if (SPLIT || cn <= 16) output_item<WK, 2, SPLIT, DEPTH>(a, p, part, s, it, cn, n0, chunks, warp);
        else output_item<WK, 4, SPLIT, DEPTH>(a, p, part, s, it, cn, n0, chunks, warp);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.T * 16; i += TO_THREADS) {
        const int t = i >> 4, r = i & 15;
        if (n0 + r >= a.N) continue;
        float sum = 0.0f;
        for (int j = 0; j < a.C; ++j) {
            const int pr = t * a.C + j;
            if (__ldg(a.ids + pr) >= static_cast<uint32_t>(a.E)) continue;
            float q = 0.0f;
            for (int l = 0; l < (SPLIT ? RUNS : 1); ++l) q = __fadd_rn(q, part[(l * P + pr) * 16 + r]);
            sum = fmaf(__ldg(a.weights + pr), q, sum);
        }
        static_cast<XT*>(a.y)[t * a.N + n0 + r] = down<XT>(sum);
    }
}

// x made ready for the MMAs where it is not: rows that do not start on 16 bytes or are
// no multiple of 8 long, copied (PLANES false), or f16 beside MXFP4 weights, as two
// bf16 planes.
template <bool PLANES>
__global__ void __launch_bounds__(256) moe_x_kernel(uint16_t* out, const uint16_t* x, int64_t T, int64_t K, int64_t Kp) {
    grid_dep_wait();
    grid_dep_launch();
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < T * Kp; i += gridDim.x * 256ll) {
        const int64_t t = i / Kp, k = i - t * Kp;
        const uint16_t v = k < K ? x[t * K + k] : 0;
        if (PLANES) {
            uint32_t hi, lo;
            split2(__half2float(__ushort_as_half(v)), 0.0f, hi, lo);
            uint16_t* o = out + t * 2 * Kp + plane_at<W_FP4>(k);
            o[0] = static_cast<uint16_t>(hi);
            o[Kp] = static_cast<uint16_t>(lo);
        } else {
            out[i] = v;
        }
    }
}

template <int WK, bool XPLANES, int NM, typename XT>
cudaError_t moe_tc_t(const LaunchCtx& c, const MoeTcArgs& a) {
    const int64_t P = static_cast<int64_t>(a.T) * a.C, plan = plan_bytes(a.E, P);
    auto kh = moe_hidden_tc_kernel<WK, XPLANES, NM>;
    constexpr int64_t ring = TH_WARPS * th_depth(WK, NM) * Feed<WK, NM>::STAGE, red = RUNS * NM * 16 * red_pitch(4) * 4;
    constexpr int64_t h_smem = ring > red ? ring : red;
    constexpr int64_t deep = TO_WARPS * to_depth(WK, true) * Feed<WK, 1>::STAGE, flat = TO_WARPS * to_depth(WK, false) * Feed<WK, 1>::STAGE;
    constexpr int64_t plan_max = plan_bytes(MOE_MAX_E, MOE_MAX_PAIRS), sums = 64 * 1024;  // bytes of sums beside the deep ring
    static_assert(2 * (plan_max + h_smem + 1024) <= 228 * 1024 && plan_max + sums + deep <= 227 * 1024 &&
                  plan_max + MOE_MAX_PAIRS * 64 + flat <= 227 * 1024, "shared memory");
    // the runs apart where their sums fit: then there are few experts to share out
    const int form = RUNS * P * 64 <= sums ? 0 : P * 64 <= sums ? 1 : 2;
    void (*const out_kernels[3])(const MoeTcArgs) = {moe_output_tc_kernel<WK, XT, true, true>, moe_output_tc_kernel<WK, XT, false, true>,
                                                     moe_output_tc_kernel<WK, XT, false, false>};
    const int64_t out_smem = plan + (form == 0 ? RUNS : 1) * P * 64 + (form == 2 ? flat : deep);
    static PerDeviceOnce setup;
    cudaError_t e = setup.run(c.eng->device, [&](int&) {
        cudaError_t q = cudaFuncSetAttribute(kh, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(plan_max + h_smem));
        for (auto k : out_kernels)
            if (q == cudaSuccess) q = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        return q;
    });
    if (e != cudaSuccess) return e;
    if ((e = launch_pdl(kh, dim3(static_cast<unsigned>((a.F + 15) / 16), static_cast<unsigned>(lmin(a.E, P))), dim3(TH_THREADS),
                        static_cast<size_t>(plan + h_smem), c.stream, a)) != cudaSuccess)
        return e;
    c.count();
    if ((e = launch_pdl(out_kernels[form], dim3(static_cast<unsigned>((a.N + 15) / 16)), dim3(TO_THREADS), static_cast<size_t>(out_smem),
                        c.stream, a)) != cudaSuccess)
        return e;
    c.count();
    return cudaGetLastError();
}

bi_status moe(bi_engine eng, void* y, const void* x, const uint32_t* ids, const float* weights, const void* wg, const uint8_t* sg,
              const void* wu, const uint8_t* su, const void* wd, const uint8_t* sd, bool fp4, int64_t t, int64_t c, int64_t k,
              int64_t f, int64_t n, int64_t e, int act, bi_dtype dt, void* stream, const char* name) {
    if (!eng) return fail(nullptr, BI_ERR_INVALID_ARG, "engine is NULL");
    if (dt != BI_F32 && dt != BI_BF16 && dt != BI_F16) return fail(eng, BI_ERR_INVALID_ARG, "dtype must be BI_F32, BI_BF16 or BI_F16");
    if (act != BI_ACT_SILU && act != BI_ACT_GELU && act != BI_ACT_RELU)
        return fail(eng, BI_ERR_INVALID_ARG, "activation must be BI_ACT_SILU, BI_ACT_GELU or BI_ACT_RELU");
    if (t < 0 || c <= 0 || k <= 0 || f <= 0 || n <= 0 || e <= 0)
        return fail(eng, BI_ERR_INVALID_ARG, "t must be >= 0, the other sizes > 0");
    if (e > MOE_MAX_E || c > MOE_MAX_PAIRS || t > MOE_MAX_PAIRS || t * c > MOE_MAX_PAIRS)
        return fail(eng, BI_ERR_UNSUPPORTED, "at most 1024 experts and t * c = 2048 choices: longer batches take the grouped matmul");
    const int64_t lim = 8388480;
    if (k > lim || f > lim || n > lim) return fail(eng, BI_ERR_UNSUPPORTED, "k, f and n are limited to 8388480");
    if (t == 0) return BI_OK;
    if (!y || !x || !ids || !weights || !wu || !wd || (fp4 && (!su || !sd)))
        return fail(eng, BI_ERR_INVALID_ARG, "y, x, ids, weights and the expert weights must not be NULL");
    if (fp4 && (wg == nullptr) != (sg == nullptr)) return fail(eng, BI_ERR_INVALID_ARG, "the gate's codes and scales go together");
    if (fp4 && !(aligned16(wg) && aligned16(sg) && aligned16(wu) && aligned16(su) && aligned16(wd) && aligned16(sd)))
        return fail(eng, BI_ERR_MISALIGNED, "codes and scales need 16-byte alignment");
    DeviceGuard g(eng->device);
    if (!g.ok) return fail(eng, BI_ERR_CUDA, "cudaSetDevice failed");
    const LaunchCtx lc = ctx(eng, stream);
    // the form is a function of the types, K, F and the weights' alignment
    if (dt != BI_F32 && (fp4 || (k % 8 == 0 && f % 8 == 0 && aligned16(wg) && aligned16(wu) && aligned16(wd)))) {
        const int64_t Fp = plane_length(f), Kp = plane_length(k);
        const bool planes = fp4 && dt == BI_F16, copy = !planes && (k % 8 != 0 || !aligned16(x));
        const int64_t hb = round256(t * c * 2 * Fp * 2), xb = planes ? t * 2 * Kp * 2 : copy ? t * Kp * 2 : 0;
        Scratch sc(eng, lc.stream, static_cast<size_t>(hb + xb));
        if (sc.err != cudaSuccess) return cuda_fail(eng, sc.err, "hidden scratch");
        MoeTcArgs a{};
        a.gate = wg; a.up = wu; a.down = wd;
        a.gate_s = sg; a.up_s = su; a.down_s = sd;
        a.x = static_cast<const uint16_t*>(x);
        a.ids = ids;
        a.weights = weights;
        a.h = static_cast<uint16_t*>(sc.ptr);
        a.y = y;
        a.T = static_cast<int>(t); a.C = static_cast<int>(c); a.E = static_cast<int>(e);
        a.act = act;
        a.K = k; a.F = f; a.N = n; a.Fp = Fp;
        a.xL = k;
        cudaError_t err = cudaSuccess;
        if (planes || copy) {
            uint16_t* xp = a.h + hb / 2;
            err = launch_pdl(planes ? moe_x_kernel<true> : moe_x_kernel<false>, dim3(static_cast<unsigned>(lmin((t * Kp + 255) / 256, 4 * lc.sm_count))),
                             dim3(256), 0, lc.stream, xp, a.x, t, k, Kp);
            if (err == cudaSuccess) lc.count();
            a.x = xp;
            a.xL = Kp;
        }
        auto gated = [&](auto nm) {
            constexpr int NM = decltype(nm)::value;
            if (fp4) return dt == BI_F16 ? moe_tc_t<W_FP4, true, NM, __half>(lc, a) : moe_tc_t<W_FP4, false, NM, __nv_bfloat16>(lc, a);
            return dt == BI_F16 ? moe_tc_t<W_F16, false, NM, __half>(lc, a) : moe_tc_t<W_BF16, false, NM, __nv_bfloat16>(lc, a);
        };
        if (err == cudaSuccess) err = wg ? gated(std::integral_constant<int, 2>()) : gated(std::integral_constant<int, 1>());
        return err == cudaSuccess ? BI_OK : cuda_fail(eng, err, name);
    }
    Scratch h(eng, lc.stream, static_cast<size_t>(round256(t * c * f * 4)));
    if (h.err != cudaSuccess) return cuda_fail(eng, h.err, "hidden scratch");
    auto go = [&](auto wtype, auto xtype) {
        using WT = decltype(wtype);
        using XT = decltype(xtype);
        MoeArgs<WT> a{};
        auto set = [&](Weights<WT>& w, const void* p, const uint8_t* s, int64_t L) {
            w.w = static_cast<const WT*>(p);
            w.s = s;
            w.L = L;
            w.vec = L % 8 == 0 && aligned16(p);
        };
        set(a.gate, wg, sg, k);
        set(a.up, wu, su, k);
        set(a.down, wd, sd, f);
        a.x = x;
        a.ids = ids;
        a.weights = weights;
        a.h = static_cast<float*>(h.ptr);
        a.y = y;
        a.T = static_cast<int>(t);
        a.C = static_cast<int>(c);
        a.E = static_cast<int>(e);
        a.act = act;
        a.xvec = k % 8 == 0 && aligned16(x);
        a.hvec = f % 8 == 0;
        a.K = k;
        a.F = f;
        a.N = n;
        return moe_t<WT, XT>(lc, a);
    };
    cudaError_t err;
    if (fp4) {
        err = go(uint8_t(), float());
    } else {
        err = dt == BI_F32 ? go(float(), float()) : dt == BI_BF16 ? go(__nv_bfloat16(), __nv_bfloat16()) : go(__half(), __half());
    }
    return err == cudaSuccess ? BI_OK : cuda_fail(eng, err, name);
}

}  // namespace
}  // namespace bi

extern "C" {

bi_status bi_moe_forward(bi_engine eng, void* y, const void* x, const uint32_t* ids, const float* weights, const void* w_gate,
                         const void* w_up, const void* w_down, int64_t t, int64_t c, int64_t k, int64_t f, int64_t n, int64_t e,
                         bi_activation activation, bi_dtype dtype, void* stream) {
    return bi::moe(eng, y, x, ids, weights, w_gate, nullptr, w_up, nullptr, w_down, nullptr, false, t, c, k, f, n, e, activation,
                   dtype, stream, "bi_moe_forward");
}

bi_status bi_moe_forward_fp4(bi_engine eng, void* y, const void* x, const uint32_t* ids, const float* weights, const uint8_t* gate_q,
                             const uint8_t* gate_s, const uint8_t* up_q, const uint8_t* up_s, const uint8_t* down_q,
                             const uint8_t* down_s, int64_t t, int64_t c, int64_t k, int64_t f, int64_t n, int64_t e,
                             bi_activation activation, bi_dtype dtype, void* stream) {
    return bi::moe(eng, y, x, ids, weights, gate_q, gate_s, up_q, up_s, down_q, down_s, true, t, c, k, f, n, e, activation, dtype,
                   stream, "bi_moe_forward_fp4");
}

}  // extern "C"
