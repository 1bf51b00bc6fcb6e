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
// h stays in f32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

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
__host__ __device__ constexpr int64_t plan_bytes(int64_t E, int64_t P) { return 8 * E + (2 * P + 2 * E + 16 + 15) / 16 * 16; }

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
    Scratch h(eng, static_cast<cudaStream_t>(stream), static_cast<size_t>(round256(t * c * f * 4)));
    if (h.err != cudaSuccess) return cuda_fail(eng, h.err, "hidden scratch");
    const LaunchCtx lc = ctx(eng, stream);
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
        err = dt == BI_F32 ? go(uint8_t(), float()) : dt == BI_BF16 ? go(uint8_t(), __nv_bfloat16()) : go(uint8_t(), __half());
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
