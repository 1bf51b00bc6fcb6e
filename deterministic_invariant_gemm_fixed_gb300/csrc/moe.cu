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
// Two forms.  16-bit weights that TMA can read (rows of a multiple of 16 bytes) and MXFP4
// weights run on tcgen05 (moe_tc.cu).  This one, for f32 and for odd sizes, is a warp to
// two weight rows in f32 FMAs, h in f32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "abi_util.h"
#include "moe.h"

namespace bi {
namespace {

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

// Weight rows [rows][L].
template <typename T>
struct Weights {
    const T* w;
    int64_t L;
    int vec;
    __device__ __forceinline__ void load(int64_t row, int64_t k, float (&v)[8]) const { load8<T>(w + row * L, k, L, vec != 0, v); }
};

// acc[r][c] += rows row0 + r of W times columns c of the operand (colp[c], of length L).
template <typename T, typename X, int NC>
__device__ __forceinline__ void dot_rows(const Weights<T>& W, int64_t row0, int nrows, const X* const (&colp)[NC], bool xvec,
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
            load8<X>(colp[c], k, W.L, xvec, x);
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

template <typename T>
struct MoeArgs {
    Weights<T> gate, up, down;  // gate.w null: no gate
    const void* x;
    const uint32_t* ids;
    const float* weights;
    float* h;                    // [P][F]
    void* y;
    int tokens, C, E, act, xvec, hvec;
    int64_t K, F, N;
};

template <typename T, int NC>
__device__ __forceinline__ void hidden_tokens(const MoeArgs<T>& a, const Plan& p, int e, int c0, int cn, int64_t f0, int nrows) {
    const T* colp[NC];
    int pair[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        pair[c] = p.list[p.first[e] + c0 + min(c, cn - 1)];
        colp[c] = static_cast<const T*>(a.x) + static_cast<int64_t>(pair[c] / a.C) * a.K;
    }
    float u[M_ROWS][NC], g[M_ROWS][NC];
    dot_rows<T, T, NC>(a.up, e * a.F + f0, nrows, colp, a.xvec != 0, u);
    if (a.gate.w != nullptr) dot_rows<T, T, NC>(a.gate, e * a.F + f0, nrows, colp, a.xvec != 0, g);
    if ((threadIdx.x & 31) != 0) return;
    for (int c = 0; c < NC && c < cn; ++c)
        for (int r = 0; r < nrows; ++r)
            a.h[pair[c] * a.F + f0 + r] = a.gate.w != nullptr ? activate(g[r][c], a.act) * u[r][c] : activate(u[r][c], a.act);
}

template <typename T>
__global__ void __launch_bounds__(M_THREADS) moe_hidden_kernel(const MoeArgs<T> a) {
    extern __shared__ __align__(16) uint8_t smem[];
    grid_dep_wait();
    grid_dep_launch();
    const Plan p = build_plan<1>(smem, a.ids, a.tokens * a.C, a.E);
    const int64_t f0 = static_cast<int64_t>(blockIdx.x) * M_BLOCK + (threadIdx.x >> 5) * M_ROWS;
    if (static_cast<int>(blockIdx.y) >= p.n || f0 >= a.F) return;
    const int e = p.active[blockIdx.y], n = static_cast<int>(p.cnt[e]);
    const int nrows = static_cast<int>(lmin(M_ROWS, a.F - f0));
    for (int c0 = 0; c0 < n; c0 += 4) {
        const int cn = min(4, n - c0);
        if (cn == 1) hidden_tokens<T, 1>(a, p, e, c0, cn, f0, nrows);
        else hidden_tokens<T, 4>(a, p, e, c0, cn, f0, nrows);
    }
}

template <typename T, int NC>
__device__ __forceinline__ void output_tokens(const MoeArgs<T>& a, const Plan& p, float* part, int e, int c0, int cn, int64_t n0,
                                              int nrows) {
    const float* colp[NC];
    int pair[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        pair[c] = p.list[p.first[e] + c0 + min(c, cn - 1)];
        colp[c] = a.h + pair[c] * a.F;
    }
    float o[M_ROWS][NC];
    dot_rows<T, float, NC>(a.down, e * a.N + n0, nrows, colp, a.hvec != 0, o);
    if ((threadIdx.x & 31) == 0)
        for (int c = 0; c < NC && c < cn; ++c)
            for (int r = 0; r < M_ROWS; ++r) part[pair[c] * M_BLOCK + r] = o[r][c];
}

template <typename T>
__global__ void __launch_bounds__(M_THREADS) moe_output_kernel(const MoeArgs<T> a) {
    extern __shared__ __align__(16) uint8_t smem[];
    grid_dep_wait();
    grid_dep_launch();
    const int P = a.tokens * a.C;
    const Plan p = build_plan<1>(smem, a.ids, P, a.E);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * M_BLOCK + warp * M_ROWS;
    if (n0 >= a.N) return;
    const int nrows = static_cast<int>(lmin(M_ROWS, a.N - n0));
    float* part = reinterpret_cast<float*>(smem + plan_bytes(a.E, P, 1)) + warp * M_ROWS;  // [P][M_BLOCK], this warp's rows
    for (int i = 0; i < p.n; ++i) {
        const int e = p.active[i], n = static_cast<int>(p.cnt[e]);
        for (int c0 = 0; c0 < n; c0 += 4) {
            const int cn = min(4, n - c0);
            if (cn == 1) output_tokens<T, 1>(a, p, part, e, c0, cn, n0, nrows);
            else output_tokens<T, 4>(a, p, part, e, c0, cn, n0, nrows);
        }
    }
    __syncwarp();
    for (int t = lane; t < a.tokens; t += 32)
        for (int r = 0; r < nrows; ++r) {
            float s = 0.0f;
            for (int j = 0; j < a.C; ++j)
                if (__ldg(a.ids + t * a.C + j) < static_cast<uint32_t>(a.E))
                    s = fmaf(__ldg(a.weights + t * a.C + j), part[(t * a.C + j) * M_BLOCK + r], s);
            static_cast<T*>(a.y)[t * a.N + n0 + r] = down<T>(s);
        }
}

template <typename T>
cudaError_t moe_t(const LaunchCtx& c, const MoeArgs<T>& a) {
    const int64_t P = static_cast<int64_t>(a.tokens) * a.C;
    const int64_t plan = plan_bytes(a.E, P, 1), out_smem = plan + P * M_BLOCK * 4;
    auto kh = moe_hidden_kernel<T>;
    auto ko = moe_output_kernel<T>;
    static PerDeviceOnce setup;
    cudaError_t e = setup.run(c.eng->device, [&](int&) {
        return cudaFuncSetAttribute(ko, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(plan_bytes(MOE_MAX_E, MOE_MAX_PAIRS, 1) + MOE_MAX_PAIRS * M_BLOCK * 4));
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

template <typename T>
cudaError_t moe_f32(const LaunchCtx& c, const MoeCall& m, float* h) {
    MoeArgs<T> a{};
    auto set = [](Weights<T>& w, const void* p, int64_t L) {
        w.w = static_cast<const T*>(p);
        w.L = L;
        w.vec = L % 8 == 0 && aligned16(p);
    };
    set(a.gate, m.gate, m.K);
    set(a.up, m.up, m.K);
    set(a.down, m.down, m.F);
    a.x = m.x;
    a.ids = m.ids;
    a.weights = m.weights;
    a.h = h;
    a.y = m.y;
    a.tokens = m.T;
    a.C = m.C;
    a.E = m.E;
    a.act = m.act;
    a.xvec = m.K % 8 == 0 && aligned16(m.x);
    a.hvec = m.F % 8 == 0;
    a.K = m.K;
    a.F = m.F;
    a.N = m.N;
    return moe_t<T>(c, a);
}

bi_status moe(bi_engine eng, const MoeCall& call, int64_t t, int64_t c, int64_t e, bool fp4, bi_dtype dt, void* stream, const char* name) {
    if (!eng) return fail(nullptr, BI_ERR_INVALID_ARG, "engine is NULL");
    MoeCall m = call;
    if (dt != BI_F32 && dt != BI_BF16 && dt != BI_F16) return fail(eng, BI_ERR_INVALID_ARG, "dtype must be BI_F32, BI_BF16 or BI_F16");
    if (m.act != BI_ACT_SILU && m.act != BI_ACT_GELU && m.act != BI_ACT_RELU)
        return fail(eng, BI_ERR_INVALID_ARG, "activation must be BI_ACT_SILU, BI_ACT_GELU or BI_ACT_RELU");
    if (t < 0 || c <= 0 || m.K <= 0 || m.F <= 0 || m.N <= 0 || e <= 0)
        return fail(eng, BI_ERR_INVALID_ARG, "t must be >= 0, the other sizes > 0");
    if (e > MOE_MAX_E || c > MOE_MAX_PAIRS || t > MOE_MAX_PAIRS || t * c > MOE_MAX_PAIRS)
        return fail(eng, BI_ERR_UNSUPPORTED, "at most 1024 experts and t * c = 2048 choices: longer batches take the grouped matmul");
    const int64_t lim = 8388480, rows = 0x7fffff00ll;
    if (m.K > lim || m.F > lim || m.N > lim || e * m.F > rows || e * m.N > rows)
        return fail(eng, BI_ERR_UNSUPPORTED, "k, f and n are limited to 8388480, e * f and e * n to 2^31 - 256");
    if (t == 0) return BI_OK;
    if (!m.y || !m.x || !m.ids || !m.weights || !m.up || !m.down || (fp4 && (!m.up_s || !m.down_s)))
        return fail(eng, BI_ERR_INVALID_ARG, "y, x, ids, weights and the expert weights must not be NULL");
    if (fp4 && (m.gate == nullptr) != (m.gate_s == nullptr)) return fail(eng, BI_ERR_INVALID_ARG, "the gate's codes and scales go together");
    if (fp4 && !(aligned16(m.gate) && aligned16(m.gate_s) && aligned16(m.up) && aligned16(m.up_s) && aligned16(m.down) && aligned16(m.down_s)))
        return fail(eng, BI_ERR_MISALIGNED, "codes and scales need 16-byte alignment");
    const uintptr_t es = static_cast<uintptr_t>(dsize(dt));
    auto off = [](const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; };
    if (off(m.y, es) || off(m.x, es) || off(m.ids, 4) || off(m.weights, 4) || (!fp4 && (off(m.gate, es) || off(m.up, es) || off(m.down, es))))
        return fail(eng, BI_ERR_MISALIGNED, "tensors need the alignment of their type");
    m.T = static_cast<int>(t);
    m.C = static_cast<int>(c);
    m.E = static_cast<int>(e);
    DeviceGuard g(eng->device);
    if (!g.ok) return fail(eng, BI_ERR_CUDA, "cudaSetDevice failed");
    const LaunchCtx lc = ctx(eng, stream);
    // the form is a function of the types, K, F and the weights' alignment: never of the batch
    const bool tc = fp4 || (dt != BI_F32 && m.K % 8 == 0 && m.F % 8 == 0 && aligned16(m.gate) && aligned16(m.up) && aligned16(m.down));
    const bool copy_x = tc && !fp4 && !aligned16(m.x);
    Scratch sc(eng, lc.stream, static_cast<size_t>(tc ? moe_tc_scratch_bytes(m, fp4, copy_x, dt) : round256(t * c * m.F * 4)));
    if (sc.err != cudaSuccess) return cuda_fail(eng, sc.err, "hidden scratch");
    cudaError_t err;
    if (tc) err = moe_tc(lc, m, fp4, copy_x, dt, sc.ptr);
    else if (dt == BI_F32) err = moe_f32<float>(lc, m, static_cast<float*>(sc.ptr));
    else if (dt == BI_BF16) err = moe_f32<__nv_bfloat16>(lc, m, static_cast<float*>(sc.ptr));
    else err = moe_f32<__half>(lc, m, static_cast<float*>(sc.ptr));
    return err == cudaSuccess ? BI_OK : cuda_fail(eng, err, name);
}

}  // namespace
}  // namespace bi

extern "C" {

bi_status bi_moe_forward(bi_engine eng, void* y, const void* x, const uint32_t* ids, const float* weights, const void* w_gate,
                         const void* w_up, const void* w_down, int64_t t, int64_t c, int64_t k, int64_t f, int64_t n, int64_t e,
                         bi_activation activation, bi_dtype dtype, void* stream) {
    const bi::MoeCall m{y, x, ids, weights, w_gate, w_up, w_down, nullptr, nullptr, nullptr, 0, 0, 0, static_cast<int>(activation), k, f, n};
    return bi::moe(eng, m, t, c, e, false, dtype, stream, "bi_moe_forward");
}

bi_status bi_moe_forward_fp4(bi_engine eng, void* y, const void* x, const uint32_t* ids, const float* weights, const uint8_t* gate_q,
                             const uint8_t* gate_s, const uint8_t* up_q, const uint8_t* up_s, const uint8_t* down_q,
                             const uint8_t* down_s, int64_t t, int64_t c, int64_t k, int64_t f, int64_t n, int64_t e,
                             bi_activation activation, bi_dtype dtype, void* stream) {
    const bi::MoeCall m{y, x, ids, weights, gate_q, up_q, down_q, gate_s, up_s, down_s, 0, 0, 0, static_cast<int>(activation), k, f, n};
    return bi::moe(eng, m, t, c, e, true, dtype, stream, "bi_moe_forward_fp4");
}

}  // extern "C"
