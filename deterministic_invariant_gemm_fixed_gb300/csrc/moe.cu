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
// weights run on tcgen05 (moe_tc.cu).  This one, for f32 and for odd sizes, is in f32
// FMAs, a warp to four weight rows and up to eight tokens at a time, h in f32: the lanes go
// along the contraction, eight elements at a time, and are added by a tree.  A hidden warp's
// rows are two of the gate's and the same two of up's; an output block has four rows, its
// warps different experts.  Bound by latency at a few tokens: 7 tokens through 2 of 8 experts
// of 1000 x 1000 in f32 read 40 MB in 16 us (hidden) and 20 MB in 16 (output), caches cold.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "abi_util.h"
#include "moe.h"

namespace bi {
namespace {

constexpr int M_WARPS = 8, M_THREADS = 32 * M_WARPS;
constexpr int M_ROWS = 4;                // weight rows of a warp
constexpr int M_COLS = 8;                // most tokens of a pass

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

// v[row * NC + column], one value for each lane: of the inner products of four weight rows
// with NC columns, the one of index lane / (32 / (4 NC)).  The lanes' sums are added by the
// tree of offsets 16, 8, .. 1, for a value the same whatever NC is.
template <typename T, typename X, int NC>
__device__ __forceinline__ float dot_rows(const T* const (&row)[M_ROWS], bool vec, const X* const (&col)[NC], bool xvec, int64_t L) {
    const int lane = threadIdx.x & 31;
    float v[M_ROWS * NC];
#pragma unroll
    for (int i = 0; i < M_ROWS * NC; ++i) v[i] = 0.0f;
#pragma unroll 2
    for (int64_t k = lane * 8; k < L; k += 256) {
        float w[M_ROWS][8];
#pragma unroll
        for (int r = 0; r < M_ROWS; ++r) load8<T>(row[r], k, L, vec, w[r]);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float x[8];
            load8<X>(col[c], k, L, xvec, x);
#pragma unroll
            for (int r = 0; r < M_ROWS; ++r)
#pragma unroll
                for (int i = 0; i < 8; ++i) v[r * NC + c] = fmaf(w[r][i], x[i], v[r * NC + c]);
        }
    }
    int n = M_ROWS * NC;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (n > 1) {  // the lanes with the offset's bit go on with the upper half of the values
            n /= 2;
            const bool upper = lane & o;
#pragma unroll
            for (int i = 0; i < M_ROWS * NC / 2; ++i)
                if (i < n) {
                    const float send = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        }
    }
    return v[0];
}

template <typename T>
struct MoeArgs {
    const T *gate, *up, *down;   // gate null: none
    const T* x;
    const uint32_t* ids;
    const float* weights;
    float* h;                    // [P][F]
    T* y;
    int tokens, C, E, act;
    int wvec, dvec, xvec, hvec;  // whether load8 may read 16 bytes at a time: gate and up, down, x, h
    int64_t K, F, N;
};

template <typename T, int NC>
__device__ __forceinline__ void hidden_tokens(const MoeArgs<T>& a, const uint16_t* list, int e, int n, int64_t f0) {
    const int lane = threadIdx.x & 31;
    const bool gated = a.gate != nullptr;
    const T* row[M_ROWS];
#pragma unroll
    for (int r = 0; r < M_ROWS; ++r) {
        const int64_t f = e * a.F + lmin(f0 + (gated ? r % 2 : r), a.F - 1);
        row[r] = (gated && r >= 2 ? a.gate : a.up) + f * a.K;
    }
    const T* col[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) col[c] = a.x + static_cast<int64_t>(list[min(c, n - 1)] / a.C) * a.K;
    const float v = dot_rows<T, T, NC>(row, a.wvec != 0, col, a.xvec != 0, a.K);
    constexpr int EACH = 32 / (M_ROWS * NC);  // lanes with the same value
    const int r = lane / EACH / NC, c = lane / EACH % NC;
    const float g = __shfl_down_sync(0xffffffffu, v, 16);  // the gate's rows are the upper half
    if (lane % EACH == 0 && c < n && f0 + r < a.F && (!gated || r < 2))
        a.h[list[c] * a.F + f0 + r] = gated ? activate(g, a.act) * v : activate(v, a.act);
}

template <typename T>
__global__ void __launch_bounds__(M_THREADS, 2) moe_hidden_kernel(const MoeArgs<T> a) {
    extern __shared__ __align__(16) uint8_t smem[];
    grid_dep_wait();
    grid_dep_launch();
    const Plan p = build_plan<1>(smem, a.ids, a.tokens * a.C, a.E);
    const int64_t f0 = (static_cast<int64_t>(blockIdx.x) * M_WARPS + (threadIdx.x >> 5)) * (a.gate ? 2 : 4);
    if (static_cast<int>(blockIdx.y) >= p.n || f0 >= a.F) return;
    const int e = p.active[blockIdx.y], n = static_cast<int>(p.cnt[e]);
    const uint16_t* list = p.list + p.first[e];
    for (int c0 = 0; c0 < n; c0 += M_COLS) {
        const int cn = min(M_COLS, n - c0);
        if (cn == 1) hidden_tokens<T, 1>(a, list + c0, e, cn, f0);
        else if (cn == 2) hidden_tokens<T, 2>(a, list + c0, e, cn, f0);
        else if (cn <= 4) hidden_tokens<T, 4>(a, list + c0, e, cn, f0);
        else hidden_tokens<T, 8>(a, list + c0, e, cn, f0);
    }
}

template <typename T, int NC>
__device__ __forceinline__ void output_tokens(const MoeArgs<T>& a, const uint16_t* list, float* part, int e, int n, int64_t n0) {
    const int lane = threadIdx.x & 31;
    const T* row[M_ROWS];
#pragma unroll
    for (int r = 0; r < M_ROWS; ++r) row[r] = a.down + (e * a.N + lmin(n0 + r, a.N - 1)) * a.F;
    const float* col[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) col[c] = a.h + list[min(c, n - 1)] * a.F;
    const float v = dot_rows<T, float, NC>(row, a.dvec != 0, col, a.hvec != 0, a.F);
    constexpr int EACH = 32 / (M_ROWS * NC);
    const int r = lane / EACH / NC, c = lane / EACH % NC;
    if (lane % EACH == 0 && c < n) part[list[c] * M_ROWS + r] = v;
}

template <typename T>
__global__ void __launch_bounds__(M_THREADS, 2) moe_output_kernel(const MoeArgs<T> a) {
    extern __shared__ __align__(16) uint8_t smem[];
    grid_dep_wait();
    grid_dep_launch();
    const int P = a.tokens * a.C, warp = threadIdx.x >> 5;
    const Plan p = build_plan<1>(smem, a.ids, P, a.E);
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * M_ROWS;
    float* part = reinterpret_cast<float*>(smem + plan_bytes(a.E, P, 1));  // [P][M_ROWS]
    int item = 0;  // (expert, up to eight of its tokens), dealt to the warps
    for (int i = 0; i < p.n; ++i) {
        const int e = p.active[i], n = static_cast<int>(p.cnt[e]);
        const uint16_t* list = p.list + p.first[e];
        for (int c0 = 0; c0 < n; c0 += M_COLS, ++item) {
            if (item % M_WARPS != warp) continue;
            const int cn = min(M_COLS, n - c0);
            if (cn == 1) output_tokens<T, 1>(a, list + c0, part, e, cn, n0);
            else if (cn == 2) output_tokens<T, 2>(a, list + c0, part, e, cn, n0);
            else if (cn <= 4) output_tokens<T, 4>(a, list + c0, part, e, cn, n0);
            else output_tokens<T, 8>(a, list + c0, part, e, cn, n0);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.tokens * M_ROWS; i += M_THREADS) {
        const int t = i / M_ROWS, r = i % M_ROWS;
        if (n0 + r >= a.N) continue;
        float s = 0.0f;
        for (int j = 0; j < a.C; ++j)
            if (__ldg(a.ids + t * a.C + j) < static_cast<uint32_t>(a.E))
                s = fmaf(__ldg(a.weights + t * a.C + j), part[(t * a.C + j) * M_ROWS + r], s);
        a.y[t * a.N + n0 + r] = down<T>(s);
    }
}

template <typename T>
cudaError_t moe_fma(const LaunchCtx& c, const MoeCall& m, float* h) {
    MoeArgs<T> a{};
    a.gate = static_cast<const T*>(m.gate);
    a.up = static_cast<const T*>(m.up);
    a.down = static_cast<const T*>(m.down);
    a.x = static_cast<const T*>(m.x);
    a.ids = m.ids;
    a.weights = m.weights;
    a.h = h;
    a.y = static_cast<T*>(m.y);
    a.tokens = m.T;
    a.C = m.C;
    a.E = m.E;
    a.act = m.act;
    a.wvec = m.K % 8 == 0 && aligned16(m.gate) && aligned16(m.up);
    a.dvec = m.F % 8 == 0 && aligned16(m.down);
    a.xvec = m.K % 8 == 0 && aligned16(m.x);
    a.hvec = m.F % 8 == 0;
    a.K = m.K;
    a.F = m.F;
    a.N = m.N;
    const int64_t P = static_cast<int64_t>(a.tokens) * a.C, plan = plan_bytes(a.E, P, 1);
    auto kh = moe_hidden_kernel<T>;
    auto ko = moe_output_kernel<T>;
    static PerDeviceOnce setup;
    cudaError_t e = setup.run(c.eng->device, [&](int&) {
        return cudaFuncSetAttribute(ko, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(plan_bytes(MOE_MAX_E, MOE_MAX_PAIRS, 1) + MOE_MAX_PAIRS * M_ROWS * 4));
    });
    if (e != cudaSuccess) return e;
    const int64_t span = M_WARPS * (a.gate ? 2 : 4);
    const dim3 gh(static_cast<unsigned>((a.F + span - 1) / span), static_cast<unsigned>(lmin(a.E, P)));
    if ((e = launch_pdl(kh, gh, dim3(M_THREADS), static_cast<size_t>(plan), c.stream, a)) != cudaSuccess) return e;
    c.count();
    const dim3 go(static_cast<unsigned>((a.N + M_ROWS - 1) / M_ROWS));
    if ((e = launch_pdl(ko, go, dim3(M_THREADS), static_cast<size_t>(plan + P * M_ROWS * 4), c.stream, a)) != cudaSuccess) return e;
    c.count();
    return cudaGetLastError();
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
    else if (dt == BI_F32) err = moe_fma<float>(lc, m, static_cast<float*>(sc.ptr));
    else if (dt == BI_BF16) err = moe_fma<__nv_bfloat16>(lc, m, static_cast<float*>(sc.ptr));
    else err = moe_fma<__half>(lc, m, static_cast<float*>(sc.ptr));
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
