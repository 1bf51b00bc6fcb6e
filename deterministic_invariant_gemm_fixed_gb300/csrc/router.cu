// Softmax router: top-k expert choice, per-expert counts, balance loss, and the
// gradient of the logits.  See include/bi.h (bi_router_forward / _backward).
//
//   p = softmax(row);  ids = the k largest logits (ties: lowest index)
//   counts[e] = times expert e was chosen;  V = rows counted
//   loss = E * sum_e counts[e] / (k V) * mean_t p[t, e]
//
// One row lives in the registers of L lanes, V consecutive experts each, so a
// row is read once and its maximum, its sum, the choice and the probabilities
// come from registers.  The sums over tokens are taken in a fixed order: a
// block owns a fixed run of rows (a function of T and E), every lane adds its
// experts' probabilities row after row in f32, the lanes and warps of the block
// are added in a fixed tree, and a second kernel adds the blocks in order.
// Counts are integers, so their order does not matter.  No result depends on
// the GPU or on scheduling.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "abi_util.h"

namespace bi {
namespace {

constexpr int RT_THREADS = 256;
constexpr int RT_WARPS = RT_THREADS / 32;
constexpr int64_t RT_BLOCKS = 1024;   // blocks aimed at: about 7 per SM for a long batch
constexpr int64_t RT_MAX_E = 1024;
constexpr int64_t RT_MAX_K = 64;
constexpr int FIN_E = 8, FIN_SLOTS = 32;  // finishing kernel: experts per block, partial sums per expert

template <typename T> __device__ __forceinline__ float up(T v);
template <> __device__ __forceinline__ float up<float>(float v) { return v; }
template <> __device__ __forceinline__ float up<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float up<__half>(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T down(float v);
template <> __device__ __forceinline__ float down<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 down<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half down<__half>(float v) { return __float2half_rn(v); }

// V consecutive elements from index e0 of a row of E; elements past E are `fill`.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T* row, int e0, int E, bool vec, float fill, float (&x)[V]) {
    constexpr int PER = 16 / sizeof(T);  // V is a multiple of PER
    if (vec && e0 + V <= E) {
#pragma unroll
        for (int i = 0; i < V; i += PER) {
            const uint4 raw = __ldg(reinterpret_cast<const uint4*>(row + e0 + i));
            const T* v = reinterpret_cast<const T*>(&raw);
#pragma unroll
            for (int j = 0; j < PER; ++j) x[i + j] = up<T>(v[j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = e0 + i < E ? up<T>(__ldg(row + e0 + i)) : fill;
    }
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A logit's place in the order of choice: larger logits have larger keys, the
// two zeros the same one; -inf and NaN are 0 (never chosen).
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    const uint32_t k = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
    return x > -INFINITY ? k : 0u;
}

struct RouteArgs {
    uint32_t* ids;        // [T, k]
    float* weights;       // [T, k]
    float* lse;           // [T]
    const void* logits;   // [T, E]
    const uint8_t* valid; // [T] or null
    float* psum;          // [blocks, E] sums of probabilities
    uint32_t* pcnt;       // [blocks, E] choices
    uint32_t* prow;       // [blocks] rows counted
    uint32_t* ticket;
    int64_t T, rows_per_block;
    int E, k, normalize, vec;
};

template <typename T, int L, int V>
__global__ void __launch_bounds__(RT_THREADS) route_kernel(const RouteArgs a) {
    constexpr int GROUPS = 32 / L;             // rows per warp
    constexpr int STEP = RT_WARPS * GROUPS;    // rows per block and step
    // choices kept per lane: slots li, li + L, ... (k is at most E <= L V)
    constexpr int SLOTS = (RT_MAX_K + L - 1) / L < V ? (RT_MAX_K + L - 1) / L : V;
    __shared__ float s_sum[RT_WARPS][L * V];
    __shared__ uint32_t s_cnt[L * V];
    __shared__ uint32_t s_rows[RT_WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grp = lane / L, li = lane % L;
    const int e0 = li * V;
    const int E = a.E;
    for (int i = threadIdx.x; i < L * V; i += RT_THREADS) s_cnt[i] = 0;
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    uint32_t rows = 0;
    const int64_t r0 = blockIdx.x * a.rows_per_block;
    const int64_t r1 = lmin(a.T, r0 + a.rows_per_block);
    for (int64_t base = r0; base < r1; base += STEP) {  // every warp runs every step: the shuffles need all lanes
        const int64_t t = base + warp * GROUPS + grp;
        const bool in = t < r1;
        bool counted = in && (a.valid == nullptr || a.valid[t] != 0);
        float x[V];
        if (counted) load_row<T, V>(static_cast<const T*>(a.logits) + t * E, e0, E, a.vec != 0, -INFINITY, x);
        else {
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = -INFINITY;
        }
        uint32_t key[V];
        float mx = -INFINITY;
        bool nan = false;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            key[i] = order_key(x[i]);
            mx = fmaxf(mx, x[i]);  // a NaN is passed over here and shows in the sum
            nan = nan || x[i] != x[i];
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) {
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            nan = __shfl_xor_sync(0xffffffffu, static_cast<int>(nan), o) != 0 || nan;
        }
        counted = counted && (mx > -INFINITY || nan);  // a row of -inf alone has no expert
        float p[V], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = counted && e0 + i < E ? __expf(x[i] - mx) : 0.0f;
            sum += p[i];
        }
        sum = group_sum<L>(sum);
        const float inv = counted ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] *= inv;
            acc[i] += p[i];
        }
        if (in && li == 0) {
            a.lse[t] = counted ? mx + logf(sum) : INFINITY;
            rows += counted;
        }
        // the choice: k times the group's largest key, the lowest index among equals
        float wsum = 0.0f;
        uint32_t my_id[SLOTS];
        float my_w[SLOTS];
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            my_id[s] = static_cast<uint32_t>(E);
            my_w[s] = 0.0f;
        }
        uint32_t best = 0;
        int bi_ = 0;
        auto scan = [&] {
            best = 0;
            bi_ = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (key[i] > best) { best = key[i]; bi_ = i; }
        };
        scan();
        for (int j = 0; j < a.k; ++j) {
            uint32_t gk = best;
            int ge = e0 + bi_;
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) {
                const uint32_t ok = __shfl_xor_sync(0xffffffffu, gk, o);
                const int oe = __shfl_xor_sync(0xffffffffu, ge, o);
                if (ok > gk || (ok == gk && oe < ge)) { gk = ok; ge = oe; }
            }
            float w = 0.0f;
            const bool mine = gk != 0 && ge / V == li;
            if (mine) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i == bi_) { w = p[i]; key[i] = 0; }
                scan();
                atomicAdd(&s_cnt[ge], 1u);
            }
            w = __shfl_sync(0xffffffffu, w, (lane & ~(L - 1)) + (gk != 0 ? ge / V : 0));
            if (gk == 0) w = 0.0f;
            wsum += w;
            if (j % L == li) {
#pragma unroll
                for (int s = 0; s < SLOTS; ++s)
                    if (s == j / L) { my_id[s] = gk != 0 ? static_cast<uint32_t>(ge) : static_cast<uint32_t>(E); my_w[s] = w; }
            }
        }
        if (in) {
#pragma unroll
            for (int s = 0; s < SLOTS; ++s) {
                const int j = s * L + li;
                if (j < a.k) {
                    const bool picked = my_id[s] != static_cast<uint32_t>(E);
                    a.ids[t * a.k + j] = my_id[s];
                    a.weights[t * a.k + j] = a.normalize && picked ? my_w[s] / wsum : my_w[s];
                }
            }
        }
    }
    // the block's sums: rows of a warp by a shuffle tree, then the warps in order
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int o = 16; o >= L; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
        if (grp == 0) s_sum[warp][e0 + i] = acc[i];
    }
    for (int o = 16; o > 0; o >>= 1) rows += __shfl_xor_sync(0xffffffffu, rows, o);
    if (lane == 0) s_rows[warp] = rows;
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += RT_THREADS) {
        float s = s_sum[0][e];
#pragma unroll
        for (int w = 1; w < RT_WARPS; ++w) s += s_sum[w][e];
        a.psum[static_cast<int64_t>(blockIdx.x) * E + e] = s;
        a.pcnt[static_cast<int64_t>(blockIdx.x) * E + e] = s_cnt[e];
    }
    if (threadIdx.x == 0) {
        uint32_t r = 0;
        for (int w = 0; w < RT_WARPS; ++w) r += s_rows[w];
        a.prow[blockIdx.x] = r;
    }
}

// Adds the blocks' sums: 8 experts per block, 32 slots per expert (slot s takes
// blocks s, s + 32, ... in order), the slots by a fixed tree.  The block that
// finishes last (a ticket) adds the experts' terms of the loss, in order of e.
__global__ void __launch_bounds__(FIN_E * FIN_SLOTS)
    route_finish_kernel(const float* psum, const uint32_t* pcnt, const uint32_t* prow, float* terms, uint32_t* ticket,
                        uint32_t* counts, uint32_t* rows_out, float* mean, float* loss, int blocks, int E, int k) {
    __shared__ float s_p[FIN_SLOTS][FIN_E];
    __shared__ uint32_t s_c[FIN_SLOTS][FIN_E];
    __shared__ uint32_t s_v[FIN_E * FIN_SLOTS / 32];
    __shared__ bool s_last;
    grid_dep_wait();
    grid_dep_launch();
    const int tid = threadIdx.x, slot = tid / FIN_E, i = tid % FIN_E, e = blockIdx.x * FIN_E + i;
    uint32_t v = 0;
    for (int b = tid; b < blocks; b += FIN_E * FIN_SLOTS) v += prow[b];
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((tid & 31) == 0) s_v[tid >> 5] = v;
    float p = 0.0f;
    uint32_t c = 0;
    if (e < E) {
#pragma unroll 4
        for (int b = slot; b < blocks; b += FIN_SLOTS) {
            p += psum[static_cast<int64_t>(b) * E + e];
            c += pcnt[static_cast<int64_t>(b) * E + e];
        }
    }
    s_p[slot][i] = p;
    s_c[slot][i] = c;
    __syncthreads();
    v = 0;
    for (int w = 0; w < FIN_E * FIN_SLOTS / 32; ++w) v += s_v[w];
    for (int o = FIN_SLOTS / 2; o > 0; o >>= 1) {
        if (slot < o) {
            s_p[slot][i] += s_p[slot + o][i];
            s_c[slot][i] += s_c[slot + o][i];
        }
        __syncthreads();
    }
    if (slot == 0 && e < E) {
        const float m = v ? s_p[0][i] / static_cast<float>(v) : 0.0f;
        mean[e] = m;
        counts[e] = s_c[0][i];
        terms[e] = static_cast<float>(s_c[0][i]) * m;
        __threadfence();
    }
    __syncthreads();
    if (tid == 0) {
        if (blockIdx.x == 0) *rows_out = v;
        s_last = atomicAdd(ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last || tid >= 32) return;
    __threadfence();
    float s = 0.0f;
    for (int q = tid; q < E; q += 32) s += __ldcg(terms + q);
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (tid == 0) *loss = v ? s * (static_cast<float>(E) / (static_cast<float>(k) * static_cast<float>(v))) : 0.0f;
}

struct RouteBackArgs {
    void* dlogits;
    const void* logits;
    const float* lse;
    const uint32_t* ids;
    const float* weights;
    const uint32_t* counts;
    const uint32_t* rows;
    const float* dweights;  // [T, k] or null
    const float* dloss;     // [1] or null
    int64_t T;
    int E, k, normalize, vec;
};

// dp[e] = q[e] (+ dweights at the chosen experts);  dL = p (dp - sum p dp), with
// q[e] = dloss E counts[e] / (k V^2).  Normalised weights are a softmax over the
// chosen logits, so their part, w (dw - sum w dw), is added to dL instead.  The
// chosen experts' values reach the lanes that own them through one row of
// shared memory per row group (kept zero between rows).  Probabilities are
// recomputed from the row's log-sum-exp: the pass reads the logits and writes
// their gradient, nothing else of that size.
template <typename T, int L, int V>
__global__ void __launch_bounds__(RT_THREADS) route_back_kernel(const RouteBackArgs a) {
    constexpr int GROUPS = 32 / L;
    constexpr int STEP = RT_WARPS * GROUPS;
    __shared__ __align__(16) float s_extra[RT_WARPS * GROUPS][L * V];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grp = lane / L, li = lane % L, e0 = li * V, E = a.E;
    float* extra = s_extra[warp * GROUPS + grp];
#pragma unroll
    for (int i = 0; i < V; ++i) extra[e0 + i] = 0.0f;
    __syncwarp();
    grid_dep_wait();
    grid_dep_launch();
    float q[V];
    {
        const uint32_t v = *a.rows;
        const float f = static_cast<float>(v);
        const float s = a.dloss != nullptr && v ? *a.dloss * static_cast<float>(E) / (static_cast<float>(a.k) * f * f) : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] = e0 + i < E ? s * static_cast<float>(a.counts[e0 + i]) : 0.0f;
    }
    const int64_t stride = static_cast<int64_t>(gridDim.x) * STEP;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * STEP; base < a.T; base += stride) {
        const int64_t t = base + warp * GROUPS + grp;
        const bool in = t < a.T;
        const float lse = in ? a.lse[t] : INFINITY;
        const bool counted = lse != INFINITY;  // false: the forward left the row out
        float x[V];
        if (counted) load_row<T, V>(static_cast<const T*>(a.logits) + t * E, e0, E, a.vec != 0, -INFINITY, x);
        else {
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = -INFINITY;
        }
        if (a.dweights != nullptr) {
            float inner = 0.0f;
            if (a.normalize && counted) {
                for (int j = li; j < a.k; j += L)
                    if (a.ids[t * a.k + j] < static_cast<uint32_t>(E)) inner += a.weights[t * a.k + j] * a.dweights[t * a.k + j];
            }
            inner = group_sum<L>(inner);
            if (counted) {
                for (int j = li; j < a.k; j += L) {
                    const uint32_t id = a.ids[t * a.k + j];
                    if (id < static_cast<uint32_t>(E)) {
                        const float dw = a.dweights[t * a.k + j];
                        extra[id] = a.normalize ? a.weights[t * a.k + j] * (dw - inner) : dw;
                    }
                }
            }
            __syncwarp();
        }
        float p[V], d[V], dot = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = counted && e0 + i < E ? __expf(x[i] - lse) : 0.0f;
            const float ex = extra[e0 + i];
            d[i] = a.normalize ? q[i] : q[i] + ex;
            dot += p[i] * d[i];
        }
        dot = group_sum<L>(dot);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float g = p[i] * (d[i] - dot);
            d[i] = counted ? (a.normalize ? g + extra[e0 + i] : g) : 0.0f;
        }
        if (a.dweights != nullptr) {
            __syncwarp();
            if (counted) {
                for (int j = li; j < a.k; j += L) {
                    const uint32_t id = a.ids[t * a.k + j];
                    if (id < static_cast<uint32_t>(E)) extra[id] = 0.0f;
                }
            }
            __syncwarp();
        }
        if (!in) continue;
        T* out = static_cast<T*>(a.dlogits) + t * E + e0;
        constexpr int PER = 16 / sizeof(T);
        if (a.vec && e0 + V <= E) {
#pragma unroll
            for (int i = 0; i < V; i += PER) {
                uint4 raw;
                T* o = reinterpret_cast<T*>(&raw);
#pragma unroll
                for (int j = 0; j < PER; ++j) o[j] = down<T>(d[i + j]);
                *reinterpret_cast<uint4*>(out + i) = raw;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (e0 + i < E) out[i] = down<T>(d[i]);
        }
    }
}

// Calls f with the lanes per row and experts per lane for E experts.
template <typename F>
cudaError_t with_layout(int64_t E, F&& f) {
#define BI_LAYOUT(L, V) return f(std::integral_constant<int, L>{}, std::integral_constant<int, V>{})
    if (E <= 8) BI_LAYOUT(1, 8);
    if (E <= 16) BI_LAYOUT(2, 8);
    if (E <= 32) BI_LAYOUT(4, 8);
    if (E <= 64) BI_LAYOUT(8, 8);
    if (E <= 128) BI_LAYOUT(16, 8);
    if (E <= 256) BI_LAYOUT(32, 8);
    if (E <= 512) BI_LAYOUT(32, 16);
    BI_LAYOUT(32, 32);
#undef BI_LAYOUT
}

int64_t lanes_for(int64_t E) { return E <= 8 ? 1 : E <= 16 ? 2 : E <= 32 ? 4 : E <= 64 ? 8 : E <= 128 ? 16 : 32; }

// Rows per block: a whole number of block steps, about RT_BLOCKS blocks.
int64_t rows_per_block(int64_t T, int64_t E) {
    const int64_t step = RT_WARPS * (32 / lanes_for(E));
    const int64_t per = (T + RT_BLOCKS - 1) / RT_BLOCKS;
    return lmax(1, (per + step - 1) / step) * step;
}

template <typename T>
cudaError_t forward_t(const LaunchCtx& c, const RouteArgs& a, int64_t blocks) {
    return with_layout(a.E, [&](auto l, auto v) {
        return launch_pdl(route_kernel<T, l.value, v.value>, dim3(static_cast<unsigned>(blocks)), dim3(RT_THREADS), 0,
                          c.stream, a);
    });
}

template <typename T>
cudaError_t backward_t(const LaunchCtx& c, const RouteBackArgs& a) {
    const int64_t step = RT_WARPS * (32 / lanes_for(a.E));
    const int64_t blocks = lmin((a.T + step - 1) / step, static_cast<int64_t>(c.sm_count) * 8);
    return with_layout(a.E, [&](auto l, auto v) {
        return launch_pdl(route_back_kernel<T, l.value, v.value>, dim3(static_cast<unsigned>(blocks)), dim3(RT_THREADS),
                          0, c.stream, a);
    });
}

bi_status check_router(bi_engine eng, int64_t t, int64_t e, int64_t k, bi_dtype dt) {
    if (!eng) return fail(nullptr, BI_ERR_INVALID_ARG, "engine is NULL");
    if (dt != BI_F32 && dt != BI_BF16 && dt != BI_F16)
        return fail(eng, BI_ERR_INVALID_ARG, "dtype must be BI_F32, BI_BF16 or BI_F16");
    if (t < 0 || e <= 0 || k <= 0 || k > e) return fail(eng, BI_ERR_INVALID_ARG, "router sizes must be t >= 0, 0 < k <= e");
    if (e > RT_MAX_E || k > RT_MAX_K || t > (int64_t(1) << 31) - 1 || t * k > 0xffffffffll)
        return fail(eng, BI_ERR_UNSUPPORTED, "the router is limited to 1024 experts, 64 choices, 2^31 - 1 rows and 2^32 - 1 slots");
    return BI_OK;
}

bool row_vectors(const void* p, int64_t E, bi_dtype dt) { return aligned16(p) && E * dsize(dt) % 16 == 0; }

}  // namespace
}  // namespace bi

using namespace bi;

extern "C" {

bi_status bi_router_forward(bi_engine eng, uint32_t* ids, float* weights, uint32_t* counts, uint32_t* rows,
                            float* mean_prob, float* loss, float* lse, const void* logits, const uint8_t* valid,
                            int64_t t, int64_t e, int64_t k, int normalize, bi_dtype dtype, void* stream) {
    bi_status st = check_router(eng, t, e, k, dtype);
    if (st != BI_OK) return st;
    if (!counts || !rows || !mean_prob || !loss || (t > 0 && (!ids || !weights || !lse || !logits)))
        return fail(eng, BI_ERR_INVALID_ARG, "the router's outputs and logits must not be NULL");
    DeviceGuard g(eng->device);
    if (!g.ok) return fail(eng, BI_ERR_CUDA, "cudaSetDevice failed");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const LaunchCtx c = ctx(eng, stream);
    cudaError_t err;
    if (t == 0) {  // nothing routed: empty sums
        err = cudaMemsetAsync(counts, 0, static_cast<size_t>(e) * 4, s);
        if (err == cudaSuccess) err = cudaMemsetAsync(mean_prob, 0, static_cast<size_t>(e) * 4, s);
        if (err == cudaSuccess) err = cudaMemsetAsync(rows, 0, 4, s);
        if (err == cudaSuccess) err = cudaMemsetAsync(loss, 0, 4, s);
        return err == cudaSuccess ? BI_OK : cuda_fail(eng, err, "bi_router_forward");
    }
    const int64_t per = rows_per_block(t, e), blocks = (t + per - 1) / per;
    // scratch: block sums | block counts | block rows | loss terms | ticket
    Scratch sc(eng, s, static_cast<size_t>(4 * (2 * blocks * e + blocks + e + 1)));
    if (sc.err != cudaSuccess) return cuda_fail(eng, sc.err, "router scratch");
    RouteArgs a{};
    a.ids = ids; a.weights = weights; a.lse = lse; a.logits = logits; a.valid = valid;
    a.psum = static_cast<float*>(sc.ptr);
    a.pcnt = reinterpret_cast<uint32_t*>(a.psum + blocks * e);
    a.prow = a.pcnt + blocks * e;
    float* terms = reinterpret_cast<float*>(a.prow + blocks);
    a.ticket = reinterpret_cast<uint32_t*>(terms + e);
    a.T = t; a.rows_per_block = per;
    a.E = static_cast<int>(e); a.k = static_cast<int>(k); a.normalize = normalize != 0;
    a.vec = row_vectors(logits, e, dtype);
    err = dtype == BI_F32 ? forward_t<float>(c, a, blocks)
        : dtype == BI_BF16 ? forward_t<__nv_bfloat16>(c, a, blocks) : forward_t<__half>(c, a, blocks);
    if (err == cudaSuccess) {
        c.count();
        err = launch_pdl(route_finish_kernel, dim3(static_cast<unsigned>((e + FIN_E - 1) / FIN_E)),
                         dim3(FIN_E * FIN_SLOTS), 0, c.stream, a.psum, a.pcnt, a.prow, terms, a.ticket, counts, rows,
                         mean_prob, loss, static_cast<int>(blocks), a.E, a.k);
        if (err == cudaSuccess) c.count();
    }
    return err == cudaSuccess ? BI_OK : cuda_fail(eng, err, "bi_router_forward");
}

bi_status bi_router_backward(bi_engine eng, void* dlogits, const void* logits, const float* lse, const uint32_t* ids,
                             const float* weights, const uint32_t* counts, const uint32_t* rows, const float* dweights,
                             const float* dloss, int64_t t, int64_t e, int64_t k, int normalize, bi_dtype dtype,
                             void* stream) {
    bi_status st = check_router(eng, t, e, k, dtype);
    if (st != BI_OK) return st;
    if (t == 0) return BI_OK;
    if (!dlogits || !logits || !lse || !ids || !weights || !counts || !rows)
        return fail(eng, BI_ERR_INVALID_ARG, "dlogits and the router's saved tensors must not be NULL");
    DeviceGuard g(eng->device);
    if (!g.ok) return fail(eng, BI_ERR_CUDA, "cudaSetDevice failed");
    const LaunchCtx c = ctx(eng, stream);
    RouteBackArgs a{};
    a.dlogits = dlogits; a.logits = logits; a.lse = lse; a.ids = ids; a.weights = weights; a.counts = counts;
    a.rows = rows; a.dweights = dweights; a.dloss = dloss;
    a.T = t; a.E = static_cast<int>(e); a.k = static_cast<int>(k); a.normalize = normalize != 0;
    a.vec = row_vectors(logits, e, dtype) && aligned16(dlogits);
    cudaError_t err = dtype == BI_F32 ? backward_t<float>(c, a)
                    : dtype == BI_BF16 ? backward_t<__nv_bfloat16>(c, a) : backward_t<__half>(c, a);
    if (err == cudaSuccess) c.count();
    return err == cudaSuccess ? BI_OK : cuda_fail(eng, err, "bi_router_backward");
}

}  // extern "C"
