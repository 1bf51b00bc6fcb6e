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
// are added in a fixed tree.  The blocks of a short batch are one cluster, whose first
// block adds the others' sums in order; those of a longer one are added by a second
// kernel, in 64 runs of every 64th block and a tree over these.  Counts are
// integers, so their order does not matter.  No result depends on the GPU or on
// scheduling.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "abi_util.h"

namespace bi {
namespace {

constexpr int RT_THREADS = 256;
constexpr int RT_WARPS = RT_THREADS / 32;
constexpr int64_t RT_BLOCKS = 608;    // blocks aimed at for a long batch: four on each of 152 SMs, one wave
constexpr int64_t RT_MAX_E = 1024;
constexpr int64_t RT_MAX_K = 64;
constexpr int FIN_E = 4, FIN_SLOTS = 64;  // finishing kernel: experts per block, partial sums per expert

template <typename T> __device__ __forceinline__ float up(T v);
template <> __device__ __forceinline__ float up<float>(float v) { return v; }
template <> __device__ __forceinline__ float up<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float up<__half>(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T down(float v);
template <> __device__ __forceinline__ float down<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 down<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half down<__half>(float v) { return __float2half_rn(v); }

// V consecutive elements of a row of E from index e0 on, as loaded: unpacked
// only when the row's turn comes, so a row's loads run under the one before.
// Elements past E, and all of them when `in` is false, are -inf.
template <typename T, int V>
struct Raw {
    uint32_t w[V * sizeof(T) / 4];
    __device__ __forceinline__ void load(const T* row, int e0, int E, bool vec, bool in) {
        constexpr int WORDS = V * sizeof(T) / 4;
        if (vec && in && e0 + V <= E) {
            if constexpr (WORDS == 2) {
                const uint2 q = __ldg(reinterpret_cast<const uint2*>(row + e0));
                w[0] = q.x; w[1] = q.y;
            } else {
#pragma unroll
                for (int i = 0; i < WORDS; i += 4) {
                    const uint4 q = __ldg(reinterpret_cast<const uint4*>(row + e0) + i / 4);
                    w[i] = q.x; w[i + 1] = q.y; w[i + 2] = q.z; w[i + 3] = q.w;
                }
            }
        } else {
            T* v = reinterpret_cast<T*>(w);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = in && e0 + i < E ? __ldg(row + e0 + i) : down<T>(-INFINITY);
        }
    }
    __device__ __forceinline__ float get(int i) const { return up<T>(reinterpret_cast<const T*>(w)[i]); }
};

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

constexpr float LOG2E = 1.44269504f, LN2 = 0.693147181f;
// 2^x, within 2 ulp.  Probabilities are 2^((x - m) log2 e), the difference taken
// first: it is exact or nearly so, and overflows for no finite logits that matter.
// The product is rounded once, so a probability 2^-d of the largest is off by up to
// 0.7 d 2^-24 of itself: the small ones have the larger error, and weigh as little in
// the sum as they are small (long f32 batch: within 1.8e-7 of 64 bits, beside 1).  A
// second product for the rounding's rest would be one more instruction per expert in
// a kernel that its instructions bound.
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The largest value of a row's L lanes (NaN passed over).
template <int L>
__device__ __forceinline__ float group_max(float v) {
    if constexpr (L == 32) {
        float y;
        asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(v));
        return y;
    } else {
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        return v;
    }
}

// loss = E / (k V) * the sum of the experts' terms counts[e] mean[e], by one warp
// in a fixed order.
__device__ __forceinline__ void write_loss(const volatile float* terms, int E, int k, uint32_t v, float* loss) {
    const int lane = threadIdx.x & 31;
    float s = 0.0f;
    for (int q = lane; q < E; q += 32) s += terms[q];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) *loss = v ? s * (static_cast<float>(E) / (static_cast<float>(k) * static_cast<float>(v))) : 0.0f;
}

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A word of another block of the cluster, at this block's address of it.
__device__ __forceinline__ uint32_t remote_u32(const void* p, uint32_t rank) {
    uint32_t at, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
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
    uint32_t* counts;     // the results, which a lone block writes itself
    uint32_t* rows;
    float* mean;
    float* loss;
    int64_t T, rows_per_block;
    int E, k, normalize, vec;
};

// The choice, k experts of a row.  For rows of one warp (more than 64 experts):
// the k-th largest of the 32 lanes' largest logits bounds the k-th largest logit
// from below, so the logits at or above it, usually a dozen, hold the choice; they
// are packed into shared memory and each ranked against the others, without a
// chain of dependent steps.  Otherwise (shorter rows, k > 32, or more than 32
// logits at or above the bound): k times the largest logit of the row's lanes.
// 8 of 256 experts, 131072 rows in f32: 245 us by the second way.
template <typename T, int L, int V, int W>  // W warps per block
__global__ void __launch_bounds__(32 * W, W == RT_WARPS && V <= 8 ? 4 : 1) route_kernel(const RouteArgs a) {
    constexpr int GROUPS = 32 / L;             // rows per warp
    constexpr int STEP = W * GROUPS;    // rows per block and step
    constexpr int MAXK = L * V < RT_MAX_K ? L * V : static_cast<int>(RT_MAX_K);
    __shared__ float s_sum[W][L * V];
    __shared__ uint32_t s_cnt[L * V];
    __shared__ uint32_t s_rows[W];
    __shared__ uint2 s_pick[W * GROUPS][MAXK];  // slot -> (expert, weight's bits)
    __shared__ __align__(16) float s_cand_v[L == 32 ? W : 1][32];
    __shared__ uint16_t s_cand_i[L == 32 ? W : 1][32];  // (place in the lane, lane)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grp = lane / L, li = lane % L;
    const int e0 = li * V;
    const int E = a.E, k = a.k;
    uint2* pick = s_pick[warp * GROUPS + grp];
    for (int i = threadIdx.x; i < L * V; i += 32 * W) s_cnt[i] = 0;
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.ticket != nullptr) *a.ticket = 0;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    uint32_t rows = 0;
    const int64_t r0 = blockIdx.x * a.rows_per_block;
    const int64_t r1 = lmin(a.T, r0 + a.rows_per_block);
    // The next row's logits and flag load under this one's arithmetic (a row that
    // is left out is loaded too, and not looked at: its flag comes no earlier).
    int64_t t = r0 + warp * GROUPS + grp;
    const T* row = static_cast<const T*>(a.logits) + t * E;
    Raw<T, V> raw;
    raw.load(row, e0, E, a.vec != 0, t < r1);
    uint32_t flag = t < r1 && a.valid != nullptr ? a.valid[t] : 1u;
    for (int64_t base = r0; base < r1; base += STEP, t += STEP) {  // every warp runs every step: the shuffles need all lanes
        const bool in = t < r1;
        bool counted = in && flag != 0;
        float x[V];
        float top = -INFINITY;  // this lane's largest
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = raw.get(i);
        if (!counted) {
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) top = fmaxf(top, x[i]);  // a NaN is passed over here and shows in the sum
        row += static_cast<int64_t>(STEP) * E;
        raw.load(row, e0, E, a.vec != 0, t + STEP < r1);
        flag = t + STEP < r1 && a.valid != nullptr ? a.valid[t + STEP] : 1u;
        const float mx = group_max<L>(top);
        if (__any_sync(0xffffffffu, mx == -INFINITY)) {  // rows of -inf alone have no expert, rows of NaN and -inf are counted
            bool nan = false;
#pragma unroll
            for (int i = 0; i < V; ++i) nan = nan || x[i] != x[i];
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) nan = __shfl_xor_sync(0xffffffffu, static_cast<int>(nan), o) != 0 || nan;
            counted = counted && (mx > -INFINITY || nan);
        }
        const float m = mx > -INFINITY ? mx : 0.0f;
        float p[V], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = exp2_approx((x[i] - m) * LOG2E);
            sum += p[i];
        }
        sum = group_sum<L>(sum);
        const float inv = counted ? __fdividef(1.0f, sum) : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(p[i], inv, acc[i]);
        if (in && li == 0) {
            a.lse[t] = counted ? fmaf(__log2f(sum), LN2, m) : INFINITY;
            rows += counted;
        }
        auto weight = [&](float v) { return exp2_approx((v - m) * LOG2E) * inv; };
        float wsum = 0.0f;
        bool done = false;
        if constexpr (L == 32) {
            if (k <= 32) {
                float most = top, bound = -INFINITY;
                for (int j = 0; j < k; ++j) {
                    bound = group_max<32>(most);
                    if (most == bound) most = -INFINITY;
                }
                bound = fmaxf(bound, -3.402823466e38f);  // -inf and NaN are no candidates
                int own = 0;
#pragma unroll
                for (int i = 0; i < V; ++i) own += x[i] >= bound;
                int at = own;  // candidates of the lanes up to this one
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, at, o);
                    if (lane >= o) at += y;
                }
                const int total = __shfl_sync(0xffffffffu, at, 31);
                if (total <= 32) {
                    done = true;
                    float* cv = s_cand_v[warp];
                    uint16_t* ce = s_cand_i[warp];
                    at -= own;
                    cv[lane] = -INFINITY;
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (x[i] >= bound) {
                            cv[at] = x[i];
                            ce[at] = static_cast<uint16_t>(i * 32 + lane);
                            ++at;
                        }
                    __syncwarp();
                    const float mine = cv[lane];  // candidates stand in order of their expert
                    int rank = 0;
                    for (int j = 0; j < total; j += 4) {
                        const float4 o = *reinterpret_cast<const float4*>(cv + j);
                        rank += o.x > mine || (o.x == mine && j < lane);
                        rank += o.y > mine || (o.y == mine && j + 1 < lane);
                        rank += o.z > mine || (o.z == mine && j + 2 < lane);
                        rank += o.w > mine || (o.w == mine && j + 3 < lane);
                    }
                    const bool chosen = lane < total && rank < k;
                    const float w = chosen ? weight(mine) : 0.0f;
                    wsum = group_sum<32>(w);
                    if (lane >= total && lane < k) pick[lane] = make_uint2(E, 0);  // choices it cannot make
                    if (chosen) {
                        const int c = ce[lane];
                        const uint32_t e = static_cast<uint32_t>((c & 31) * V + (c >> 5));
                        pick[rank] = make_uint2(e, __float_as_uint(w));
                        atomicAdd(&s_cnt[e], 1u);
                    }
                }
            }
        }
        if (!done) {
            float best;
            int at;
            auto scan = [&] {
                best = -INFINITY;
                at = 0;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (x[i] > best) { best = x[i]; at = i; }
            };
            scan();
            for (int j = 0; j < k; ++j) {
                float gv = best;
                int ge = e0 + at;
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) {
                    const float ov = __shfl_xor_sync(0xffffffffu, gv, o);
                    const int oe = __shfl_xor_sync(0xffffffffu, ge, o);
                    if (ov > gv || (ov == gv && oe < ge)) { gv = ov; ge = oe; }
                }
                const bool can = gv > -INFINITY;
                const float w = can ? weight(gv) : 0.0f;
                wsum += w;
                if (j % L == li) pick[j] = make_uint2(can ? ge : E, __float_as_uint(w));
                if (can && ge / V == li) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (i == at) x[i] = -INFINITY;
                    scan();
                    atomicAdd(&s_cnt[ge], 1u);
                }
            }
        }
        __syncwarp();
        if (in) {
            uint32_t* ids = a.ids + t * k;
            float* weights = a.weights + t * k;
            for (int j = li; j < k; j += L) {
                const uint2 q = pick[j];
                const float w = __uint_as_float(q.y);
                ids[j] = q.x;
                weights[j] = a.normalize && q.x != static_cast<uint32_t>(E) ? __fdividef(w, wsum) : w;
            }
        }
        __syncwarp();  // pick and cand are free again
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
    uint32_t v = 0;
    for (int w = 0; w < W; ++w) v += s_rows[w];
    for (int e = threadIdx.x; e < E; e += 32 * W) {
        float s = s_sum[0][e];
#pragma unroll
        for (int w = 1; w < W; ++w) s += s_sum[w][e];
        if (a.psum != nullptr) {
            a.psum[static_cast<int64_t>(blockIdx.x) * E + e] = s;
            a.pcnt[static_cast<int64_t>(blockIdx.x) * E + e] = s_cnt[e];
        } else {
            s_sum[0][e] = s;
        }
    }
    if (a.psum != nullptr) {
        if (threadIdx.x == 0) a.prow[blockIdx.x] = v;
        return;
    }
    // a short batch: the grid is one block, or one cluster whose first block adds
    // the others' sums, in order, from their shared memory
    __shared__ uint32_t s_v;
    if (threadIdx.x == 0) s_v = v;
    __syncthreads();
    if (gridDim.x > 1) cluster_barrier();
    if (blockIdx.x == 0) {
        for (uint32_t b = 1; b < gridDim.x; ++b) v += remote_u32(&s_v, b);
        for (int e = threadIdx.x; e < E; e += 32 * W) {
            float s = s_sum[0][e];
            uint32_t n = s_cnt[e];
            for (uint32_t b = 1; b < gridDim.x; ++b) {
                s += __uint_as_float(remote_u32(&s_sum[0][e], b));
                n += remote_u32(&s_cnt[e], b);
            }
            const float m = v ? s / static_cast<float>(v) : 0.0f;
            a.mean[e] = m;
            a.counts[e] = n;
            s_sum[0][e] = static_cast<float>(n) * m;
        }
        __syncthreads();
        if (warp == 0) write_loss(s_sum[0], E, k, v, a.loss);
        if (threadIdx.x == 0) *a.rows = v;
    }
    if (gridDim.x > 1) cluster_barrier();  // no block leaves while its sums may be read
}

// Adds the blocks' sums: FIN_E experts per block, FIN_SLOTS slots each (slot s takes
// blocks s, s + FIN_SLOTS, ... in order), the slots by a fixed tree.  The block that
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
    // (at most RT_BLOCKS blocks: all loads of a thread in flight at once)
    constexpr int ROW_TURNS = static_cast<int>((RT_BLOCKS + FIN_E * FIN_SLOTS - 1) / (FIN_E * FIN_SLOTS));
    constexpr int TURNS = static_cast<int>((RT_BLOCKS + FIN_SLOTS - 1) / FIN_SLOTS);
    uint32_t v = 0;
#pragma unroll
    for (int q = 0; q < ROW_TURNS; ++q) {
        const int b = tid + q * FIN_E * FIN_SLOTS;
        v += b < blocks ? prow[b] : 0u;
    }
    float ps[TURNS];
    uint32_t cs[TURNS];
#pragma unroll
    for (int q = 0; q < TURNS; ++q) {
        const int b = slot + q * FIN_SLOTS;
        const bool in = e < E && b < blocks;
        ps[q] = in ? psum[static_cast<int64_t>(b) * E + e] : 0.0f;
        cs[q] = in ? pcnt[static_cast<int64_t>(b) * E + e] : 0u;
    }
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((tid & 31) == 0) s_v[tid >> 5] = v;
    float p = 0.0f;
    uint32_t c = 0;
#pragma unroll
    for (int q = 0; q < TURNS; ++q) {
        p += ps[q];
        c += cs[q];
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
    write_loss(terms, E, k, v, loss);
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
// recomputed from the row, with its maximum and its sum, as in the forward: the pass
// reads the logits and writes their gradient, nothing else of that size.  (From the
// log-sum-exp they would be off by its rounding: 2^-24 of the logits' size, 2e-2 of
// the gradient at logits of 1e6.)  The log-sum-exp says which rows were left out.
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
    const T* logits = static_cast<const T*>(a.logits);
    // the next row's operands load under this one's arithmetic
    int64_t t = static_cast<int64_t>(blockIdx.x) * STEP + warp * GROUPS + grp;
    struct Slot {  // the row's choice li
        uint32_t id;
        float w, dw;
    };
    auto load_slot = [&](int64_t row) {
        Slot z{0xffffffffu, 0.0f, 0.0f};
        if (row < a.T && li < a.k) {
            z.id = a.ids[row * a.k + li];
            z.dw = a.dweights[row * a.k + li];
            if (a.normalize) z.w = a.weights[row * a.k + li];
        }
        return z;
    };
    Slot slot{0xffffffffu, 0.0f, 0.0f};
    if (a.dweights != nullptr) slot = load_slot(t);
    Raw<T, V> raw;
    float lse_next = t < a.T ? a.lse[t] : INFINITY;
    raw.load(logits + t * E, e0, E, a.vec != 0, t < a.T);
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * STEP; base < a.T; base += stride, t += stride) {
        const bool in = t < a.T;
        const float lse = lse_next;
        const bool counted = lse != INFINITY;  // false: the forward left the row out
        float p[V], d[V], dot = 0.0f;
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) top = fmaxf(top, raw.get(i));
        top = group_max<L>(top);
        const float m = top > -INFINITY ? top : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = exp2_approx((raw.get(i) - m) * LOG2E);
            sum += p[i];
        }
        const float inv = __fdividef(1.0f, group_sum<L>(sum));
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = counted ? p[i] * inv : 0.0f;
        lse_next = t + stride < a.T ? a.lse[t + stride] : INFINITY;
        raw.load(logits + (t + stride) * E, e0, E, a.vec != 0, t + stride < a.T);
        float ex[V];
#pragma unroll
        for (int i = 0; i < V; ++i) ex[i] = 0.0f;
        if (a.dweights != nullptr) {
            const Slot now = slot;
            slot = load_slot(t + stride);
            float inner = 0.0f;
            if (a.normalize) {
                if (counted && now.id < static_cast<uint32_t>(E)) inner = now.w * now.dw;
                for (int j = li + L; j < a.k; j += L) {  // more choices than lanes
                    if (counted && a.ids[t * a.k + j] < static_cast<uint32_t>(E))
                        inner += a.weights[t * a.k + j] * a.dweights[t * a.k + j];
                }
                inner = group_sum<L>(inner);
            }
            if (counted) {
                if (now.id < static_cast<uint32_t>(E)) extra[now.id] = a.normalize ? now.w * (now.dw - inner) : now.dw;
                for (int j = li + L; j < a.k; j += L) {
                    const uint32_t id = a.ids[t * a.k + j];
                    const float dw = a.dweights[t * a.k + j];
                    if (id < static_cast<uint32_t>(E)) extra[id] = a.normalize ? a.weights[t * a.k + j] * (dw - inner) : dw;
                }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < V; ++i) ex[i] = extra[e0 + i];
            __syncwarp();
            if (counted) {
                if (now.id < static_cast<uint32_t>(E)) extra[now.id] = 0.0f;
                for (int j = li + L; j < a.k; j += L) {
                    const uint32_t id = a.ids[t * a.k + j];
                    if (id < static_cast<uint32_t>(E)) extra[id] = 0.0f;
                }
            }
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            d[i] = a.normalize ? q[i] : q[i] + ex[i];
            dot = fmaf(p[i], d[i], dot);
        }
        dot = group_sum<L>(dot);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float g = p[i] * (d[i] - dot);
            d[i] = counted ? (a.normalize ? g + ex[i] : g) : 0.0f;  // (0 * dloss is no 0 for every dloss)
        }
        if (!in) continue;
        T* out = static_cast<T*>(a.dlogits) + t * E + e0;
        if (a.vec && e0 + V <= E) {
            constexpr int WORDS = V * sizeof(T) / 4;
            uint32_t w[WORDS];
#pragma unroll
            for (int i = 0; i < V; ++i) reinterpret_cast<T*>(w)[i] = down<T>(d[i]);
            if constexpr (WORDS == 2) {
                *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
            } else {
#pragma unroll
                for (int i = 0; i < WORDS; i += 4)
                    reinterpret_cast<uint4*>(out)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
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
    if (E <= 128) BI_LAYOUT(32, 4);
    if (E <= 256) BI_LAYOUT(32, 8);
    if (E <= 512) BI_LAYOUT(32, 16);
    BI_LAYOUT(32, 32);
#undef BI_LAYOUT
}

int64_t lanes_for(int64_t E) { return E <= 8 ? 1 : E <= 16 ? 2 : E <= 32 ? 4 : E <= 64 ? 8 : 32; }

// Warps of a block in the short-batch form, as far as 48 KB of shared memory go.
constexpr int short_warps(int V) { return V <= 16 ? 16 : RT_WARPS; }
int short_warps_for(int64_t E) { return E <= 512 ? short_warps(16) : short_warps(32); }

// How the rows are dealt.  Up to SHORT_STEPS steps of one cluster of up to
// SHORT_BLOCKS large blocks: one launch, the sums through the cluster's shared
// memory (64 rows of 64 experts 7 us; 16384 rows of 8, with the gradient, 13.5 us
// against 17.5 with a second kernel).  Longer batches: about RT_BLOCKS blocks of RT_WARPS warps and a
// second kernel that adds their sums.  Either way a function of T and E.
struct Deal {
    int64_t per, blocks;  // rows per block (whole block steps), blocks
    bool is_short;
};
constexpr int64_t SHORT_BLOCKS = 8, SHORT_STEPS = 4;
Deal deal_rows(int64_t T, int64_t E) {
    const int64_t rows = 32 / lanes_for(E), step = short_warps_for(E) * rows;
    if (T <= SHORT_BLOCKS * SHORT_STEPS * step) {
        int64_t n = 1;  // a power of two: a cluster
        while (n < SHORT_BLOCKS && n * step < T) n *= 2;
        const int64_t per = (T + n * step - 1) / (n * step) * step;
        return {per, n, true};
    }
    const int64_t small = RT_WARPS * rows, per = ((T + RT_BLOCKS - 1) / RT_BLOCKS + small - 1) / small * small;
    return {per, (T + per - 1) / per, false};
}

template <typename T>
cudaError_t forward_t(const LaunchCtx& c, const RouteArgs& a, const Deal& d) {
    return with_layout(a.E, [&](auto l, auto v) {
        constexpr int L = l.value, V = v.value, W = short_warps(V);
        if (!d.is_short)
            return launch_pdl(route_kernel<T, L, V, RT_WARPS>, dim3(static_cast<unsigned>(d.blocks)), dim3(RT_THREADS), 0,
                              c.stream, a);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(d.blocks));
        cfg.blockDim = dim3(32 * W);
        cfg.stream = c.stream;
        cudaLaunchAttribute at[2];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        at[1].id = cudaLaunchAttributeClusterDimension;
        at[1].val.clusterDim.x = static_cast<unsigned>(d.blocks);
        at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = d.blocks > 1 ? 2 : 1;
        return cudaLaunchKernelEx(&cfg, route_kernel<T, L, V, W>, a);
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
    const Deal d = deal_rows(t, e);
    const int64_t per = d.per, blocks = d.blocks;
    // scratch (a long batch): block sums | block counts | block rows | loss terms | ticket
    Scratch sc(eng, s, !d.is_short ? static_cast<size_t>(4 * (2 * blocks * e + blocks + e + 1)) : 0);
    if (sc.err != cudaSuccess) return cuda_fail(eng, sc.err, "router scratch");
    RouteArgs a{};
    a.ids = ids; a.weights = weights; a.lse = lse; a.logits = logits; a.valid = valid;
    float* terms = nullptr;
    if (!d.is_short) {
        a.psum = static_cast<float*>(sc.ptr);
        a.pcnt = reinterpret_cast<uint32_t*>(a.psum + blocks * e);
        a.prow = a.pcnt + blocks * e;
        terms = reinterpret_cast<float*>(a.prow + blocks);
        a.ticket = reinterpret_cast<uint32_t*>(terms + e);
    }
    a.counts = counts; a.rows = rows; a.mean = mean_prob; a.loss = loss;
    a.T = t; a.rows_per_block = per;
    a.E = static_cast<int>(e); a.k = static_cast<int>(k); a.normalize = normalize != 0;
    a.vec = row_vectors(logits, e, dtype);
    err = dtype == BI_F32 ? forward_t<float>(c, a, d)
        : dtype == BI_BF16 ? forward_t<__nv_bfloat16>(c, a, d) : forward_t<__half>(c, a, d);
    if (err == cudaSuccess) c.count();
    if (err == cudaSuccess && !d.is_short) {
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
