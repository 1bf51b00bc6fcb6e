// What the kernels of the few-token expert layer share: limits, the choices by expert,
// the activation (moe.cu: entry points and f32 FMAs; moe_tc.cu: tcgen05).
#pragma once

#include "bi_internal.h"
#include "moe_ring.h"

namespace bi {

struct MoeCall {
    void* y;                     // [T][N]
    const void* x;               // [T][K]
    const uint32_t* ids;         // [T][C]
    const float* weights;        // [T][C]
    const void *gate, *up, *down;  // [E][F][K] twice (gate may be null), [E][N][F]; MXFP4: codes
    const uint8_t *gate_s, *up_s, *down_s;  // MXFP4: scales
    int T, C, E, act;
    int64_t K, F, N;
};

// tcgen05 forms (moe_tc.cu): 16-bit weights on 16 bytes with K and F multiples of 8, or
// MXFP4 weights with x and y of any type.  copy_x: x is not on 16 bytes.
int64_t moe_tc_scratch_bytes(const MoeCall& m, bool fp4, bool copy_x, bi_dtype dt);
cudaError_t moe_tc(const LaunchCtx& c, const MoeCall& m, bool fp4, bool copy_x, bi_dtype dt, void* scratch);

#ifdef __CUDACC__

// What a launch executes once is as slow as its way from memory: the rarer activations
// and the list of several passes an expert (moe_tc.cu) are functions of their own and the
// long lists' code lies apart, so that what every launch runs through stays short (MXFP4, 4
// tokens: 34 us; with all of it inlined, 42).
static __device__ __noinline__ float activate_other(float v, int act) {
    if (act == BI_ACT_GELU) return 0.5f * v * (1.0f + tanhf(0.79788456f * (v + 0.044715f * v * v * v)));
    return fmaxf(v, 0.0f) + (v != v ? v : 0.0f);  // relu; NaN stays
}
__device__ __forceinline__ float activate(float v, int act) {
    return act == BI_ACT_SILU ? v / (1.0f + expf(-v)) : activate_other(v, act);
}

// The choices of a call by expert, built by every block in its shared memory.  Expert
// e's choices, in ascending order, have the places first[e] .. first[e] + cnt[e] - 1, first[e]
// a multiple of ALIGN; list[place] is the choice.  cnt and first are set for the
// experts with choices only.
struct Plan {
    uint32_t* cnt;     // [E]
    uint32_t* first;   // [E]
    uint16_t* list;    // [places]
    uint16_t* active;  // [E] experts with choices
    int n;             // how many
};

__device__ __forceinline__ uint32_t lane_prefix(uint32_t v) {  // inclusive sum over the lanes
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t w = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += w;
    }
    return v;
}

template <int ALIGN>
__device__ __forceinline__ void build_long_plan(const Plan p, uint32_t* cursor, uint32_t* n, const uint32_t* __restrict__ ids, int P, int E) {
    const int lane = threadIdx.x & 31;
    const uint32_t below = (1u << lane) - 1u;
    for (int e = threadIdx.x; e < E; e += blockDim.x) p.cnt[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < P; i += blockDim.x) {
        const uint32_t e = __ldg(ids + i);
        if (e < static_cast<uint32_t>(E)) atomicAdd(p.cnt + e, 1u);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        uint32_t run = 0, act = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {  // prefix sums over the experts
            const int e = e0 + lane;
            const uint32_t c = e < E ? p.cnt[e] : 0u, room = (c + ALIGN - 1) / ALIGN * ALIGN, sum = lane_prefix(room);
            const uint32_t has = __ballot_sync(0xffffffffu, c != 0);
            if (e < E) p.first[e] = cursor[e] = run + sum - room;
            if (c) p.active[act + __popc(has & below)] = static_cast<uint16_t>(e);
            run += __shfl_sync(0xffffffffu, sum, 31);
            act += __popc(has);
        }
        __syncwarp();
        for (int i0 = 0; i0 < P; i0 += 32) {  // the lists, in order: every block's are the same
            const int i = i0 + lane;
            const uint32_t e = i < P ? __ldg(ids + i) : 0xffffffffu;
            const bool in = e < static_cast<uint32_t>(E);
            const uint32_t same = __match_any_sync(0xffffffffu, in ? e : 0xffffffffu);
            const uint32_t at = in ? cursor[e] + __popc(same & below) : 0u;
            if (in) p.list[at] = static_cast<uint16_t>(i);
            __syncwarp();
            if (in && __ffs(same) - 1 == lane) cursor[e] = at + __popc(same);
            __syncwarp();
        }
        if (lane == 0) *n = act;
    }
    __syncthreads();
}

template <int ALIGN>
__device__ __forceinline__ Plan build_plan(uint8_t* smem, const uint32_t* __restrict__ ids, int P, int E) {
    Plan p;
    p.cnt = reinterpret_cast<uint32_t*>(smem);
    p.first = p.cnt + E;
    uint32_t* cursor = p.first + E;
    p.active = reinterpret_cast<uint16_t*>(cursor + E);
    p.list = p.active + E;
    p.n = 0;
    uint32_t* n = reinterpret_cast<uint32_t*>(smem + plan_bytes(E, P, ALIGN)) - 1;
    if (__builtin_expect(P > 32, 0)) {
        build_long_plan<ALIGN>(p, cursor, n, ids, P, E);
    } else {  // one warp, a choice per lane, no passes over the experts
        if (threadIdx.x < 32) {
            const int lane = threadIdx.x;
            const uint32_t below = (1u << lane) - 1u;
            const uint32_t e = lane < P ? __ldg(ids + lane) : 0xffffffffu;
            const bool in = e < static_cast<uint32_t>(E);
            const uint32_t same = __match_any_sync(0xffffffffu, in ? e : 0xffffffffu);
            const int leader = __ffs(same) - 1;
            const bool lead = in && leader == lane;
            const uint32_t c = lead ? __popc(same) : 0u, room = (c + ALIGN - 1) / ALIGN * ALIGN, start = lane_prefix(room) - room;
            const uint32_t leads = __ballot_sync(0xffffffffu, lead), at = __shfl_sync(0xffffffffu, start, leader);
            if (lead) {
                p.cnt[e] = c;
                p.first[e] = start;
                p.active[__popc(leads & below)] = static_cast<uint16_t>(e);
            }
            if (in) p.list[at + __popc(same & below)] = static_cast<uint16_t>(lane);
            if (lane == 0) *n = __popc(leads);
        }
        __syncthreads();
    }
    p.n = static_cast<int>(*n);
    return p;
}

#endif

}  // namespace bi
