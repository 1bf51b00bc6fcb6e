// The adapters among a 256-row tile's rows (AdapterPlan), found by the warps of one
// block in shared memory.
#pragma once

#include "adapter.h"

namespace bi {

struct PlanSmem {
    uint4 masks[ADAPTER_TILE][2];  // the result: for entry e the rows of its adapter, a bit each, at masks[slot[e]] ...
    uint32_t ids[ADAPTER_TILE];    // ... and the adapter's index
    uint16_t slot[ADAPTER_TILE];
    uint32_t count;
    uint32_t g_id[ADAPTER_TILE], g_mask[ADAPTER_TILE];  // per 32 rows the groups of rows with one adapter
    uint32_t g_n[8], g_new[8];
};

// WARPS warps (8 % WARPS == 0), this one `warp`; `sync` is a barrier among them.
// Rows of 32 with the same adapter are found by a match; the first of them stands
// for its group.  With up to 256 adapters it leaves the group's bits in the
// adapter's own place of a table, whose used places are the entries.  With more
// it looks for its adapter among the groups of the rows before (then it is no new
// entry), and gathers the bits of the groups after: with an adapter of its own for
// every row some 4 us, where the table takes 1.
template <int WARPS, typename Sync>
__device__ __forceinline__ void plan_tile(const uint32_t* row_ids, int64_t M, uint32_t G, int64_t tile, int warp, PlanSmem& sm,
                                          Sync&& sync) {
    constexpr int PER = 8 / WARPS;
    const int lane = threadIdx.x & 31;
    uint32_t id[PER];
    bool lead[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int64_t row = tile * ADAPTER_TILE + (warp + i * WARPS) * 32 + lane;
        id[i] = row < M ? row_ids[row] : G;
    }
    if (G <= ADAPTER_TILE) {
        for (uint32_t i = warp * 32 + lane; i < 2 * G; i += WARPS * 32) sm.masks[i >> 1][i & 1] = make_uint4(0, 0, 0, 0);
        sync();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t same = __match_any_sync(0xffffffffu, id[i]);
            if (id[i] < G && (same & ((1u << lane) - 1)) == 0)
                reinterpret_cast<uint32_t*>(sm.masks[id[i]])[warp + i * WARPS] = same;
        }
        sync();
        uint32_t used[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t g = (warp + i * WARPS) * 32 + lane;
            bool any = false;
            if (g < G) {
                const uint4 a = sm.masks[g][0], b = sm.masks[g][1];
                any = (a.x | a.y | a.z | a.w | b.x | b.y | b.z | b.w) != 0;
            }
            used[i] = __ballot_sync(0xffffffffu, any);
            if (lane == 0) sm.g_new[warp + i * WARPS] = __popc(used[i]);
        }
        sync();
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int q = warp + i * WARPS;
            if ((used[i] >> lane) & 1u) {
                uint32_t at = __popc(used[i] & ((1u << lane) - 1));
                for (int w = 0; w < q; ++w) at += sm.g_new[w];
                sm.ids[at] = 32 * q + lane;
                sm.slot[at] = static_cast<uint16_t>(32 * q + lane);
            }
        }
        if (warp == 0 && lane == 0) {
            uint32_t n = 0;
            for (int w = 0; w < 8; ++w) n += sm.g_new[w];
            sm.count = n;
        }
        sync();
        return;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int q = warp + i * WARPS;
        const uint32_t same = __match_any_sync(0xffffffffu, id[i]);
        lead[i] = id[i] < G && (same & ((1u << lane) - 1)) == 0;
        const uint32_t leads = __ballot_sync(0xffffffffu, lead[i]);
        if (lead[i]) {
            const int k = 32 * q + __popc(leads & ((1u << lane) - 1));
            sm.g_id[k] = id[i];
            sm.g_mask[k] = same;
        }
        if (lane == 0) sm.g_n[q] = __popc(leads);
    }
    sync();
    uint32_t mask[PER][8], fresh[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int q = warp + i * WARPS;
        bool is_new = lead[i];
        if (lead[i]) {
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                mask[i][w] = 0;
                for (uint32_t j = 0; j < sm.g_n[w]; ++j)
                    if (sm.g_id[32 * w + j] == id[i]) {
                        mask[i][w] = sm.g_mask[32 * w + j];
                        break;
                    }
                if (w < q && mask[i][w] != 0) is_new = false;
            }
        }
        fresh[i] = __ballot_sync(0xffffffffu, is_new);
        if (lane == 0) sm.g_new[q] = __popc(fresh[i]);
    }
    sync();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int q = warp + i * WARPS;
        if ((fresh[i] >> lane) & 1u) {
            uint32_t at = __popc(fresh[i] & ((1u << lane) - 1));
            for (int w = 0; w < q; ++w) at += sm.g_new[w];
            sm.ids[at] = id[i];
            sm.slot[at] = static_cast<uint16_t>(at);
            sm.masks[at][0] = make_uint4(mask[i][0], mask[i][1], mask[i][2], mask[i][3]);
            sm.masks[at][1] = make_uint4(mask[i][4], mask[i][5], mask[i][6], mask[i][7]);
        }
    }
    if (warp == 0 && lane == 0) {
        uint32_t n = 0;
        for (int w = 0; w < 8; ++w) n += sm.g_new[w];
        sm.count = n;
    }
    sync();
}

// Copies the tile's plan to global memory, thread `tid` of `threads`.
__device__ __forceinline__ void plan_store(const AdapterPlan& plan, int64_t tile, const PlanSmem& sm, int tid, int threads) {
    const int n = static_cast<int>(sm.count);
    uint4* masks = reinterpret_cast<uint4*>(plan.masks + tile * ADAPTER_TILE * 8);
    for (int i = tid; i < 2 * n; i += threads) masks[i] = sm.masks[sm.slot[i >> 1]][i & 1];
    for (int i = tid; i < n; i += threads) plan.ids[tile * ADAPTER_TILE + i] = sm.ids[i];
    if (tid < 8) plan.over[tile * 8 + tid] = 0;  // set by the finish kernel
    if (tid == 0) plan.count[tile] = sm.count;
}

}  // namespace bi
