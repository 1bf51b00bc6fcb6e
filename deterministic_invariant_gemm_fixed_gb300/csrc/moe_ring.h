// Sizes of the few-token expert layer's lists in shared memory, and of the tcgen05 kernels'
// ring behind them (moe_tc.cu).  Plain C++: a host test goes over every call's sizes.
#pragma once

#include <cstdint>

namespace bi {

constexpr int64_t MOE_MAX_PAIRS = 2048;  // token choices of a call
constexpr int64_t MOE_MAX_E = 1024;

constexpr int64_t plan_places(int64_t E, int64_t P, int64_t align) { return P + (align - 1) * (E < P ? E : P); }
// (a multiple of 16, the last four bytes n)
constexpr int64_t plan_bytes(int64_t E, int64_t P, int64_t align) { return (14 * E + 2 * plan_places(E, P, align) + 4 + 15) / 16 * 16; }
constexpr int64_t passes_bytes(int64_t most) { return (4 * most + 4 + 15) / 16 * 16; }

constexpr int PARTS = 8;                   // MXFP4 rows of a token
constexpr int PLACES = 128 / PARTS;        // tokens whose rows are one piece of scales: an expert's places start on it
constexpr int H_PLANES = 3;                // 16-bit parts of a hidden value
constexpr int T_LIMIT = 227 * 1024;
constexpr int T_BARS = 512;
constexpr int T_EX = 2 * 16 * 64 * 4;      // the epilogue's exchange between the gate's and up's warps
constexpr int A_BYTES = 128 * 128;         // weights of a stage
constexpr int MAX_STAGES = 12;
constexpr int SF_WARPS = 4;                // MXFP4: warps that put the weights' scales in place

struct MoeRing {
    int cap;        // most columns of a pass
    int passes;     // room for them
    int stage;      // bytes of a stage
    int depth;      // stages
    int64_t fixed;  // bytes before the first
};
// T tokens with P choices in all, E experts.
constexpr MoeRing moe_ring(bool fp4, bool out, int T, int64_t P, int64_t E) {
    MoeRing r{};
    const int tokens16 = (T + 15) / 16 * 16;
    // (output kernel: three parts of 64 choices are 192 columns of the MMA; with 32 or 48 choices a pass 64
    // tokens over 64 experts take 138 us for 141, but 96 over 8 179 and 181 for 171)
    r.cap = fp4 ? (T <= PLACES ? PLACES : 2 * PLACES) : out ? (tokens16 < 64 ? tokens16 : 64) : (tokens16 < 256 ? tokens16 : 256);
    r.stage = A_BYTES + (fp4 ? 1024 + r.cap * (PARTS * 128) + r.cap / PLACES * 1024 : r.cap * 128 * (out ? H_PLANES : 1));
    const int64_t active = E < P ? E : P;  // experts, at most
    // (choices shared out among the active experts make at most one pass each that is not full)
    r.passes = static_cast<int>(fp4 || out ? active + P / r.cap : active * ((T + r.cap - 1) / r.cap));
    r.fixed = plan_bytes(E, P, fp4 ? PLACES : 1) + passes_bytes(r.passes) + T_EX + T_BARS + 1024;
    const int64_t depth = (T_LIMIT - r.fixed) / r.stage;
    r.depth = static_cast<int>(depth < MAX_STAGES ? depth : MAX_STAGES);
    return r;
}

// Of the warps that put the weights' scales in place, those at work.  They take the uses of
// the ring in turn, so one that waits for use n knows no more than that use n - turn - depth
// has been consumed (its wait before), while the parity it waits by means the right phase only
// if use n - 2 depth has: no more warps than stages.
constexpr int moe_scale_warps(int depth) { return depth < SF_WARPS ? depth : SF_WARPS; }

}  // namespace bi
