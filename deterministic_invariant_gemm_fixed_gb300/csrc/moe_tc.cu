// The few-token expert layer on tcgen05 (see moe.cu for the layer and its other form).
//
//   D [128 weight rows x tokens] = A [128 x K] B [tokens x K]^T
//
// The weights are the A operand: a decoding step is bound by reading them, and
// this way each goes from memory to shared memory by TMA and on to the tensor cores without an
// instruction of its own; the tokens, few, are the MMA's N.  A block takes 128 weight
// rows of one expert at a time (hidden kernel: 64 of the gate's and 64 of up's, whose
// products meet in the epilogue) and walks such units, one block per SM, the copies
// running ahead from unit to unit.  A column's element is one ascending chain over the
// contraction in one f32 accumulator, whatever the number of tokens beside it.
//
// 16-bit weights: kind::f16, stages of 64.  The tokens of the hidden kernel are all tokens
// of the batch, straight from x (up to 256 at a time): columns of tokens that chose
// other experts are thrown away.  For a few tokens that costs nothing next to gathering; with 256
// a stage brings twice as much of x as of the weights, and the ring is shorter.  h enters the output
// kernel as three 16-bit parts, each what the ones before left: all 24 bits of its f32
// value.  They are N columns of their own, added in the epilogue from the smallest up: a sum of the
// tensor cores cuts off what it shifts out, once for every MMA into it.  (Two parts into
// one sum leave 2^-17 of h in bf16: 64 tokens, 64 experts of 2048 x 1408, 3.7 results of
// 1000 are not the 64-bit value's rounding, here 2.4; 138 and 141 us.)  f16 has not h's range:
// there h is kept in f32, and a kernel between the two scales each choice's by a power of
// two, its largest to 2^14 (its parts stop at 2^-39 of the largest), which the sums are
// multiplied back by.
//
// MXFP4 weights: kind::mxf4 with block scales, stages of 256, the codes as they lie in
// memory: no weight is ever expanded.  Its other operand has to be MXFP4 too, so a token's
// x (and h) is written as a sum of PARTS rows in MXFP4.  Each part rounds what the parts
// before left, per block of 32, by a scale 2^s at least a quarter of the largest of it:
// up to 4 the codes are at most 1 apart, so at most 2^s / 2 is left where more than 2^(s+1)
// was, and the next scale is 2^(s-3).  Three bits a part: eight leave at most 2^-23 of the
// block's largest value.  (By scales that use codes up to 6, which are 2 apart there, a part
// gains two bits: twelve parts.)  The parts are N columns of their own, added in the
// epilogue from the smallest up.  A kernel of its own makes them, of x and of h: in the
// hidden kernel's epilogue, which has 128 threads per SM, they took longer than all
// else (f16, 96 tokens, 8 experts of 4096 x 4096: 200 us for that kernel, 97 without).
//
// Sums of the output kernel's units go to memory once per choice, and a third, small
// kernel adds every token's choices in order.  (A block that adds up a tile once it has
// finished the tile's last unit is late for its next unit, and so the last again: that
// kernel took 182 against 55 us for 64 tokens, 64 experts of 2048 x 1408.)
//
// Bound by reading the weights where there are many: 64 tokens through 6 of 64 experts of
// 2048 x 1408 in bf16 read 450 MB in 85 us (hidden) and 228 MB in 56 (output), caches cold,
// set-up and ends included.  One token's 104 MB take 29 us over the three kernels, a third
// of it set-up and ends.  MXFP4 with many tokens (96, 2 of 8 experts of 4096 x 4096: 86 us for
// 220 MB) is bound by the tokens' rows, 1 KB a token and stage beside the weights' 16 KB.
#include "abi_util.h"
#include "fp4.h"
#include "moe.h"
#include "tc_common.cuh"

#include <cuda_fp4.h>

#include <type_traits>

namespace bi {
namespace {

constexpr int t_threads(bool fp4) { return 192 + (fp4 ? 32 * SF_WARPS : 0); }
constexpr int SF_COL = 256, SF_COLS = 24;  // tensor memory: accumulator, then two stages of scales (A 8, B 16)

struct TcArgs {
    MoeCall m;
    uint16_t* h;        // 16-bit weights: planes [H_PLANES][P][Fp]
    float* hf;          // not bf16: h itself, [places][F], which a kernel of its own makes the next operand of
    const float* unscale;  // f16 weights, output kernel: [P] by which a place's sums are multiplied
    float* part;        // [P][Nq] the choices' sums
    int64_t Fp, Nq;
    int P, tiles, chunks;  // choices; row tiles of an expert; stages of the contraction
    int cap, passes;       // most columns of a pass; most passes
    int stage, depth;      // ring: bytes of a stage, stages
    uint32_t fmt;          // 16-bit weights: 0 f16, 1 bf16
    int* status;
    unsigned long long wait_limit;
};

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar, uint32_t lead) {
    asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar), "r"(lead)
                 : "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory"); }
__device__ __forceinline__ void mma_16(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 e, %6, 0;\n\t"
        "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(DESC_HI), "r"(idesc), "r"(acc), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t acc,
                                         uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %7, 0;\n\tsetp.ne.b32 e, %8, 0;\n\t"
        "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %4, [%5], [%6], p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(DESC_HI), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint32_t saddr, uint32_t lead) {
    constexpr uint32_t HI = (128u >> 4) | (1u << 14);
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b64 d;\n\tsetp.ne.b32 e, %3, 0;\n\tmov.b64 d, {%1, %2};\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}\n" ::"r"(taddr),
        "r"(((saddr & 0x3FFFFu) >> 4) | (1u << 16)), "r"(HI), "r"(lead)
        : "memory");
}
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
    uint32_t v;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(taddr));
    return v;
}

// The passes of a call: an expert and up to cap columns, from column c0 of its own on.  A
// column is a token of the batch (16-bit weights, hidden kernel) or one of the expert's
// choices.  Experts with more of them have several passes, each as long as another
// expert's: what the blocks share out is passes, so that an expert with many tokens does
// not keep one block busy after the others.
struct Passes {
    uint16_t *e, *c0;  // c0 null: all 0
    int n;
};
template <bool CHOICES>
__device__ __noinline__ void build_many_passes(const Passes q, uint32_t* n, const Plan p, int tokens, int cap) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        uint32_t run = 0;
        for (int s0 = 0; s0 < p.n; s0 += 32) {
            const int s = s0 + lane, e = s < p.n ? p.active[s] : 0;
            const uint32_t all = s < p.n ? (CHOICES ? p.cnt[e] : static_cast<uint32_t>(tokens)) : 0u, mine = (all + cap - 1) / cap;
            const uint32_t sum = lane_prefix(mine);
            for (uint32_t i = 0; i < mine; ++i) {
                q.e[run + sum - mine + i] = static_cast<uint16_t>(e);
                q.c0[run + sum - mine + i] = static_cast<uint16_t>(i * cap);
            }
            run += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (lane == 0) *n = run;
    }
    __syncthreads();
}
template <bool CHOICES>
__device__ __forceinline__ Passes build_passes(uint8_t* smem, int64_t most, const Plan& p, int tokens, int choices, int cap) {
    if ((CHOICES ? choices : tokens) <= cap) return Passes{p.active, nullptr, p.n};  // a pass for each expert
    Passes q{reinterpret_cast<uint16_t*>(smem), reinterpret_cast<uint16_t*>(smem) + most, 0};
    uint32_t* n = reinterpret_cast<uint32_t*>(smem + passes_bytes(most)) - 1;
    build_many_passes<CHOICES>(q, n, p, tokens, cap);
    q.n = static_cast<int>(*n);
    return q;
}

// A block's units: (pass, row tile), tiles of one pass next to one another, or in the
// output kernel (row tile, pass).
template <bool FP4, bool OUT>
struct Walk {
    int u, e, tile, n, c0;  // n: the pass's columns
    __device__ __forceinline__ bool more(const TcArgs& a, const Passes& q) const { return u < q.n * a.tiles; }
    __device__ __forceinline__ void open(const TcArgs& a, const Plan& p, const Passes& q) {
        if (!more(a, q)) return;
        const int pass = OUT ? u % q.n : u / a.tiles;
        tile = OUT ? u / q.n : u % a.tiles;
        e = q.e[pass];
        c0 = q.c0 ? q.c0[pass] : 0;
        n = min(a.cap, (FP4 || OUT ? static_cast<int>(p.cnt[e]) : a.m.T) - c0);
    }
    __device__ __forceinline__ void next(const TcArgs& a, const Plan& p, const Passes& q) {
        u += gridDim.x;
        open(a, p, q);
    }
};

// One part of a block of 32: the byte of the smallest scale of which the largest
// magnitude is at most four times.
__device__ __forceinline__ uint32_t part_scale(uint32_t amax_bits) {
    const uint32_t e = amax_bits >> 23, exact = (amax_bits & 0x7fffffu) == 0 ? 1u : 0u;
    return e == 255u ? 255u : e < 1u + exact ? 0u : e - 1u - exact;
}
__device__ __forceinline__ float part_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// h of a lane's row for n tokens, places step apart.
__device__ __forceinline__ void hidden_out(const TcArgs& a, const float (&r)[8], int64_t place, int step, int n, int64_t row) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (j >= n || row >= a.m.F) continue;
        if (a.hf) {
            a.hf[(place + j * step) * a.m.F + row] = r[j];
            continue;
        }
        // eight bits of the 24 a plane, cut off so that no plane leaves bf16's range
        float v = r[j];
        uint16_t* o = a.h + (place + j * step) * a.Fp + row;
#pragma unroll
        for (int x = 0; x < H_PLANES; ++x) {
            const __nv_bfloat16 b = __float2bfloat16_rz(v);
            o[x * static_cast<int64_t>(a.P) * a.Fp] = __bfloat16_as_ushort(b);
            v -= __bfloat162float(b);
        }
    }
}

template <bool FP4, bool OUT>
__global__ void __launch_bounds__(t_threads(FP4), 1)
    moe_tc_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmSB, const __grid_constant__ CUtensorMap tmB8, const TcArgs a) {
    constexpr int ALIGN = FP4 ? PLACES : 1;
    constexpr int BPARTS = !FP4 && OUT ? H_PLANES : 1;  // planes of B
    extern __shared__ __align__(16) uint8_t smem_raw[];
    const MoeCall& m = a.m;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    uint8_t* after = smem_raw + plan_bytes(m.E, a.P, ALIGN) + passes_bytes(a.passes);
    float* ex = reinterpret_cast<float*>(after);
    uint64_t* bars = reinterpret_cast<uint64_t*>(after + T_EX);
    const uint32_t bar0 = smem_u32(bars), sbase = (bar0 + T_BARS + 1023u) & ~1023u;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (MAX_STAGES + s); };
    const uint32_t tfull = bar0 + 8u * (2 * MAX_STAGES), tempty = tfull + 8, drain = tfull + 16;
    uint32_t* slot = reinterpret_cast<uint32_t*>(bars + 2 * MAX_STAGES + 3);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(slot + 1);

    if (warp == 2 && lane < (FP4 ? 5 : 4)) prefetch_map(lane == 0 ? &tmA0 : lane == 1 ? &tmA1 : lane == 2 ? &tmB : lane == 3 ? &tmB8 : &tmSB);
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.depth; ++s) {
            mbar_init(full_bar(s), FP4 ? 2 : 1);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(tfull, 1);
        mbar_init(tempty, 4);
        mbar_init(drain, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(slot), 0);
    // Behind another kernel of the layer, which waited for all before it and let this one
    // start only then, ids and weights are complete already: the lists are made and the first
    // weights fetched while that kernel ends.
    constexpr bool EARLY = FP4 || OUT;
    if (!EARLY) {
        grid_dep_wait();
        grid_dep_launch();
    }
    const Plan p = build_plan<ALIGN>(smem_raw, m.ids, a.P, m.E);
    const Passes q = build_passes<FP4 || OUT>(smem_raw + plan_bytes(m.E, a.P, ALIGN), a.passes, p, m.T, a.P, a.cap);
    const int64_t R = OUT ? m.N : m.F;       // rows of an expert
    const bool gated = !OUT && m.gate != nullptr;
    const int span = gated ? 64 : 128;       // rows of a tile, of each of the two matrices or of the one
    Walk<FP4, OUT> w;
    w.u = blockIdx.x;
    w.open(a, p, q);
    const int sfa_at = A_BYTES, b_at = A_BYTES + (FP4 ? 1024 : 0), b_bytes = a.cap * (FP4 ? PARTS : BPARTS) * 128;
    const int sfb_at = b_at + b_bytes;

    if (warp == 0) {
        // ------------------------------------------------------------ copies, a lane each
        // Lanes 30 and 31: 64 weight rows each.  From lane 0: B's boxes of 128 or 16 rows, then
        // (MXFP4) B's scales, 16 tokens a box.  What a lane copies is found once per pass:
        // a stage costs its wait and the copy (found anew for each stage: 0.37 us a stage).
        const bool wlane = lane >= 30;
        const CUtensorMap* map = nullptr;
        uint32_t to = 0, bytes = 0;
        int y = 0, xs = 0;
        bool has = false;
        auto aim = [&](const Walk<FP4, OUT>& x) {
            const int cols = x.n, nb = ((FP4 ? PARTS : 1) * cols + 15) / 16, big = nb / 8, each = big + nb % 8;
            const int sf = FP4 ? (cols + PLACES - 1) / PLACES : 0;
            const int first = FP4 || OUT ? static_cast<int>(p.first[x.e]) + x.c0 : x.c0;
            bytes = A_BYTES + nb * BPARTS * 2048 + sf * 1024;
            xs = FP4 ? 128 : 64;
            if (wlane) {
                const int64_t r = x.e * R + static_cast<int64_t>(x.tile) * span;
                map = lane == 30 ? &tmA0 : &tmA1;
                to = sbase + (lane - 30) * (A_BYTES / 2);
                y = static_cast<int>(gated ? r : r + (lane - 30) * 64);
                has = true;
            } else if (lane < each * BPARTS) {
                const int part = BPARTS == 1 ? 0 : lane / each, i = lane - part * each, b = i < big ? i * 8 : big * 8 + i - big;
                map = i < big ? &tmB8 : &tmB;
                to = sbase + b_at + (part * nb + b) * 2048;
                y = FP4 ? first * PARTS + b * 16 : part * a.P + first + b * 16;
                has = true;
            } else {
                map = &tmSB;
                to = sbase + sfb_at + (lane - each) * 1024;
                y = first / PLACES + lane - each;
                xs = 256;
                has = FP4 && lane < each + sf;
            }
        };
        struct At { Walk<FP4, OUT> x; int c, s; uint32_t ph; };
        // up to `limit` stages from `at` on: the weights, with the expected bytes, or the rest, or both
        auto stages = [&](At& at, int limit, bool weights, bool rest) {
            int made = 0;
            bool ok = true;
            while (ok && made < limit && at.x.more(a, q)) {
                aim(at.x);
                const bool mine = has && (wlane ? weights : rest);
                for (; at.c < a.chunks && made < limit; ++at.c, ++made) {
                    if (weights) {
                        ok = __all_sync(0xffffffffu, mbar_wait_fast(empty_bar(at.s), at.ph ^ 1u, abort_flag, a, DEV_TIMEOUT_PRODUCER));
                        if (!ok) break;
                        if (lane == 31) mbar_expect_tx(full_bar(at.s), bytes);
                        __syncwarp();
                    }
                    if (mine) tma_2d(to + at.s * a.stage, map, at.c * xs, y, full_bar(at.s));
                    if (++at.s == a.depth) { at.s = 0; at.ph ^= 1u; }
                }
                if (at.c == a.chunks) {
                    at.c = 0;
                    at.x.next(a, p, q);
                }
            }
            return made;
        };
        At at{w, 0, 0, 0u};
        if (EARLY) {
            At again = at;
            const int made = stages(at, FP4 ? a.depth : min(a.depth, 4), true, false);  // (16-bit: four stages are fetched by the time the other ends)
            grid_dep_wait();
            grid_dep_launch();
            stages(again, made, false, true);
        }
        stages(at, 0x7fffffff, true, true);
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        const uint32_t lead = elect_lane();
        int s = 0, sf = 0;
        uint32_t ph = 0, it = 0;
        bool ok = true;
        for (; ok && w.more(a, q); w.next(a, p, q), ++it) {
            if (it) ok = __all_sync(0xffffffffu, mbar_wait_fast(tempty, (it - 1) & 1u, abort_flag, a, DEV_TIMEOUT_MMA));
            if (!ok) break;
            tc_fence_after();
            const int cols = w.n;
            const uint32_t N = ((FP4 ? PARTS : 1) * cols + 15) / 16 * 16 * BPARTS;
            for (int c = 0; c < a.chunks; ++c) {
                ok = __all_sync(0xffffffffu, mbar_wait_fast(full_bar(s), ph, abort_flag, a, DEV_TIMEOUT_MMA));
                if (!ok) break;
                tc_fence_after();
                const uint32_t st = sbase + s * a.stage, da = desc_lo(st, false), db = desc_lo(st + b_at, false);
                if constexpr (FP4) {
                    const uint32_t ta = tmem + SF_COL + sf * SF_COLS, tb = ta + 8;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        scales_to_tmem(ta + k * 4, st + sfa_at + k * 512, lead);
                        scales_to_tmem(tb + k * 8, st + sfb_at + k * 512, lead);
                        if (cols > PLACES) scales_to_tmem(tb + k * 8 + 4, st + sfb_at + 1024 + k * 512, lead);
                    }
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint32_t id = (kk & 1) * 2;
                        mma_mxf4(tmem, da + kk * K_STEP, db + kk * K_STEP,
                                 (id << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | (1u << 23) | (1u << 27) | (id << 29), ta + (kk >> 1) * 4,
                                 tb + (kk >> 1) * 8, (c | kk) != 0 ? 1u : 0u, lead);
                    }
                    sf ^= 1;
                } else {
                    const uint32_t idesc = (1u << 4) | (a.fmt << 7) | (a.fmt << 10) | ((N >> 3) << 17) | (8u << 24);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_16(tmem, da + kk * K_STEP, db + kk * K_STEP, idesc, (c | kk) != 0 ? 1u : 0u, lead);
                }
                commit(empty_bar(s), lead);
                if (++s == a.depth) { s = 0; ph ^= 1u; }
            }
            if (!ok) break;
            commit(tfull, lead);
        }
        __syncwarp();
        if (lead) {
            commit(drain, 1u);
            mbar_drain(drain, 0);
        }
        __syncwarp();
    } else if (FP4 && warp >= 6) {
        // ------------------------------------------------------------ the weights' scales
        // A lane has rows lane and lane + 32 of either half of the tile, wherever their
        // bytes lie, and puts them side by side in the order that the tensor cores take.
        // Loaded for BATCH stages at once: the fence that hands a stage on waits for the
        // loads in flight too (loads between the fences: 1.1 us a stage); and by up to SF_WARPS
        // warps in turn, each taking as long over a stage as the tensor cores over several
        // (never more warps than stages: moe_scale_warps).
        constexpr int BATCH = 4;
        const int turn = moe_scale_warps(a.depth), first = warp - 6;
        const int64_t Lp = fp4_padded(OUT ? m.F : m.K), all = m.E * R;
        const uint8_t* s0 = OUT ? m.down_s : gated ? m.gate_s : m.up_s;
        const uint8_t* s1 = OUT ? m.down_s : m.up_s;
        int s = 0, c = 0;
        uint32_t ph = 0;
        uint32_t v[BATCH][8];
        bool have[BATCH];
        const uint8_t* at[4];
        auto rows = [&] {
            const int64_t r = w.e * R + static_cast<int64_t>(w.tile) * span;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t row = lmin(r + lane + (j & 1) * 32 + (j >= 2 && !gated ? 64 : 0), all - 1);
                at[j] = (j < 2 ? s0 : s1) + fp4_scale_at(row, 0, Lp);
            }
        };
        auto ahead = [&](int n) {  // the walk n stages on
            for (; n > 0 && w.more(a, q); --n)
                if (++c == a.chunks) { c = 0; w.next(a, p, q); }
        };
        auto load = [&](uint32_t (&x)[8], bool& got) {
            got = w.more(a, q);
            if (!got) return;
            rows();
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = __ldg(reinterpret_cast<const uint32_t*>(at[j & 3] + static_cast<int64_t>(2 * c + (j >> 2)) * 512));
            ahead(turn);
        };
        ahead(first);
        auto step = [&](int n) {  // the ring's stage n uses on
            for (s += n; s >= a.depth; s -= a.depth) ph ^= 1u;
        };
        step(first);
        bool go = first < turn;
        while (go) {
#pragma unroll
            for (int i = 0; i < BATCH; ++i) load(v[i], have[i]);
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                go = go && have[i] && __all_sync(0xffffffffu, mbar_wait_fast(empty_bar(s), ph ^ 1u, abort_flag, a, DEV_TIMEOUT_PRODUCER));
                if (!go) continue;
                const uint32_t to = sbase + s * a.stage + sfa_at + lane * 16;
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(v[i][0]), "r"(v[i][1]), "r"(v[i][2]), "r"(v[i][3]) : "memory");
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + 512), "r"(v[i][4]), "r"(v[i][5]), "r"(v[i][6]), "r"(v[i][7]) : "memory");
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) arrive(full_bar(s));
                step(turn);
            }
        }
    } else if (warp >= 2 && warp < 6) {
        // ------------------------------------------------------------ epilogue
        if (EARLY) grid_dep_wait();
        const int quad = warp & 3;
        uint32_t it = 0;
        int k = 0;  // exchanges so far: the buffers take turns over all units
        auto meet = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
        auto all_warps = [](int ok) {
            uint32_t r;
            asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.and.pred q, 1, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}\n"
                         : "=r"(r) : "r"(ok) : "memory");
            return r != 0;
        };
        for (; w.more(a, q); w.next(a, p, q), ++it) {
            // the four warps go on or give up together: they meet below
            if (!all_warps(__all_sync(0xffffffffu, mbar_wait(tfull, it & 1u, abort_flag, a, DEV_TIMEOUT_EPILOGUE)))) break;
            tc_fence_after();
            const uint32_t tb = tmem + (static_cast<uint32_t>(quad * 32) << 16);
            auto drained = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(tempty);
            };
            // the choices of this pass: places i0 .. i0 + items - 1 of the expert's
            int i0 = w.c0, items = w.n;
            if (!FP4 && !OUT) {
                const int n = static_cast<int>(p.cnt[w.e]);
                i0 = items = 0;
                for (int i = lane; i < n; i += 32) {
                    const int tok = p.list[p.first[w.e] + i] / m.C;
                    i0 += tok < w.c0;
                    items += tok >= w.c0 && tok < w.c0 + a.cap;
                }
                i0 = __reduce_add_sync(0xffffffffu, i0);
                items = __reduce_add_sync(0xffffffffu, items);
            }
            const uint16_t* mine = p.list + p.first[w.e] + i0;
            const int place = static_cast<int>(p.first[w.e]) + i0;
            const int half = gated ? quad & 1 : quad;
            const int64_t row = static_cast<int64_t>(w.tile) * span + half * 32 + lane;  // of the hidden layer or the output
            for (int b = 0; b < items; b += 16) {
                const int cnt = min(16, items - b);
                float v[16];
                if constexpr (FP4) {
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        v[j] = v[j + 1] = 0.0f;
                        if (j >= cnt) continue;
                        uint32_t r[16];  // two tokens' parts
                        static_assert(PARTS == 8, "two tokens per load");
                        __syncwarp();
                        tmem_ld16(tb + (b + j) * PARTS, r);
#pragma unroll
                        for (int x = 7; x >= 0; --x) {
                            v[j] = __fadd_rn(v[j], __uint_as_float(r[x]));
                            v[j + 1] = __fadd_rn(v[j + 1], __uint_as_float(r[8 + x]));
                        }
                    }
                } else if constexpr (OUT) {
                    const int plane = (items + 15) / 16 * 16;  // columns of a part
                    uint32_t r[H_PLANES][16];
                    __syncwarp();
#pragma unroll
                    for (int x = 0; x < H_PLANES; ++x) tmem_get16(tb + x * plane + b, r[x]);
                    tmem_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {  // the smallest first
                        v[j] = __uint_as_float(r[H_PLANES - 1][j]);
#pragma unroll
                        for (int x = H_PLANES - 2; x >= 0; --x) v[j] = __fadd_rn(__uint_as_float(r[x][j]), v[j]);
                    }
                } else {
                    // a lane finds a token's column for all
                    const int mycol = mine[min(b + lane, items - 1)] / m.C - w.c0;
                    uint32_t r[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        r[j] = 0;
                        const int col = __shfl_sync(0xffffffffu, mycol, j);
                        if (j < cnt) r[j] = tmem_ld1(tb + col);
                    }
                    tmem_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
                }
                if (b + 16 >= items) drained();  // the last of the accumulator: the next pass's MMAs may start
                if (OUT) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (j < cnt && row < R)
                            __stcg(a.part + mine[b + j] * a.Nq + row, a.unscale ? v[j] * __ldg(a.unscale + place + b + j) : v[j]);
                    continue;
                }
                float r[8] = {};
                if (gated) {
                    // warps 0 and 1 have the gate's rows, 2 and 3 up's: they swap half, the
                    // first two finish the even tokens, the others the odd ones
                    float* e = ex + (k++ & 1) * (16 * 64) + half * 32 + lane;
                    const bool odd = quad >= 2;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (2 * j < cnt) e[(2 * j + (odd ? 0 : 1)) * 64] = odd ? v[2 * j] : v[2 * j + 1];
                    meet();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (2 * j >= cnt) break;
                        const float other = e[(2 * j + (odd ? 1 : 0)) * 64];
                        r[j] = odd ? activate(other, m.act) * v[2 * j + 1] : activate(v[2 * j], m.act) * other;
                    }
                    hidden_out(a, r, place + b + (odd ? 1 : 0), 2, (cnt + (odd ? 0 : 1)) / 2, row);
                } else {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) r[j] = 8 * x + j < cnt ? activate(v[8 * x + j], m.act) : 0.0f;
                        if (cnt > 8 * x) hidden_out(a, r, place + b + 8 * x, 1, min(8, cnt - 8 * x), row);
                    }
                }
            }
            if (items == 0) drained();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) settle_copies();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// Rows as their parts, at the places of the choices: x [T][K] (each token at those of its
// C choices), or with BY_PLACE h [places][K] (C = 1, T choices).  A warp to 128 elements of a
// row.
constexpr int X_THREADS = 128;
template <typename T, bool BY_PLACE>
__global__ void __launch_bounds__(X_THREADS) moe_parts_kernel(const T* x, const uint32_t* ids, uint8_t* xq, uint8_t* xs, int T_, int C, int E,
                                                              int64_t K) {
    extern __shared__ __align__(16) uint8_t smem[];
    if (!BY_PLACE) grid_dep_wait();  // (h's is behind the hidden kernel: the ids are complete)
    const int P = T_ * C, lane = threadIdx.x & 31;
    const Plan p = build_plan<PLACES>(smem, ids, P, E);
    uint16_t* place = reinterpret_cast<uint16_t*>(smem + plan_bytes(E, P, PLACES));  // of each choice
    for (int i = threadIdx.x; i < P; i += X_THREADS) place[i] = 0xffff;              // none
    __syncthreads();
    for (int s = threadIdx.x >> 5; s < p.n; s += X_THREADS / 32) {
        const int e = p.active[s];
        for (int i = lane; i < static_cast<int>(p.cnt[e]); i += 32) place[p.list[p.first[e] + i]] = static_cast<uint16_t>(p.first[e] + i);
    }
    __syncthreads();
    if (BY_PLACE) grid_dep_wait();
    grid_dep_launch();
    const int64_t Kp = fp4_padded(K), per = Kp / 128;
    for (int64_t i = blockIdx.x * int64_t(X_THREADS / 32) + (threadIdx.x >> 5); i < T_ * per; i += gridDim.x * int64_t(X_THREADS / 32)) {
        const int64_t t = i / per, k = (i - t * per) * 128 + lane * 4;
        if (BY_PLACE && place[t] == 0xffff) continue;
        const T* row = x + (BY_PLACE ? static_cast<int64_t>(place[t]) : t) * K;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = k + j < K ? static_cast<float>(row[k + j]) : 0.0f;
        uint32_t word[PARTS], bytes[PARTS / 4];
#pragma unroll
        for (int part = 0; part < PARTS; ++part) {
            uint32_t mx = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) mx = max(mx, __float_as_uint(v[j]) & 0x7fffffffu);
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const uint32_t byte = part_scale(mx);
            const float inv = byte == 255u ? 0.0f : part_inverse(byte), scale = fp4_scale_value(byte);
            word[part] = 0;
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const float a = __fmul_rn(v[j], inv), b = __fmul_rn(v[j + 1], inv);
                const uint32_t c = byte == 255u ? 0u : __nv_cvt_float2_to_fp4x2(make_float2(a, b), __NV_E2M1, cudaRoundNearest);
                word[part] |= c << (4 * j);
                // exact: the rest of a rounding to nearest (taken before the scale: the code of a
                // value near 2^128 may stand for 2^128)
                v[j] = byte == 255u ? 0.0f : __fmul_rn(__fsub_rn(a, fp4_code_value(c & 15u)), scale);
                v[j + 1] = byte == 255u ? 0.0f : __fmul_rn(__fsub_rn(b, fp4_code_value(c >> 4)), scale);
            }
            if (part % 4 == 0) bytes[part / 4] = 0;
            bytes[part / 4] |= byte << (8 * (part % 4));
        }
        for (int j = 0; j < C; ++j) {
            const uint32_t at = place[t * C + j];
            if (at == 0xffffu) continue;
            const int64_t r = static_cast<int64_t>(at) * PARTS;
            uint8_t* q = xq + r * (Kp / 2) + k / 2;
            uint8_t* s = xs + fp4_scale_at(r, k >> 5, Kp);  // (the rows of a place: 16 bytes apart)
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
                *reinterpret_cast<uint16_t*>(q + part * (Kp / 2)) = static_cast<uint16_t>(word[part]);
                if ((lane & 7) == 0) s[part * 16] = static_cast<uint8_t>(bytes[part / 4] >> (8 * (part % 4)));
            }
        }
    }
}

// y[t] = sum over j of weights[t,j] * part[t,j], four columns per thread.
template <typename T>
__global__ void __launch_bounds__(128) moe_sum_kernel(T* y, const float* part, const uint32_t* ids, const float* weights, int T_, int C, int E,
                                                      int64_t N, int64_t Nq) {
    grid_dep_wait();
    grid_dep_launch();
    const int64_t per = (N + 3) / 4, i = blockIdx.x * 128ll + threadIdx.x;
    if (i >= T_ * per) return;
    const int64_t t = i / per, n0 = (i - t * per) * 4;
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int j = 0; j < C; ++j) {
        const int64_t pr = t * C + j;
        const bool in = __ldg(ids + pr) < static_cast<uint32_t>(E);
        const float w = __ldg(weights + pr);
        const float4 d = in ? __ldg(reinterpret_cast<const float4*>(part + pr * Nq + n0)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (in) {
            s[0] = fmaf(w, d.x, s[0]);
            s[1] = fmaf(w, d.y, s[1]);
            s[2] = fmaf(w, d.z, s[2]);
            s[3] = fmaf(w, d.w, s[3]);
        }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x)
        if (n0 + x < N) y[t * N + n0 + x] = static_cast<T>(s[x]);
}

// f16 weights: a choice's h, scaled by a power of two, in f16 planes.  A block per place
// (places that no choice has hold anything, and are not read).
__global__ void __launch_bounds__(256) moe_planes_kernel(uint16_t* h, float* unscale, const float* hf, int64_t F, int64_t Fp, int P) {
    __shared__ uint32_t top[8];
    grid_dep_wait();
    grid_dep_launch();
    const float* v = hf + blockIdx.x * F;
    uint32_t mx = 0;
    for (int64_t f = threadIdx.x; f < F; f += 256) mx = max(mx, __float_as_uint(v[f]) & 0x7fffffffu);
    mx = __reduce_max_sync(0xffffffffu, mx);
    if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = mx;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = max(mx, top[i]);
    const uint32_t e = mx >> 23, field = e == 255u ? 127u : min(max(268u - e, 1u), 253u);
    const float scale = __uint_as_float(field << 23);
    uint16_t* o = h + blockIdx.x * Fp;
    for (int64_t f = threadIdx.x; f < F; f += 256) {
        float x = v[f] * scale;
#pragma unroll
        for (int i = 0; i < H_PLANES; ++i) {
            const __half b = __float2half_rn(x);
            o[i * P * Fp + f] = __half_as_ushort(b);
            x -= __half2float(b);
        }
    }
    if (threadIdx.x == 0) unscale[blockIdx.x] = __uint_as_float((254u - field) << 23);
}

// rows of 16-bit x copied to rows of Kp (zeros past K)
__global__ void __launch_bounds__(256) moe_copy_kernel(uint16_t* out, const uint16_t* x, int64_t T, int64_t K, int64_t Kp) {
    grid_dep_wait();
    grid_dep_launch();
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < T * Kp; i += gridDim.x * 256ll) {
        const int64_t t = i / Kp, k = i - t * Kp;
        out[i] = k < K ? x[t * K + k] : 0;
    }
}

// [rows][inner] of 16-bit (box 64 x box_rows) or 8-bit (box 128 x box_rows) elements, pitch bytes apart.
cudaError_t row_map(CUtensorMap* mp, bool bytes, const void* ptr, uint64_t inner, uint64_t rows, uint64_t pitch, uint32_t box_rows) {
    auto enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    cuuint64_t dims[2] = {inner, rows}, strides[1] = {pitch};
    cuuint32_t box[2] = {bytes ? 128u : 64u, box_rows}, es[2] = {1, 1};
    return enc(mp, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess : cudaErrorInvalidValue;
}
cudaError_t word_map(CUtensorMap* mp, const void* ptr, uint64_t pieces, uint64_t words) {
    auto enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    cuuint64_t dims[2] = {words, pieces}, strides[1] = {words * 4};
    cuuint32_t box[2] = {256, 1}, es[2] = {1, 1};
    return enc(mp, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess : cudaErrorInvalidValue;
}

// Scratch, part by part.
struct Room {
    int64_t x, xs, h, hs, hf, scale, part, bytes;  // offsets, and all
    int64_t places, Kp, Fp, Nq;
};
Room room(const MoeCall& m, bool fp4, bool copy_x, bool f16) {
    Room r{};
    const int64_t P = static_cast<int64_t>(m.T) * m.C;
    r.places = (plan_places(m.E, P, PLACES) + PLACES - 1) / PLACES * PLACES;
    r.Kp = fp4 ? fp4_padded(m.K) : (m.K + 63) / 64 * 64;
    r.Fp = fp4 ? fp4_padded(m.F) : (m.F + 7) / 8 * 8;
    r.Nq = (m.N + 127) / 128 * 128;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t o = at;
        at += round256(bytes);
        return o;
    };
    const int64_t rows = r.places * PARTS;
    r.x = take(fp4 ? rows * (r.Kp / 2) : copy_x ? m.T * r.Kp * 2 : 0);
    r.xs = take(fp4 ? rows / 128 * r.Kp * 4 : 0);
    r.h = take(fp4 ? rows * (r.Fp / 2) : H_PLANES * P * r.Fp * 2);
    r.hs = take(fp4 ? rows / 128 * r.Fp * 4 : 0);
    r.hf = take(fp4 ? r.places * m.F * 4 : f16 ? P * m.F * 4 : 0);
    r.scale = take(!fp4 && f16 ? P * 4 : 0);
    r.part = take(P * r.Nq * 4);
    r.bytes = at;
    return r;
}

template <bool FP4, bool OUT>
cudaError_t launch(const LaunchCtx& c, TcArgs a, const CUtensorMap& a0, const CUtensorMap& a1, const CUtensorMap& b, const CUtensorMap& sb,
                   const CUtensorMap& b8) {
    auto kern = moe_tc_kernel<FP4, OUT>;
    static PerDeviceOnce setup;
    cudaError_t e = setup.run(c.eng->device, [&](int&) {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T_LIMIT);
    });
    if (e != cudaSuccess) return e;
    const int64_t rows = OUT ? a.m.N : a.m.F, len = OUT ? a.m.F : a.m.K;
    const int span = !OUT && a.m.gate ? 64 : 128;
    a.tiles = static_cast<int>((rows + span - 1) / span);
    a.chunks = static_cast<int>(FP4 ? fp4_padded(len) / 256 : (len + 63) / 64);
    const MoeRing ring = moe_ring(FP4, OUT, a.m.T, a.P, a.m.E);
    a.cap = ring.cap;
    a.passes = ring.passes;
    a.stage = ring.stage;
    a.depth = ring.depth;
    if (a.depth < 2) return cudaErrorInvalidConfiguration;
    const int64_t units = static_cast<int64_t>(a.tiles) * a.passes;  // at most
    e = launch_pdl(kern, dim3(static_cast<unsigned>(lmin(units, c.sm_count))), dim3(t_threads(FP4)), static_cast<size_t>(ring.fixed + a.depth * a.stage),
                   c.stream, a0, a1, b, sb, b8, a);
    if (e != cudaSuccess) return e;
    c.count();
    return cudaGetLastError();
}

template <typename T, bool BY_PLACE>
cudaError_t parts(const LaunchCtx& c, const MoeCall& m, const T* x, uint8_t* xq, uint8_t* xs, int T_, int C, int64_t K) {
    const int64_t P = static_cast<int64_t>(T_) * C, smem = plan_bytes(m.E, P, PLACES) + (2 * P + 15) / 16 * 16;
    static PerDeviceOnce setup;
    const cudaError_t q = setup.run(c.eng->device, [&](int&) {
        return cudaFuncSetAttribute(moe_parts_kernel<T, BY_PLACE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(plan_bytes(MOE_MAX_E, MOE_MAX_PAIRS, PLACES) + 2 * MOE_MAX_PAIRS));
    });
    if (q != cudaSuccess) return q;
    const int64_t blocks = (T_ * (fp4_padded(K) / 128) + X_THREADS / 32 - 1) / (X_THREADS / 32);
    const cudaError_t e = launch_pdl(moe_parts_kernel<T, BY_PLACE>, dim3(static_cast<unsigned>(lmin(blocks, 8 * c.sm_count))), dim3(X_THREADS),
                                     static_cast<size_t>(smem), c.stream, x, m.ids, xq, xs, T_, C, m.E, K);
    if (e == cudaSuccess) c.count();
    return e;
}

template <bool FP4>
cudaError_t moe_form(const LaunchCtx& c, const MoeCall& m, bool copy_x, bi_dtype dt, uint8_t* scratch) {
    const bool f16 = !FP4 && dt == BI_F16;
    const Room r = room(m, FP4, copy_x, f16);
    TcArgs a{};
    a.m = m;
    a.P = m.T * m.C;
    a.h = reinterpret_cast<uint16_t*>(scratch + r.h);
    a.part = reinterpret_cast<float*>(scratch + r.part);
    a.Fp = r.Fp;
    a.Nq = r.Nq;
    a.fmt = dt == BI_BF16;
    if (FP4 || f16) a.hf = reinterpret_cast<float*>(scratch + r.hf);
    a.status = c.status;
    a.wait_limit = c.wait_limit_ns;
    CUtensorMap gate, up, down, mx, mh, mx8, mh8, sx, sh;
    cudaError_t e;
    const int64_t rows = r.places * PARTS, ef = m.E * m.F, en = m.E * m.N;
    if (FP4) {
        uint8_t *xq = scratch + r.x, *xs = scratch + r.xs;
        e = dt == BI_F32    ? parts<float, false>(c, m, static_cast<const float*>(m.x), xq, xs, m.T, m.C, m.K)
            : dt == BI_BF16 ? parts<__nv_bfloat16, false>(c, m, static_cast<const __nv_bfloat16*>(m.x), xq, xs, m.T, m.C, m.K)
                            : parts<__half, false>(c, m, static_cast<const __half*>(m.x), xq, xs, m.T, m.C, m.K);
        if (e != cudaSuccess) return e;
        if ((e = row_map(&up, true, m.up, r.Kp / 2, ef, r.Kp / 2, 64)) != cudaSuccess) return e;
        if (m.gate && (e = row_map(&gate, true, m.gate, r.Kp / 2, ef, r.Kp / 2, 64)) != cudaSuccess) return e;
        if ((e = row_map(&down, true, m.down, r.Fp / 2, en, r.Fp / 2, 64)) != cudaSuccess) return e;
        if ((e = row_map(&mx, true, xq, r.Kp / 2, rows, r.Kp / 2, 16)) != cudaSuccess) return e;
        if ((e = row_map(&mh, true, scratch + r.h, r.Fp / 2, rows, r.Fp / 2, 16)) != cudaSuccess) return e;
        if ((e = row_map(&mx8, true, xq, r.Kp / 2, rows, r.Kp / 2, 128)) != cudaSuccess) return e;
        if ((e = row_map(&mh8, true, scratch + r.h, r.Fp / 2, rows, r.Fp / 2, 128)) != cudaSuccess) return e;
        if ((e = word_map(&sx, xs, rows / 128, r.Kp)) != cudaSuccess) return e;
        if ((e = word_map(&sh, scratch + r.hs, rows / 128, r.Fp)) != cudaSuccess) return e;
    } else {
        const void* x = m.x;
        int64_t pitch = m.K;
        if (copy_x) {
            uint16_t* xc = reinterpret_cast<uint16_t*>(scratch + r.x);
            e = launch_pdl(moe_copy_kernel, dim3(static_cast<unsigned>(lmin((m.T * r.Kp + 255) / 256, 4 * c.sm_count))), dim3(256), 0, c.stream, xc,
                           static_cast<const uint16_t*>(m.x), static_cast<int64_t>(m.T), m.K, r.Kp);
            if (e != cudaSuccess) return e;
            c.count();
            x = xc;
            pitch = r.Kp;
        }
        if ((e = row_map(&up, false, m.up, m.K, ef, m.K * 2, 64)) != cudaSuccess) return e;
        if (m.gate && (e = row_map(&gate, false, m.gate, m.K, ef, m.K * 2, 64)) != cudaSuccess) return e;
        if ((e = row_map(&down, false, m.down, m.F, en, m.F * 2, 64)) != cudaSuccess) return e;
        if ((e = row_map(&mx, false, x, m.K, m.T, pitch * 2, 16)) != cudaSuccess) return e;
        if ((e = row_map(&mh, false, a.h, m.F, static_cast<int64_t>(H_PLANES) * a.P, r.Fp * 2, 16)) != cudaSuccess) return e;
        if ((e = row_map(&mx8, false, x, m.K, m.T, pitch * 2, 128)) != cudaSuccess) return e;
        if ((e = row_map(&mh8, false, a.h, m.F, static_cast<int64_t>(H_PLANES) * a.P, r.Fp * 2, 128)) != cudaSuccess) return e;
        sx = sh = mx;
    }
    if (!m.gate) gate = up;
    if ((e = launch<FP4, false>(c, a, gate, up, mx, sx, mx8)) != cudaSuccess) return e;
    if (FP4 && (e = parts<float, true>(c, m, a.hf, scratch + r.h, scratch + r.hs, a.P, 1, m.F)) != cudaSuccess) return e;
    if (f16) {
        float* unscale = reinterpret_cast<float*>(scratch + r.scale);
        e = launch_pdl(moe_planes_kernel, dim3(static_cast<unsigned>(a.P)), dim3(256), 0, c.stream, a.h, unscale, a.hf, m.F, a.Fp, a.P);
        if (e != cudaSuccess) return e;
        c.count();
        a.unscale = unscale;
    }
    if ((e = launch<FP4, true>(c, a, down, down, mh, sh, mh8)) != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>((m.T * ((m.N + 3) / 4) + 127) / 128));
    auto sum = [&](auto* y) {
        auto kern = moe_sum_kernel<std::remove_pointer_t<decltype(y)>>;
        return launch_pdl(kern, grid, dim3(128), 0, c.stream, y, a.part, m.ids, m.weights, m.T, m.C, m.E, m.N, a.Nq);
    };
    e = dt == BI_F32 ? sum(static_cast<float*>(m.y)) : dt == BI_BF16 ? sum(static_cast<__nv_bfloat16*>(m.y)) : sum(static_cast<__half*>(m.y));
    if (e != cudaSuccess) return e;
    c.count();
    return cudaGetLastError();
}

}  // namespace

int64_t moe_tc_scratch_bytes(const MoeCall& m, bool fp4, bool copy_x, bi_dtype dt) { return room(m, fp4, copy_x, dt == BI_F16).bytes; }

cudaError_t moe_tc(const LaunchCtx& c, const MoeCall& m, bool fp4, bool copy_x, bi_dtype dt, void* scratch) {
    return fp4 ? moe_form<true>(c, m, copy_x, dt, static_cast<uint8_t*>(scratch)) : moe_form<false>(c, m, copy_x, dt, static_cast<uint8_t*>(scratch));
}

}  // namespace bi
