// Low-rank adapters on the tensor cores: the narrow product (h and u) and the
// adapters' gradients.  The wide product runs inside the projection's own kernel
// (tc.cu, mode ADAPTER).
#include "adapter.h"
#include "adapter_parts.cuh"
#include "adapter_plan.cuh"
#include "tc_common.cuh"

namespace bi {
namespace {

constexpr int BK = 64;  // contraction block: one 128-byte swizzle row of 16-bit data

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar, uint32_t lead) {
    asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar), "r"(lead)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
template <int COLS>
__device__ __forceinline__ void tmem_alloc(uint32_t slot) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <int COLS>
__device__ __forceinline__ void tmem_free(uint32_t base) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(COLS) : "memory");
}
// kind::f16, f32 accumulation; format 0 f16, 1 bf16.
__device__ __forceinline__ uint32_t instr_desc(int fmt, bool a_mn, bool b_mn, int n, int m = 128) {
    const uint32_t f = static_cast<uint32_t>(fmt);
    return (1u << 4) | (f << 7) | (f << 10) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// One 64-wide contraction block: four K = 16 MMAs, the operands' descriptors (low
// words; the high words do not change) advancing by astep, bstep.  The issuing
// thread's own instructions are what a small tile waits for (a block's four MMAs
// of N = 64 take 130 cycles), so this is one asm statement without 64-bit
// arithmetic.
__device__ __forceinline__ void mma_block(uint32_t d_tmem, uint32_t a, uint32_t ahi, uint32_t astep, uint32_t b, uint32_t bhi,
                                          uint32_t bstep, uint32_t idesc, uint32_t acc, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, q, e;\n\t.reg .b64 da, db;\n\t.reg .b32 x, y;\n\t"
        "setp.ne.b32 p, %8, 0;\n\tsetp.eq.b32 q, 0, 0;\n\tsetp.ne.b32 e, %9, 0;\n\t"
        "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%4, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %7, p;\n\t"
        "add.u32 x, %1, %3;\n\tadd.u32 y, %4, %6;\n\tmov.b64 da, {x, %2};\n\tmov.b64 db, {y, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %7, q;\n\t"
        "add.u32 x, x, %3;\n\tadd.u32 y, y, %6;\n\tmov.b64 da, {x, %2};\n\tmov.b64 db, {y, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %7, q;\n\t"
        "add.u32 x, x, %3;\n\tadd.u32 y, y, %6;\n\tmov.b64 da, {x, %2};\n\tmov.b64 db, {y, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %7, q;\n\t}\n" ::"r"(d_tmem),
        "r"(a), "r"(ahi), "r"(astep), "r"(b), "r"(bhi), "r"(bstep), "r"(idesc), "r"(acc), "r"(lead)
        : "memory");
}
// Before a CTA that gave up (a wait ran out) lets its shared memory go, it waits for
// the copies it has issued: the last min(issued, stages) fills, fill f on stage f %
// stages in phase f / stages.
template <typename Bar>
__device__ __forceinline__ void drain_copies(Bar&& full_bar, int issued, int stages) {
    for (int f = max(0, issued - stages); f < issued; ++f) mbar_drain(full_bar(f % stages), (f / stages) & 1);
}
// The MMAs issued by the electing lane have finished before the CTA goes on.
template <typename P>
__device__ __forceinline__ void drain_mmas(uint32_t bar, uint32_t lead, volatile int* abort_flag, const P& p) {
    mma_commit(bar, lead);
    if (!mbar_wait_fast(bar, 0, abort_flag, p, DEV_TIMEOUT_MMA)) mbar_drain(bar, 0);
}

// ---------------------------------------------------------------- narrow product
//
// A CTA takes 128 rows and one 512-element piece of the contraction, and for
// these the adapters among its rows, four groups of 16 ranks (64 accumulator
// columns) at a time: D [128 rows x 64] += X [128 x 64] P^T, P the groups' rows
// stacked.  Every row is multiplied with every adapter of the tile, and reads
// back its own adapter's columns; the other products are thrown away.  With rows in
// runs, a few adapters to a tile, they are free: the pass is bound by reading X
// once (8192 rows of 4096: 67 MB, 10 us at the copy rate) and the tensor cores idle
// beside it, while sorting the rows first would read and write X once more.  They
// are not where a tile's rows have many adapters: X passes through shared memory
// once per four groups, ceil(adapters ceil(R / 16) / 4) times, and the wide product
// takes as many masked MMAs (8192 rows of 4096 x 4096 in random order, the whole
// forward: 64 adapters of rank 16 417 us, 128 of rank 256 3600, in runs 163 and 316).
// 128 rows x 512 elements is a unit
// small enough that a batch of 8192 rows gives 512 of them, and one of 64 rows
// with an own adapter each 128.
//
// Roles: warp 0 TMA, warp 1 MMA, warps 2-5 plan and epilogue; two CTAs per SM, so
// one CTA's set-up and drain run beside the other's loads.  Every CTA finds its
// tile's adapters itself, while the first blocks of X are on their way (a kernel
// of its own took 3 to 9 us before this one could start); the first CTA of each
// tile leaves them in the plan for the kernels after.
constexpr int NP_THREADS = 192, NP_STAGES = 4;
constexpr int NP_A = 128 * 128, NP_B = 64 * 128, NP_STAGE = NP_A + NP_B;
constexpr int NP_BARS = 2 * NP_STAGES + 6;
constexpr int NP_SMEM = 1024 + NP_STAGES * NP_STAGE + static_cast<int>(sizeof(PlanSmem)) + NP_BARS * 8 + 16 + 128 * 8 + 256;
static_assert(NP_SMEM <= 113 * 1024, "two CTAs per SM");
constexpr int NP_KB = static_cast<int>(ADAPTER_PIECE / BK);

struct NarrowParams {
    AdapterPlan plan;
    const uint32_t* ids;
    uint32_t G;
    float* partial;
    int64_t M;
    int R, rp, num_kb, fmt;
    int* status;
    unsigned long long wait_limit;
};

__global__ void __launch_bounds__(NP_THREADS, 2)
    narrow_tc_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmP, const NarrowParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t sbase = smem_u32(smem);
    PlanSmem& pl = *reinterpret_cast<PlanSmem*>(smem + NP_STAGES * NP_STAGE);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + NP_STAGES * NP_STAGE + sizeof(PlanSmem));
    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (NP_STAGES + s); };
    auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * NP_STAGES + b); };
    auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * NP_STAGES + 2 + b); };
    const uint32_t drain_bar = bar0 + 8u * (2 * NP_STAGES + 4), list_bar = drain_bar + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NP_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile uint32_t* s_count = tmem_slot + 2;
    uint32_t* s_ent = tmem_slot + 4;  // the tile's entries with a row in this half: their masks' place
    uint32_t* s_id = s_ent + 128;     // ... and adapter

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int64_t tile = blockIdx.x >> 1;
    const int half = blockIdx.x & 1;
    const int row0 = static_cast<int>(blockIdx.x) * 128;
    if (threadIdx.x == 0) {
        for (int s = 0; s < NP_STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 4);
        }
        mbar_init(drain_bar, 1);
        mbar_init(list_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<128>(smem_u32(tmem_slot));
    tc_fence_before();
    __syncthreads();  // this CTA has its TMEM before a dependent kernel may start and ask for some
    tc_fence_after();
    grid_dep_wait();
    grid_dep_launch();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(tmem_slot), 0);
    const int rg = p.rp / 16;  // groups of 16 ranks per adapter
    const int pieces = (p.num_kb + NP_KB - 1) / NP_KB;  // this CTA's: blockIdx.y, + gridDim.y, ...
    int fills = 0;  // stages the producer has filled
    auto piece_blocks = [&](int piece) { return min(NP_KB, p.num_kb - piece * NP_KB); };

    if (warp == 0) {  // a lane for each of a stage's copies, as in the small tiles' kernel below
        // the first blocks of X need no list: their bytes are expected and the
        // copies issued now, the stages' own arrivals follow with the adapters'
        // (the first CTA of a tile and piece; others may have no adapters left)
        const int early = blockIdx.z == 0 ? min(NP_STAGES, piece_blocks(blockIdx.y)) : 0;
        if (lane < early) {
            asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(full_bar(lane)), "r"(NP_A) : "memory");
            tma_load_2d(sbase + lane * NP_STAGE, &tmX, (static_cast<int>(blockIdx.y) * NP_KB + lane) * BK, row0, full_bar(lane));
        }
        __syncwarp();
        const bool listed = __all_sync(0xffffffffu, mbar_wait_fast(list_bar, 0, abort_flag, p, DEV_TIMEOUT_PRODUCER));
        const int groups = listed ? static_cast<int>(*s_count) * rg : 0, batches = (groups + 3) / 4;
        int s = 0;
        uint32_t ph = 0;
        if (static_cast<int>(blockIdx.z) >= batches && lane == 0) {  // nothing to multiply: let the early copies land
            for (int kb = 0; kb < early; ++kb) mbar_expect_tx(full_bar(kb), 0);
            drain_copies(full_bar, early, NP_STAGES);
        }
        for (int piece = blockIdx.y; piece < pieces; piece += gridDim.y)
        for (int q = blockIdx.z; q < batches; q += gridDim.z) {
            const int n = min(4, groups - 4 * q);
            const int gi = 4 * q + lane, e = gi / rg, r16 = (gi - e * rg) * 16;
            const int g = lane < n ? static_cast<int>(s_id[e]) : 0;
            const int kb0 = piece * NP_KB, nkb = piece_blocks(piece);
            for (int kb = 0; kb < nkb; ++kb) {
                const uint32_t a = sbase + s * NP_STAGE;
                const bool have_x = fills < early;
                if (!have_x && !__all_sync(0xffffffffu, mbar_wait_fast(empty_bar(s), ph ^ 1u, abort_flag, p, DEV_TIMEOUT_PRODUCER)))
                    goto done_p;
                if (lane == 0) mbar_expect_tx(full_bar(s), (have_x ? 0 : NP_A) + n * 2048);
                __syncwarp();
                if (!have_x && lane == 4) tma_load_2d(a, &tmX, (kb0 + kb) * BK, row0, full_bar(s));
                if (lane < n) tma_load_3d(a + NP_A + lane * 2048, &tmP, (kb0 + kb) * BK, r16, g, full_bar(s));
                ++fills;
                if (++s == NP_STAGES) { s = 0; ph ^= 1u; }
            }
        }
    done_p:;
    } else if (warp == 1) {
        const uint32_t lead = elect_lane();
        const bool listed = __all_sync(0xffffffffu, mbar_wait_fast(list_bar, 0, abort_flag, p, DEV_TIMEOUT_MMA));
        const int groups = listed ? static_cast<int>(*s_count) * rg : 0, batches = (groups + 3) / 4;
        int s = 0, ab = 0;
        uint32_t ph = 0, aph = 0;
        for (int piece = blockIdx.y; piece < pieces; piece += gridDim.y)
        for (int q = blockIdx.z; q < batches; q += gridDim.z) {
            const int nkb = piece_blocks(piece);
            const uint32_t idesc = instr_desc(p.fmt, false, false, 16 * min(4, groups - 4 * q));
            if (!__all_sync(0xffffffffu, mbar_wait_fast(tempty_bar(ab), aph ^ 1u, abort_flag, p, DEV_TIMEOUT_MMA))) goto done_m;
            tc_fence_after();
            for (int kb = 0; kb < nkb; ++kb) {
                if (!__all_sync(0xffffffffu, mbar_wait_fast(full_bar(s), ph, abort_flag, p, DEV_TIMEOUT_MMA))) goto done_m;
                tc_fence_after();
                const uint32_t a = sbase + s * NP_STAGE, b = a + NP_A;
                mma_block(tmem_base + ab * 64, desc_lo(a, false), DESC_HI, K_STEP, desc_lo(b, false), DESC_HI, K_STEP, idesc,
                          kb != 0 ? 1u : 0u, lead);
                mma_commit(empty_bar(s), lead);
                if (++s == NP_STAGES) { s = 0; ph ^= 1u; }
            }
            mma_commit(tfull_bar(ab), lead);
            if (++ab == 2) { ab = 0; aph ^= 1u; }
        }
    done_m:
        // the MMAs issued above have finished before the CTA leaves, and with
        // them the copies they waited for
        drain_mmas(drain_bar, lead, abort_flag, p);
    } else if (warp >= 2) {
        const int w = warp & 3;  // the TMEM lanes a warp may read
        auto sync4 = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
        plan_tile<4>(p.ids, p.M, p.G, tile, warp - 2, pl, sync4);
        if (half == 0 && blockIdx.y == 0 && blockIdx.z == 0) plan_store(p.plan, tile, pl, threadIdx.x - 64, 128);
        if (warp == 2) {  // those with a row in this CTA's half
            uint32_t total = 0;
            for (uint32_t i0 = 0; i0 < pl.count; i0 += 32) {
                const uint32_t i = i0 + lane;
                const uint32_t place = i < pl.count ? pl.slot[i] : 0;
                const uint4 m = i < pl.count ? pl.masks[place][half] : make_uint4(0, 0, 0, 0);
                const bool has = (m.x | m.y | m.z | m.w) != 0;
                const uint32_t b = __ballot_sync(0xffffffffu, has);
                if (has) {
                    const uint32_t at = total + __popc(b & ((1u << lane) - 1));
                    s_ent[at] = place;
                    s_id[at] = pl.ids[i];
                }
                total += __popc(b);
            }
            if (lane == 0) *s_count = total;
            __syncwarp();
            if (lane == 0) mbar_arrive(list_bar);
        }
        sync4();
        const int groups = static_cast<int>(*s_count) * rg, batches = (groups + 3) / 4;
        const int64_t row = row0 + 32 * w + lane;
        int ab = 0;
        uint32_t aph = 0;
        bool going = true;
        for (int piece = blockIdx.y; piece < pieces && going; piece += gridDim.y)
        for (int q = blockIdx.z; q < batches; q += gridDim.z) {
            const int n = min(4, groups - 4 * q);
            bool ok = mbar_wait_fast(tfull_bar(ab), aph, abort_flag, p, DEV_TIMEOUT_EPILOGUE);
            going = __all_sync(0xffffffffu, ok);
            if (!going) break;
            tc_fence_after();
            for (int i = 0; i < n; ++i) {
                const int gi = 4 * q + i;
                const uint32_t mask = reinterpret_cast<const uint32_t*>(&pl.masks[s_ent[gi / rg]][half])[w];
                if (mask == 0) continue;  // the same for the whole warp
                __syncwarp();
                uint32_t v[16];
                tmem_ld16(tmem_base + (static_cast<uint32_t>(32 * w) << 16) + ab * 64 + 16 * i, v);
                if ((mask >> lane) & 1u) {
                    float4* dst = reinterpret_cast<float4*>(p.partial + (static_cast<int64_t>(piece) * p.M + row) * p.rp +
                                                            (gi % rg) * 16);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        dst[j] = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                             __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty_bar(ab));
            if (++ab == 2) { ab = 0; aph ^= 1u; }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort_flag != 0 && threadIdx.x == 0) drain_copies(full_bar, fills, NP_STAGES);
    if (warp == 1) {
        tc_fence_after();
        tmem_free<128>(tmem_base);
    }
}

// ---------------------------------------------------------------- small tiles
//
// The projection with its adapters' terms by tiles of 128 rows x 64 columns, one
// per CTA (cta_group::1), for few rows or narrow outputs.  A decoding batch is
// bound by reading W once (4096 x 4096: 33.5 MB, 5 us at the copy rate); 256-column
// tiles would read it with a quarter of the SMs.  Every output element is the
// same chain as in the CTA-pair kernel (64-wide blocks of the contraction
// ascending, then the adapter's ranks ascending, high part before remainder), so
// its bits are the same.  Measured, bf16 4096 x 4096, rank 16: see
// adapter_small_tiles.
//
// Up to 64 rows take MMAs of 64 rows, which read half as much of A: a block's MMAs
// of M = 128, N = 64 are bound by their operands' reads from shared memory.
// The rows' inner products (up to rank 64) stay in shared memory, and a ring
// stage then carries four adapters' 16 ranks of B: a batch in which every row has
// an adapter of its own reads little besides these.
//
// Where the pieces of h are few (up to SM_FUSE sums for the tile's rows) the
// epilogue warps add them up and lay them out in shared memory themselves, in the
// finish kernel's order, and the first CTA of the row writes h: one launch less.
//
// The base product needs nothing of the kernel just before this one, so it starts
// under it (programmatic launch): only the adapters' part waits for that kernel
// (grid_dep_wait).  x and w are complete, because the narrow product (and the
// finish kernel) waited for whatever came before it ere it let this one start: this
// kernel is launched behind one of these two only.  The kernel behind it is let in
// after that wait, like everywhere.
constexpr int SM_THREADS = 192, SM_COLS = 64, SM_B = 64 * 128, SM_MAX_STAGES = 12;
constexpr int SM_BARS = 2 * SM_MAX_STAGES + 3;
constexpr int SM_TAIL = SM_BARS * 8 + 16 + 128 * 4 + 128 * 16 + 64;  // barriers, slots, adapter list and masks, rows beyond f16

struct SmallParams {
    AdapterPlan plan;
    void* out;
    const void* bias;
    int64_t M, C;
    AdapterFar far;  // the pieces of h and what makes s h of them (fused), and the terms beyond f16
    float* h;        // fused
    uint32_t G;
    int fused;
    int a_bytes;  // of one A tile's rows that exist (a multiple of 8 rows)
    int R, num_kb, stages, resident;  // resident: 32-rank parts of h kept in shared memory (0: streamed)
    int* status;
    unsigned long long wait_limit;
};

// Sixteen ranks of one adapter: the high parts' MMA and the remainders' (64 bytes on
// in the rows of h), on the accumulator lanes that `off` does not exclude.
__device__ __forceinline__ void mma_masked(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint4 off, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t.reg .b32 x;\n\t"
        "setp.eq.b32 p, 0, 0;\n\tsetp.ne.b32 e, %9, 0;\n\t"
        "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, {%5, %6, %7, %8}, p;\n\t"
        "add.u32 x, %1, 4;\n\tmov.b64 da, {x, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, {%5, %6, %7, %8}, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a), "r"(b), "r"(DESC_HI), "r"(idesc), "r"(off.x), "r"(off.y), "r"(off.z), "r"(off.w), "r"(lead)
        : "memory");
}

template <int FMT, int AR, bool B_MN>
__global__ void __launch_bounds__(SM_THREADS, 1)
    small_rows_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                      const __grid_constant__ CUtensorMap tmH, const __grid_constant__ CUtensorMap tmQ, const SmallParams p) {
    constexpr int A_BYTES = AR * 128, STAGE = A_BYTES + SM_B;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t sbase = smem_u32(smem);
    const int stages = p.stages;
    const uint32_t hbase = sbase + stages * STAGE;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + stages * STAGE + p.resident * A_BYTES);
    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (SM_MAX_STAGES + s); };
    const uint32_t done_bar = bar0 + 8u * (2 * SM_MAX_STAGES), h_bar = done_bar + 8, list_bar = done_bar + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + SM_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile uint32_t* s_count = tmem_slot + 2;
    // per adapter of this half the accumulator lanes that are not its rows', and its index
    uint4* s_off = reinterpret_cast<uint4*>((reinterpret_cast<uintptr_t>(tmem_slot + 4) + 15) & ~uintptr_t(15));
    uint32_t* s_id = reinterpret_cast<uint32_t*>(s_off + 128);
    uint32_t* s_over = s_id + 128;  // fused: a bit per row with a rank beyond f16
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int row0 = static_cast<int>(blockIdx.y) * 128, col0 = static_cast<int>(blockIdx.x) * SM_COLS;
    const int rg = (p.R + 15) / 16;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(done_bar, 1);
        mbar_init(h_bar, 1);
        mbar_init(list_bar, 1);
        *abort_flag = 0;
        for (int i = 0; i < 4; ++i) s_over[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<64>(smem_u32(tmem_slot));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(tmem_slot), 0);
    int issued = 0;  // stages the producer has filled
    bool h_issued = false;

    if (warp == 0) {
        // the whole warp runs this: lane 0 expects a stage's bytes, then a lane for
        // each of its copies issues them side by side (one lane issuing four copies
        // per stage, with their addresses, took 0.2 us a copy)
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        auto claim = [&](uint32_t bytes) {  // the next stage, free and expecting `bytes`
            ok = __all_sync(0xffffffffu, mbar_wait_fast(empty_bar(s), ph ^ 1u, abort_flag, p, DEV_TIMEOUT_PRODUCER));
            if (!ok) return;
            ++issued;
            if (lane == 0) mbar_expect_tx(full_bar(s), bytes);
            __syncwarp();
        };
        auto advance = [&] {
            if (++s == stages) { s = 0; ph ^= 1u; }
        };
        const CUtensorMap* map = lane == 0 ? &tmX : &tmW;
        const uint32_t to = sbase + (lane == 0 ? 0 : A_BYTES);
        const uint32_t bytes = p.a_bytes + SM_B;
        for (int kb = 0; kb < p.num_kb && ok; ++kb) {
            claim(bytes);
            if (!ok) break;
            const int kx = kb * BK;
            if (lane < 2) tma_load_2d(to + s * STAGE, map, B_MN && lane ? col0 : kx, lane == 0 ? row0 : (B_MN ? kx : col0), full_bar(s));
            advance();
        }
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait_fast(list_bar, 0, abort_flag, p, DEV_TIMEOUT_PRODUCER));
        if (ok) {
            grid_dep_wait();
            const int steps = static_cast<int>(*s_count) * rg;
            if (p.resident && steps) {
                h_issued = !p.fused;
                if (h_issued && lane == 0) {
                    mbar_expect_tx(h_bar, p.resident * p.a_bytes);
                    for (int c = 0; c < p.resident; ++c) tma_load_2d(hbase + c * A_BYTES, &tmH, c * 64, row0, h_bar);
                }
                for (int f = 0; f < steps && ok; f += 4) {
                    const int n = min(4, steps - f);
                    const int e = (f + lane) / rg, jr = f + lane - e * rg;
                    const int g = lane < n ? static_cast<int>(s_id[e]) : 0;
                    claim(n * 2048);
                    if (!ok) break;
                    if (lane < n) tma_load_3d(sbase + s * STAGE + A_BYTES + lane * 2048, &tmQ, col0, jr * 16, g, full_bar(s));
                    advance();
                }
            } else {
                for (int f = 0; f < steps && ok;) {  // one 32-rank part of one adapter
                    const int e = f / rg, jr = f - e * rg, n = min(2, rg - jr);
                    claim(p.a_bytes + n * 2048);
                    if (!ok) break;
                    const uint32_t a = sbase + s * STAGE;
                    if (lane < n) tma_load_3d(a + A_BYTES + lane * 2048, &tmQ, col0, (jr + lane) * 16, static_cast<int>(s_id[e]), full_bar(s));
                    if (lane == n) tma_load_2d(a, &tmH, (jr / 2) * 64, row0, full_bar(s));
                    f += n;
                    advance();
                }
            }
        }
    } else if (warp == 1) {
        const uint32_t idesc = instr_desc(FMT, false, B_MN, SM_COLS, AR), idesc_q = instr_desc(FMT, false, true, SM_COLS, AR);
        // the whole warp runs this, one lane issues: warp-uniform code keeps the
        // descriptors in uniform registers, where the MMA takes them from
        const uint32_t lead = elect_lane();
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        auto take = [&] {
            ok = __all_sync(0xffffffffu, mbar_wait_fast(full_bar(s), ph, abort_flag, p, DEV_TIMEOUT_MMA));
            tc_fence_after();
        };
        auto release = [&] {
            mma_commit(empty_bar(s), lead);
            if (++s == stages) { s = 0; ph ^= 1u; }
        };
        for (int kb = 0; kb < p.num_kb && ok; ++kb) {
            take();
            if (!ok) break;
            const uint32_t a = sbase + s * STAGE, b = a + A_BYTES;
            mma_block(tmem_base, desc_lo(a, false), DESC_HI, K_STEP, desc_lo(b, B_MN), DESC_HI, B_MN ? MN_STEP_16 : K_STEP, idesc,
                      kb != 0 ? 1u : 0u, lead);
            release();
        }
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait_fast(list_bar, 0, abort_flag, p, DEV_TIMEOUT_MMA));
        if (ok) {
            const int steps = static_cast<int>(*s_count) * rg;
            if (p.resident && steps) ok = __all_sync(0xffffffffu, mbar_wait_fast(h_bar, 0, abort_flag, p, DEV_TIMEOUT_MMA));
            // step f: 16-rank group jr of adapter e; four steps per stage (h resident),
            // or up to two of one 32-rank part
            const uint32_t h_desc = desc_lo(hbase, false);
            int e = 0, jr = 0;
            uint4 off = s_off[0], next = s_off[1];
            for (int f = 0; f < steps && ok;) {
                take();
                if (!ok) break;
                const uint32_t st = sbase + s * STAGE;
                const int n = p.resident ? min(4, steps - f) : min(2, rg - jr);
                const uint32_t a0 = p.resident ? h_desc : desc_lo(st, false), b0 = desc_lo(st + A_BYTES, true);
                for (int i = 0; i < n; ++i) {
                    const uint32_t part = p.resident ? static_cast<uint32_t>(jr >> 1) * (A_BYTES >> 4) : 0u;
                    mma_masked(tmem_base, a0 + part + (jr & 1) * K_STEP, b0 + i * MN_STEP_16, idesc_q, off, lead);
                    if (++jr == rg) {
                        jr = 0;
                        off = next;
                        next = s_off[min(++e + 1, 127)];
                    }
                }
                f += n;
                release();
            }
        }
        __syncwarp();
        drain_mmas(done_bar, lead, abort_flag, p);
    } else if (warp >= 2) {
        const int w = warp & 3;
        if (warp == 2) {  // the adapters of this half of the plan tile, in the plan's order
            grid_dep_wait();
            grid_dep_launch();
            const int64_t tile = blockIdx.y >> 1;
            const int half = blockIdx.y & 1;
            const uint32_t n = p.plan.count[tile];
            uint4 m[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                m[q] = q * 32 + lane < n
                           ? *reinterpret_cast<const uint4*>(p.plan.masks + (tile * ADAPTER_TILE + q * 32 + lane) * 8 + 4 * half)
                           : make_uint4(0, 0, 0, 0);
            uint32_t total = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const bool has = (m[q].x | m[q].y | m[q].z | m[q].w) != 0;
                const uint32_t b = __ballot_sync(0xffffffffu, has);
                if (has) {
                    const uint32_t at = total + __popc(b & ((1u << lane) - 1));
                    // 64 rows: row i is lane 32 (i / 16) + i % 16
                    s_off[at] = AR == 64 ? make_uint4(~m[q].x, ~(m[q].x >> 16), ~m[q].y, ~(m[q].y >> 16))
                                         : make_uint4(~m[q].x, ~m[q].y, ~m[q].z, ~m[q].w);
                    s_id[at] = p.plan.ids[tile * ADAPTER_TILE + q * 32 + lane];
                }
                total += __popc(b);
            }
            __syncwarp();
            if (lane == 0) {
                *s_count = total;
                mbar_arrive(list_bar);
            }
            __syncwarp();
        }
        constexpr int RPW = AR / 4;  // rows per warp: 32, or 16 in the first lanes of a 64-row tile's
        const int64_t row = row0 + RPW * w + lane;
        uint32_t over = 0;  // f16: this lane's row has terms beyond the MMAs'
        if (FMT == 0 && !p.fused) {
            grid_dep_wait();
            if (row < p.M) over = p.far.over[row >> 5];
        }
        if (p.fused) {  // s h of the tile's rows, 8 ranks (16 bytes of each part) per thread and turn
            grid_dep_wait();
            const int per_row = p.resident * 4;
            const int rows = static_cast<int>(lmin(AR, p.M - row0));
            for (int i = threadIdx.x - 64; i < rows * per_row; i += 128) {
                const int row = i / per_row, r0 = (i % per_row) * 8;
                const uint32_t g = p.far.ids[row0 + row];
                float v[8], sv[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = 0.0f;
                if (g < p.G && r0 < p.far.rp)
                    sum_pieces8(p.far.partial + static_cast<int64_t>(row0 + row) * p.far.rp + r0, p.M * p.far.rp, p.far.pieces, v);
                const float s = g < p.G && p.far.scales != nullptr ? p.far.scales[g] : 1.0f;
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const bool is_rank = r0 + u < p.R;  // past R the padding stays 0 whatever the scale
                    if (is_rank && p.h != nullptr && blockIdx.x == 0) p.h[static_cast<int64_t>(row0 + row) * p.R + r0 + u] = v[u];
                    sv[u] = is_rank ? v[u] * s : 0.0f;
                }
                uint32_t w_hi[4], w_lo[4];
                if (two_parts8<FMT>(sv, w_hi, w_lo)) atomicOr(&s_over[row >> 5], 1u << (row & 31));
                const uint32_t at = hbase + (r0 / 32) * A_BYTES + row * 128;
                const uint32_t c = (r0 % 32) / 8;  // 16-byte piece of the high parts; the remainders' is 4 on
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + ((c ^ (row & 7)) * 16)), "r"(w_hi[0]),
                             "r"(w_hi[1]), "r"(w_hi[2]), "r"(w_hi[3]) : "memory");
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + (((c + 4) ^ (row & 7)) * 16)), "r"(w_lo[0]),
                             "r"(w_lo[1]), "r"(w_lo[2]), "r"(w_lo[3]) : "memory");
            }
            fence_proxy_async_smem();
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (threadIdx.x == 64) mbar_arrive(h_bar);
            if (FMT == 0) over = s_over[(row - row0) >> 5];
        }
        const bool far = ((over >> (row & 31)) & 1u) != 0;
        bool ok = mbar_wait_fast(done_bar, 0, abort_flag, p, DEV_TIMEOUT_EPILOGUE);
        ok = __all_sync(0xffffffffu, ok && *abort_flag == 0);
        if (ok) {
            tc_fence_after();
            using O = OutT<FMT>;
            using T = typename O::T;
            T* dst = static_cast<T*>(p.out) + row * p.C + col0;
            if (row0 + RPW * w < p.M) {
#pragma unroll
                for (int c = 0; c < SM_COLS; c += 16) {
                    if (col0 + c >= p.C) break;
                    uint32_t v[16];
                    tmem_ld16(tmem_base + (static_cast<uint32_t>(32 * w) << 16) + c, v);
                    if (row < p.M && lane < RPW) {
                        float f[16];
                        const int have = static_cast<int>(lmin(16, p.C - col0 - c));  // 8 or 16
#pragma unroll
                        for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(v[i]);
                        if (FMT == 0 && far) {
                            float t[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) t[i] = f[i];
                            add_far_terms(p.far, row, col0 + c, t);
#pragma unroll
                            for (int i = 0; i < 16; ++i) f[i] = t[i];
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            if (p.bias != nullptr && i < have) f[i] = __fadd_rn(f[i], O::load(p.bias, col0 + c + i));
                        }
#pragma unroll
                        for (int i = 0; i < 16; i += 8)
                            if (i < have)
                                *reinterpret_cast<uint4*>(dst + c + i) =
                                    make_uint4(O::pack(f[i], f[i + 1]), O::pack(f[i + 2], f[i + 3]), O::pack(f[i + 4], f[i + 5]),
                                               O::pack(f[i + 6], f[i + 7]));
                    }
                    __syncwarp();
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort_flag != 0 && threadIdx.x == 0) {
        drain_copies(full_bar, issued, stages);
        if (h_issued) mbar_drain(h_bar, 0);
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_free<64>(tmem_base);
    }
}

constexpr int SM_LIMIT = 227 * 1024;  // shared memory of one CTA

template <int FMT, int AR, bool B_MN>
cudaError_t small_rows_t(const LaunchCtx& c, const CUtensorMap& x, const CUtensorMap& w, const CUtensorMap& h,
                         const CUtensorMap& q, SmallParams p, dim3 grid) {
    auto kern = small_rows_kernel<FMT, AR, B_MN>;
    static PerDeviceOnce setup;
    const cudaError_t e = setup.run(c.eng->device, [&](int&) {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SM_LIMIT);
    });
    if (e != cudaSuccess) return e;
    // a whole SM's shared memory where the tiles leave SMs over, else half
    const int budget = int64_t(grid.x) * grid.y <= c.sm_count ? SM_LIMIT : SM_LIMIT / 2 - 1024;
    constexpr int STAGE = AR * 128 + SM_B;
    const int pad = 1024 + SM_TAIL;  // alignment, barriers and lists
    p.resident = p.R <= 64 ? (p.R + 31) / 32 : 0;
    p.stages = min(SM_MAX_STAGES, (budget - pad - p.resident * AR * 128) / STAGE);
    const int bytes = pad + p.resident * AR * 128 + p.stages * STAGE;
    const cudaError_t r = launch_pdl(kern, grid, dim3(SM_THREADS), bytes, c.stream, x, w, h, q, p);
    if (r == cudaSuccess) c.count();
    return r;
}

template <int FMT>
cudaError_t small_rows_fmt(const LaunchCtx& c, int dx, int64_t M, const CUtensorMap& x, const CUtensorMap& w,
                           const CUtensorMap& h, const CUtensorMap& q, const SmallParams& p, dim3 grid) {
    if (M <= 64)
        return dx ? small_rows_t<FMT, 64, false>(c, x, w, h, q, p, grid) : small_rows_t<FMT, 64, true>(c, x, w, h, q, p, grid);
    return dx ? small_rows_t<FMT, 128, false>(c, x, w, h, q, p, grid) : small_rows_t<FMT, 128, true>(c, x, w, h, q, p, grid);
}

// ---------------------------------------------------------------- small tiles, f32
//
// The 3xTF32 product of the CTA-pair kernel (operands split into hi and lo parts,
// both K-major) by tiles of 128 rows x 64 columns on single CTAs: per 32-wide
// block and K = 8 step lo hi and hi lo into one accumulator, hi hi into another,
// in the pair kernel's order, so the bits are the same.  Two accumulators make two
// chains of dependent MMAs; a block takes 0.3 us of them, the pairs' 256 x 256
// tile 1.14 us.  999 x 1000 x 1000: 36 us on 16 pairs, 15 on 128 CTAs.
constexpr int SF_STAGE = 2 * (128 * 128 + SM_B), SF_STAGES = 4, SF_BARS = 2 * SF_STAGES + 1;
constexpr int SF_SMEM = 1024 + SF_STAGES * SF_STAGE + SF_BARS * 8 + 16;

struct SmallF32Params {
    float* out;
    const float* bias;
    int64_t M, C, ldo;
    int num_kb;
    int* status;
    unsigned long long wait_limit;
};

__device__ __forceinline__ void mma_tf32(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 e, %6, 0;\n\t"
        "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::tf32 [%0], da, db, %4, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a), "r"(b), "r"(DESC_HI), "r"(idesc), "r"(acc), "r"(lead)
        : "memory");
}

__global__ void __launch_bounds__(SM_THREADS, 1)
    small_f32_kernel(const __grid_constant__ CUtensorMap tmAh, const __grid_constant__ CUtensorMap tmAl,
                     const __grid_constant__ CUtensorMap tmBh, const __grid_constant__ CUtensorMap tmBl, const SmallF32Params p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t sbase = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SF_STAGES * SF_STAGE);
    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (SF_STAGES + s); };
    const uint32_t done_bar = bar0 + 8u * (2 * SF_STAGES);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + SF_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int row0 = static_cast<int>(blockIdx.y) * 128, col0 = static_cast<int>(blockIdx.x) * SM_COLS;
    constexpr int A_HI = 0, B_HI = 128 * 128, A_LO = B_HI + SM_B, B_LO = A_LO + 128 * 128;
    if (threadIdx.x == 0) {
        for (int s = 0; s < SF_STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<128>(smem_u32(tmem_slot));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(tmem_slot), 0);
    grid_dep_wait();
    grid_dep_launch();
    int issued = 0;  // stages the producer has filled
    if (warp == 0) {  // a lane for each of a block's four copies
        const CUtensorMap* map = lane == 0 ? &tmAh : lane == 1 ? &tmBh : lane == 2 ? &tmAl : &tmBl;
        const uint32_t to = sbase + (lane == 0 ? A_HI : lane == 1 ? B_HI : lane == 2 ? A_LO : B_LO);
        int s = 0;
        uint32_t ph = 0;
        for (int kb = 0; kb < p.num_kb; ++kb) {
            if (!__all_sync(0xffffffffu, mbar_wait_fast(empty_bar(s), ph ^ 1u, abort_flag, p, DEV_TIMEOUT_PRODUCER))) break;
            ++issued;
            if (lane == 0) mbar_expect_tx(full_bar(s), SF_STAGE);
            __syncwarp();
            if (lane < 4) tma_load_2d(to + s * SF_STAGE, map, kb * 32, lane & 1 ? col0 : row0, full_bar(s));
            if (++s == SF_STAGES) { s = 0; ph ^= 1u; }
        }
    } else if (warp == 1) {
        const uint32_t lead = elect_lane();
        const uint32_t idesc = instr_desc(2, false, false, SM_COLS);  // 2: tf32 in kind::tf32
        int s = 0;
        uint32_t ph = 0;
        for (int kb = 0; kb < p.num_kb; ++kb) {
            if (!__all_sync(0xffffffffu, mbar_wait_fast(full_bar(s), ph, abort_flag, p, DEV_TIMEOUT_MMA))) break;
            tc_fence_after();
            const uint32_t st = sbase + s * SF_STAGE;
            const uint32_t ah = desc_lo(st + A_HI, false), bh = desc_lo(st + B_HI, false), al = desc_lo(st + A_LO, false),
                           bl = desc_lo(st + B_LO, false);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const uint32_t acc = (kb | kk) != 0 ? 1u : 0u, o = kk * K_STEP;
                mma_tf32(tmem_base + SM_COLS, al + o, bh + o, idesc, acc, lead);
                mma_tf32(tmem_base + SM_COLS, ah + o, bl + o, idesc, 1u, lead);
                mma_tf32(tmem_base, ah + o, bh + o, idesc, acc, lead);
            }
            mma_commit(empty_bar(s), lead);
            if (++s == SF_STAGES) { s = 0; ph ^= 1u; }
        }
        drain_mmas(done_bar, lead, abort_flag, p);
    } else if (warp >= 2) {
        const int w = warp & 3;
        bool ok = mbar_wait_fast(done_bar, 0, abort_flag, p, DEV_TIMEOUT_EPILOGUE);
        ok = __all_sync(0xffffffffu, ok && *abort_flag == 0);
        if (ok && row0 + 32 * w < p.M) {
            tc_fence_after();
            const int64_t row = row0 + 32 * w + lane;
            float* dst = p.out + row * p.ldo + col0;
            const uint32_t t = tmem_base + (static_cast<uint32_t>(32 * w) << 16);
#pragma unroll
            for (int c = 0; c < SM_COLS; c += 16) {
                if (col0 + c >= p.C) break;
                uint32_t v[16], x[16];
                tmem_ld16(t + c, v);
                tmem_ld16(t + SM_COLS + c, x);
                if (row < p.M) {
                    float f[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        f[i] = __uint_as_float(v[i]);
                        // an infinite hi hi sum is the result: the cross terms of an
                        // infinite operand carry no value
                        if (!isinf(f[i])) f[i] = __fadd_rn(f[i], __uint_as_float(x[i]));
                        if (p.bias != nullptr && col0 + c + i < p.C) f[i] = __fadd_rn(f[i], p.bias[col0 + c + i]);
                    }
#pragma unroll
                    for (int i = 0; i < 16; i += 4)  // C is a multiple of 4
                        if (col0 + c + i < p.C) *reinterpret_cast<float4*>(dst + c + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
                }
                __syncwarp();
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort_flag != 0 && threadIdx.x == 0) drain_copies(full_bar, issued, SF_STAGES);
    if (warp == 1) {
        tc_fence_after();
        tmem_free<128>(tmem_base);
    }
}

// ---------------------------------------------------------------- gradients
//
// A CTA takes one chunk (at most 1024) of one adapter's sorted rows, 128 columns
// of z and up to 64 ranks: D [128 columns x 4 rank_run] += z^T v, both operands
// with the output index contiguous, 64 rows per block.  The rows lie anywhere in
// z: four warps copy them 16 bytes at a time (cp.async) into the swizzled tiles,
// rows past the chunk's end as zeros, so rows of other adapters are never read.
// v comes in four 16-bit parts whose products stand in columns of their own and
// are added at the end, and each 512 rows have an accumulator of their own (the
// tensor core's accumulation rounds towards zero, an error that grows with the
// length: dA of 8192 x 4096 rows was off by 1.3e-6 with one, 0.9e-6 with two), so
// dA and dB keep f32's precision.  z is read once per 64 ranks, which bounds the pass (8192 rows of 4096: 67 MB, 10 us at the copy
// rate); two CTAs per SM keep about 190 KB in flight.
constexpr int GT_THREADS = 160, GT_ROWS = 64;
constexpr int GT_A = 2 * 8192;  // 64 rows x 128 columns, two 64-column atoms
__host__ __device__ constexpr int gt_atoms(int run) { return 4 * run / 64; }
__host__ __device__ constexpr int gt_stage(int run) { return GT_A + gt_atoms(run) * 8192; }
// two CTAs per SM, or (more ranks, whose two accumulators fill the tensor memory) one
__host__ __device__ constexpr int gt_ctas(int run) { return run > 32 ? 1 : 2; }
__host__ __device__ constexpr int gt_stages(int run) { return (run > 32 ? 196608 : 98304) / gt_stage(run); }
__host__ __device__ constexpr int gt_smem(int run) { return 1024 + gt_stages(run) * gt_stage(run) + 256; }
static_assert(gt_stages(16) == 4 && gt_stages(32) == 3 && gt_stages(48) == 4 && gt_stages(64) == 4, "ring depths");
constexpr int GT_HALF = 8;  // blocks per accumulator

struct GradParams {
    AdapterGradJob job[2];  // v4 [M, vcols], z [M, C]
    const uint32_t* off;
    const uint32_t* perm;
    AdapterChunks ch;
    int64_t vcols;
    uint32_t chunk0, strips0, strips;  // block x: strip x % strips (job 0's first) of chunk chunk0 + x / strips
    int R, G, fmt;
    int* status;
    unsigned long long wait_limit;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
    const int n = in ? 16 : 0;  // 0: the 16 bytes are filled with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

template <int RUN>
__global__ void __launch_bounds__(GT_THREADS, gt_ctas(RUN)) grad_tc_kernel(const GradParams p) {
    constexpr int ATOMS = gt_atoms(RUN), STAGE = gt_stage(RUN), STAGES = gt_stages(RUN), LAG = STAGES - 1;
    constexpr int ACC = 4 * RUN <= 128 ? 4 * RUN : 256, COLS = 2 * ACC;  // TMEM columns of an accumulator, of both
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t sbase = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE);
    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    const uint32_t done_bar = bar0 + 8u * (2 * STAGES);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t chunk = p.chunk0 + blockIdx.x / p.strips;
    if (chunk >= p.ch.first[p.G]) return;
    int g = 0;  // the last adapter whose first chunk is <= chunk
    for (int hi = p.G - 1; g < hi;) {
        const int mid = (g + hi + 1) >> 1;
        if (p.ch.first[mid] <= chunk) g = mid; else hi = mid - 1;
    }
    const uint32_t j = chunk - p.ch.first[g], nchunks = p.ch.first[g + 1] - p.ch.first[g];
    const uint32_t s0 = p.off[g] + j * static_cast<uint32_t>(ADAPTER_CHUNK);
    const uint32_t s1 = min(p.off[g + 1], s0 + static_cast<uint32_t>(ADAPTER_CHUNK));
    const int blocks = static_cast<int>((s1 - s0 + GT_ROWS - 1) / GT_ROWS);
    const uint32_t strip = blockIdx.x % p.strips;
    const AdapterGradJob& jb = p.job[strip >= p.strips0];
    const int64_t C = jb.C;
    const int64_t c0 = static_cast<int64_t>(strip >= p.strips0 ? strip - p.strips0 : strip) * 128;
    const int r0 = blockIdx.y * 64;

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 128);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 4) tmem_alloc<COLS>(smem_u32(tmem_slot));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(tmem_slot), 0);

    if (warp < 4) {
        // thread t copies 16-byte piece t % 8 of each 128-byte atom row, rows t / 8 + 16 i
        const int piece = tid & 7, rr = tid >> 3;
        const uint32_t sw = static_cast<uint32_t>((piece ^ (rr & 7)) * 16);  // rr + 16 i has the same low bits
        const bool in0 = c0 + piece * 8 < C, in1 = c0 + 64 + piece * 8 < C;
        const uint16_t* z = static_cast<const uint16_t*>(jb.z);
        const uint16_t* zc = z + c0 + piece * 8;
        const uint16_t* vc = static_cast<const uint16_t*>(jb.v4) + static_cast<int64_t>(blockIdx.y) * (4 * RUN) + piece * 8;
        uint32_t row[4];
        auto rows_of = [&](int b) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t s = s0 + b * GT_ROWS + rr + 16 * i;
                row[i] = b < blocks && s < s1 ? p.perm[s] : 0xffffffffu;
            }
        };
        rows_of(0);
        bool ok = true;
        int st = 0, st_done = 0;
        uint32_t ph = 0;
        for (int b = 0; b < blocks + LAG; ++b) {
            if (b < blocks) {
                ok = ok && mbar_wait_fast(empty_bar(st), ph ^ 1u, abort_flag, p, DEV_TIMEOUT_PRODUCER);
                if (ok) {
                    const uint32_t a = sbase + st * STAGE;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool in = row[i] != 0xffffffffu;
                        const int64_t m = in ? row[i] : 0;
                        const uint32_t dst = a + (rr + 16 * i) * 128 + sw;
                        copy16(dst, in && in0 ? zc + m * C : z, in && in0);
                        copy16(dst + 8192, in && in1 ? zc + m * C + 64 : z, in && in1);
#pragma unroll
                        for (int q = 0; q < ATOMS; ++q) copy16(dst + GT_A + q * 8192, vc + m * p.vcols + q * 64, in);
                    }
                }
                rows_of(b + 1);
                if (++st == STAGES) { st = 0; ph ^= 1u; }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (b >= LAG) {
                asm volatile("cp.async.wait_group %0;" ::"n"(LAG) : "memory");
                fence_proxy_async_smem();
                mbar_arrive(full_bar(st_done));
                if (++st_done == STAGES) st_done = 0;
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        // epilogue: this thread's column, ranks ascending, the parts added from the smallest
        ok = mbar_wait_fast(done_bar, 0, abort_flag, p, DEV_TIMEOUT_EPILOGUE) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
            tc_fence_after();
            const int64_t col = c0 + 32 * warp + lane;
            float* dst = nchunks > 1 ? jb.parts + static_cast<int64_t>(p.ch.part[g] + j) * p.R * C
                                     : jb.out + static_cast<int64_t>(g) * p.R * C;
            const uint32_t t = tmem_base + (static_cast<uint32_t>(32 * warp) << 16);
            for (int q = 0; q < RUN && r0 + q < p.R; q += 16) {
                float sum[16];
                for (int half = 0; half < (blocks > GT_HALF ? 2 : 1); ++half) {
                    const uint32_t th = t + half * ACC + q;
                    uint32_t v0[16], v1[16], v2[16], v3[16];
                    tmem_ld16(th, v0);
                    tmem_ld16(th + RUN, v1);
                    tmem_ld16(th + 2 * RUN, v2);
                    tmem_ld16(th + 3 * RUN, v3);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float a = __uint_as_float(v0[i]), m = __uint_as_float(v1[i]), l = __uint_as_float(v2[i]);
                        const float z3 = __uint_as_float(v3[i]);
                        const float r = p.fmt ? m + (l + z3)
                                              : fmaf(a, 0x1p11f, fmaf(fmaf(z3, 0x1p-11f, l), 0x1p-11f, m));
                        sum[i] = half == 0 ? r : sum[i] + r;
                    }
                }
                if (col < C) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (r0 + q + i < p.R) dst[static_cast<int64_t>(r0 + q + i) * C + col] = sum[i];
                }
                __syncwarp();
            }
        }
    } else {
        const uint32_t lead = elect_lane();
        const uint32_t idesc = instr_desc(p.fmt, true, true, 4 * RUN);
        int s = 0;
        uint32_t ph = 0;
        for (int b = 0; b < blocks; ++b) {
            if (!__all_sync(0xffffffffu, mbar_wait_fast(full_bar(s), ph, abort_flag, p, DEV_TIMEOUT_MMA))) break;
            tc_fence_after();
            const uint32_t a = sbase + s * STAGE, v = a + GT_A;
            mma_block(tmem_base + (b < GT_HALF ? 0 : ACC), desc_lo(a, true), DESC_HI, MN_STEP_16, desc_lo(v, true), DESC_HI, MN_STEP_16,
                      idesc, b % GT_HALF != 0 ? 1u : 0u, lead);
            mma_commit(empty_bar(s), lead);
            if (++s == STAGES) { s = 0; ph ^= 1u; }
        }
        drain_mmas(done_bar, lead, abort_flag, p);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_free<COLS>(tmem_base);
    }
}

template <int RUN>
cudaError_t grad_run(const LaunchCtx& c, const GradParams& p, dim3 grid) {
    static PerDeviceOnce setup;
    const cudaError_t e = setup.run(c.eng->device, [](int&) {
        return cudaFuncSetAttribute(grad_tc_kernel<RUN>, cudaFuncAttributeMaxDynamicSharedMemorySize, gt_smem(RUN));
    });
    if (e != cudaSuccess) return e;
    const cudaError_t r = launch_plain(grad_tc_kernel<RUN>, grid, dim3(GT_THREADS), gt_smem(RUN), c.stream, p);
    if (r == cudaSuccess) c.count();
    return r;
}

}  // namespace

cudaError_t tc_adapter_narrow(const LaunchCtx& c, bi_dtype dt, float* partial, const void* z, const void* pw,
                              const uint32_t* ids, const AdapterPlan& plan, int64_t M, int64_t L, int R, int64_t G) {
    static PerDeviceOnce setup;
    cudaError_t e = setup.run(c.eng->device, [](int&) {
        return cudaFuncSetAttribute(narrow_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, NP_SMEM);
    });
    if (e != cudaSuccess) return e;
    CUtensorMap x, w;
    if ((e = make_map(&x, dt, z, L, M, 1, 128)) != cudaSuccess) return e;
    if ((e = make_map(&w, dt, pw, L, R, G, 16, true)) != cudaSuccess) return e;
    NarrowParams p{};
    p.plan = plan; p.ids = ids; p.G = static_cast<uint32_t>(G); p.partial = partial; p.M = M; p.R = R; p.rp = (R + 15) / 16 * 16;
    p.num_kb = static_cast<int>((L + BK - 1) / BK);
    p.fmt = dt == BI_BF16 ? 1 : 0;
    p.status = c.status; p.wait_limit = c.wait_limit_ns;
    const int64_t tiles = (M + 127) / 128, pieces = (L + ADAPTER_PIECE - 1) / ADAPTER_PIECE;
    // A CTA per tile and piece, or, where those are more than the two CTAs that fit
    // an SM, several pieces one after the other (its set-up once: 8192 rows of 4096
    // in 18 us with a CTA per piece).  Where they are fewer, the batches of four
    // 16-rank groups (at most one adapter per row) are split among CTAs as well.
    const int64_t slots = 2 * int64_t(c.sm_count);
    const int64_t each = (tiles * pieces + slots - 1) / slots, gy = (pieces + each - 1) / each;
    const int64_t most = (lmin(lmin(G, M), 128) * (p.rp / 16) + 3) / 4;
    const int64_t want = (2 * slots + tiles * gy - 1) / (tiles * gy);
    const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(gy), static_cast<unsigned>(lmin(most, want)));
    e = launch_pdl(narrow_tc_kernel, grid, dim3(NP_THREADS), NP_SMEM, c.stream, x, w, p);
    if (e == cudaSuccess) c.count();
    return e;
}

// Which tiles (both give the same bits).  A wave of CTA pairs takes 300 ns per
// contraction block; single CTAs take 80 ns, or what their operands take to come
// from L2, 7/6 ns per tile and block, if that is more.  Measured, bf16, K = 4096,
// the whole call, single CTAs against pairs: N = 4096, 64 rows 16.5 us against 35,
// 512 rows 26.7 against 33.1; N = 11008, 128 rows 31 against 37, 256 rows 53
// against 38.
bool adapter_small_tiles(const LaunchCtx& c, int64_t M, int64_t C) {
    const int64_t pairs = (M + 255) / 256 * ((C + 255) / 256), tiles = (M + 127) / 128 * ((C + 63) / 64);
    const int64_t wave_p = (pairs + c.sm_count / 2 - 1) / (c.sm_count / 2), wave_s = (tiles + c.sm_count - 1) / c.sm_count;
    return (M + 127) / 128 <= 65535 && lmax(480 * wave_s, 7 * tiles) < 1800 * wave_p;
}

// Sums of pieces that a small tile's CTA takes on itself: 64 KB of L2 reads.
constexpr int64_t SM_FUSE = 16384;
bool adapter_small_fuses(const LaunchCtx& c, int64_t M, int64_t C, int64_t L, int R) {
    const int64_t pieces = (L + ADAPTER_PIECE - 1) / ADAPTER_PIECE, rp = (R + 15) / 16 * 16;
    return (!c.eng || c.eng->tile_cols == 0) && R <= 64 && adapter_small_tiles(c, M, C) &&
           lmin(M, 128) * rp * pieces <= SM_FUSE;
}

cudaError_t tc_adapter_rows_small(const LaunchCtx& c, bi_dtype dt, int dx, void* out, const void* z, const void* w,
                                  const void* bias, const void* hh, const void* q, const AdapterPlan& plan,
                                  const AdapterPieces& src, int64_t M, int64_t K, int64_t N, int R, int64_t G, bool fuse) {
    const int64_t L = dx ? N : K, C = dx ? K : N;
    const uint32_t ar = static_cast<uint32_t>(lmin(128, (M + 7) / 8 * 8));
    CUtensorMap mx, mw, mh, mq;
    cudaError_t e;
    if ((e = make_map(&mx, dt, z, L, M, 1, ar)) != cudaSuccess) return e;
    if ((e = make_map(&mw, dt, w, N, K, 1, 64)) != cudaSuccess) return e;
    if (!fuse && (e = make_map(&mh, dt, hh, adapter_part_cols(R), M, 1, ar)) != cudaSuccess) return e;
    if ((e = make_map(&mq, dt, q, C, R, G, 16, true)) != cudaSuccess) return e;
    SmallParams p{};
    if (fuse) mh = mx;  // not read
    p.far = {src.partial, src.ids, src.scales, q, plan.over, M, C, src.pieces, (R + 15) / 16 * 16, R};
    p.h = src.h; p.G = static_cast<uint32_t>(G); p.fused = fuse;
    p.plan = plan; p.out = out; p.bias = bias; p.M = M; p.C = C; p.R = R; p.a_bytes = static_cast<int>(ar) * 128;
    p.num_kb = static_cast<int>((L + BK - 1) / BK);
    p.status = c.status; p.wait_limit = c.wait_limit_ns;
    const dim3 grid(static_cast<unsigned>((C + SM_COLS - 1) / SM_COLS), static_cast<unsigned>((M + 127) / 128));
    return dt == BI_BF16 ? small_rows_fmt<1>(c, dx, M, mx, mw, mh, mq, p, grid)
                         : small_rows_fmt<0>(c, dx, M, mx, mw, mh, mq, p, grid);
}

// A wave of pairs takes 1.14 us per 32-wide block, one of single CTAs 0.3 us, or
// what their 48 KB per block take from L2, 4.8 ns per tile.
bool tf32x3_small_tiles(const LaunchCtx& c, int64_t rows, int64_t cols, int64_t depth) {
    const int64_t pairs = (rows + 255) / 256 * ((cols + 255) / 256), tiles = (rows + 127) / 128 * ((cols + 63) / 64);
    const int64_t wave_p = (pairs + c.sm_count / 2 - 1) / (c.sm_count / 2), wave_s = (tiles + c.sm_count - 1) / c.sm_count;
    return c.eng->tile_cols == 0 && depth <= TF32X3_PIECE && (rows + 127) / 128 <= 65535 &&
           lmax(3000 * wave_s, 48 * tiles) < 11400 * wave_p;
}

cudaError_t tc_tf32x3_small(const LaunchCtx& c, const float* a_hi, const float* a_lo, int64_t lda, const float* b_hi,
                            const float* b_lo, int64_t ldb, float* out, int64_t ldo, const float* bias, int64_t rows,
                            int64_t cols, int64_t depth) {
    static PerDeviceOnce setup;
    cudaError_t e = setup.run(c.eng->device, [](int&) {
        return cudaFuncSetAttribute(small_f32_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SF_SMEM);
    });
    if (e != cudaSuccess) return e;
    CUtensorMap ah, al, bh, bl;
    if ((e = make_map32(&ah, a_hi, depth, rows, lda, 128)) != cudaSuccess) return e;
    if ((e = make_map32(&al, a_lo, depth, rows, lda, 128)) != cudaSuccess) return e;
    if ((e = make_map32(&bh, b_hi, depth, cols, ldb, 64)) != cudaSuccess) return e;
    if ((e = make_map32(&bl, b_lo, depth, cols, ldb, 64)) != cudaSuccess) return e;
    SmallF32Params p{};
    p.out = out; p.bias = bias; p.M = rows; p.C = cols; p.ldo = ldo;
    p.num_kb = static_cast<int>((depth + 31) / 32);
    p.status = c.status; p.wait_limit = c.wait_limit_ns;
    const dim3 grid(static_cast<unsigned>((cols + SM_COLS - 1) / SM_COLS), static_cast<unsigned>((rows + 127) / 128));
    e = launch_pdl(small_f32_kernel, grid, dim3(SM_THREADS), SF_SMEM, c.stream, ah, al, bh, bl, p);
    if (e == cudaSuccess) c.count();
    return e;
}

cudaError_t tc_adapter_grad(const LaunchCtx& c, bi_dtype dt, const AdapterGradJob* jobs, int count, const uint32_t* off,
                            const uint32_t* perm, const AdapterChunks& ch, int64_t M, int R, int64_t G) {
    GradParams p{};
    int64_t strips = 0;
    for (int i = 0; i < count; ++i) {
        p.job[i] = jobs[i];
        strips += (jobs[i].C + 127) / 128;
        if (i == 0) p.strips0 = static_cast<uint32_t>(strips);
    }
    p.off = off; p.perm = perm; p.ch = ch; p.vcols = adapter_grad_cols(R); p.R = R; p.G = static_cast<int>(G);
    p.fmt = dt == BI_BF16 ? 1 : 0;
    p.status = c.status; p.wait_limit = c.wait_limit_ns;
    p.strips = static_cast<uint32_t>(strips);
    const int64_t chunks = AdapterChunks::max_chunks(M, G);
    const int64_t slice = ((int64_t(1) << 31) - 1) / strips;  // chunks per launch
    for (int64_t q = 0; q < chunks; q += slice) {
        p.chunk0 = static_cast<uint32_t>(q);
        const dim3 grid(static_cast<unsigned>(lmin(slice, chunks - q) * strips), static_cast<unsigned>((R + 63) / 64));
        const int run = adapter_rank_run(R);
        const cudaError_t e = run == 16 ? grad_run<16>(c, p, grid) : run == 32 ? grad_run<32>(c, p, grid)
                            : run == 48 ? grad_run<48>(c, p, grid) : grad_run<64>(c, p, grid);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace bi
