// The MXFP4 product: out [rows][cols] = a [rows][depth] b [cols][depth]^T (+ bias),
// operands as fp4.cu lays them out, on tcgen05.mma.kind::mxf4 with block scales.
//
// A persistent grid of CTA pairs, each running M256 x N256 x K64 MMAs on 256 x 256
// output tiles: CTA r of the pair holds rows [128r, 128r + 128) of A and columns
// [128r, 128r + 128) of B in its shared memory and rows [128r, 128r + 128) of the
// accumulator in its tensor memory.  A ring stage is 256 contraction elements (one
// 128-byte swizzle row of codes per operand row): 16 KB of A, 16 KB of B, 1 KB of A's
// scales (this CTA's rows) and 2 KB of B's (all 256 columns, which each CTA of the
// pair scales by).  The scales are stored in the order the tensor cores want, so
// tcgen05.cp takes them from shared memory to tensor memory as they are: six copies
// and four MMAs per stage.
//
// Every output element is one chain of 64-wide blocks in ascending order in one f32
// accumulator; a result kept in f32 takes pieces of TC_PIECE_ROWS elements, a launch
// each, every one after the first adding to the output.  No split, no atomics, one tile
// shape for every batch: a row's result does not depend on the rows beside it.
//
// Tensor memory has 512 columns: two 256-column accumulators and the scales do not
// fit, so the accumulators overlap: [0, 256) and [192, 448), scales (two stages of 24
// columns) from 448 on.  The epilogue of a tile drains the 64 shared columns first;
// then the next tile's MMAs start and the other 192 columns are stored beside them.
//
// Bound by the ring's feed from L2, 70 KB per pair and stage for 33.6 MFLOP: 8192 x 4096 x
// 12288 takes 128 us (6.4 PFLOP/s), the tensor pipe 60 % busy.  One token's stage takes
// 0.39 us, a batch's 0.4.
#include "abi_util.h"
#include "fp4.h"
#include "tc_common.cuh"

namespace bi {
namespace {

constexpr int F_THREADS = 192;
constexpr int F_BKE = 256;                 // contraction elements per stage
constexpr int F_TILE = 128 * 128;          // bytes of one CTA's codes of an operand per stage
constexpr int F_SFA = 1024, F_SFB = 2048;  // scales of 128 rows, of 256 columns
constexpr int F_STAGE = 2 * F_TILE + F_SFA + F_SFB;
static_assert(F_STAGE % 1024 == 0, "stages start on the swizzle's atom");
constexpr int F_OUT = 4 * 2 * 32 * 128;    // output staging: two slices of 32 rows x 128 bytes per epilogue warp
constexpr int F_BIAS = 4 * 256 * 4;        // the tile's bias in f32, a copy per epilogue warp
constexpr int F_BARS = 256;
constexpr int F_LIMIT = 227 * 1024;
constexpr int F_STAGES = (F_LIMIT - 1024 - F_OUT - F_BIAS - F_BARS) / F_STAGE;
constexpr int F_SMEM = 1024 + F_STAGES * F_STAGE + F_OUT + F_BIAS + F_BARS;
static_assert(F_STAGES == 5 && F_SMEM <= F_LIMIT, "ring depth");
constexpr int F_ACC1 = 192, F_SHARED = 64;  // second accumulator's column; columns both have
constexpr int F_SF = 448, F_SF_STAGE = 24;  // scales' first column; columns per stage (A 8, B 16)
static_assert(F_ACC1 + F_SHARED == 256 && F_ACC1 + 256 == F_SF && F_SF + 2 * F_SF_STAGE <= 512, "tensor memory");

struct Fp4Params {
    void* out;
    int64_t ldo, rows, cols;
    const void* bias;
    int units_m, num_n;
    int wide;       // a sweep over the columns is shared by 32 row tiles, not 16
    int kb0, nkb;   // the stages of this launch
    int accum;      // f32: add to what the output holds
    int tma_out;    // the output's rows are multiples of 16 bytes: stored by TMA
    int* status;
    unsigned long long wait_limit;
};

// tcgen05.cp of one 512-byte piece of scales to 4 tensor-memory columns of both CTAs.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t saddr, uint32_t lead) {
    constexpr uint32_t HI = (128u >> 4) | (1u << 14);  // 8 rows of 16 bytes after 8 rows; no swizzle
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b64 d;\n\tsetp.ne.b32 e, %3, 0;\n\tmov.b64 d, {%1, %2};\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n\t}\n" ::"r"(taddr),
        "r"(((saddr & 0x3FFFFu) >> 4) | (1u << 16)), "r"(HI), "r"(lead)
        : "memory");
}
// One M256 x N256 x K64 MMA; scales at sfa, sfb, the byte pair given by the descriptor.
__device__ __forceinline__ void mma_fp4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t acc,
                                        uint32_t lead) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %7, 0;\n\tsetp.ne.b32 e, %8, 0;\n\t"
        "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %4, [%5], [%6], p;\n\t}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(DESC_HI), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc), "r"(lead)
        : "memory");
}
// Instruction descriptor: e2m1 operands (1), K-major, e8m0 scales; `id`: the first of
// the two scale bytes (of four) that this MMA's 64 elements have.
__host__ __device__ constexpr uint32_t fp4_idesc(uint32_t id) {
    return (id << 4) | (1u << 7) | (1u << 10) | ((256u >> 3) << 17) | (1u << 23) | ((256u >> 7) << 27) | (id << 29);
}

template <int OUT>  // 0 f16, 1 bf16, 2 f32
__global__ void __launch_bounds__(F_THREADS, 1)
    fp4_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                    const __grid_constant__ CUtensorMap tmO, const Fp4Params p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t sbase = smem_u32(smem);
    const uint32_t ostage = sbase + F_STAGES * F_STAGE;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + F_STAGES * F_STAGE + F_OUT + F_BIAS);
    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };                 // CTA 0: both CTAs' copies of a stage
    auto empty_bar = [&](int s) { return bar0 + 8u * (F_STAGES + s); };   // each CTA: CTA 0's commit
    auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * F_STAGES + b); };
    const uint32_t tover_bar = bar0 + 8u * (2 * F_STAGES + 2);            // CTA 0: shared columns drained, 8 warps
    const uint32_t drain_bar = bar0 + 8u * (2 * F_STAGES + 3);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * F_STAGES + 4);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    const int lane = threadIdx.x & 31;
    const uint32_t crank = blockIdx.x & 1u;
    const int cidx = static_cast<int>(blockIdx.x >> 1), ncl = static_cast<int>(gridDim.x >> 1);
    const int tiles = p.units_m * p.num_n;

    if (warp == 2 && lane < 5) prefetch_map(lane == 0 ? &tmA : lane == 1 ? &tmB : lane == 2 ? &tmSA : lane == 3 ? &tmSB : &tmO);
    if (threadIdx.x == 0) {
        for (int s = 0; s < F_STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) mbar_init(tfull_bar(b), 1);
        mbar_init(tover_bar, 8);
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(tmem_slot), 0);
    grid_dep_wait();
    grid_dep_launch();

    if (warp == 0) {
        // ------------------------------------------------------------ producer (both CTAs): a lane per copy
        const CUtensorMap* map = lane == 0 ? &tmA : lane == 1 ? &tmB : lane == 2 ? &tmSA : &tmSB;
        const uint32_t to = sbase + (lane < 2 ? lane * F_TILE : lane == 2 ? 2 * F_TILE : 2 * F_TILE + F_SFA);
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int t = cidx; ok && t < tiles; t += ncl) {
            int mp, nb;
            dense_raster(t, p.units_m, p.num_n, mp, nb, p.wide ? 32 : 16);
            const int y = lane == 0 ? mp * 256 + static_cast<int>(crank) * 128
                        : lane == 1 ? nb * 256 + static_cast<int>(crank) * 128
                        : lane == 2 ? mp * 2 + static_cast<int>(crank) : nb * 2;
            for (int kb = 0; kb < p.nkb; ++kb) {
                ok = __all_sync(0xffffffffu, mbar_wait_fast(empty_bar(s), ph ^ 1u, abort_flag, p, DEV_TIMEOUT_PRODUCER));
                if (!ok) break;
                if (crank == 0 && lane == 0) mbar_expect_tx(full_bar(s), 2 * F_STAGE);
                __syncwarp();
                if (lane < 4)
                    tma_load_2d_pair(to + s * F_STAGE, map, (p.kb0 + kb) * (lane < 2 ? 128 : 256), y, mapa_rank(full_bar(s), 0));
                if (++s == F_STAGES) { s = 0; ph ^= 1u; }
            }
        }
        // CTA 0's MMA warp takes every copy of both CTAs before it finishes, unless a wait
        // gave up (see the teardown)
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (CTA 0)
        if (crank == 0) {
            const uint32_t lead = elect_lane();
            int s = 0, it = 0, sf = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = cidx; ok && t < tiles; t += ncl, ++it) {
                if (it > 0)  // the tile before has left the shared columns (and the one before that all of its own)
                    ok = __all_sync(0xffffffffu, mbar_wait_fast(tover_bar, (it - 1) & 1, abort_flag, p, DEV_TIMEOUT_MMA));
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem + (it & 1) * F_ACC1;
                for (int kb = 0; kb < p.nkb; ++kb) {
                    ok = __all_sync(0xffffffffu, mbar_wait_fast(full_bar(s), ph, abort_flag, p, DEV_TIMEOUT_MMA));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t st = sbase + s * F_STAGE, sfa = st + 2 * F_TILE, sfb = sfa + F_SFA;
                    const uint32_t ta = tmem + F_SF + sf * F_SF_STAGE, tb = ta + 8;
#pragma unroll
                    for (int a = 0; a < 2; ++a) {  // 128 elements of the stage
                        copy_scales(ta + a * 4, sfa + a * 512, lead);
                        copy_scales(tb + a * 8, sfb + a * 512, lead);
                        copy_scales(tb + a * 8 + 4, sfb + 1024 + a * 512, lead);
                    }
                    const uint32_t da = desc_lo(st, false), db = desc_lo(st + F_TILE, false);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_fp4(d, da + kk * K_STEP, db + kk * K_STEP, fp4_idesc((kk & 1) * 2), ta + (kk >> 1) * 4, tb + (kk >> 1) * 8,
                                (kb | kk) != 0 ? 1u : 0u, lead);
                    mma_commit_pair_lead(empty_bar(s), 0x3, lead);
                    sf ^= 1;
                    if (++s == F_STAGES) { s = 0; ph ^= 1u; }
                }
                if (!ok) break;
                mma_commit_pair_lead(tfull_bar(it & 1), 0x3, lead);
            }
            __syncwarp();
            if (lead) {
                mma_commit_pair(drain_bar);
                mbar_drain(drain_bar, 0);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------ epilogue (both CTAs)
        constexpr int OES = OUT == 2 ? 4 : 2, CPS = 128 / OES, SLICES = 256 / CPS;
        using O = OutT<OUT == 1 ? 1 : 0>;
        const int qd = warp & 3;
        const uint32_t over = mapa_rank(tover_bar, 0);
        int it = 0, oslot = 0;
        float* bias = reinterpret_cast<float*>(smem + F_STAGES * F_STAGE + F_OUT) + qd * 256;
        for (int t = cidx; t < tiles; t += ncl, ++it) {
            int mp, nb;
            dense_raster(t, p.units_m, p.num_n, mp, nb, p.wide ? 32 : 16);
            const int64_t row0 = static_cast<int64_t>(mp) * 256 + crank * 128 + qd * 32, orow = row0 + lane;
            const int64_t col0 = static_cast<int64_t>(nb) * 256;
            if (p.bias != nullptr) {  // this warp's copy of the tile's
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t c = col0 + i * 32 + lane;
                    bias[i * 32 + lane] = c < p.cols ? (OUT == 2 ? static_cast<const float*>(p.bias)[c] : O::load(p.bias, c)) : 0.0f;
                }
                __syncwarp();
            }
            if (!__all_sync(0xffffffffu, mbar_wait(tfull_bar(it & 1), (it >> 1) & 1, abort_flag, p, DEV_TIMEOUT_EPILOGUE))) break;
            tc_fence_after();
            const uint32_t tbase = tmem + (static_cast<uint32_t>(qd * 32) << 16) + (it & 1) * F_ACC1;
            const int first = (it & 1) ? 0 : F_ACC1 / CPS;  // the slices of the shared columns come first
            for (int i = 0; i < SLICES; ++i) {
                const int cs = (first + i) % SLICES * CPS;
                const bool any = col0 + cs < p.cols && row0 < p.rows;
                const uint32_t buf = ostage + static_cast<uint32_t>(qd * 8192 + (oslot & 1) * 4096);
                uint32_t v[CPS];
                if (any) {
                    __syncwarp();
#pragma unroll
                    for (int c16 = 0; c16 < CPS; c16 += 16) tmem_get16(tbase + cs + c16, v + c16);
                    tmem_wait();
                }
                if (i == F_SHARED / CPS - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(over);
                }
                if (any) {
                    if (p.tma_out) {
                        if (lane == 0) bulk_wait_read<1>();  // the slice staged two slices ago has been read
                        __syncwarp();
                    }
                    float* f = reinterpret_cast<float*>(v);
                    if (OUT == 2 && p.accum && orow < p.rows) {  // the pieces before
                        const float* prev = static_cast<const float*>(p.out) + orow * p.ldo + col0 + cs;
#pragma unroll
                        for (int j = 0; j < CPS; ++j)
                            if (col0 + cs + j < p.cols) f[j] = __fadd_rn(prev[j], f[j]);
                    }
                    if (p.bias != nullptr) {
#pragma unroll
                        for (int j = 0; j < CPS; j += 4) {
                            const float4 b = *reinterpret_cast<const float4*>(bias + cs + j);
                            f[j] = __fadd_rn(f[j], b.x);
                            f[j + 1] = __fadd_rn(f[j + 1], b.y);
                            f[j + 2] = __fadd_rn(f[j + 2], b.z);
                            f[j + 3] = __fadd_rn(f[j + 3], b.w);
                        }
                    }
                    const uint32_t at = buf + static_cast<uint32_t>(lane * 128);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {  // 16-byte chunks of the row's 128 bytes
                        uint32_t w[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            w[x] = OUT == 2 ? v[(4 * j + x) % CPS] : O::pack(f[(8 * j + 2 * x) % CPS], f[(8 * j + 2 * x + 1) % CPS]);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + static_cast<uint32_t>((j ^ (lane & 7)) * 16)),
                                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                                     : "memory");
                    }
                }
                if (any && p.tma_out) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&tmO, buf, static_cast<int>(col0) + cs, static_cast<int>(row0));
                        bulk_commit();
                    }
                    ++oslot;
                } else if (any) {  // rows that TMA cannot store, one after the other, a lane to a column
                    __syncwarp();
                    const int rows = static_cast<int>(lmin(32, p.rows - row0));
#pragma unroll 8
                    for (int r = 0; r < rows; ++r) {
#pragma unroll
                        for (int x = 0; x < CPS; x += 32) {
                            const int cc = x + lane;
                            if (col0 + cs + cc >= p.cols) continue;
                            const uint8_t* from = smem + (buf - sbase) + r * 128 + (((cc * OES / 16) ^ (r & 7)) * 16) + cc * OES % 16;
                            const int64_t o = (row0 + r) * p.ldo + col0 + cs + cc;
                            if (OUT == 2) static_cast<uint32_t*>(p.out)[o] = *reinterpret_cast<const uint32_t*>(from);
                            else static_cast<uint16_t*>(p.out)[o] = *reinterpret_cast<const uint16_t*>(from);
                        }
                    }
                    __syncwarp();
                }
            }
        }
        if (lane == 0) bulk_wait<0>();
    }

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) settle_copies();
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// Codes [rows][pitch bytes], box {128 bytes, 128 rows}, 128-byte swizzle; scales
// [row pieces][words], box {256 words, n pieces}.  Zeros past the end.
cudaError_t code_map(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t pitch) {
    auto enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    cuuint64_t dims[2] = {pitch, rows}, strides[1] = {pitch};
    cuuint32_t box[2] = {128, 128}, es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess : cudaErrorInvalidValue;
}
cudaError_t scale_map(CUtensorMap* m, const void* ptr, uint64_t pieces, uint64_t words, uint32_t n) {
    auto enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    cuuint64_t dims[2] = {words, pieces}, strides[1] = {words * 4};
    cuuint32_t box[2] = {256, n}, es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess : cudaErrorInvalidValue;
}

template <int OUT>
cudaError_t product_t(const LaunchCtx& c, void* out, const uint8_t* a, const uint8_t* as, const uint8_t* b, const uint8_t* bs,
                      const void* bias, int64_t rows, int64_t cols, int64_t depth) {
    auto kern = fp4_pair_kernel<OUT>;
    static PerDeviceOnce setup;  // per device: the shared-memory opt-in and the co-resident pairs
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cudaError_t e = setup.run(c.eng->device, [&](int& pairs) {
        cudaError_t q = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, F_SMEM);
        if (q != cudaSuccess) return q;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(128);
        cfg.blockDim = dim3(F_THREADS);
        cfg.dynamicSmemBytes = F_SMEM;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        q = cudaOccupancyMaxActiveClusters(&pairs, kern, &cfg);
        return q == cudaSuccess && pairs < 1 ? cudaErrorInvalidConfiguration : q;
    });
    if (e != cudaSuccess) return e;
    const int64_t depth_p = fp4_padded(depth), esize = OUT == 2 ? 4 : 2;
    CUtensorMap ma, mb, msa, msb, mo;
    if ((e = code_map(&ma, a, rows, depth_p / 2)) != cudaSuccess) return e;
    if ((e = code_map(&mb, b, cols, depth_p / 2)) != cudaSuccess) return e;
    if ((e = scale_map(&msa, as, (rows + 127) / 128, depth_p, 1)) != cudaSuccess) return e;
    if ((e = scale_map(&msb, bs, (cols + 127) / 128, depth_p, 2)) != cudaSuccess) return e;
    Fp4Params p{};
    p.out = out;
    p.ldo = cols;
    p.rows = rows;
    p.cols = cols;
    p.units_m = static_cast<int>((rows + 255) / 256);
    p.num_n = static_cast<int>((cols + 255) / 256);
    // 32 row tiles to a sweep over the columns, which reads b from memory once per group, while
    // a's codes of them stay in L2 (up to 32 MB: depth 8192), else 16: 8192 x 4096 x 12288 128
    // against 134 us, 65536 x 2048 x 8192 432 against 456; 8192 x 12288 x 12288 332 against 319.
    // (The number itself as a parameter: one token 13.7 against 13.3 us.)
    p.wide = 32 * 256 * (depth_p / 2) <= (32 << 20);
    p.tma_out = cols * esize % 16 == 0 && aligned16(out);
    if (!p.tma_out) mo = ma;
    else if ((e = make_out_map(&mo, OUT, out, cols, rows, cols)) != cudaSuccess) return e;
    p.status = c.status;
    p.wait_limit = c.wait_limit_ns;
    const int64_t tiles = static_cast<int64_t>(p.units_m) * p.num_n;
    const int64_t all = depth_p / F_BKE, piece = OUT == 2 ? TC_PIECE_ROWS / F_BKE : all;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * lmin(tiles, setup.value[c.eng->device])));
    cfg.blockDim = dim3(F_THREADS);
    cfg.dynamicSmemBytes = F_SMEM;
    cfg.stream = c.stream;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    for (int64_t k0 = 0; k0 < all; k0 += piece) {
        p.kb0 = static_cast<int>(k0);
        p.nkb = static_cast<int>(lmin(piece, all - k0));
        p.accum = k0 > 0;
        p.bias = k0 + piece >= all ? bias : nullptr;  // after the last piece
        if ((e = cudaLaunchKernelEx(&cfg, kern, ma, mb, msa, msb, mo, p)) != cudaSuccess) return e;
        c.count();
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t tc_fp4_product(const LaunchCtx& c, bi_dtype out_dt, void* out, const uint8_t* a, const uint8_t* as, const uint8_t* b,
                           const uint8_t* bs, const void* bias, int64_t rows, int64_t cols, int64_t depth) {
    return out_dt == BI_F32    ? product_t<2>(c, out, a, as, b, bs, bias, rows, cols, depth)
           : out_dt == BI_BF16 ? product_t<1>(c, out, a, as, b, bs, bias, rows, cols, depth)
                               : product_t<0>(c, out, a, as, b, bs, bias, rows, cols, depth);
}

}  // namespace bi
