// Low-rank adapters beside a shared projection: what the scalar kernels
// (adapter.cu) and the tensor-core kernels (adapter_tc.cu) share.
#pragma once

#include "bi_internal.h"

namespace bi {

constexpr int64_t ADAPTER_MAX_RANK = 256;
// h and u contract in pieces of this many elements, each an own sum, the pieces
// added in order: a decoding batch then has pieces enough to fill the GPU, and
// the piece length does not depend on the batch, so neither does a row's value.
constexpr int64_t ADAPTER_PIECE = 512;
// dA and dB contract in chunks of this many rows of one adapter (sorted by row
// index), the chunks added in order.
constexpr int64_t ADAPTER_CHUNK = 1024;
constexpr int ADAPTER_TILE = 256;  // rows per plan tile

// Which adapters the rows of each 256-row tile have: per tile the number of
// distinct ones, and for each its index and a bit per row.
struct AdapterPlan {
    uint32_t* count;  // [tiles]
    uint32_t* ids;    // [tiles][256]
    uint32_t* masks;  // [tiles][256][8]
    uint32_t* over;   // [tiles][8] a bit per row: an inner product of it is beyond f16 (adapter_parts.cuh)
    static int64_t tiles(int64_t M) { return (M + ADAPTER_TILE - 1) / ADAPTER_TILE; }
    static int64_t words(int64_t M) { return tiles(M) * (1 + 256 + 256 * 8 + 8); }
    static AdapterPlan at(void* p, int64_t M) {
        AdapterPlan r;
        r.masks = static_cast<uint32_t*>(p);  // 16-byte aligned masks first
        r.ids = r.masks + tiles(M) * 256 * 8;
        r.over = r.ids + tiles(M) * 256;
        r.count = r.over + tiles(M) * 8;
        return r;
    }
};

// Chunks of the sorted rows (dA, dB): first[g] = chunks of adapters before g;
// part[g] = the same over the adapters of two chunks or more, whose chunk
// results go through the partial sums (an adapter of one chunk writes its
// result itself).  At most 2 M / ADAPTER_CHUNK partial slots.
struct AdapterChunks {
    uint32_t* first;  // [G + 1]
    uint32_t* part;   // [G + 1]
    static int64_t words(int64_t G) { return 2 * (G + 1); }
    static AdapterChunks at(void* p, int64_t G) {
        AdapterChunks r;
        r.first = static_cast<uint32_t*>(p);
        r.part = r.first + G + 1;
        return r;
    }
    static int64_t max_chunks(int64_t M, int64_t G) { return M / ADAPTER_CHUNK + lmin(G, M); }
    static int64_t max_parts(int64_t M) { return 2 * (M / ADAPTER_CHUNK); }
};

// Tensor-core formats of an inner product v (h or u, scaled), 16-bit.
// Two parts, for the wide product: row m holds per 32 ranks 32 high parts and 32
// remainders, v ~ hi + lo (bf16: to 2^-17 of v, f16: to 2^-22 of v or, for small
// ones, 2^-25; beyond f16's 65504 both are 0 and the epilogue adds the term).
inline int64_t adapter_part_cols(int64_t R) { return (R + 31) / 32 * 64; }
// Four parts, for dA and dB: row m holds per 64 ranks four runs of rank_run
// columns whose products are summed apart.  bf16: v = p1 + p2 + p3, together f32's
// 24 bits (p0 = 0).  f16, whose exponent is narrow: v = 2^11 p0 + p1 + 2^-11 p2 +
// 2^-22 p3, p0 for magnitudes beyond 65504 only (up to 2^27); a part that would be
// subnormal is 0 and its value left to the next one, because the tensor core
// aligns a sum's products by exponents that a subnormal factor overstates (a
// part of 2^-24 took the sum's last bits with it: 2^-17 of the result).
__host__ __device__ inline int adapter_rank_run(int R) { return R > 64 ? 64 : (R + 15) / 16 * 16; }
__host__ __device__ inline int64_t adapter_grad_cols(int R) { return (R + 63) / 64 * 4 * adapter_rank_run(R); }

// The narrow product's pieces, and what makes h (u) of them.
struct AdapterPieces {
    const float* partial;
    const uint32_t* ids;
    const float* scales;
    float* h;  // fused small tiles only: receives the unscaled sums (nullable)
    int pieces;
};
// The wide product on the tensor cores: forward (dx = 0) or dX with the shared
// product, its bias and the adapters' terms in one pass (tc.cu).
cudaError_t tc_adapter_rows(const LaunchCtx& c, bi_dtype dt, int dx, void* out, const void* z, const void* w,
                            const void* bias, const void* hh, const void* q, const AdapterPlan& plan,
                            const AdapterPieces& src, int64_t M, int64_t K, int64_t N, int R, int64_t G);
// The same by 128 x 64 tiles on single CTAs (adapter_tc.cu): identical bits, for
// outputs that the 256 x 256 tiles of CTA pairs spread over too few SMs.
bool adapter_small_tiles(const LaunchCtx& c, int64_t M, int64_t C);
// ... and whether they also add up the pieces of h (then no finish kernel runs).
bool adapter_small_fuses(const LaunchCtx& c, int64_t M, int64_t C, int64_t L, int R);
cudaError_t tc_adapter_rows_small(const LaunchCtx& c, bi_dtype dt, int dx, void* out, const void* z, const void* w,
                                  const void* bias, const void* hh, const void* q, const AdapterPlan& plan,
                                  const AdapterPieces& src, int64_t M, int64_t K, int64_t N, int R, int64_t G, bool fuse);
// The shared product of f32 adapters, as bi_forward / bi_backward_dx compute it
// (engine.cu), with the 3xTF32 tiles chosen by their number: single CTAs' 128 x
// 64 tiles (adapter_tc.cu; contractions up to one piece) give the same bits.
bi_status adapter_projection_f32(bi_engine eng, const LaunchCtx& c, int dx, void* out, const void* z, const void* w,
                                 const void* bias, int64_t m, int64_t k, int64_t n, int tensor_cores);
bool tf32x3_small_tiles(const LaunchCtx& c, int64_t rows, int64_t cols, int64_t depth);
cudaError_t tc_tf32x3_small(const LaunchCtx& c, const float* a_hi, const float* a_lo, int64_t lda, const float* b_hi,
                            const float* b_lo, int64_t ldb, float* out, int64_t ldo, const float* bias, int64_t rows,
                            int64_t cols, int64_t depth);
// The narrow product on the tensor cores (adapter_tc.cu): partial[piece][m][rp] =
// the piece's sum of z[m,l] p[g][r,l], rp = R rounded up to 16 the row stride.
// Also makes the plan of the rows' adapters.
cudaError_t tc_adapter_narrow(const LaunchCtx& c, bi_dtype dt, float* partial, const void* z, const void* p,
                              const uint32_t* ids, const AdapterPlan& plan, int64_t M, int64_t L, int R, int64_t G);
// dA and dB on the tensor cores: out[g][r,c] (or its chunks' partial slots) =
// sum over the adapter's sorted rows of v[m,r] z[m,c], v in four parts [M,
// adapter_grad_cols(R)]; up to two such products in one launch.
struct AdapterGradJob {
    float* out;
    float* parts;
    const void* v4;
    const void* z;
    int64_t C;
};
struct AdapterGradJobs {
    AdapterGradJob job[2];
};
cudaError_t tc_adapter_grad(const LaunchCtx& c, bi_dtype dt, const AdapterGradJob* jobs, int count, const uint32_t* off,
                            const uint32_t* perm, const AdapterChunks& ch, int64_t M, int R, int64_t G);

}  // namespace bi
