// The inner products of the adapters (h and u, scaled) on their way into the wide
// product on the tensor cores: the sum of their pieces, their two 16-bit parts, and
// the terms that f16 parts cannot carry.  The finish kernel, the small tiles and the
// CTA pairs use the same code, so their results have the same bits.
#pragma once

#include "adapter.h"
#include "tc_common.cuh"

namespace bi {

// v = the pieces' sums at p, p + step, ... (eight ranks), added in order, the loads
// of four pieces in flight.
__device__ __forceinline__ void sum_pieces8(const float* p, int64_t step, int pieces, float (&v)[8]) {
    for (int q0 = 0; q0 < pieces; q0 += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q0 + q >= pieces) break;
            a[q] = reinterpret_cast<const float4*>(p + (q0 + q) * step)[0];
            b[q] = reinterpret_cast<const float4*>(p + (q0 + q) * step)[1];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q0 + q >= pieces) break;
            const float t[8] = {a[q].x, a[q].y, a[q].z, a[q].w, b[q].x, b[q].y, b[q].z, b[q].w};
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = q0 + q == 0 ? t[u] : v[u] + t[u];
        }
    }
}

// Values that f16 (FMT 0) has no number for, infinities among them, stay out of the
// MMAs: the epilogue adds their terms in f32 (add_far_terms).  bf16 has f32's range.
template <int FMT>
__device__ __forceinline__ bool beyond_parts(float v) { return FMT == 0 && fabsf(v) > 65504.0f; }

// v ~ hi + lo, 0 for what is beyond; true if there is such a one.  A part that would
// be an infinity's remainder is 0, so an infinity stays one.
template <int FMT>
__device__ __forceinline__ bool two_parts8(const float (&v)[8], uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    using O = OutT<FMT>;
    bool far = false;
#pragma unroll
    for (int u = 0; u < 8; u += 2) {
        const bool f0 = beyond_parts<FMT>(v[u]), f1 = beyond_parts<FMT>(v[u + 1]);
        far = far || f0 || f1;
        const float a = f0 ? 0.0f : v[u], b = f1 ? 0.0f : v[u + 1];
        hi[u / 2] = O::pack(a, b);
        const float h0 = O::load(&hi[u / 2], 0), h1 = O::load(&hi[u / 2], 1);
        lo[u / 2] = O::pack(isinf(h0) ? 0.0f : a - h0, isinf(h1) ? 0.0f : b - h1);
    }
    return far;
}

// What the epilogues need to add the terms of ranks beyond f16.
struct AdapterFar {
    const float* partial;  // pieces of h or u [pieces][M][rp]
    const uint32_t* ids;
    const float* scales;
    const void* q;         // [G, R, C] f16
    const uint32_t* over;  // a bit per row: it has such ranks
    int64_t M, C;
    int pieces, rp, R;
};

// f[0..15], columns c.. of row m, += the row's terms beyond f16, ranks ascending, in
// f32 FMAs; the values are taken from their pieces again, in the finish's order.  Rows
// without such a rank (all but a few, or the scales are out of place) never come here.
static __device__ __noinline__ void add_far_terms(const AdapterFar a, int64_t m, int64_t c, float* f) {
    const uint32_t g = a.ids[m];
    const float s = a.scales != nullptr ? a.scales[g] : 1.0f;
    const __half* q = static_cast<const __half*>(a.q) + static_cast<int64_t>(g) * a.R * a.C + c;
    const int n = static_cast<int>(lmin(16, a.C - c));
    for (int r = 0; r < a.R; ++r) {
        float v = a.partial[m * a.rp + r];
        for (int p = 1; p < a.pieces; ++p) v += a.partial[(p * a.M + m) * a.rp + r];
        v *= s;
        if (!beyond_parts<0>(v)) continue;
        for (int i = 0; i < n; ++i) f[i] = fmaf(v, __half2float(q[r * a.C + i]), f[i]);
    }
}

}  // namespace bi
