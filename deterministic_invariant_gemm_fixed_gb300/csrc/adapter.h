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
// distinct ones (in order of their first row), and for each its index and a bit
// per row.
struct AdapterPlan {
    uint32_t* count;  // [tiles]
    uint32_t* ids;    // [tiles][256]
    uint32_t* masks;  // [tiles][256][8]
    static int64_t tiles(int64_t M) { return (M + ADAPTER_TILE - 1) / ADAPTER_TILE; }
    static int64_t words(int64_t M) { return tiles(M) * (1 + 256 + 256 * 8); }
    static AdapterPlan at(void* p, int64_t M) {
        AdapterPlan r;
        r.masks = static_cast<uint32_t*>(p);  // 16-byte aligned masks first
        r.ids = r.masks + tiles(M) * 256 * 8;
        r.count = r.ids + tiles(M) * 256;
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

}  // namespace bi
