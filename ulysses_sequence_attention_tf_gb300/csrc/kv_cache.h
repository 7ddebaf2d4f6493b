// kv_cache.h -- internal interface of the paged key-value cache: appending rows and
// attention over them.  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "relayout.h"

namespace tfu {

struct KvCache {
    uint8_t* codes[2];      // K, V: e4m3 [pages][Hkv][page][D]
    float* scales[2];       // [pages][Hkv]
    const int32_t* table;   // [N][max_pages], rows table_stride apart
    const int32_t* lens;    // [N]
    const int32_t* starts;  // [N + 1]
    int64_t table_stride;
    uint32_t pages, Hkv, page, D, N, max_pages;
};

// [rows, heads, D] views of P head groups: base addresses and byte strides.
struct RowView {
    uint8_t* base[kMaxShards];
    int64_t t, h;
};

enum class Rope : int { kNone = 0, kInterleaved = 1, kHalfSplit = 2 };

struct KvAppendParams {
    KvCache c;
    RowView src[2];        // K, V rows
    RowView q, q_out;      // q.base[0] null: no queries
    const void* weight[2]; // RMSNorm weights of K and Q, or null
    const float* table;    // cos/sin [table_rows][D/2][2]
    uint32_t table_rows;
    float eps;
    Rope rope;
    uint32_t P, T, Hl, Hkl;
    uint32_t units;        // upper bound of the (sequence, page) pairs that get rows
    uint32_t slices;       // CTAs of a unit (set by the launch)
};

// Attention over long caches is split along the keys: chunk c of a sequence is keys
// [c * chunk, (c + 1) * chunk).  A sequence of one chunk is written at once; the
// others leave sums relative to their own reference, and a second kernel joins them:
// per (sequence, key head, row, chunk) D unnormalised fp32 values, reference and sum.
struct KvAttendParams {
    KvCache c;
    RowView q, out;
    float* part;             // [N][Hkv][row_cap][chunks][D], or null for one chunk
    float2* part_stat;       // [N][Hkv][row_cap][chunks] (reference in log2 units, sum)
    uint32_t chunk, chunks;  // keys of a chunk, chunks of the longest sequence
    uint32_t row_cap;        // rows (token, query head) of a key head, rounded up to row tiles
    uint32_t unit;           // rows of a CTA
    bool tiles;              // many rows: kv_attend_tiles.cu
    float* lse[kMaxShards];  // [Hl][T] per group, or null
    const float* slopes;     // [P * Hl] or null
    float scale, cap;
    uint32_t P, T, Hl, Hkl, shared;
    uint32_t max_tokens, max_len;
    uint32_t causal;
};

constexpr uint32_t kTileRows = 256;  // rows of a CTA of the tile kernel

cudaError_t launch_kv_append(const KvAppendParams& p, bool bf16, cudaStream_t stream);
cudaError_t launch_kv_attend(const KvAttendParams& p, bool bf16, cudaStream_t stream, int* launches);

// the tile kernel alone (kv_attend_tiles.cu)
cudaError_t launch_kv_tiles(const KvAttendParams& p, bool bf16, cudaStream_t stream);

// Status word of the cache kernels: 0, or 1 when a length, a start or a page number
// of some sequence was out of range and the sequence (or the page) was left out.
cudaError_t read_kv_append_status(unsigned* out, bool clear);
cudaError_t read_kv_attend_status(unsigned* out, bool clear);
cudaError_t read_kv_tiles_status(unsigned* out, unsigned* waits, bool clear);  // *waits: 1 when a bounded wait gave up

}  // namespace tfu
