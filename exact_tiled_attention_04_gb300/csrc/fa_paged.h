// Declarations shared by the host entry points of the paged key/value cache
// (fa_paged_api.cu) and its kernels.  Not part of the public C ABI.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "fa_kv4.h"  // launches that overlap with the kernel before them

namespace fa {

// A cache as the kernels see it (fa_paged_cache_t in 32-bit sizes).
struct PagedCache {
    uint16_t* pages[2];      // keys, values: [num_pages, H_kv, page, d]
    const int32_t* table;    // [B, max_pages]
    int32_t* lengths;        // [B]
    int num_pages, page, B, max_pages, H_kv, d;
    int capacity;            // max_pages * page
    int unwaited;            // 1: read behind another kernel's wait for what wrote it (attention behind a prefix)
};

struct RowsView {
    uint16_t* data;
    long long row, head;  // strides in elements
};

struct PagedAppendParams {
    PagedCache c;
    RowsView k, v, q, q_out, k_out;  // q, q_out, k_out: data may be nullptr
    const int32_t* cu;               // [B + 1] or nullptr: n rows for each sequence
    const float* table;              // [table_rows, rot] or nullptr (rot = 0)
    const int32_t* positions;        // [T] or nullptr
    int32_t* lengths_out;            // [B]
    DevStatus* status;
    long long T, first_position, table_rows;
    int n, H, rot;
    int whole;   // 1: a block has all rows of a sequence (and advances its length)
    int parts;   // warps that share a token's rows
};
// interleaved: pairs of neighbouring channels.
cudaError_t launch_paged_append(const PagedAppendParams& p, int sms, bool f16, bool interleaved, cudaStream_t stream);

// Attention over the cache.  Rows: the R = N_q * group query rows of a
// key/value head, row r = g * N_q + i (query head g of the group, query i), in
// blocks of `rows_per_block`.  A unit is one (sequence, key/value head, row
// block); its keys are cut into tiles of 128, and the tiles of all units, in
// order, into runs of equal length, one per CTA.
struct PagedFwdParams : FwdParams {
    PagedCache c;
    int rows, row_blocks;
    int ctas;
    int parts_always;  // 1: every unit's result is a partial one (behind a prefix)
    // workspace: partial results.  Slots 2 i and 2 i + 1: of CTA i's first unit,
    // where another CTA began it, and of its last; behind them, with
    // parts_always, one for each unit that one CTA has alone.
    float4* part_ml;   // [slots, rows_per_block]: reference, exact sum, rounded sum
    float* unit_o;     // [slots, rows_per_block, d]
    // the prefix's partial results, `splits` slabs of [B * H_kv * rows] rows
    // (FwdParams::o_part, ml_part; splits = 0: no prefix)
};
// The smallest block that holds the rows, or 32 (4 rows: 32 sequences of up to
// 16384 slots, d = 128, 169.4 us, in blocks of 16 171.6; 64 behind a prefix 42.3, 45.9;
// four short ones, d = 64, 7.6, 8.1).
constexpr int paged_rows_per_block(int64_t rows) { return rows <= 4 ? 4 : rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }
cudaError_t launch_paged_fwd_bf16(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PagedFwdParams& p,
                                  cudaStream_t stream);
cudaError_t launch_paged_fwd_f16(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PagedFwdParams& p,
                                 cudaStream_t stream);

// The prefix that all sequences share, by the packed forward kernel
// (fa_packed_fwd.cuh).  A tile of 128 query rows holds the `rows` rows that `seqs`
// sequences (as many as fit) have for one key/value head; a block has two tiles (or,
// where one holds all sequences, one) and a partition of the keys, and leaves a
// partial result.  The key/value tiles come from pages as in the kernel above.
struct PrefixFwdParams : FwdParams {
    const int32_t* pages;  // numbers of the prefix's pages
    int page, n_pages;
    int B, rows, seqs;
    int blocks;            // blocks along the sequences, per key/value head
    int pair;              // 1: two tiles
    int negate;            // as in PackedFwdParams
};
// q: [B, H_kv, rows, d] with boxes of `rows` rows x 1 x `seqs` sequences.
cudaError_t launch_prefix_fwd_bf16(int d, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                   const PrefixFwdParams& p, cudaStream_t stream);
cudaError_t launch_prefix_fwd_f16(int d, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                  const PrefixFwdParams& p, cudaStream_t stream);

}  // namespace fa
