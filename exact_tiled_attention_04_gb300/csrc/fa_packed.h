// Declarations shared by the host entry points of attention over packed
// sequences (fa_packed_api.cu) and its kernels.  Not part of the public C ABI.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "fa_bwd_internal.h"
#include "fa_internal.h"

namespace fa {

// The sequences of a packed batch: sequence s has query rows cu_q[s] ..
// cu_q[s + 1] - 1 and key rows cu_k[s] .. cu_k[s + 1] - 1, read on the device.
struct PackedSeqs {
    const int32_t* cu_q;  // [B + 1]
    const int32_t* cu_k;
    int B;
    int Tq, Tk;           // rows of the tensors
    int causal;
    int max_level;        // above every level of find_block
};

// Forward launch.  A CTA has two tiles of 128 query rows of one sequence, with
// one key/value head: the same rows of two query heads (head_step = 1,
// tile_step = 0: groups of an even number of heads) or 256 rows of one head
// (head_step = 0, tile_step = 128).
struct PackedFwdParams : FwdParams {
    PackedSeqs seqs;
    int units;                 // heads, or pairs of heads
    int tile_step, head_step;
    int negate;                // 1: the scale is negative (scale_log2 holds its magnitude, never 0)
    long long o_row, o_head;   // strides of the output in elements
};
cudaError_t launch_packed_fwd_bf16(int d, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                   const PackedFwdParams& p, unsigned int grid, cudaStream_t stream);
cudaError_t launch_packed_fwd_f16(int d, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                  const PackedFwdParams& p, unsigned int grid, cudaStream_t stream);

// Backward: prep, main and dQ conversion as for a batch (fa_bwd_internal.h),
// with two differences.  The statistics and the dQ accumulator have whole
// blocks of 128 rows for every sequence (padded_row, fa_packed.cuh).  And a tile
// of 128 rows that reaches behind its sequence must not use the next one's rows
// (an infinity there, times a weight of 0, is a NaN) nor write them: the main
// kernel zeroes them in shared memory and stores such a block's rows one by one.
struct PackedMaps {  // of the whole tensors; dq: over the accumulator
    CUtensorMap q, k, v, dout, dk, dv, dq;
};
struct PackedAuxParams {
    PackedSeqs seqs;
    int H;
    int tiles;             // blocks of 128 rows per head of the statistics and of the accumulator
    const uint16_t* o;
    const uint16_t* dout;
    long long o_row, o_head, dout_row, dout_head;
    const float* lse;      // [H, Tq]
    float* stats;          // [H, tiles] blocks of kStatFloatsPerTile
    float* dq_acc;         // [H, 128 tiles, d]
    uint16_t* dq;
    long long dq_row, dq_head;
    float scale;
};
struct PackedBwdParams : BwdParams {
    PackedSeqs seqs;
    int tiles;
    uint16_t *dk, *dv;
    long long dk_row, dk_head, dv_row, dv_head;
};
cudaError_t launch_packed_prep(const PackedAuxParams& p, int d, bool f16, cudaStream_t stream);
cudaError_t launch_packed_dq(const PackedAuxParams& p, int d, bool f16, cudaStream_t stream);
cudaError_t launch_packed_bwd_bf16(int d, const PackedMaps& m, const PackedBwdParams& p, unsigned int grid, cudaStream_t stream);
cudaError_t launch_packed_bwd_f16(int d, const PackedMaps& m, const PackedBwdParams& p, unsigned int grid, cudaStream_t stream);

}  // namespace fa
