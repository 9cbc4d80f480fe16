// Backward pass over packed sequences: the two memory-bound kernels around the
// main one (fa_bwd_kernel.cuh).
//   prep: per query row D = dO . O, the negated base-2 log-sum-exp and a zeroed
//         row of the fp32 dQ accumulator;
//   dq:   dQ = scale * accumulator in the input dtype.
// What bounds them: memory.  For 16384 rows of 32 heads, d = 128: prep 82 us for 537
// MB (6.5 TB/s: o and dO read, the accumulator's zeros written), dq 56 us for 403
// MB (7.2 TB/s, part of the accumulator being in L2 still).
// A block has one tile of 128 rows of one head; rows of 16-byte chunks, d / 8
// lanes a row, so that a warp reads whole lines whatever the strides.
#include <cmath>
#include <cstdint>

#include "fa_kv4.h"
#include "fa_packed.cuh"
#include "fa_packed.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kAuxThreads = 256;

// The tile's sequence and its first row there; false: no sequence has rows in it.
__device__ __forceinline__ bool find_tile(const PackedSeqs& p, int tile, int& q0, int& first, int& rows) {
    int lo = 0, hi = p.B;  // the last sequence that begins at or before the tile
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        const int at = min(max(p.cu_q[mid], 0), p.Tq);
        if (padded_row(at, mid) / 128 <= tile) lo = mid;
        else hi = mid;
    }
    int nq, k0, nk;
    seq_rows(p, lo, q0, nq, k0, nk);
    first = 128 * tile - static_cast<int>(padded_row(q0, lo));
    rows = min(nq - first, 128);
    return first >= 0 && rows > 0;
}

template <int D, bool F16>
__global__ void __launch_bounds__(kAuxThreads) fa_packed_prep_kernel(const PackedAuxParams p) {
    grid_wait();
    grid_release();
    constexpr int kLanes = D / 8;                  // lanes of a row
    constexpr int kStep = kAuxThreads / kLanes;    // rows at a time
    const int tile = static_cast<int>(blockIdx.x), head = static_cast<int>(blockIdx.y);
    int q0, first, rows;
    if (!find_tile(p.seqs, tile, q0, first, rows)) return;
    const int c = static_cast<int>(threadIdx.x) % kLanes;
    float* st = p.stats + (static_cast<size_t>(head) * p.tiles + tile) * kStatFloatsPerTile;
    float* acc = p.dq_acc + (static_cast<size_t>(head) * p.tiles + tile) * 128 * D + c * 8;
#pragma unroll 4
    for (int r = static_cast<int>(threadIdx.x) / kLanes; r < 128; r += kStep) {
        float sum = 0.0f;
        if (r < rows) {
            const size_t row = static_cast<size_t>(q0 + first + r);
            const uint4 o = *reinterpret_cast<const uint4*>(p.o + row * p.o_row + head * p.o_head + c * 8);
            const uint4 g = *reinterpret_cast<const uint4*>(p.dout + row * p.dout_row + head * p.dout_head + c * 8);
            const uint32_t ow[4] = {o.x, o.y, o.z, o.w}, gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sum += widen_lo16<F16>(ow[i]) * widen_lo16<F16>(gw[i]) + widen_lo16<F16>(ow[i] >> 16) * widen_lo16<F16>(gw[i] >> 16);
            float4* z = reinterpret_cast<float4*>(acc + static_cast<size_t>(r) * D);
            z[0] = z[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (c == 0) {
            // rows behind the sequence's end and rows that see no key: weight 0
            float neg = -INFINITY;
            if (r < rows) {
                const float lse = p.lse[static_cast<size_t>(head) * p.seqs.Tq + q0 + first + r];
                if (lse != -INFINITY) neg = -lse * 1.4426950408889634f;
            }
            st[r] = neg;
            st[128 + r] = sum;
        }
    }
}

template <int D, bool F16>
__global__ void __launch_bounds__(kAuxThreads) fa_packed_dq_kernel(const PackedAuxParams p) {
    grid_wait();
    grid_release();
    constexpr int kLanes = D / 8, kStep = kAuxThreads / kLanes;
    const int tile = static_cast<int>(blockIdx.x), head = static_cast<int>(blockIdx.y);
    int q0, first, rows;
    if (!find_tile(p.seqs, tile, q0, first, rows)) return;
    const int c = static_cast<int>(threadIdx.x) % kLanes;
    const float* acc = p.dq_acc + (static_cast<size_t>(head) * p.tiles + tile) * 128 * D + c * 8;
    const float s = p.scale;
#pragma unroll 4
    for (int r = static_cast<int>(threadIdx.x) / kLanes; r < rows; r += kStep) {
        const float4 a = *reinterpret_cast<const float4*>(acc + static_cast<size_t>(r) * D);
        const float4 b = *reinterpret_cast<const float4*>(acc + static_cast<size_t>(r) * D + 4);
        *reinterpret_cast<uint4*>(p.dq + static_cast<size_t>(q0 + first + r) * p.dq_row + head * p.dq_head + c * 8) =
            make_uint4(pack_16x2<F16>(a.x * s, a.y * s), pack_16x2<F16>(a.z * s, a.w * s),
                       pack_16x2<F16>(b.x * s, b.y * s), pack_16x2<F16>(b.z * s, b.w * s));
    }
}

}  // namespace

cudaError_t launch_packed_prep(const PackedAuxParams& p, int d, bool f16, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(p.tiles), static_cast<unsigned>(p.H));
    auto kern = d == 64 ? (f16 ? fa_packed_prep_kernel<64, true> : fa_packed_prep_kernel<64, false>)
                        : (f16 ? fa_packed_prep_kernel<128, true> : fa_packed_prep_kernel<128, false>);
    return launch_dependent(kern, grid, kAuxThreads, 0, stream, p);
}

cudaError_t launch_packed_dq(const PackedAuxParams& p, int d, bool f16, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(p.tiles), static_cast<unsigned>(p.H));
    auto kern = d == 64 ? (f16 ? fa_packed_dq_kernel<64, true> : fa_packed_dq_kernel<64, false>)
                        : (f16 ? fa_packed_dq_kernel<128, true> : fa_packed_dq_kernel<128, false>);
    return launch_dependent(kern, grid, kAuxThreads, 0, stream, p);
}

}  // namespace fa
