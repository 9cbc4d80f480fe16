// Which block of which sequence a CTA of a packed launch works on (device code
// shared by the forward and the backward kernel).
//
// The lengths are on the device, and a grid that follows them would need a
// kernel or a copy ahead of every call.  Instead each CTA finds its own block,
// with one warp, while the others set the CTA up.  Blocks are numbered by their
// work, heaviest first (in batches of up to kMostByWork sequences), so that a long
// sequence's last blocks do not begin at the end of the launch: with a mask block r of a sequence sees about r blocks
// of keys more than its first one, so blocks with the same `level` (first
// level of the sequence + r) cost about the same, and the number of blocks at
// or above a level is a sum over the sequences.  A binary search over the
// levels (their number is the logarithm of the longest sequence's blocks) and a
// prefix sum over the sequences find block `index`.  It takes one warp 2.2 us
// (16 sequences), which the loading of the block before hides in the forward kernel.
#pragma once

#include <cstdint>

#include "fa_packed.h"
#include "fa_ptx.cuh"

namespace fa {

struct SeqBlock {
    int q0, nq, k0, nk;  // the sequence's first query row, queries, first key row, keys
    int s;               // sequence
    int r;               // its block, -1: none, -2: nor has any `index` behind it
    int base;            // its first row in arrays that give every sequence whole blocks of 128 rows (padded_row)
};

// Rows of sequence s clamped to the tensors, whatever the offsets hold.
__device__ __forceinline__ void seq_rows(const PackedSeqs& p, int s, int& q0, int& nq, int& k0, int& nk) {
    q0 = min(max(p.cu_q[s], 0), p.Tq);
    nq = min(max(p.cu_q[s + 1], q0), p.Tq) - q0;
    k0 = min(max(p.cu_k[s], 0), p.Tk);
    nk = min(max(p.cu_k[s + 1], k0), p.Tk) - k0;
}

// A sequence's first row where each sequence begins on a multiple of 128 rows
// and has room for its rows rounded up to 128: no sum over the sequences
// before it is needed (the next one begins at least 128 ceil(n / 128) later).
__host__ __device__ __forceinline__ long long padded_row(long long first, long long s) {
    return (first & ~127ll) + 128ll * s;
}

// kKeys: blocks of keys (backward), else of queries (forward).  `rows`: a
// block's rows.  The blocks of sequence s have levels lo, lo + 1, .. with the
// mask and all lo without it.
template <bool kKeys>
__device__ __forceinline__ void seq_levels(const PackedSeqs& p, int rows, int nq, int nk, int& nb, int& lo) {
    const int qb = (nq + rows - 1) / rows, kb = (nk + rows - 1) / rows;
    if (kKeys) {
        nb = kb;  // keys from the sequence's end: the last block is seen by the last rows alone
        lo = p.causal ? 0 : qb;
    } else {
        nb = qb;
        lo = p.causal ? max(0, nk - nq) / rows : kb;
    }
}

// In batches of more sequences than kMostByWork the search by work, which reads
// all offsets many times, costs more than its order gains, and blocks go by the
// sequences' order, heaviest first within each.  Sequence s has the places from
// first_row / rows + s on (as in padded_row, no sum is needed), and the last
// sequence that begins at or before a place is found by a 32-way search; some
// places have no block.  Measured (24000 rows, H = 16/4, d = 128, causal, us by order
// and by work), forward: 100 sequences of 240 rows 99, 110; 300 of 80 106, 220;
// 1000 of 24 304, 1621; 4000 of 6 1165, 20540; 48 of 20 to 4000 rows (37325 in all) 296, 298.
// Backward: 1000 of 24 770, 1060; 48 of 20 to 4000 1127, 1069.
constexpr int kMostByWork = 64;

template <bool kKeys>
__device__ __forceinline__ SeqBlock find_in_order(const PackedSeqs& p, int rows, int units, unsigned int index, int& unit) {
    const int lane = static_cast<int>(threadIdx.x) % 32;
    const int T = kKeys ? p.Tk : p.Tq;
    const int32_t* cu = kKeys ? p.cu_k : p.cu_q;
    auto place_of = [&](int s) { return min(max(cu[s], 0), T) / rows + s; };
    const int places = min(max(cu[p.B], 0), T) / rows + p.B;
    SeqBlock out;
    out.r = -2;
    unit = 0;
    if (static_cast<unsigned long long>(places) * static_cast<unsigned>(units) <= index) return out;
    out.r = -1;
    int place;
    lpt_item(index, units, places, unit, place);
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, s = lo + (lane + 1) * step;
        const unsigned int begun = __ballot_sync(0xffffffffu, s < hi && place_of(s) <= place);
        lo += __popc(begun) * step;
        hi = min(hi, lo + step);
    }
    seq_rows(p, lo, out.q0, out.nq, out.k0, out.nk);
    const int nb = ((kKeys ? out.nk : out.nq) + rows - 1) / rows, r = place - place_of(lo);
    out.s = lo;
    out.base = static_cast<int>(padded_row(out.q0, lo));
    if (r >= 0 && r < nb) out.r = kKeys || !p.causal ? r : nb - 1 - r;
    return out;
}

// The block numbered blockIdx.x among `units` (heads) times the batch's
// blocks.  One whole warp.  Blocks of one unit's group (lpt_item) are taken
// together, so that the heads in flight share keys in L2.
template <bool kKeys>
__device__ __forceinline__ SeqBlock find_block(const PackedSeqs& p, int rows, int units, unsigned int index, int& unit) {
    if (p.B > kMostByWork) return find_in_order<kKeys>(p, rows, units, index, unit);
    const int lane = static_cast<int>(threadIdx.x) % 32;
    // a batch of at most 32 sequences stays in registers
    int nb0 = 0, lo0 = 0;
    if (lane < p.B) {
        int q0, nq, k0, nk;
        seq_rows(p, lane, q0, nq, k0, nk);
        seq_levels<kKeys>(p, rows, nq, nk, nb0, lo0);
    }
    auto at = [&](int s, int& nb, int& lo) {
        if (s < 32) {
            nb = nb0;
            lo = lo0;
            return;
        }
        int q0, nq, k0, nk;
        seq_rows(p, s, q0, nq, k0, nk);
        seq_levels<kKeys>(p, rows, nq, nk, nb, lo);
    };
    auto above = [&](int level) {  // blocks at `level` or above it
        int n = 0;
        for (int s = lane; s < p.B; s += 32) {
            int nb, lo;
            at(s, nb, lo);
            n += p.causal ? min(max(lo + nb - level, 0), nb) : (lo >= level ? nb : 0);
        }
        return __reduce_add_sync(0xffffffffu, n);
    };
    SeqBlock out;
    out.r = -2;
    unit = 0;
    const int total = above(0);
    if (total == 0 || static_cast<unsigned long long>(total) * static_cast<unsigned>(units) <= index) return out;
    int rank;
    lpt_item(index, units, total, unit, rank);
    // the level of block `rank`: above(level + 1) <= rank < above(level)
    int level = 0, past = p.max_level, higher = 0;
    while (past - level > 1) {
        const int mid = (level + past) / 2, n = above(mid);
        if (n > rank) {
            level = mid;
        } else {
            past = mid;
            higher = n;
        }
    }
    int left = rank - higher;
    for (int s0 = 0; s0 < p.B; s0 += 32) {
        const int s = s0 + lane;
        int nb = 0, lo = 0, n = 0;
        if (s < p.B) {
            at(s, nb, lo);
            n = p.causal ? (lo <= level && level < lo + nb ? 1 : 0) : (lo == level ? nb : 0);
        }
        int sum = n;  // inclusive over the lanes
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        const unsigned int hit = __ballot_sync(0xffffffffu, left < sum);
        if (hit != 0u) {
            const int src = __ffs(static_cast<int>(hit)) - 1;
            const int r = p.causal ? level - lo : left - (sum - n);
            out.r = __shfl_sync(0xffffffffu, r, src);
            out.s = s0 + src;
            seq_rows(p, s0 + src, out.q0, out.nq, out.k0, out.nk);
            out.base = static_cast<int>(padded_row(out.q0, s0 + src));
            if (kKeys && p.causal) out.r = (out.nk + rows - 1) / rows - 1 - out.r;
            return out;
        }
        left -= __shfl_sync(0xffffffffu, sum, 31);
    }
    return out;
}

}  // namespace fa
