// Forward kernel over packed sequences, sm_103a: the products, the softmax and
// their overlap are those of the forward kernel (fa_fwd_kernel.cuh: one CTA =
// two tiles of 128 query rows against one key/value head, two softmax
// warpgroups, an issuing warp for each).  What differs is the work around them.
//
// Packed batches have many short sequences, and a CTA that does one block of
// rows pays 9 us beside the block's key tiles (time stamps: 0.9 from the CTA
// before it on the SM, 2.2 to find its block, 2.4 until Q and K have landed,
// 1.7 to write O, 1.5 to tear down), as much as five tiles take.  So a CTA goes through
// many blocks without a pause.  The grid has a CTA for every block; a running
// CTA takes the next one's place before that one starts (cluster launch
// control), so blocks still begin in the grid's order, heaviest first, on the
// SM that is free first.
//   warps 0-7  softmax of tiles 0 and 1, as there; O leaves by 4 KB of shared
//              memory a warp, so that the query tiles are free for the next block
//   warp  8    issuer of tile 0, owner of tensor memory
//   warp  9    TMA producer, in the next block's tiles while this one ends
//   warp 10    issuer of tile 1
//   warp 11    asks for the next block, finds its sequence (find_block), and
//              zeroes what a sequence's last value tile has of the next one
// All ring and score barriers count tiles over the CTA's whole life.
//
// Rows past a sequence's end are the next sequence's.  Their scores are masked
// and their queries not stored; a value row, however, enters the product with
// weight 0, and 0 x infinity is not 0.  So a sequence's last value tile lands on a
// barrier of its own, and warp 11 hands it on with those rows zeroed.
//
// The same kernel (kPrefix) goes over the pages of a prefix that a batch of
// sequences shares: a block's rows are those of several sequences, its keys a
// partition of the prefix, its result a partial one (PrefixFwdParams).
//
// What bounds it: the tensor cores and, beside them, the exponentials, as in the
// forward kernel; below some 1000 rows a sequence the ends of the blocks.
// Measured (bf16, causal, H = 32 over 8, d = 128): sequences of 16384, 8191, 4096
// and 1000 rows 2.00 to 2.04 ms, 1450 to 1420 TFLOP/s (2.09 to 2.11 ms, 1380 to 1370, in
// longer runs, on several boxes); 16 of 17 to 2048 rows 143 us, 870 TFLOP/s;
// 64 of 128 rows 43 us at d = 64 (67 with a CTA per block).  Uniform lengths, against
// the batch's kernel: 1 x 8192 400 us (444), 16 x 512 62 us (98); without the mask
// 1 x 8192 774 us (750, as there the last wave's key range is split over idle SMs,
// which takes the lengths on the host).
//
// Every wait is bounded as in the forward kernel, those for a whole block (warp 11's
// for its loads, the others' for the next one, behind places without one) by kSweepLimits.
#pragma once

#include <cmath>
#include <cstdint>

#include "fa_fwd_kernel.cuh"
#include "fa_packed.cuh"
#include "fa_packed.h"
#include "fa_paged.h"

namespace fa {
namespace packed {

template <int D, bool F16>
struct Cfg : FwdCfg<false, D, F16> {
    using Base = FwdCfg<false, D, F16>;
    // A K stage less than there (d = 128), whose place the rows of O take on
    // their way out: 4 KB a warp, 32 rows of 64 channels.
    static constexpr int kKStages = D == 128 ? 2 : 4;
    static constexpr int kVStages = Base::kVStages;
    static constexpr int kOffV = Base::kOffK + kKStages * Base::kTileBytes;
    static constexpr int kOffRows = kOffV + kVStages * Base::kTileBytes;
    static constexpr int kOffBar = kOffRows + 8 * 4096;
    // barriers
    static constexpr int kBarQFull = 0;
    static constexpr int kBarQEmpty = 1;                             // both issuers' last scores of a block
    static constexpr int kBarKFull = 2;
    static constexpr int kBarKEmpty = kBarKFull + kKStages;
    static constexpr int kBarVFull = kBarKEmpty + kKStages;
    static constexpr int kBarVEmpty = kBarVFull + kVStages;
    static constexpr int kBarVRaw = kBarVEmpty + kVStages;     // a sequence's last value tile
    static constexpr int kBarSFull = kBarVRaw + 1;                   // [2] (not kStageDone)
    static constexpr int kBarSFree = kBarSFull + 2;                  // [2] kEarlyS: S_w read (4 warps)
    static constexpr int kBarPFull = kBarSFree + 2;                  // [2 tiles][2 halves]
    static constexpr int kBarOFull = kBarPFull + 4;                  // [2]
    static constexpr int kBarOFree = kBarOFull + 2;                  // [2] O_w read (4 warps)
    static constexpr int kBarDrain = kBarOFree + 2;                  // [2]
    static constexpr int kBarNext = kBarDrain + 2;                   // answer to the request for a block
    static constexpr int kBarBlockFull = kBarNext + 1;               // [2] a block's description
    static constexpr int kBarBlockEmpty = kBarBlockFull + 2;         // [2] every reader is done with the block
    static constexpr int kBarLoaded = kBarBlockEmpty + 2;            // the loads of a block are about to end
    static constexpr int kNumBars = kBarLoaded + 1;
    // Key tiles left to load when the next block is asked for.  Asking takes 1
    // us and finding the sequence 2, a tile 1.8; asked for at a block's start,
    // the last blocks lay with CTAs that had a long one before them (one
    // sequence of 8192, causal, H = 32/8, d = 128: 555 us, against 450 us).
    static constexpr int kAskAhead = 2;
    static constexpr int kOffAnswer = (kOffBar + kNumBars * 8 + 15) / 16 * 16;  // 16 bytes
    static constexpr int kOffBlocks = kOffAnswer + 16;               // int [2][8]
    static constexpr int kOffTmemSlot = kOffBlocks + 64;
    static constexpr int kOffAbort = kOffTmemSlot + 4;
    static constexpr int kOffTurnFlags = kOffAbort + 4;              // [2][4] u32
    static constexpr size_t kSmemBytes = static_cast<size_t>(kOffTurnFlags + 32) + 1024;  // alignment slack
    static_assert(kSmemBytes <= 232448, "shared memory budget exceeded");
};

// Instruction descriptor: the product of -A and B.
constexpr uint32_t kNegateA = 1u << 13;

// A block as its readers see it (kPrefix: q0 the first sequence, nq 0, k0 the
// first key tile, nk the prefix's keys, row0 the partition, head the key/value head).
struct Block {
    int q0, nq, k0, nk, row0, head;  // head of tile 0; row0: first row within the sequence; nq < 0: no more blocks
    int T;                           // key tiles that its last row sees
};

__device__ __forceinline__ Block block_of(const int4* in) {
    const int4 x = in[0], y = in[1];
    return {x.x, x.y, x.z, x.w, y.x, y.y, y.z};
}

// Ask for the CTA that would start next: its index, or the answer that there is
// none, arrives at `answer` (16 bytes) as transaction bytes on `bar`.
__device__ __forceinline__ void request_next(uint32_t answer, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     answer),
                 "r"(bar)
                 : "memory");
}
// The answer: true and the CTA's blockIdx.x, which will not start.
__device__ __forceinline__ bool read_next(uint32_t answer, unsigned int& index) {
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
        : "=r"(got), "=r"(x)
        : "r"(answer)
        : "memory");
    index = x;
    return got != 0u;
}

// Epilogue of a block, by one softmax warp: its 32 rows of O / lq (lane r has row
// r) by way of `stage` (4 KB of its own) as whole lines, the rows past `have`
// left out.  Not inlined: it runs once per block, and as a call it leaves the
// softmax loop's registers as they are (inlined, 312 to 388 bytes were spilled
// there at d = 128).  Straight from the lanes, a row each, 64 sequences of 128
// rows (H = 32/8, d = 128, causal) took 78 us, by shared memory 74.
template <int D, bool F16>
__device__ __noinline__ void store_rows(uint16_t* out, long long row_stride, int have, bool any, uint32_t tO, float inv_l,
                                        uint8_t* stage, uint32_t o_free) {
    const int lane = static_cast<int>(threadIdx.x) % 32;
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
        uint32_t o[2][32];
        if (any) {
            tmem_ld32(tO + 64u * h, o[0]);
            tmem_ld32(tO + 64u * h + 32u, o[1]);
            tmem_ld_wait(o[0]);
            tmem_ld_wait(o[1]);
        } else {  // no visible key: O = 0 (and lse = -inf)
#pragma unroll
            for (int e = 0; e < 32; ++e) o[0][e] = o[1][e] = 0u;
        }
        if (h == D / 64 - 1 && any) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free);
        }
        if (h > 0) __syncwarp();  // the rows before have been read
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const uint32_t(&x)[32] = o[c / 4];
            const int e = (c % 4) * 8;
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) =
                make_uint4(pack_16x2<F16>(u2f(x[e]) * inv_l, u2f(x[e + 1]) * inv_l),
                           pack_16x2<F16>(u2f(x[e + 2]) * inv_l, u2f(x[e + 3]) * inv_l),
                           pack_16x2<F16>(u2f(x[e + 4]) * inv_l, u2f(x[e + 5]) * inv_l),
                           pack_16x2<F16>(u2f(x[e + 6]) * inv_l, u2f(x[e + 7]) * inv_l));
        }
        __syncwarp();
        uint16_t* row = out + (lane / 8) * row_stride + 64 * h + (lane % 8) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + lane / 8;
            if (r < have)
                *reinterpret_cast<uint4*>(row) = *reinterpret_cast<const uint4*>(stage + r * 128 + (((lane ^ r) & 7) << 4));
            row += 4 * row_stride;
        }
    }
    __syncwarp();  // (the next block's rows go to the same place)
}

// Epilogue of a prefix's block: the warp's 32 rows of O as they are, lane r's row
// to row `out_row` of the partition's slab (-1: not a query row) by way of
// `stage`, and their statistics.
template <int D>
__device__ __noinline__ void store_part(float* o_part, float4* ml_part, long long out_row, uint32_t tO, float4 ml,
                                        uint8_t* stage, uint32_t o_free) {
    const int lane = static_cast<int>(threadIdx.x) % 32;
    if (out_row >= 0) ml_part[out_row] = ml;
#pragma unroll 1
    for (int q = 0; q < D / 32; ++q) {
        uint32_t o[32];
        tmem_ld32(tO + 32u * q, o);
        tmem_ld_wait(o);
        if (q == D / 32 - 1) tc_fence_before();
        __syncwarp();  // the rows before have been read (and, the last time, all loads are done)
        if (q == D / 32 - 1 && lane == 0) mbar_arrive(o_free);
#pragma unroll
        for (int c = 0; c < 8; ++c)
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) =
                make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + lane / 8;
            const long long row = __shfl_sync(0xffffffffu, out_row, r);
            if (row >= 0)
                *reinterpret_cast<uint4*>(o_part + row * D + 32 * q + (lane % 8) * 4) =
                    *reinterpret_cast<const uint4*>(stage + r * 128 + (((lane ^ r) & 7) << 4));
        }
    }
    __syncwarp();
}

template <int D, bool F16, bool kCausal, bool kPrefix, class Params>
__global__ void __launch_bounds__(kThreads, 1)
    fa_packed_fwd_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v, const Params p) {
    using C = Cfg<D, F16>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw_u32 & 1023u)) & 1023u;
    uint8_t* smem = smem_raw + pad;
    const uint32_t sbase = raw_u32 + pad;

    const int warp = static_cast<int>(threadIdx.x) / 32;
    const int lane = static_cast<int>(threadIdx.x) % 32;
    auto bar = [&](int i) -> uint32_t { return sbase + C::kOffBar + 8u * static_cast<uint32_t>(i); };
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::kOffAbort);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffTmemSlot);

    int tiles = 2;  // of a block; with one, the second issuer and warpgroup sit out
    if constexpr (kPrefix) tiles = 1 + p.pair;

    if (threadIdx.x == 0) {
        const unsigned int abort_gen = *reinterpret_cast<volatile unsigned int*>(&p.status->abort_gen);
        mbar_init(bar(C::kBarQFull), 1);
        mbar_init(bar(C::kBarQEmpty), tiles);
        for (int s = 0; s < C::kKStages; ++s) {
            mbar_init(bar(C::kBarKFull + s), 1);
            mbar_init(bar(C::kBarKEmpty + s), tiles);  // the issuers' commits
        }
        for (int s = 0; s < C::kVStages; ++s) {
            mbar_init(bar(C::kBarVFull + s), 1);
            mbar_init(bar(C::kBarVEmpty + s), tiles);
        }
        mbar_init(bar(C::kBarVRaw), 1);
        for (int w = 0; w < 2; ++w) {
            mbar_init(bar(C::kBarSFull + w), 1);
            mbar_init(bar(C::kBarSFree + w), 4);  // one arrival per softmax warp
            mbar_init(bar(C::kBarPFull + 2 * w + 0), 4);
            mbar_init(bar(C::kBarPFull + 2 * w + 1), 4);
            mbar_init(bar(C::kBarOFull + w), 1);
            mbar_init(bar(C::kBarOFree + w), 4);
            mbar_init(bar(C::kBarDrain + w), 1);
            mbar_init(bar(C::kBarBlockFull + w), 1);
            mbar_init(bar(C::kBarBlockEmpty + w), 5 * tiles + 1);  // softmax warps, issuers, producer
        }
        mbar_init(bar(C::kBarNext), 1);
        mbar_init(bar(C::kBarLoaded), 1);
        volatile uint32_t* tf = reinterpret_cast<volatile uint32_t*>(smem + C::kOffTurnFlags);
        for (int i = 0; i < 8; ++i) tf[i] = i < 4 ? 1u : 0u;
        *abort_flag = (abort_gen == p.gen) ? 1u : 0u;
        mbar_init_fence();
    }
    if (warp == kLoadWarp && lane == 0) {
        tma_prefetch_desc(&map_q);
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    // set up beside the kernel before; what it wrote is read behind this wait
    grid_wait();
    grid_release();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const bool skip = *abort_flag != 0u;

    // Block n of the CTA, for one of its readers; false when there is none (or the CTA gives up).
    auto block_info = [&](int n) { return reinterpret_cast<const int4*>(smem + C::kOffBlocks + (n & 1) * 32); };
    auto read_block = [&](int n, Block& b) -> bool {
        if (!wait_phase(bar(C::kBarBlockFull + (n & 1)), (n >> 1) & 1, abort_flag, p, 80, true, kSweepLimits)) return false;
        b = block_of(block_info(n));
        return b.nq >= 0;
    };
    auto done_block = [&](int n) { mbar_arrive(bar(C::kBarBlockEmpty + (n & 1))); };

    if (skip) {
        // nothing issued: go straight to the teardown
    } else if (warp >= 8) {
        regs_decrease<C::kOtherRegs>();
        if (warp == kTransposeWarp) {
            // ------------------------------------------------- blocks, tails
            unsigned int index = blockIdx.x;
            bool more = true, ok = true;
            int n = 0, tails = 0, asked = 0;
            // An index that has no block, nor any behind it: the grid is for all of the tensors' rows, of which the
            // offsets may use a few, and the places behind are taken without a search (1000 rows in use of 131072,
            // H = 32/8, d = 128, causal, in 3 and in 72 sequences: 39 and 70 us, by a search each 73 and 153).
            unsigned int past = 0xffffffffu;
            int tail_stage = -1, tail_rows = 0;  // of the block published last
            int G = 0;                           // key tiles of the blocks published
            while (ok) {
                Block b{};
                b.nq = -1;
                if (n > 0) {
                    ok = __all_sync(0xffffffffu, wait_phase(bar(C::kBarLoaded), (n - 1) & 1, abort_flag, p, 87, true, kSweepLimits));
                    if (!ok) break;
                }
                while (more) {
                    if (n > 0 || asked > 0) {  // (the first block is the CTA's own)
                        if (lane == 0) {
                            mbar_arrive_expect_tx(bar(C::kBarNext), 16);
                            request_next(sbase + C::kOffAnswer, bar(C::kBarNext));
                        }
                        ok = __all_sync(0xffffffffu, wait_phase(bar(C::kBarNext), (asked - 1) & 1, abort_flag, p, 81, false));
                        if (!ok) break;
                        more = read_next(sbase + C::kOffAnswer, index);
                        fence_proxy_async_smem();  // read before the next answer may be written
                        __syncwarp();
                        if (!more) break;
                    }
                    ++asked;
                    if constexpr (kPrefix) {
                        const int i = static_cast<int>(index), split = i % p.splits, rest = i / p.splits;
                        const int t0 = split * p.tiles_per_split;
                        b = {rest % p.blocks * tiles * p.seqs, 0, t0, p.Nkv, split, rest / p.blocks,
                             min(p.tiles_per_split, p.n_kv_tiles - t0)};
                        break;
                    } else if (index < past) {
                        int unit;
                        const SeqBlock f = find_block<false>(p.seqs, kTileM + p.tile_step, p.units, index, unit);
                        if (f.r >= 0) {
                            b = {f.q0, f.nq, f.k0, f.nk, f.r * (kTileM + p.tile_step), unit * (1 + p.head_step), 0};
                            int seen = f.nk;
                            if (kCausal) seen = min(f.nk, min(b.row0 + kTileM + p.tile_step, f.nq) + f.nk - f.nq);
                            b.T = seen <= 0 ? 0 : (seen + kTileN - 1) / kTileN;
                            break;
                        }
                        // (the grid is as large as any lengths need)
                        if (f.r == -2) past = index;
                    }
                }
                if (!ok) break;
                ok = __all_sync(0xffffffffu, wait_phase(bar(C::kBarBlockEmpty + (n & 1)), ((n >> 1) & 1) ^ 1, abort_flag, p, 82));
                if (!ok) break;
                if (lane == 0) {
                    int4* out = reinterpret_cast<int4*>(smem + C::kOffBlocks + (n & 1) * 32);
                    out[0] = make_int4(b.q0, b.nq, b.k0, b.nk);
                    out[1] = make_int4(b.row0, b.head, b.T, 0);
                    mbar_arrive(bar(C::kBarBlockFull + (n & 1)));
                }
                __syncwarp();
                // the last value tile of the block before, where its sequence ends in it
                if (tail_stage >= 0) {
                    ok = __all_sync(0xffffffffu, wait_phase(bar(C::kBarVRaw), tails & 1, abort_flag, p, 83));
                    if (!ok) break;
                    ++tails;
                    for (int a = 0; a < C::kAtoms; ++a) {
                        uint4* rows = reinterpret_cast<uint4*>(smem + C::kOffV + tail_stage * C::kTileBytes + a * C::kAtomBytes);
                        for (int i = tail_rows * 8 + lane; i < kTileN * 8; i += 32) rows[i] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::kBarVFull + tail_stage));
                }
                if (b.nq < 0) break;
                tail_stage = -1;
                G += b.T;
                const int end = b.nk - ((kPrefix ? b.k0 : 0) + b.T - 1) * kTileN;  // keys of the last tile
                if (b.T > 0 && end < kTileN) {
                    tail_stage = (G - 1) % C::kVStages;
                    tail_rows = end;
                }
                ++n;
            }
        } else if (warp == kLoadWarp) {
            // ------------------------------------------------- TMA producer
            // (a prefix's boxes are dealt to the lanes, a page of 64 channels each)
            if (lane == 0 || kPrefix) {
                const uint64_t keep = policy_evict_last();
                const uint64_t once = policy_evict_first();
                int G = 0, m = 0, tails = 0;  // tiles, blocks with tiles, and sequences' last tiles so far
                int nk = 0, nv = 0;           // K and V tiles whose loads were issued
                int last_tail = -C::kVStages;  // V tile that went to the barrier of its own
                bool ok = true;
                Block b;
                // every lane's wait, or the one lane's
                auto all = [&](bool got) -> bool { return kPrefix ? __all_sync(0xffffffffu, got) : got; };
                for (int n = 0; ok && all(read_block(n, b)); ++n) {
                    const bool tail = b.nk - ((kPrefix ? b.k0 : 0) + b.T - 1) * kTileN < kTileN;
                    // tile j's rows of K or V
                    [[maybe_unused]] int id = 0, pages = 0;  // (a prefix: this lane's page of the tile, and how many it has)
                    auto load = [&](uint32_t dst, const CUtensorMap* map, uint32_t full, int j) {
                        if constexpr (kPrefix) {
                            if (lane == 0)
                                mbar_arrive_expect_tx(full, static_cast<uint32_t>(pages * p.page * C::kAtoms * 128));
                            __syncwarp();
                            const int mine = lane / C::kAtoms, a = lane % C::kAtoms;
                            if (mine < pages)
                                tma_load_4d(dst + a * C::kAtomBytes + mine * p.page * 128, map, full, a * C::kAtomElems, 0,
                                            b.head, id, keep);
                            __syncwarp();
                        } else {
                            mbar_arrive_expect_tx(full, C::kTileBytes);
                            for (int a = 0; a < C::kAtoms; ++a)
                                tma_load_3d(dst + a * C::kAtomBytes, map, full, a * C::kAtomElems, b.k0 + j * kTileN,
                                            b.head / p.group, keep);
                        }
                    };
                    if (lane == 0 && b.T <= C::kAskAhead) mbar_arrive(bar(C::kBarLoaded));
                    for (int j = 0; j < b.T; ++j, ++G) {
                        if (lane == 0 && j > 0 && j == b.T - C::kAskAhead) mbar_arrive(bar(C::kBarLoaded));
                        if constexpr (kPrefix) {
                            const int page0 = (b.k0 + j) * (kTileN / p.page);
                            pages = min(kTileN / p.page, p.n_pages - page0);
                            id = lane / C::kAtoms < pages ? p.pages[page0 + lane / C::kAtoms] : 0;
                        }
                        const int ks = G % C::kKStages;
                        ok = all(wait_phase(bar(C::kBarKEmpty + ks), ((G / C::kKStages) & 1) ^ 1, abort_flag, p, 1));
                        if (!ok) break;
                        load(sbase + C::kOffK + ks * C::kTileBytes, &map_k, bar(C::kBarKFull + ks), j);
                        nk = G + 1;
                        if (j == 0) {
                            ok = all(wait_phase(bar(C::kBarQEmpty), (m & 1) ^ 1, abort_flag, p, 84));
                            if (!ok) break;
                            if constexpr (kPrefix) {
                                if (lane == 0) {
                                    mbar_arrive_expect_tx(bar(C::kBarQFull),
                                                          static_cast<uint32_t>(tiles * C::kAtoms * p.rows * p.seqs * 128));
                                    for (int w = 0; w < tiles; ++w)
                                        for (int a = 0; a < C::kAtoms; ++a)
                                            tma_load_4d(sbase + C::kOffQ + w * C::kTileBytes + a * C::kAtomBytes, &map_q,
                                                        bar(C::kBarQFull), a * C::kAtomElems, 0, b.head, b.q0 + w * p.seqs, keep);
                                }
                                __syncwarp();
                            } else {
                                mbar_arrive_expect_tx(bar(C::kBarQFull), 2u * C::kTileBytes);
                                for (int w = 0; w < 2; ++w)
                                    for (int a = 0; a < C::kAtoms; ++a)
                                        tma_load_3d(sbase + C::kOffQ + w * C::kTileBytes + a * C::kAtomBytes, &map_q,
                                                    bar(C::kBarQFull), a * C::kAtomElems, b.q0 + b.row0 + w * p.tile_step,
                                                    b.head + w * p.head_step, once);
                            }
                            ++m;
                        }
                        const int vs = G % C::kVStages;
                        ok = all(wait_phase(bar(C::kBarVEmpty + vs), ((G / C::kVStages) & 1) ^ 1, abort_flag, p, 2));
                        if (!ok) break;
                        uint32_t vbar = bar(C::kBarVFull + vs);
                        if (tail && j + 1 == b.T) {
                            // the tail before has been handed on (long ago where its stage was loaded again since)
                            if (G - last_tail < C::kVStages)
                                ok = all(wait_phase(bar(C::kBarVFull + last_tail % C::kVStages),
                                                    (last_tail / C::kVStages) & 1, abort_flag, p, 86));
                            if (!ok) break;
                            vbar = bar(C::kBarVRaw);
                            last_tail = G;
                            ++tails;
                        }
                        load(sbase + C::kOffV + vs * C::kTileBytes, &map_v, vbar, j);
                        nv = G + 1;
                    }
                    if (lane == 0) done_block(n);
                }
                // Drain: every load has landed before the CTA may exit.
                if (m > 0) wait_phase(bar(C::kBarQFull), (m - 1) & 1, abort_flag, p, 3, false);
                for (int s = 0; s < C::kKStages && s < nk; ++s) {
                    const int last = s + ((nk - 1 - s) / C::kKStages) * C::kKStages;
                    wait_phase(bar(C::kBarKFull + s), (last / C::kKStages) & 1, abort_flag, p, 3, false);
                }
                if (tails > 0) wait_phase(bar(C::kBarVRaw), (tails - 1) & 1, abort_flag, p, 3, false);
                for (int s = 0; s < C::kVStages && s < nv; ++s) {
                    const int last = s + ((nv - 1 - s) / C::kVStages) * C::kVStages;
                    if (last == last_tail) continue;  // (its other barrier is warp 11's to complete)
                    wait_phase(bar(C::kBarVFull + s), (last / C::kVStages) & 1, abort_flag, p, 3, false);
                }
            }
        } else if (lane == 0 && (warp == kMmaWarp || tiles == 2)) {
            // ------------------------------------------ tensor-core issuers
            const int w = (warp == kMmaWarp) ? 0 : 1;
            const uint32_t dS = tmem + 128u * static_cast<uint32_t>(w);
            const uint32_t dO = tmem + C::kColO + static_cast<uint32_t>(D * w);
            const uint32_t dP = C::kEarlyS ? tmem + C::kColP + 64u * static_cast<uint32_t>(w) : dS;
            const uint32_t sQ = sbase + C::kOffQ + w * C::kTileBytes;
            constexpr bool kDescAdd = D == 128;  // see the forward kernel
            const uint64_t dQ0 = smem_desc_sw128(sQ, 16, 1024);
            const uint32_t idesc_qk = C::kIdescQK | (p.negate ? kNegateA : 0u);
            auto issue_qk = [&](int ks) {
                const uint32_t sK = sbase + C::kOffK + ks * C::kTileBytes;
                const uint64_t dK0 = smem_desc_sw128(sK, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < C::kQkSteps; ++kk) {
                    const uint32_t off = (kk * 32) / 128 * C::kAtomBytes + (kk * 32) % 128;
                    const uint64_t da = kDescAdd ? dQ0 + (off >> 4) : smem_desc_sw128(sQ + off, 16, 1024);
                    const uint64_t db = kDescAdd ? dK0 + (off >> 4) : smem_desc_sw128(sK + off, 16, 1024);
                    mma_ss<false>(dS, da, db, idesc_qk, kk > 0 ? 1u : 0u);
                }
            };
            auto issue_pv = [&](int vs, bool accumulate, int k0, int k1) {
                const uint32_t sV = sbase + C::kOffV + vs * C::kTileBytes;
#pragma unroll
                for (int kk = k0; kk < k1; ++kk) {
                    const uint64_t db = kDescAdd ? smem_desc_sw128(sV, C::kAtomBytes, 1024) + ((kk * C::kUmmaK * 128) >> 4)
                                                 : smem_desc_sw128(sV + kk * C::kUmmaK * 128, C::kAtomBytes, 1024);
                    mma_ts<false>(dO, dP + kk * 8, db, C::kIdescPV, (accumulate || kk > 0) ? 1u : 0u);
                }
            };
            // scores of tile G; `last`: the block's last, behind which its queries are free
            auto scores = [&](int G, bool last) -> bool {
                const int ks = G % C::kKStages;
                if (!wait_phase(bar(C::kBarKFull + ks), (G / C::kKStages) & 1, abort_flag, p, 7)) return false;
                tc_fence_after();
                issue_qk(ks);
                if (!C::kStageDone) tc_commit(bar(C::kBarSFull + w));
                tc_commit(bar(C::kBarKEmpty + ks));
                if (last) tc_commit(bar(C::kBarQEmpty));
                return true;
            };
            int G = 0, m = 0;  // tiles and blocks with tiles so far
            bool ok = true;
            Block b;
            for (int n = 0; ok && read_block(n, b); ++n) {
                const int T = b.T;
                if (T > 0) {
                    ok = wait_phase(bar(C::kBarQFull), m & 1, abort_flag, p, 4);
                    // (kEarlyS) the block before has been read out of S
                    if (ok && C::kEarlyS && G > 0) ok = wait_phase(bar(C::kBarSFree + w), (G - 1) & 1, abort_flag, p, 14);
                    if (ok) ok = scores(G, T == 1);
                }
                for (int j = 0; ok && j < T; ++j) {
                    const int g = G + j, vs = g % C::kVStages;
                    if (C::kEarlyS && j + 1 < T) {
                        // S(j+1) as soon as the softmax has read S(j)
                        ok = wait_phase(bar(C::kBarSFree + w), g & 1, abort_flag, p, 14) && scores(g + 1, j + 2 == T);
                        if (!ok) break;
                    }
                    ok = wait_phase(bar(C::kBarVFull + vs), (g / C::kVStages) & 1, abort_flag, p, 5);
                    if (!ok) break;
                    // O of the block before has been read
                    if (j == 0 && m > 0) ok = wait_phase(bar(C::kBarOFree + w), (m - 1) & 1, abort_flag, p, 85);
                    if (ok) ok = wait_phase(bar(C::kBarPFull + 2 * w), g & 1, abort_flag, p, 6);
                    if (!ok) break;
                    tc_fence_after();
                    issue_pv(vs, j > 0, 0, C::kPvSteps / 2);
                    ok = wait_phase(bar(C::kBarPFull + 2 * w + 1), g & 1, abort_flag, p, 6);
                    if (!ok) break;
                    tc_fence_after();
                    issue_pv(vs, true, C::kPvSteps / 2, C::kPvSteps);
                    tc_commit(bar(C::kBarVEmpty + vs));
                    if (j + 1 == T) {
                        tc_commit(bar(C::kBarOFull + w));
                    } else if (!C::kEarlyS) {
                        ok = scores(g + 1, j + 2 == T);
                    }
                }
                G += T;
                if (T > 0) ++m;
                done_block(n);
            }
            // every tensor-core operation has completed before tensor memory is released
            tc_commit(bar(C::kBarDrain + w));
            wait_phase(bar(C::kBarDrain + w), 0, abort_flag, p, 9, false);
        }
    } else if (warp < 4 * tiles) {
        // ------------------------------------------------ softmax warpgroups
        // The forward kernel's loop (its comments there) in less code: a short
        // sequence's tiles are full, masked, first and last ones in turn, and
        // with a path of its own for each the instruction cache did not hold
        // them (16 sequences of 512, causal, d = 128: 3.5 warps in a scheduler's
        // ten waited for instructions).  Masked scores are -inf, so that their weights
        // come out as 0 by the same path; a negative scale is taken into the
        // product (kNegateA), so that the reference is a maximum; and the maximum
        // comes with the scores, so that nothing is gained by exponentials ahead of it.
        regs_increase<C::kSoftmaxRegs>();
        const int w = warp / 4;
        const int wi = warp % 4;
        const int t = wi * 32 + lane;
        const uint32_t lane_off = static_cast<uint32_t>(wi * 32) << 16;
        const uint32_t tS = tmem + lane_off + 128u * static_cast<uint32_t>(w);
        const uint32_t tO = tmem + lane_off + C::kColO + static_cast<uint32_t>(D * w);
        const uint32_t tP = C::kEarlyS ? tmem + lane_off + C::kColP + 64u * static_cast<uint32_t>(w) : tS;
        const float c = p.scale_log2;
        volatile uint32_t* const turn_mine = reinterpret_cast<volatile uint32_t*>(smem + C::kOffTurnFlags) + 4 * w + wi;
        volatile uint32_t* const turn_other =
            reinterpret_cast<volatile uint32_t*>(smem + C::kOffTurnFlags) + 4 * (1 - w) + wi;
        int G = 0, m = 0;  // tiles and blocks with tiles so far; G counts on inside a block
        // hand the turn to the other warpgroup after this one's tile G, warp to
        // warp through shared counters, with the mask too (by barriers 16384
        // causal keys and shorter sequences beside them took 2073 us, so 2014)
        auto pass_turn = [&]() { *turn_other = static_cast<uint32_t>(G + 1 + w); };
        bool ok = true;
        for (int n = 0; ok; ++n) {
            int row_limit, T;
            {
                Block b;
                if (!__all_sync(0xffffffffu, read_block(n, b))) break;
                if constexpr (kPrefix) {
                    row_limit = b.nk - b.k0 * kTileN;  // keys from the partition's first tile on
                } else {
                    const int i = b.row0 + w * p.tile_step + t;  // this thread's row of the sequence
                    row_limit = kCausal ? max(-1, min(b.nk, i + 1 + b.nk - b.nq)) : b.nk;
                }
                T = b.T;
            }
            float m_ref = -INFINITY, l = 0.0f, lq = 0.0f;
            for (int j = 0; j < T; ++j, ++G) {
                bool got = C::kStageDone ? wait_phase(bar(C::kBarKEmpty + G % C::kKStages), (G / C::kKStages) & 1,
                                                      abort_flag, p, 10)
                                         : wait_phase(bar(C::kBarSFull + w), G & 1, abort_flag, p, 10);
                ok = __all_sync(0xffffffffu, got);
                if (!ok) break;
                if (C::kTakeTurns && tiles == 2) {
                    got = wait_flag(turn_mine, static_cast<uint32_t>(G + 1), abort_flag, p, 13);
                    ok = __all_sync(0xffffffffu, got);
                    if (!ok) break;
                }
                tc_fence_after();

                // the scores and each 32-key quarter's maximum (reducing load)
                uint32_t s[4][32];
                float qmax[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld32_max(tS + 32u * q, s[q], qmax[q]);
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld_wait_red(s[q], qmax[q]);
                if constexpr (C::kEarlyS) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::kBarSFree + w));
                }
                float mx = fmaxf(fmax3(qmax[0], qmax[1], qmax[2]), qmax[3]);
                const int valid = row_limit - j * kTileN;  // keys of this tile that the row sees
                if (kCausal ? __any_sync(0xffffffffu, valid < kTileN) : (valid < kTileN)) {
                    // the others' weights are 2^-inf
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (q * 32 + e >= valid) s[q][e] = 0xff800000u;
                    mx = row_extreme<true>(s);
                }

                // lazy reference, as in the forward kernel
                const float m_new = fmaxf(m_ref, mx * c);
                const bool need = m_new > m_ref + kRescaleThreshold;  // always true on the first tile
                const float alpha = need ? ex2(m_ref - m_new) : 1.0f;
                if (need) {
                    l *= alpha;
                    lq *= alpha;
                    m_ref = m_new;
                }
                const float shift = (m_ref == -INFINITY) ? 0.0f : m_ref;
                const uint64_t c2 = f2_pack(c, c);
                const uint64_t ns2 = f2_pack(-shift, -shift);
                uint64_t acc[4] = {0, 0, 0, 0};
                // (kEarlyS: the first half's exponentials run ahead of the wait below)
                uint32_t pw[32];
                if constexpr (C::kEarlyS) exp_half_regs<F16>(s, c2, ns2, 0, pw, acc);
                // kEarlyS: P_w and O_w hold the tile before's product until it completes
                if (C::kEarlyS && j > 0) {
                    ok = __all_sync(0xffffffffu, wait_phase(bar(C::kBarVEmpty + (G - 1) % C::kVStages),
                                                            ((G - 1) / C::kVStages) & 1, abort_flag, p, 15));
                    if (!ok) break;
                }
                if (j > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll 1
                    for (int q = 0; q < D / 32; ++q) {
                        uint32_t o[32];
                        tmem_ld32(tO + 32u * q, o);
                        tmem_ld_wait(o);
                        const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float x0, x1;
                            f2_unpack(f2_mul(f2_pack(u2f(o[e]), u2f(o[e + 1])), a2), x0, x1);
                            o[e] = f2u(x0);
                            o[e + 1] = f2u(x1);
                        }
                        tmem_st32(tO + 32u * q, o);
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (C::kEarlyS && h == 0) tmem_st32(tP, pw);
                    else exp_half<false, F16, false>(s, c2, ns2, 0, tP, h, acc);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::kBarPFull + 2 * w + h));
                    if (C::kTakeTurns && tiles == 2 && h == C::kTurnAfterHalf && lane == 0) pass_turn();
                }
                const float tsum = sum8(acc);
                const float pmax = ex2(fmaf(mx, c, -shift));
                const float pmax_r = widen_lo16<F16>(pack_16x2<F16>(pmax, 0.0f));
                l += tsum;
                lq += tsum + (pmax_r - pmax);
            }
            if (!ok) break;

            if (T > 0) {
                ok = __all_sync(0xffffffffu, wait_phase(bar(C::kBarOFull + w), m & 1, abort_flag, p, 11));
                if (!ok) break;
                tc_fence_after();
            }
            if constexpr (kPrefix) {
                const Block b = block_of(block_info(n));
                const int seq = b.q0 + w * p.seqs + t / p.rows;
                const long long row = t < p.rows * p.seqs && seq < p.B
                                          ? (static_cast<long long>(seq) * p.H_kv + b.head) * p.rows + t % p.rows : -1;
                const long long slab = b.row0 * p.part_rows;
                store_part<D>(p.o_part + slab * D, reinterpret_cast<float4*>(p.ml_part) + slab, row, tO,
                              make_float4(m_ref, l, lq, 0.0f), smem + C::kOffRows + warp * 4096, bar(C::kBarOFree + w));
            } else {
                const Block b = block_of(block_info(n));
                const int head = b.head + w * p.head_step;
                const int row0 = b.row0 + w * p.tile_step;  // the tile's first row of the sequence
                if (p.lse != nullptr && row0 + t < b.nq)
                    p.lse[static_cast<size_t>(head) * p.seqs.Tq + b.q0 + row0 + t] =
                        (l > 0.0f ? m_ref + log2f(l) : -INFINITY) * 0.69314718055994531f;
                store_rows<D, F16>(static_cast<uint16_t*>(p.out) + static_cast<size_t>(b.q0 + row0 + wi * 32) * p.o_row +
                                       static_cast<size_t>(head) * p.o_head,
                                   p.o_row, b.nq - (row0 + wi * 32), T > 0, tO, lq > 0.0f ? 1.0f / lq : 0.0f,
                                   smem + C::kOffRows + warp * 4096, bar(C::kBarOFree + w));
            }
            if (T > 0) ++m;
            __syncwarp();
            if (lane == 0) done_block(n);
        }
    }

    // --------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// `grid`: CTAs enough for any lengths.
template <int D, bool F16, bool kCausal>
cudaError_t launch_variant(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PackedFwdParams& p,
                           unsigned int grid, cudaStream_t stream) {
    using C = Cfg<D, F16>;
    auto kern = fa_packed_fwd_kernel<D, F16, kCausal, false, PackedFwdParams>;
    static SmemAllowed allowed;
    const cudaError_t e = allow_smem_regs(reinterpret_cast<const void*>(kern), static_cast<int>(C::kSmemBytes),
                                          static_cast<int>(kLaunchRegs), allowed);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(grid), kThreads, C::kSmemBytes, stream, q, k, v, p);
}

// A prefix.  (The kernel behind it relies on this one to let it be set up only
// behind its own wait.)
template <int D, bool F16>
cudaError_t launch_prefix(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PrefixFwdParams& p,
                          cudaStream_t stream) {
    using C = Cfg<D, F16>;
    auto kern = fa_packed_fwd_kernel<D, F16, false, true, PrefixFwdParams>;
    static SmemAllowed allowed;
    const cudaError_t e = allow_smem_regs(reinterpret_cast<const void*>(kern), static_cast<int>(C::kSmemBytes),
                                          static_cast<int>(kLaunchRegs), allowed);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(static_cast<unsigned>(p.H_kv * p.blocks * p.splits)), kThreads, C::kSmemBytes, stream, q,
                            k, v, p);
}

}  // namespace packed
}  // namespace fa
