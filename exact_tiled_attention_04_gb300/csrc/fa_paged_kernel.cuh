// Attention of short query blocks (decode steps, drafts) over a paged
// key/value cache, sm_103a: the online softmax of "FlashAttention dissected",
// section "Algorithmic core in pseudocode", over key partitions (its section
// "Interaction with the KV cache during inference").
//
// The products are those of the decode kernel (fa_decode_kernel.cuh), keys on
// the tensor-memory lanes:  S^T = K_j Q^T (128 keys x NR rows), P^T = 2^(c S^T -
// m), O^T += V_j^T P^T, with one reference maximum per row for the warpgroup.
//
// What bounds it: reading the cache.  Sequences have different lengths, known
// on the device alone, so the tiles of all units are cut into equal runs, one
// per CTA (one CTA an SM): none idles because a sequence is short, and a long
// one is shared by many.  A CTA goes through the units of its run without a
// pause: the loading warp is up to a ring ahead, in the next unit's keys while
// the softmax still ends this one, Q, S^T and O^T have two buffers each, and two
// softmax warpgroups take the units in turn, as the ends of one (its last
// product, the sums over 128 threads, its rows' way out) take as long as three of
// its tiles (64 sequences of up to 512 slots behind a prefix of 8192: 52.5 us
// against 60.7 with one).  A warp issues the scores and another the products with
// V: one thread's instructions for both, 1.2 us a tile, were more than the tile's
// 64 KB take (1.45 us on all SMs, less on some): 64 sequences of 256 slots 16.5 us
// against 17.7.  K's stage of the ring is free a product before V's.
// Of a unit cut between CTAs each leaves a partial result, at most two a CTA,
// which a second kernel adds up in order, so results do not depend on timing.
//
// Measured: 32 sequences of up to 16384 slots (H = 32 over 8, d = 128, bf16, pages
// of 64) 164 to 165 us, 6.7 TB/s of keys and values; 64 of 128, 512, 1024 and 4096
// slots 11.5, 25.8, 46.8 and 159 us, about 7 us and their bytes (32 of 16384 in pages of
// 128, 64, 32 and 16: 307, 310, 316 and 336 us; d = 64 163, 165, 173 and 207); of more than 32
// rows a head each block of 32 is a unit that reads the head's keys and values again (16 of 4096
// slots, 32, 64, 96 and 128 rows 52, 92, 130 and 168 us; d = 64 38, 67, 95 and 121); four of up to 1000
// (8 over 2, d = 64) 7.2 to 7.5 us, the depth of the two kernels: set-up, the run's place, the
// first tile, the unit's end, the second kernel.
//
// Pages.  A tile of 128 keys is 128 / page boxes of a tensor map over
// [pages, H_kv, page, d] each for K and V, one per lane of the loading warp.  Pages behind the
// last one in use are not loaded and a number outside the pool reads as
// zeros.  Value rows behind a sequence's end hold anything; their weight is 0, but 0 x
// infinity is not, so the softmax threads zero them in shared memory.
#pragma once

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "fa_decode_kernel.cuh"
#include "fa_paged.h"

namespace fa {
namespace paged {

// NV: query rows of a block, 4, 8, 16 or 32; the products' N is at least 16.
template <int D, bool F16, int NV>
struct Cfg {
    static constexpr int NR = NV < 16 ? 16 : NV;
    static constexpr int kAtomElems = 64;
    static constexpr int kAtoms = D / kAtomElems;
    static constexpr int kAtomBytes = 128 * 128;            // 128 keys x 128 bytes
    static constexpr int kTileBytes = kAtoms * kAtomBytes;  // 128 keys x D
    static constexpr int kRowAtomBytes = NR * 128;          // NR rows x 128 bytes
    static constexpr int kQBytes = kAtoms * kRowAtomBytes;
    static constexpr int kUmmaK = 16;
    static constexpr int kQkSteps = D / kUmmaK;
    static constexpr int kPvSteps = 128 / kUmmaK;
    static constexpr int kStages = D == 128 ? 3 : 6;  // of K, and of V
    // Softmax warpgroups: two take the run's units in turn (at 32 rows their
    // registers would not fit).
    static constexpr int kGroups = NR == 16 ? 2 : 1;
    // Issuers of the scores (and owner of tensor memory) and of the products with V.
    static constexpr int kMmaWarp = 4 * kGroups, kLoadWarp = kMmaWarp + 1, kPvWarp = kMmaWarp + 2;
    static constexpr int kThreads = (kPvWarp + 1) * 32;
    static constexpr uint32_t kFmt = F16 ? 0u : 1u;
    static constexpr uint32_t kIdescQK = instr_desc(kFmt, false, false, 128, NR);
    static constexpr uint32_t kIdescPV = instr_desc(kFmt, true, false, 128, NR);
    // tensor memory
    static constexpr uint32_t kColS = 0;       // [2] x NR
    static constexpr uint32_t kColO = 2 * NR;  // [2] x NR
    static constexpr uint32_t kTmemCols = 4 * NR;
    static_assert(kTmemCols == 64 || kTmemCols == 128, "columns are allocated in powers of two");
    // shared memory; V first: at d = 64 the padded half of V^T is read 16 KB
    // past a V tile, which stays inside the V and K rings
    static constexpr int kOffV = 0;                             // [kStages]
    static constexpr int kOffK = kOffV + kStages * kTileBytes;  // [kStages]
    static constexpr int kOffQ = kOffK + kStages * kTileBytes;  // [2] x kAtoms x NR rows
    static constexpr int kOffP = kOffQ + 2 * kQBytes;           // [2] x 2 atoms x NR rows
    // of a group, floats: row maxima, sums l and lq of each warp [3][4][NV]; references [NV]
    static constexpr int kRedFloats = 13 * NV;
    static constexpr int kOffRed = kOffP + 2 * 2 * kRowAtomBytes;  // [kGroups]
    static constexpr int kOffBar = kOffRed + kGroups * kRedFloats * 4;
    // barriers
    static constexpr int kBarQFull = 0;                   // [2] a unit's Q landed
    static constexpr int kBarQEmpty = kBarQFull + 2;      // [2] its last scores are computed
    static constexpr int kBarFull = kBarQEmpty + 2;           // [K, V][kStages] a tile landed
    static constexpr int kBarEmpty = kBarFull + 2 * kStages;  // [K, V][kStages] its product is done
    static constexpr int kBarS = kBarEmpty + 2 * kStages;     // [kGroups][2] S^T buffer ready, by the group's own count of tiles
    static constexpr int kBarP = kBarS + 2 * kGroups;     // [2] P^T buffer written (4 warps)
    static constexpr int kBarPFree = kBarP + 2;           // [2] the product reading it is done
    static constexpr int kBarO = kBarPFree + 2;           // [2] every product of a unit is done
    static constexpr int kBarOFree = kBarO + 2;           // [2] its O^T was read (4 warps)
    static constexpr int kBarDrain = kBarOFree + 2;       // both issuers' last products are done
    static constexpr int kNumBars = kBarDrain + 1;
    static constexpr int kOffTmemSlot = kOffBar + kNumBars * 8;
    static constexpr int kOffAbort = kOffTmemSlot + 4;
    static constexpr int kOffPlan = kOffAbort + 4;        // int [8]: the CTA's run
    static constexpr int kOffQuery = kOffPlan + 32;       // uint8 [128]: query index of each of a head's rows
    static constexpr int kSmemUsed = kOffQuery + 128;
    static constexpr size_t kSmemBytes = static_cast<size_t>(kSmemUsed) + 1024;  // alignment slack
    static_assert(kSmemBytes <= 232448, "shared memory budget exceeded");
    static_assert(kOffQ % 1024 == 0 && kOffP % 1024 == 0, "operand tiles must be 1024-byte aligned");
};

// A word that a kernel before wrote.  Where no wait of this kernel's own lies
// between (c.unwaited: behind a prefix's kernel; the second kernel), from L2, as the
// SM's L1 may hold what was there before; else by way of L1, which saves the page
// numbers' way (2 % of a step over long sequences).
__device__ __forceinline__ int word_of(const int32_t* at, bool unwaited) { return unwaited ? __ldcg(at) : *at; }
__device__ __forceinline__ int length_of(const PagedCache& c, int b, bool unwaited) {
    return min(max(word_of(c.lengths + b, unwaited), 0), c.capacity);
}
__device__ __forceinline__ int length_of(const PagedCache& c, int b) { return length_of(c, b, c.unwaited != 0); }
__device__ __forceinline__ int tiles_of(int len) { return (len + 127) / 128; }

// Tiles of a run, all CTAs' alike (the tiles of all units number less than 2^31).
__device__ __forceinline__ int run_of(int total, int ctas) { return max(1, (total + ctas - 1) / ctas); }

// Tiles of one unit of each of the sequences before `b`, and of all, by one warp.
struct Spread {
    int before, total;  // in tiles of one unit each
    int len;            // of sequence b
};
__device__ __forceinline__ Spread spread_of(const PagedCache& c, int b, bool unwaited) {
    const int lane = static_cast<int>(threadIdx.x) % 32;
    int before = 0, total = 0, len = 0;
    for (int s = lane; s < c.B; s += 32) {
        const int l = length_of(c, s, unwaited), n = tiles_of(l);
        total += n;
        if (s < b) before += n;
        if (s == b) len = l;
    }
    return {static_cast<int>(__reduce_add_sync(0xffffffffu, before)), static_cast<int>(__reduce_add_sync(0xffffffffu, total)),
            static_cast<int>(__reduce_max_sync(0xffffffffu, len))};
}

// Position in a CTA's run: tiles pos .. end - 1 of all units', unit u of
// sequence b next, from its tile t on.
struct Cursor {
    int pos, end, b, u, t, len;

    __device__ __forceinline__ bool valid() const { return pos < end; }
    __device__ __forceinline__ int tiles() const { return tiles_of(len); }
    __device__ __forceinline__ int last() const { return min(tiles(), t + end - pos); }  // behind the segment's last tile
    __device__ __forceinline__ void next(const PagedCache& c, int units) {
        const int n = last() - t;
        const bool ended = t + n == tiles();
        pos += n;
        t = 0;
        if (!ended || !valid()) return;
        if (++u < units) return;
        u = 0;
        do len = length_of(c, ++b);
        while (len == 0);  // (pos < end: a sequence with tiles follows)
    }
};

// The run of CTA blockIdx.x, by one warp.
__device__ __forceinline__ Cursor first_of(const PagedCache& c, int units, int ctas) {
    const int lane = static_cast<int>(threadIdx.x) % 32;
    const Spread all = spread_of(c, 0, c.unwaited != 0);
    Cursor k{};
    const int total = all.total * units, run = run_of(total, ctas);
    const long long pos = static_cast<long long>(blockIdx.x) * run;
    if (pos >= total) return k;  // pos = end = 0
    k.pos = static_cast<int>(pos);
    k.end = min(total - k.pos, run) + k.pos;
    int left = k.pos;
    for (int s0 = 0; s0 < c.B; s0 += 32) {
        const int s = s0 + lane;
        const int len = s < c.B ? length_of(c, s) : 0;
        int sum = tiles_of(len) * units;
        const int mine = sum;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        const unsigned int hit = __ballot_sync(0xffffffffu, left < sum);
        if (hit != 0u) {
            const int src = __ffs(static_cast<int>(hit)) - 1;
            const int in = __shfl_sync(0xffffffffu, left - (sum - mine), src);
            k.b = s0 + src;
            k.len = __shfl_sync(0xffffffffu, len, src);
            k.u = in / tiles_of(k.len);
            k.t = in % tiles_of(k.len);
            return k;
        }
        left -= __shfl_sync(0xffffffffu, sum, 31);
    }
    return k;
}

// NV consecutive TMEM columns of this warp's 32 lanes (one per thread), the wait
// for them, and back.
template <int NV>
__device__ __forceinline__ void ld_cols(uint32_t taddr, uint32_t (&r)[NV]) {
    if constexpr (NV >= 16) {
        tmem_ld_cols<NV>(taddr, r);
        tmem_ld_cols_wait<NV>(r);
    } else if constexpr (NV == 8) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                     :
                     : "memory");
    } else {
        static_assert(NV == 4, "4, 8, 16 or 32 columns");
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(taddr));
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3])
                     :
                     : "memory");
    }
}
template <int NV>
__device__ __forceinline__ void st_cols(uint32_t taddr, const uint32_t (&r)[NV]) {
    if constexpr (NV >= 16) {
        tmem_st_cols<NV>(taddr, r);
    } else if constexpr (NV == 8) {
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                     "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    } else {
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                     "r"(r[2]), "r"(r[3])
                     : "memory");
    }
}

// One CTA per run.  map_q: [B * H_kv, R, d] (d first), boxes of NR rows.
template <int D, bool F16, bool kCausal, int NV>
__global__ void __launch_bounds__((Cfg<D, F16, NV>::kThreads), 1)
    fa_paged_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, const PagedFwdParams p) {
    using C = Cfg<D, F16, NV>;
    constexpr int NR = C::NR;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw_u32 & 1023u)) & 1023u;
    uint8_t* smem = smem_raw + pad;
    const uint32_t sbase = raw_u32 + pad;

    const int warp = static_cast<int>(threadIdx.x) / 32;
    const int lane = static_cast<int>(threadIdx.x) % 32;
    const int units = p.c.H_kv * p.row_blocks;  // of a sequence
    auto bar = [&](int i) -> uint32_t { return sbase + C::kOffBar + 8u * static_cast<uint32_t>(i); };
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::kOffAbort);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffTmemSlot);
    int* plan = reinterpret_cast<int*>(smem + C::kOffPlan);

    if (threadIdx.x == 0) {
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar(C::kBarQFull + b), 1);
            mbar_init(bar(C::kBarQEmpty + b), 1);
            for (int g = 0; g < C::kGroups; ++g) mbar_init(bar(C::kBarS + 2 * g + b), 1);
            mbar_init(bar(C::kBarP + b), 4);
            mbar_init(bar(C::kBarPFree + b), 1);
            mbar_init(bar(C::kBarO + b), 1);
            mbar_init(bar(C::kBarOFree + b), 4);
        }
        for (int s = 0; s < 2 * C::kStages; ++s) {
            mbar_init(bar(C::kBarFull + s), 1);
            mbar_init(bar(C::kBarEmpty + s), 1);
        }
        mbar_init(bar(C::kBarDrain), 2);
        *abort_flag = (*reinterpret_cast<volatile unsigned int*>(&p.status->abort_gen) == p.gen) ? 1u : 0u;
        mbar_init_fence();
    }
    if constexpr (NV < NR) {  // rows that only the products have
        for (int i = static_cast<int>(threadIdx.x); i < 4 * C::kRowAtomBytes / 16; i += C::kThreads)
            reinterpret_cast<uint4*>(smem + C::kOffP)[i] = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    if (kCausal && threadIdx.x < 128) smem[C::kOffQuery + threadIdx.x] = static_cast<uint8_t>(threadIdx.x % p.Nq);
    if (warp == C::kMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    if (warp == C::kLoadWarp) {
        if (lane == 0) {
            tma_prefetch_desc(&map_q);
            tma_prefetch_desc(&map_k);
            tma_prefetch_desc(&map_v);
        }
        // Lengths, pages and q may come from the kernel before.  Behind a
        // prefix's kernel, which reads them too and lets this one be set up
        // behind its own wait for whatever wrote them, this one waits at its end
        // instead, for the second kernel's sake.
        if (!p.parts_always) grid_wait();
        grid_release();
        const Cursor k = first_of(p.c, units, p.ctas);
        if (lane == 0) {
            plan[0] = k.pos;
            plan[1] = k.end;
            plan[2] = k.b;
            plan[3] = k.u;
            plan[4] = k.t;
            plan[5] = k.len;
        }
    } else if (!p.parts_always) {
        grid_wait();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const bool skip = *abort_flag != 0u;  // an earlier CTA of this launch gave up
    const Cursor start{plan[0], plan[1], plan[2], plan[3], plan[4], plan[5]};

    if (skip) {
        // nothing (the device error word already reports the failure)
    } else if (warp == C::kLoadWarp) {
        // ---------------------------------------------------------- producer
        const uint64_t once = policy_evict_first();  // a unit reads every byte once (see Measured for row blocks)
        const int pages = 128 / p.c.page;            // of a tile
        // this lane's box of K's or V's tile: 64 channels of page `mine` (8 pages at most, 2 boxes each)
        const int mine = lane / C::kAtoms, atom = lane % C::kAtoms;
        const uint32_t box = static_cast<uint32_t>(atom * C::kAtomBytes + mine * p.c.page * 128);
        int it = 0, keys = 0, seg = 0;  // tiles, their K loads issued, units
        bool ok = true;
        for (Cursor k = start; ok && k.valid(); k.next(p.c, units), ++seg) {
            const int kvh = k.u / p.row_blocks, rb = k.u % p.row_blocks;
            const int32_t* table = p.c.table + static_cast<size_t>(k.b) * p.c.max_pages;
            if (seg >= 2) ok = __all_sync(0xffffffffu, wait_phase(bar(C::kBarQEmpty + (seg & 1)), ((seg >> 1) & 1) ^ 1,
                                                                  abort_flag, p, 70));
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(C::kBarQFull + (seg & 1)), C::kQBytes);
                for (int a = 0; a < C::kAtoms; ++a)
                    tma_load_3d(sbase + C::kOffQ + (seg & 1) * C::kQBytes + a * C::kRowAtomBytes, &map_q,
                                bar(C::kBarQFull + (seg & 1)), a * C::kAtomElems, rb * NR, k.b * p.c.H_kv + kvh, once);
            }
            for (int j = k.t; j < k.last(); ++j, ++it) {
                const int s = it % C::kStages;
                const int have = min(pages, (k.len - j * 128 + p.c.page - 1) / p.c.page);  // pages of the tile in use
                const int id = mine < have ? word_of(table + j * pages + mine, p.c.unwaited != 0) : 0;
                // (K's stage is free when the scores are computed, a product before V's)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    if (ok) ok = __all_sync(0xffffffffu, wait_phase(bar(C::kBarEmpty + v * C::kStages + s),
                                                                    ((it / C::kStages) & 1) ^ 1, abort_flag, p, 60));
                    if (!ok) break;
                    const uint32_t full = bar(C::kBarFull + v * C::kStages + s);
                    if (lane == 0)
                        mbar_arrive_expect_tx(full, static_cast<uint32_t>(have * p.c.page) * (C::kAtoms * 128u));
                    __syncwarp();
                    if (mine < have)
                        tma_load_4d(sbase + (v ? C::kOffV : C::kOffK) + s * C::kTileBytes + box, v ? &map_v : &map_k, full,
                                    atom * C::kAtomElems, 0, kvh, id, once);
                    __syncwarp();
                    if (v == 0) ++keys;
                }
                if (!ok) break;
            }
        }
        // every issued load has landed before the CTA may exit
        if (lane == 0) {
            for (int s = 0; s < C::kStages; ++s) {
                if (s < keys) wait_phase(bar(C::kBarFull + s), ((keys - 1 - s) / C::kStages) & 1, abort_flag, p, 61, false);
                if (s < it)
                    wait_phase(bar(C::kBarFull + C::kStages + s), ((it - 1 - s) / C::kStages) & 1, abort_flag, p, 61, false);
            }
            for (int b = 0; b < 2 && b < seg; ++b) {
                const int last = b + ((seg - 1 - b) / 2) * 2;
                wait_phase(bar(C::kBarQFull + b), (last >> 1) & 1, abort_flag, p, 61, false);
            }
        }
    } else if (warp == C::kMmaWarp) {
        // ------------------------------------------------------------ scores
        // (Descriptors of a stage or a buffer by adding its offset / 16: one thread's
        // instructions are what a tile costs here.)
        if (lane == 0 && start.valid()) {
            const uint64_t dK0 = smem_desc_sw128(sbase + C::kOffK, 16, 1024);
            const uint64_t dQ0 = smem_desc_sw128(sbase + C::kOffQ, 16, 1024);
            const int total = start.end - start.pos;
            uint32_t stage = 0, phase = 0;
            int seg = 0, scored[C::kGroups] = {};  // units; tiles of each softmax group
            Cursor k = start;
            int j = k.t;
            for (int it = 0; it < total; ++it) {
                bool ok = true;
                if (j == k.t) ok = wait_phase(bar(C::kBarQFull + (seg & 1)), (seg >> 1) & 1, abort_flag, p, 62);
                if (ok) ok = wait_phase(bar(C::kBarFull + stage), phase, abort_flag, p, 63);
                // the scores before in this buffer were read before their P^T was published
                if (ok && it >= 2) ok = wait_phase(bar(C::kBarP + (it & 1)), ((it >> 1) & 1) ^ 1, abort_flag, p, 64);
                if (!ok) break;
                tc_fence_after();
                const uint64_t dK = dK0 + stage * (C::kTileBytes >> 4);
                const uint64_t dQ = dQ0 + (seg & 1) * (C::kQBytes >> 4);
#pragma unroll
                for (int kk = 0; kk < C::kQkSteps; ++kk) {
                    const uint32_t koff = (kk * 32) / 128 * C::kAtomBytes + (kk * 32) % 128;
                    const uint32_t qoff = (kk * 32) / 128 * C::kRowAtomBytes + (kk * 32) % 128;
                    mma_ss<false>(tmem + C::kColS + NR * (it & 1), dK + (koff >> 4), dQ + (qoff >> 4), C::kIdescQK,
                                  kk > 0 ? 1u : 0u);
                }
                if (C::kGroups == 2 && (seg & 1)) tc_commit(bar(C::kBarS + 2 + (scored[C::kGroups - 1]++ & 1)));
                else tc_commit(bar(C::kBarS + (scored[0]++ & 1)));
                tc_commit(bar(C::kBarEmpty + stage));  // K is no longer read
                if (++stage == C::kStages) {
                    stage = 0;
                    phase ^= 1;
                }
                if (++j == k.last()) {
                    tc_commit(bar(C::kBarQEmpty + (seg & 1)));
                    k.next(p.c, units);
                    j = k.t;
                    ++seg;
                }
            }
            tc_commit(bar(C::kBarDrain));
            wait_phase(bar(C::kBarDrain), 0, abort_flag, p, 65, false);
        }
    } else if (warp == C::kPvWarp) {
        // ------------------------------------------------ products with V
        if (lane == 0 && start.valid()) {
            const uint64_t dV0 = smem_desc_sw128(sbase + C::kOffV, C::kAtomBytes, 1024);
            const uint64_t dP0 = smem_desc_sw128(sbase + C::kOffP, 16, 1024);
            const int total = start.end - start.pos;
            uint32_t stage = 0, phase = 0;
            int seg = 0;
            Cursor k = start;
            int j = k.t;
            for (int it = 0; it < total; ++it) {
                const int b = it & 1;
                const bool first = j == k.t;
                bool ok = true;
                if (first && seg >= 2)  // O^T of the unit before the last one has been read
                    ok = wait_phase(bar(C::kBarOFree + (seg & 1)), ((seg >> 1) & 1) ^ 1, abort_flag, p, 71);
                if (ok) ok = wait_phase(bar(C::kBarFull + C::kStages + stage), phase, abort_flag, p, 73);
                if (ok) ok = wait_phase(bar(C::kBarP + b), (it >> 1) & 1, abort_flag, p, 74);
                if (!ok) break;
                tc_fence_after();
                // O^T += V^T P^T: A = V read MN-major (d contiguous, its two
                // 64-element blocks 16 KB apart), B = P^T K-major
                const uint64_t dV = dV0 + stage * (C::kTileBytes >> 4);
                const uint64_t dP = dP0 + b * (2 * C::kRowAtomBytes >> 4);
#pragma unroll
                for (int kk = 0; kk < C::kPvSteps; ++kk) {
                    const uint32_t poff = (kk * 32) / 128 * C::kRowAtomBytes + (kk * 32) % 128;
                    mma_ss<false>(tmem + C::kColO + NR * (seg & 1), dV + (kk * C::kUmmaK * 128 >> 4), dP + (poff >> 4),
                                  C::kIdescPV, (!first || kk > 0) ? 1u : 0u);
                }
                tc_commit(bar(C::kBarPFree + b));
                tc_commit(bar(C::kBarEmpty + C::kStages + stage));  // V is no longer read
                if (++stage == C::kStages) {
                    stage = 0;
                    phase ^= 1;
                }
                if (++j == k.last()) {
                    tc_commit(bar(C::kBarO + (seg & 1)));
                    k.next(p.c, units);
                    j = k.t;
                    ++seg;
                }
            }
            tc_commit(bar(C::kBarDrain));
            wait_phase(bar(C::kBarDrain), 0, abort_flag, p, 65, false);
        }
    } else {
        // ----------------------------------------------- softmax warpgroups
        const int group = warp / 4, gwarp = warp % 4;  // of the units seg, every kGroups-th one
        const int t = static_cast<int>(threadIdx.x) % 128;  // key t of each tile; lane t of O^T
        const uint32_t lane_base = static_cast<uint32_t>(gwarp * 32) << 16;
        const uint32_t named = kDecNamedBar + static_cast<uint32_t>(group);
        const uint32_t tS = tmem + lane_base + C::kColS;
        const float c = p.scale_log2;
        float* red = reinterpret_cast<float*>(smem + C::kOffRed) + group * C::kRedFloats;
        float* ref = red + 12 * NV;            // the references, for the unit's result
        float* inv = red;                      // 1 / lq then, where the maxima were
        constexpr int kLanesPerRow = 32 / NV;  // after warp_reduce_rows
        // key t's 16-bit slot in row n of a P^T buffer (see the decode kernel)
        const int pch = (t % 64) / 8;
        uint8_t* pkey = smem + C::kOffP + (t / 64) * C::kRowAtomBytes + (t % 8) * 2;
        bool ok = true;
        int it = 0, mine = 0, seg = 0;  // tiles, those of this group, units
        for (Cursor k = start; ok && k.valid(); k.next(p.c, units), ++seg) {
            if (C::kGroups == 2 && (seg & 1) != group) {
                it += k.last() - k.t;
                continue;
            }
            const int row0 = (k.u % p.row_blocks) * NV;
            const int rows = min(p.rows - row0, NV);
            const uint32_t tO = tmem + lane_base + C::kColO + NR * (seg & 1);
            float m[NV], l[NV], lq[NV];  // reference maxima (base 2, scaled), sums
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                m[n] = -INFINITY;
                l[n] = 0.0f;
                lq[n] = 0.0f;
            }
            const int first = k.t, last = k.last();
            for (int j = first; j < last; ++j, ++it, ++mine) {
                const int b = it & 1, s_ = it % C::kStages;
                const int key = j * 128 + t;
                uint32_t s[NV];
                if (ok) ok = wait_phase(bar(C::kBarS + 2 * group + (mine & 1)), (mine >> 1) & 1, abort_flag, p, 66,
                                        true, kSweepLimits);  // (behind the other group's unit)
                ok = __all_sync(0xffffffffu, ok);  // the TMEM loads below are warp-wide
                if (ok) {
                    tc_fence_after();
                    ld_cols<NV>(tS + NR * b, s);
                } else {
#pragma unroll
                    for (int n = 0; n < NV; ++n) s[n] = 0u;
                }
                // scores in base 2; of keys that a row does not see -inf (rows past the last are not stored)
                float x[NV];
#pragma unroll
                for (int n = 0; n < NV; ++n) x[n] = u2f(s[n]) * c;
                if (j * 128 + 128 > k.len || (kCausal && j * 128 + 127 > k.len - p.Nq)) {
                    if (kCausal) {
                        const int late = key - k.len + p.Nq;  // rows of query indexes below it do not see the key
#pragma unroll
                        for (int n = 0; n < NV; ++n)
                            if (key >= k.len || late > static_cast<int>(smem[C::kOffQuery + row0 + n])) x[n] = -INFINITY;
                    } else if (key >= k.len) {
#pragma unroll
                        for (int n = 0; n < NV; ++n) x[n] = -INFINITY;
                    }
                }
                bool need = !ok;
#pragma unroll
                for (int n = 0; n < NV; ++n) need |= x[n] - m[n] > kRescaleThreshold;
                // (a unit's first tile always sets the references: no vote)
                if (j == first || named_barrier_or(named, 128, need)) {
                    if (named_barrier_or(named, 128, !ok)) {  // every thread leaves together
                        ok = false;
                        break;
                    }
                    // the tile's row maxima over its 128 keys
                    float v[NV];
#pragma unroll
                    for (int n = 0; n < NV; ++n) v[n] = x[n];
                    const float r = warp_reduce_rows<NV, true>(v, lane);
                    if (lane % kLanesPerRow == 0) red[gwarp * NV + lane / kLanesPerRow] = r;
                    named_barrier_sync(named, 128);
                    float alpha[NV];
#pragma unroll
                    for (int n = 0; n < NV; ++n) {
                        const float tmax = fmaxf(fmaxf(red[n], red[NV + n]), fmaxf(red[2 * NV + n], red[3 * NV + n]));
                        float mn = fmaxf(m[n], tmax);
                        // no weight yet (no visible key, or scores of -inf alone): the least finite
                        // reference, below any score that follows (0 would hide scores far below 0)
                        if (mn == -INFINITY) mn = -FLT_MAX;
                        alpha[n] = ex2(m[n] - mn);      // 0 while m was -inf
                        l[n] *= alpha[n];
                        lq[n] *= alpha[n];
                        m[n] = mn;
                        if (t == 0) ref[n] = mn;
                    }
                    if (j > first) {  // O^T holds tiles < j: rescale it once the last product into it is done
                        ok = __all_sync(0xffffffffu, wait_phase(bar(C::kBarPFree + (b ^ 1)), ((it - 1) >> 1) & 1,
                                                                abort_flag, p, 67));
                        if (ok) {
                            tc_fence_after();
                            uint32_t o[NV];
                            ld_cols<NV>(tO, o);
#pragma unroll
                            for (int n = 0; n < NV; ++n) o[n] = f2u(u2f(o[n]) * alpha[n]);
                            st_cols<NV>(tO, o);
                            tmem_st_wait();
                        }
                    }
                }
                // P^T buffer b was last read by the product of tile it - 2
                if (ok && it >= 2) ok = wait_phase(bar(C::kBarPFree + b), ((it - 2) >> 1) & 1, abort_flag, p, 68);
                ok = __all_sync(0xffffffffu, ok);
                if (ok && key >= k.len) {  // value rows behind the sequence's end, and of pages not loaded
                    ok = wait_phase(bar(C::kBarFull + C::kStages + s_), (it / C::kStages) & 1, abort_flag, p, 72);
#pragma unroll 1
                    for (int a = 0; ok && a < C::kAtoms; ++a) {
                        uint4* row = reinterpret_cast<uint4*>(smem + C::kOffV + s_ * C::kTileBytes + a * C::kAtomBytes + t * 128);
#pragma unroll
                        for (int i = 0; i < 8; ++i) row[i ^ (t & 7)] = make_uint4(0u, 0u, 0u, 0u);  // (all banks at a time)
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                if (ok) {
                    uint8_t* pbuf = pkey + b * 2 * C::kRowAtomBytes;
#pragma unroll
                    for (int n = 0; n < NV; n += 2) {
                        const float p0 = ex2(x[n] - m[n]), p1 = ex2(x[n + 1] - m[n + 1]);
                        l[n] += p0;
                        l[n + 1] += p1;
                        const uint32_t w2 = pack_16x2<F16>(p0, p1);
                        lq[n] += widen_lo16<F16>(w2);
                        lq[n + 1] += widen_lo16<F16>(w2 >> 16);
                        *reinterpret_cast<uint16_t*>(pbuf + n * 128 + ((pch ^ (n & 7)) << 4)) =
                            static_cast<uint16_t>(w2 & 0xFFFFu);
                        *reinterpret_cast<uint16_t*>(pbuf + (n + 1) * 128 + ((pch ^ ((n + 1) & 7)) << 4)) =
                            static_cast<uint16_t>(w2 >> 16);
                    }
                    fence_proxy_async_smem();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C::kBarP + b));
                }
            }

            // --------------------------------------------- the unit's result
            // l and lq over the 128 keys of the warpgroup, while the last product runs
            const float rl = warp_reduce_rows<NV, false>(l, lane);
            const float rq = warp_reduce_rows<NV, false>(lq, lane);
            if (lane % kLanesPerRow == 0) {
                red[4 * NV + gwarp * NV + lane / kLanesPerRow] = rl;
                red[8 * NV + gwarp * NV + lane / kLanesPerRow] = rq;
            }
            const bool whole = first == 0 && last == k.tiles();
            const bool final = whole && !p.parts_always;
            const long long unit = static_cast<long long>(k.b) * units + k.u;
            // first row of the output, or of the partial result's slot
            const long long at = final ? (static_cast<long long>(k.b) * p.c.H_kv + k.u / p.row_blocks) * p.rows + row0
                                       : (whole ? 2ll * p.ctas + unit : 2ll * blockIdx.x + (seg == 0 ? 0 : 1)) * NV;
            named_barrier_sync(named, 128);
            if (t < rows) {
                const float* a = red + 4 * NV + t;
                const float* q = red + 8 * NV + t;
                const float L = (a[0] + a[NV]) + (a[2 * NV] + a[3 * NV]);
                const float LQ = (q[0] + q[NV]) + (q[2 * NV] + q[3 * NV]);
                if (final) {
                    inv[t] = LQ == 0.0f ? 0.0f : 1.0f / LQ;
                    if (p.lse != nullptr) p.lse[at + t] = L == 0.0f ? -INFINITY : (ref[t] + log2f(L)) * 0.69314718055994531f;
                } else {
                    // a row that sees no key here gets weight 0 (m = -inf)
                    p.part_ml[at + t] = make_float4(L == 0.0f ? -INFINITY : ref[t], L, LQ, 0.0f);
                }
            }
            if (ok) ok = wait_phase(bar(C::kBarO + (seg & 1)), (seg >> 1) & 1, abort_flag, p, 69);
            ok = __all_sync(0xffffffffu, ok);
            if (named_barrier_or(named, 128, !ok)) {  // (and `inv` is written)
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t o[NV];
            ld_cols<NV>(tO, o);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::kBarOFree + (seg & 1)));
            if (t < D) {
                if (final) {
                    uint16_t* out = static_cast<uint16_t*>(p.out) + at * D + t;
#pragma unroll
                    for (int n = 0; n < NV; ++n)
                        if (n < rows) out[n * D] = static_cast<uint16_t>(pack_16x2<F16>(u2f(o[n]) * inv[n], 0.0f) & 0xFFFFu);
                } else {
                    float* out = p.unit_o + at * D + t;
#pragma unroll
                    for (int n = 0; n < NV; ++n)
                        if (n < rows) out[n * D] = u2f(o[n]);
                }
            }
            // `red` is written again after the next unit's votes, which all threads reach
        }
    }

    // --------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (warp == C::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
    if (p.parts_always) grid_wait();
}

constexpr int kJoinThreads = 256;
constexpr int kJoinAhead = 16;  // partial rows whose loads are in flight

// A row's partial results added up in order, as consecutive tiles of the online
// softmax are:  M = max m_s,  O = sum 2^(m_s - M) O_s / sum 2^(m_s - M) lq_s,
// lse = ln 2 (M + log2 sum 2^(m_s - M) l_s).  By one warp, D / 32 channels a lane.
template <int D>
struct Joined {
    static constexpr int kPer = D / 32;
    float M = -INFINITY, L = 0.0f, LQ = 0.0f, acc[kPer] = {};

    // `parts` of them: part i's statistics and row by stats(i) and row(i).
    template <int kAhead, class Stats, class Row>
    __device__ __forceinline__ void add_by(int parts, Stats stats, Row row) {
        const int lane = static_cast<int>(threadIdx.x) % 32;
        for (int i0 = 0; i0 < parts; i0 += kAhead) {
            const int here = min(kAhead, parts - i0);
            float4 ml = make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
            if (lane < here) ml = stats(i0 + lane);
            float o[kAhead][kPer];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {  // (those past the last repeat it)
                const float* src = row(i0 + min(k, here - 1)) + lane * kPer;
                if constexpr (kPer == 4) {
                    const float4 y = *reinterpret_cast<const float4*>(src);
                    o[k][0] = y.x, o[k][1] = y.y, o[k][2] = y.z, o[k][3] = y.w;
                } else {
                    const float2 y = *reinterpret_cast<const float2*>(src);
                    o[k][0] = y.x, o[k][1] = y.y;
                }
            }
            float most = ml.x;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
            most = fmaxf(most, M);
            const float ref = most == -INFINITY ? 0.0f : most;
            const float old = ex2(M - ref), w = ex2(ml.x - ref);
            float l = w * ml.y, q = w * ml.z;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                l += __shfl_xor_sync(0xffffffffu, l, off);
                q += __shfl_xor_sync(0xffffffffu, q, off);
            }
            M = most;
            L = L * old + l;
            LQ = LQ * old + q;
#pragma unroll
            for (int x = 0; x < kPer; ++x) acc[x] *= old;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const float f = __shfl_sync(0xffffffffu, w, k);
                if (k < here && f != 0.0f) {  // (0 times what a part without keys holds)
#pragma unroll
                    for (int x = 0; x < kPer; ++x) acc[x] += f * o[k][x];
                }
            }
        }
    }
    template <class Stats, class Row>
    __device__ __forceinline__ void add(int parts, Stats stats, Row row) {
        if (parts <= 4) add_by<4>(parts, stats, row);
        else add_by<kJoinAhead>(parts, stats, row);
    }
};

// spread_of for a warp of a block whose first row is of sequence b0, the lengths
// read by all warps together: in larger batches than kJoinAlone each warp's own
// pass over them would take longer than its rows (2048 sequences of 256 slots 355 us,
// by each warp 405; 128 27.3, 26.6).
constexpr int kJoinAlone = 256;
__device__ __forceinline__ Spread spread_by_block(const PagedCache& c, int b0, int b) {
    __shared__ int parts[2][kJoinThreads / 32];
    const int lane = static_cast<int>(threadIdx.x) % 32;
    int before = 0, total = 0;
    for (int s = static_cast<int>(threadIdx.x); s < c.B; s += kJoinThreads) {
        const int n = tiles_of(length_of(c, s, true));
        total += n;
        if (s < b0) before += n;
    }
    total = static_cast<int>(__reduce_add_sync(0xffffffffu, total));
    before = static_cast<int>(__reduce_add_sync(0xffffffffu, before));
    if (lane == 0) {
        parts[0][threadIdx.x / 32] = before;
        parts[1][threadIdx.x / 32] = total;
    }
    __syncthreads();
    before = total = 0;
#pragma unroll
    for (int i = 0; i < kJoinThreads / 32; ++i) {
        before += parts[0][i];
        total += parts[1][i];
    }
    // (a block has 8 rows, so at most 7 sequences begin behind its first one's)
    const int s = b0 + lane;
    before += static_cast<int>(__reduce_add_sync(0xffffffffu, s < b ? tiles_of(length_of(c, s, true)) : 0));
    return {before, total, length_of(c, b, true)};
}

// The second kernel: rows whose keys several CTAs shared, or that have a
// prefix, a warp each.  The lengths are read ahead of the wait: the kernel
// before let this one be set up behind its own wait for whatever wrote them.
// kMany: more than kJoinAlone sequences.
template <int D, bool F16, bool kMany>
__global__ void __launch_bounds__(kJoinThreads) fa_paged_join_kernel(const PagedFwdParams p, int rows_per_block) {
    const int lane = static_cast<int>(threadIdx.x) % 32;
    const long long row = static_cast<long long>(blockIdx.x) * (kJoinThreads / 32) + threadIdx.x / 32;
    const long long total_rows = static_cast<long long>(p.c.B) * p.c.H_kv * p.rows;
    [[maybe_unused]] const long long per_sequence = static_cast<long long>(p.c.H_kv) * p.rows;
    Spread sp;
    if constexpr (kMany)
        sp = spread_by_block(p.c, static_cast<int>(static_cast<long long>(blockIdx.x) * (kJoinThreads / 32) / per_sequence),
                             static_cast<int>(min(row, total_rows - 1) / per_sequence));
    if (row >= total_rows) {
        grid_wait();
        return;
    }
    const int units = p.c.H_kv * p.row_blocks;
    const int r = static_cast<int>(row % p.rows);
    const long long head = row / p.rows;  // b * H_kv + key/value head
    const int b = static_cast<int>(head / p.c.H_kv);
    const int u = static_cast<int>(head % p.c.H_kv) * p.row_blocks + r / rows_per_block;
    const int n = r % rows_per_block;
    if constexpr (!kMany) sp = spread_of(p.c, b, true);
    const int tiles = tiles_of(sp.len);
    const int run = run_of(sp.total * units, p.ctas);
    const int begin = sp.before * units + u * tiles;  // the unit's first tile among all
    const int c0 = begin / run, c1 = tiles > 0 ? (begin + tiles - 1) / run : c0 - 1;  // its CTAs
    const bool whole = c0 == c1;
    grid_wait();
    grid_release();
    if (whole && !p.parts_always) return;  // written by its CTA
    Joined<D> j;
    j.add(p.splits, [&](int i) { return *reinterpret_cast<const float4*>(p.ml_part + (i * total_rows + row) * 4); },
          [&](int i) { return p.o_part + (i * total_rows + row) * D; });
    auto slot = [&](int i) -> long long {
        if (whole) return 2ll * p.ctas + static_cast<long long>(b) * units + u;
        // a CTA whose run starts inside or with the unit has it as its first
        const int cta = c0 + i;
        return 2ll * cta + (i == 0 && begin != c0 * run ? 1 : 0);
    };
    j.add(c1 - c0 + 1, [&](int i) { return p.part_ml[slot(i) * rows_per_block + n]; },
          [&](int i) { return p.unit_o + (slot(i) * rows_per_block + n) * D; });
    const float inv = j.LQ == 0.0f ? 0.0f : 1.0f / j.LQ;
    constexpr int kPer = Joined<D>::kPer;
    uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + row * D + lane * kPer);
#pragma unroll
    for (int x = 0; x < kPer; x += 2) dst[x / 2] = pack_16x2<F16>(j.acc[x] * inv, j.acc[x + 1] * inv);
    if (lane == 0 && p.lse != nullptr)
        p.lse[row] = j.L == 0.0f ? -INFINITY : (j.M + log2f(j.L)) * 0.69314718055994531f;
}

template <int D, bool F16, bool kCausal, int NV>
cudaError_t launch_variant(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PagedFwdParams& p,
                           cudaStream_t stream) {
    using C = Cfg<D, F16, NV>;
    auto kern = fa_paged_kernel<D, F16, kCausal, NV>;
    static SmemAllowed allowed;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), static_cast<int>(C::kSmemBytes), allowed);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kern, dim3(static_cast<unsigned>(p.ctas)), C::kThreads, C::kSmemBytes, stream, q, k, v, p);
    if (e != cudaSuccess) return e;
    const long long rows = static_cast<long long>(p.c.B) * p.c.H_kv * p.rows;
    auto join = p.c.B > kJoinAlone ? fa_paged_join_kernel<D, F16, true> : fa_paged_join_kernel<D, F16, false>;
    return launch_dependent(join, dim3(static_cast<unsigned>((rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32))), kJoinThreads, 0,
                            stream, p, NV);
}

template <int D, bool F16, bool kCausal>
cudaError_t launch_rows(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PagedFwdParams& p,
                        cudaStream_t stream) {
    switch (paged_rows_per_block(p.rows)) {
        case 4: return launch_variant<D, F16, kCausal, 4>(q, k, v, p, stream);
        case 8: return launch_variant<D, F16, kCausal, 8>(q, k, v, p, stream);
        case 16: return launch_variant<D, F16, kCausal, 16>(q, k, v, p, stream);
        default: return launch_variant<D, F16, kCausal, 32>(q, k, v, p, stream);
    }
}

template <int D, bool F16>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PagedFwdParams& p,
                   cudaStream_t stream) {
    return p.causal ? launch_rows<D, F16, true>(q, k, v, p, stream) : launch_rows<D, F16, false>(q, k, v, p, stream);
}

}  // namespace paged
}  // namespace fa
