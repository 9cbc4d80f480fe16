// Attention weight received by the keys of a prompt, sm_103a (include/fa.h,
// fa_fwd_weights):
//
//   w[j] = sum over rows i of 2^(c s_ij - lse2_i),  s = q_i . k_j
//
// the column sums of the attention map that the forward pass (whose lse it
// takes) never writes; the map is recomputed tile by tile as the backward
// pass does ("FlashAttention dissected", section "Memory complexity: from
// O(N^2) to O(N)").
//
// The keys sit on the 128 tensor-memory lanes (S^T = K Q^T), so a thread
// owns a key and its sum runs along the thread's own columns: no reduction
// across threads, no atomics, one fixed order of additions.  A step's 128
// terms are added first and then added to the running sum, which keeps the
// rounding of a sum over 10^5 rows near 2^-22 of it.
//
// One CTA owns 256 keys of one key/value head (two tiles of 128, resident in
// shared memory, so a query tile that was loaded serves two products) and
// sweeps the rows of the head's query heads, 128 a step:
//   warps 0-15   four warpgroups; product n (step n / 2, key tile n % 2) goes
//                to warpgroup n % 4, which owns 128 columns of tensor memory
//                and gives them back once its second 64 are in registers
//   warps 16, 17 tensor-core issuers, one thread per key tile; 16 owns the
//                tensor memory
//   warp 18      TMA producer
// Bound by the exponentials, the products and the issue slots alike: 128 x 128
// scores take 512 clocks of the first two at d = 128 (32 exponentials a clock
// and SM; the products half of that at d = 64) and about 350 issue slots.
// Each issuer's barrier waits, about 180 clocks a product, and the commits, 35
// each, come on top: two issuers hide one another's, and a query stage is
// given back by the warps that read the scores instead of by a commit.
// Measured at B = 2, H = 32/8, N = 8192, d = 128, causal: 375 to 408 us on
// different boxes, 1465 to 1347 TFLOP/s (tensor pipe and exponentials 67 % busy
// each); on the first, one issuer 588 us;
// keys in tensor memory and three buffers 566; products of 64 rows, whose
// columns are free sooner, 800 (an N = 64 product takes 48 clocks a step
// instead of 32).
//
// Causal: the rows below a tile's diagonal are swept from the first one that
// sees any of its keys; only the first steps are masked.  When the key blocks
// do not fill the GPU, the CTAs of one thread-block cluster share the steps
// of a key block and add their sums in order through distributed shared
// memory.
#pragma once

#include <cmath>
#include <cstdint>

#include "fa_fwd_kernel.cuh"
#include "fa_kv4.h"

namespace fa {

constexpr int kWtWarpgroups = 4;
constexpr int kWtSoftmaxWarps = 4 * kWtWarpgroups;
constexpr int kWtMmaWarp = kWtSoftmaxWarps;  // and the next: one issuer per key tile
constexpr int kWtLoadWarp = kWtMmaWarp + 2;
constexpr int kWtThreads = (kWtLoadWarp + 1) * 32;

template <int D, bool F16>
struct WtCfg {
    static constexpr int kAtoms = D / 64;
    static constexpr int kAtomBytes = 128 * 128;
    static constexpr int kTileBytes = kAtoms * kAtomBytes;
    static constexpr int kSteps = D / 16;
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr uint32_t kFmt = F16 ? 0u : 1u;
    static constexpr uint32_t kIdesc = instr_desc(kFmt, false, false, 128, 128);
    static constexpr int kOffK = 0;                                  // two tiles
    static constexpr int kOffQ = kOffK + 2 * kTileBytes;             // [kStages]
    static constexpr int kOffLse = kOffQ + kStages * kTileBytes;     // float [kStages][128]: -lse2 of the rows
    static constexpr int kOffSum = kOffLse + kStages * 128 * 4;  // float [warpgroup][128]
    static constexpr int kOffBar = kOffSum + kWtWarpgroups * 128 * 4;
    static constexpr int kBarK = 0;
    static constexpr int kBarFull = 1;                    // [kStages] a query tile and its lse landed
    static constexpr int kBarEmpty = kBarFull + kStages;  // [kStages] its scores were read
    static constexpr int kBarS = kBarEmpty + kStages;     // [warpgroups] scores ready
    static constexpr int kBarSFree = kBarS + kWtWarpgroups;  // [warpgroups] scores read
    static constexpr int kBarDrain = kBarSFree + kWtWarpgroups;  // [2] an issuer's products are done
    static constexpr int kNumBars = kBarDrain + 2;
    static constexpr int kOffTmemSlot = kOffBar + kNumBars * 8;
    static constexpr int kOffAbort = kOffTmemSlot + 4;
    static constexpr size_t kSmemBytes = static_cast<size_t>(kOffAbort + 4) + 1024;
    static_assert(kSmemBytes <= 232448, "shared memory budget exceeded");
};

// Adds 2^(c r_i + neg_i) for 64 rows to the two pairs of sums; rows before
// first_col are hidden (kMasked), whatever their scores are.
template <bool kMasked>
__device__ __forceinline__ void add_weights(const uint32_t (&r)[2][32], const float* neg, uint64_t c2, int first_col,
                                            uint64_t (&sum)[2]) {
#pragma unroll
    for (int i = 0; i < 64; i += 4) {
        const float4 n4 = *reinterpret_cast<const float4*>(neg + i);
        const uint32_t* x4 = &r[i / 32][i % 32];
        float x[4];
        f2_unpack(f2_fma(f2_pack(u2f(x4[0]), u2f(x4[1])), c2, f2_pack(n4.x, n4.y)), x[0], x[1]);
        f2_unpack(f2_fma(f2_pack(u2f(x4[2]), u2f(x4[3])), c2, f2_pack(n4.z, n4.w)), x[2], x[3]);
        if constexpr (kMasked) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < first_col) x[e] = -INFINITY;
        }
        sum[0] = f2_add(sum[0], f2_pack(ex2(x[0]), ex2(x[1])));
        sum[1] = f2_add(sum[1], f2_pack(ex2(x[2]), ex2(x[3])));
    }
}

// grid = B * H_kv * ceil(N_kv / 256) * p.splits, clusters of p.splits.
template <int D, bool F16>
__global__ void __launch_bounds__(kWtThreads, 1)
    fa_weights_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                      const WeightsParams p) {
    using C = WtCfg<D, F16>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw_u32 & 1023u)) & 1023u;
    uint8_t* smem = smem_raw + pad;
    const uint32_t sbase = raw_u32 + pad;
    const int warp = static_cast<int>(threadIdx.x) / 32, lane = static_cast<int>(threadIdx.x) % 32;

    const int n_blocks = (p.Nkv + 255) / 256;
    const unsigned int split = blockIdx.x % static_cast<unsigned>(p.splits);
    const unsigned int item = blockIdx.x / static_cast<unsigned>(p.splits);
    int kvh, block;  // causal: a head's first key block is its heaviest
    if (p.causal) {
        lpt_item(item, static_cast<int>(gridDim.x) / p.splits / n_blocks, n_blocks, kvh, block);
    } else {
        kvh = static_cast<int>(item / static_cast<unsigned>(n_blocks));
        block = static_cast<int>(item % static_cast<unsigned>(n_blocks));
    }
    const int key0 = block * 256;
    const int tiles = p.Nkv - key0 > 128 ? 2 : 1;
    // rows first_row .. Nq - 1 of every query head, 128 a step
    int first_row = p.first_query;
    if (p.causal) first_row = max(first_row, min(key0 - p.causal_offset, p.Nq));
    const int per_head = (p.Nq - first_row + 127) / 128;
    const int all = per_head * p.group;
    const int share = (all + p.splits - 1) / p.splits;
    const int begin = min(static_cast<int>(split) * share, all);
    const int T = min(share, all - begin);
    const long long head0 = static_cast<long long>(kvh / p.H_kv) * p.H + static_cast<long long>(kvh % p.H_kv) * p.group;

    auto bar = [&](int i) -> uint32_t { return sbase + C::kOffBar + 8u * static_cast<uint32_t>(i); };
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::kOffAbort);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffTmemSlot);
    FwdParams wp;  // what a bounded wait reports to
    wp.status = p.status;
    wp.gen = p.gen;

    if (threadIdx.x == 0) {
        mbar_init(bar(C::kBarK), 1);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(bar(C::kBarFull + s), 2);  // the query tile, and its rows' lse
            mbar_init(bar(C::kBarEmpty + s), static_cast<uint32_t>(4 * tiles));
        }
        for (int w = 0; w < kWtWarpgroups; ++w) {
            mbar_init(bar(C::kBarS + w), 1);
            mbar_init(bar(C::kBarSFree + w), 4);
        }
        for (int i = 0; i < 2; ++i) mbar_init(bar(C::kBarDrain + i), 1);
        *abort_flag = (*reinterpret_cast<volatile unsigned int*>(&p.status->abort_gen) == p.gen) ? 1u : 0u;
        mbar_init_fence();
    }
    if (warp == kWtMmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const bool skip = *abort_flag != 0u;
    grid_release();
    grid_wait();

    if (warp == kWtLoadWarp) {
        if (T > 0 && !skip) {
            const uint64_t keep = policy_evict_last(), once = policy_evict_first();
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(C::kBarK), static_cast<uint32_t>(tiles) * C::kTileBytes);
                for (int i = 0; i < tiles; ++i)
                    for (int a = 0; a < C::kAtoms; ++a)
                        tma_load_3d(sbase + C::kOffK + i * C::kTileBytes + a * C::kAtomBytes, &map_k, bar(C::kBarK),
                                    a * 64, key0 + 128 * i, kvh, once);
            }
            int head = begin / per_head, block_in_head = begin - head * per_head;
            // lse of rows lane + 32 i of a step, -inf behind the last; asked for a step ahead
            float lse[4];
            auto load_lse = [&] {
                const float* src = p.lse + (head0 + head) * p.Nq;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = first_row + 128 * block_in_head + lane + 32 * i;
                    lse[i] = head < p.group && row < p.Nq ? src[row] : -INFINITY;
                }
            };
            load_lse();
            int issued = 0;
            for (int j = 0; j < T; ++j) {
                const int s = j % C::kStages;
                if (!__all_sync(0xffffffffu,
                                wait_phase(bar(C::kBarEmpty + s), ((j / C::kStages) & 1) ^ 1, abort_flag, wp, 90)))
                    break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(C::kBarFull + s), C::kTileBytes);
                    for (int a = 0; a < C::kAtoms; ++a)
                        tma_load_3d(sbase + C::kOffQ + s * C::kTileBytes + a * C::kAtomBytes, &map_q,
                                    bar(C::kBarFull + s), a * 64, first_row + 128 * block_in_head,
                                    static_cast<int>(head0) + head, keep);
                }
                float* neg = reinterpret_cast<float*>(smem + C::kOffLse) + s * 128;
#pragma unroll
                for (int i = 0; i < 4; ++i)  // -lse2; -inf where a row counts nothing
                    neg[lane + 32 * i] = lse[i] == -INFINITY ? -INFINITY : lse[i] * -1.4426950408889634f;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::kBarFull + s));
                if (++block_in_head == per_head) {
                    block_in_head = 0;
                    ++head;
                }
                load_lse();
                issued = j + 1;
            }
            if (lane == 0) {
                wait_phase(bar(C::kBarK), 0, abort_flag, wp, 91, false);
                for (int s = 0; s < C::kStages && s < issued; ++s) {
                    const int last = s + ((issued - 1 - s) / C::kStages) * C::kStages;
                    wait_phase(bar(C::kBarFull + s), (last / C::kStages) & 1, abort_flag, wp, 92, false);
                }
            }
        }
    } else if (warp >= kWtMmaWarp) {
        const int i = warp - kWtMmaWarp;  // key tile
        if (lane == 0 && T > 0 && !skip && i < tiles) {
            // a k-step's descriptor is the tile's plus a constant
            const uint64_t dk0 = smem_desc_sw128(sbase + C::kOffK + i * C::kTileBytes, 16, 1024);
            const uint64_t dq0 = smem_desc_sw128(sbase + C::kOffQ, 16, 1024);
            bool ok = wait_phase(bar(C::kBarK), 0, abort_flag, wp, 93);
            for (int j = 0; ok && j < T; ++j) {
                const int s = j % C::kStages, n = j * tiles + i, w = n % kWtWarpgroups;
                ok = wait_phase(bar(C::kBarFull + s), (j / C::kStages) & 1, abort_flag, wp, 94) &&
                     wait_phase(bar(C::kBarSFree + w), ((n / kWtWarpgroups) & 1) ^ 1, abort_flag, wp, 95);
                if (!ok) break;
                tc_fence_after();
                const uint64_t dq = dq0 + static_cast<uint64_t>((s * C::kTileBytes) >> 4);
#pragma unroll
                for (int kk = 0; kk < C::kSteps; ++kk) {
                    constexpr uint32_t kAtom = C::kAtomBytes;
                    const uint32_t off = ((kk * 32) / 128 * kAtom + (kk * 32) % 128) >> 4;
                    mma_ss<false>(tmem + 128u * w, dk0 + off, dq + off, C::kIdesc, kk > 0 ? 1u : 0u);
                }
                tc_commit(bar(C::kBarS + w));
            }
            tc_commit(bar(C::kBarDrain + i));
            wait_phase(bar(C::kBarDrain + i), 0, abort_flag, wp, 96, false);
        }
    } else {
        const int wg = warp / 4, t = static_cast<int>(threadIdx.x) % 128;
        const int tile = tiles == 2 ? wg % 2 : 0;
        const int key = key0 + 128 * tile + t;
        const uint32_t tS = tmem + (static_cast<uint32_t>((warp % 4) * 32) << 16) + 128u * wg;
        float total = 0.0f;
        if (T > 0 && !skip) {
            // products n = wg, wg + 4, .. of T * tiles; their steps j = n / tiles are row blocks
            // `block_in_head` of the query heads
            const int products = T * tiles, ahead = kWtWarpgroups / tiles;
            int block_in_head = (begin + wg / tiles) % per_head;
            const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2);
            const int diagonal = p.causal ? key - p.causal_offset - first_row : -1;  // first row that sees the key
            uint32_t turn = 0;
            for (int n = wg; n < products; n += kWtWarpgroups, ++turn) {
                const int j = n / tiles, stage = j % C::kStages;
                const float* neg = reinterpret_cast<const float*>(smem + C::kOffLse) + stage * 128;
                const int first_col = diagonal - 128 * block_in_head;  // of this step
                for (block_in_head += ahead; block_in_head >= per_head;) block_in_head -= per_head;
                const bool masked = __any_sync(0xffffffffu, first_col > 0);
                if (!__all_sync(0xffffffffu,
                                wait_phase(bar(C::kBarFull + stage), (j / C::kStages) & 1, abort_flag, wp, 98) &&
                                    wait_phase(bar(C::kBarS + wg), turn & 1, abort_flag, wp, 97)))
                    break;
                tc_fence_after();
                uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t r[2][32];
                    tmem_ld32(tS + 64u * q, r[0]);
                    tmem_ld32(tS + 64u * q + 32u, r[1]);
                    tmem_ld_wait(r[0]);
                    tmem_ld_wait(r[1]);
                    if (q == 1) {  // the scores are in registers: the next product may start
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(C::kBarSFree + wg));
                    }
                    if (masked)
                        add_weights<true>(r, neg + 64 * q, c2, first_col - 64 * q, sum);
                    else
                        add_weights<false>(r, neg + 64 * q, c2, 0, sum);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::kBarEmpty + stage));  // the rows' lse was read
                float a0, a1;
                f2_unpack(f2_add(sum[0], sum[1]), a0, a1);
                total += a0 + a1;
            }
        }
        reinterpret_cast<float*>(smem + C::kOffSum)[wg * 128 + t] = total;
    }
    tc_fence_before();
    if (p.splits > 1)
        cluster_sync_all();
    else
        __syncthreads();
    // the warpgroups and every CTA of the cluster add up in order
    if (split == 0 && threadIdx.x < 256) {
        const int tile = static_cast<int>(threadIdx.x) / 128, t = static_cast<int>(threadIdx.x) % 128;
        const int key = key0 + 128 * tile + t;
        if (key < p.Nkv) {
            const long long at = static_cast<long long>(kvh) * p.weight_stride + key;
            float s = 0.0f;
            // one tile: the four warpgroups took its products in turn; two: those of its parity
            for (int r = 0; r < p.splits; ++r)
                for (int w = tile; w < kWtWarpgroups; w += tiles) {
                    const int i = w * 128 + t;
                    float v;
                    if (p.splits > 1)
                        asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                     : "=f"(v)
                                     : "r"(mapa_shared(sbase + C::kOffSum + 4u * static_cast<uint32_t>(i),
                                                       static_cast<uint32_t>(r)))
                                     : "memory");
                    else
                        v = reinterpret_cast<float*>(smem + C::kOffSum)[i];
                    s += v;
                }
            p.weight_out[at] = (p.weight_in != nullptr ? p.weight_in[at] : 0.0f) + s;
        }
    }
    if (p.splits > 1)
        cluster_sync_all();  // no CTA leaves while its sums may be read
    else
        __syncthreads();
    if (warp == kWtMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, bool F16>
cudaError_t launch_weights_variant(const CUtensorMap& q, const CUtensorMap& k, const WeightsParams& p,
                                   unsigned int grid, cudaStream_t stream) {
    using C = WtCfg<D, F16>;
    auto kern = fa_weights_kernel<D, F16>;
    static SmemAllowed allowed;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), static_cast<int>(C::kSmemBytes), allowed);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kWtThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.splits);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.splits > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kern, q, k, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace fa
