// Attention over the 4-bit key/value cache, sm_103a (include/fa.h,
// fa_kv4_fwd): the online softmax of "FlashAttention dissected", section
// "Algorithmic core in pseudocode", over key partitions (its section
// "Interaction with the KV cache during inference").
//
// Mathematics.  Per key/value head, with the R = N_q * group query rows of
// its query heads: S^T = K Q^T (keys x rows), P = 2^(c S - ref), O^T = V^T P^T.
// A stored value is e2m1 x e4m3, exact in fp16, so both products run in fp16
// whatever the type of q: a row of q is scaled by a power of two to
// [2^14, 2^15), which is exact (values below 2^-28 of the row's largest lose
// bits, less than the fp32 accumulation does), and the power goes into c.
//
// Layout.  fa_kv4_tiles.cuh: how a warp reads a slab of 32 slots and keeps a
// block of up to 4, 8 or 16 rows.
//
// What bounds it: reading the cache.  Groups of eight slabs (32 keys each, one
// per warp) arrive by four bulk copies (codes and scales of K and V) in a
// ring that a ninth warp refills (a copy holds up the warp that asks for it;
// by the warp that finished a group last, 65536 slots took 109 us, by the
// ninth 104, at B = 8, H = 32/8, d = 128); two blocks an SM keep 147 KB in
// flight.
//
// Work split.  The slabs of all units (sequence, key/value head, block of
// rows), in order, are cut into equal runs, one per CTA, from the lengths on
// the device: no CTA idles because a sequence is short, and a long one is
// shared by many.  A run that ends one unit and begins another takes about as
// long as one of a group more, so a unit counts a group more than it has;
// where a CTA gets two groups or fewer of a full cache it does not, as runs
// then often end with their unit.  (Counted against not, at d = 128, H = 32/8:
// N = 2048 B = 8 10.7 / 10.0 us; N = 2560 13.2 / 14.7; N = 4096 B = 5 13.6 /
// 14.7, B = 8, where every unit is cut into four equal runs, 15.3 / 15.3; N =
// 16384 33.6 / 35.0; d = 64 alike.  With 8 rows a head, 2560 slots 15.6 / 17.8,
// 16384 38.3 / 40.0, but B = 8 N = 4096 19.1 / 17.9; with 16, N = 4096 B = 5
// 19.5 / 20.8, 8192 33.0 / 34.5, 16384 53.3 / 53.1, but 2048 17.1 / 15.4 and
// 2560 19.6 / 17.5: there the rule counts where it had better not.)
//
// A CTA whose run holds a whole unit writes its output; of a unit cut between
// CTAs each leaves a partial result (at most two per CTA: the unit it starts
// inside and the one it ends inside), which the second kernel adds up in
// order, so results do not depend on timing.  (The last CTA to arrive adding
// them up, counted by an atomic, took longer: 44.3 against 40.6 us at B = 8,
// H = 32/8, 16384 slots, d = 128, and 69 against 54 us for one sequence of
// 131071.)  The second kernel also forms the accumulated weights from the
// scores, which the first leaves in the workspace (4 bytes a score, against
// the 72 of reading a key again at d = 128).
//
// A cache of at most kWholeSlots slots, or twice that where there are as many
// units as SMs, is not cut: a CTA per unit, and no second kernel unless
// weights are asked for.  Whole against cut, in us, d = 128 and H = 32/8:
// 512 slots B = 1 5.5 / 6.9, B = 8 5.8 / 7.2, B = 64 16.1 / 18.6, B = 256 45.8 /
// 45.5; 1024 slots B = 1 7.6 / 6.9, B = 24 12.0 / 15.4, B = 64 22.5 / 26.6, B =
// 256 68.6 / 69.9; d = 64 and 8 or 16 rows a head alike.  64 units of 1024
// slots, which the rule cuts, are 6 % sooner whole there (7.9 / 8.3), and up to
// 24 % with 16 rows at d = 64 (7.9 / 9.8).
//
// What is left (B = 8, H = 32/8, d = 128): 16384 slots take 33.8 us, 65536
// 104 (5.8 TB/s); 49152 more cost what reading them does, so 11 us do not
// depend on the length: 1.5 from the wait to the first copy, 1.7 until it is
// there, up to 7 between the first and the last block's end (about 3 between
// their mean and the last), 1.7 for the second kernel.
//
// Every wait is bounded as in the forward kernel; a warp that gives up skips
// its remaining slabs but still reaches the block's barriers.
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "fa_fwd_kernel.cuh"
#include "fa_kv4.h"
#include "fa_kv4_tiles.cuh"

namespace fa {
namespace {

using namespace kv4;

constexpr int kLoadWarp = kWarps;
constexpr int kWholeSlots = 2 * kWarps * kSlab;
constexpr int kThreads4 = (kWarps + 1) * 32;

// R: query rows per block, 4 (layout Paired), 8 or 16 (layout Wide).
template <int D, int R>
struct Kv4Cfg {
    static constexpr int kRows = R;
    static constexpr int kStages = D == 128 ? 2 : 4;  // the same bytes in flight (two at d = 64: 68.1, four 66.9 us
                                                      // at B = 8, H = 32/8, 65536 slots)
    static constexpr int kCodeBytes = kSlab * D / 2;
    static constexpr int kScaleBytes = kSlab * D / 16;
    static constexpr int kStageBytes = 2 * kWarps * (kCodeBytes + kScaleBytes);  // a group: a slab per warp
    static constexpr int kQTiles = R <= 8 ? 1 : 2;           // 8-column tiles of Q^T
    static constexpr int kSums = R * D / 128;                // float4 accumulators of O^T per lane
    static constexpr int kOffRing = 0;  // [stages] K codes, V codes, K scales, V scales of kWarps slabs
    static constexpr int kOffO = kOffRing + kStages * kStageBytes;          // float4 [warps][kSums][32]
    static constexpr int kOffMl = kOffO + kWarps * kSums * 32 * 16;         // float4 [warps][kRows]
    static constexpr int kOffQ = kOffMl + kWarps * kRows * 16;              // uint4 [kQTiles][D / 32][32]
    static constexpr int kOffC = kOffQ + kQTiles * (D / 32) * 32 * 16;      // float [kRows]: score factors
    static constexpr int kOffBar = kOffC + kRows * 4;
    static constexpr int kOffAbort = kOffBar + 2 * kStages * 8;  // behind [stages] landed, [stages] read
    static constexpr int kSmemBytes = (kOffAbort + 4 + 15) / 16 * 16;
    static constexpr int kCtasPerSm = R <= 8 ? 2 : 1;
    static_assert(kOffQ % 16 == 0 && kOffBar % 8 == 0 && kOffO % 16 == 0, "alignment");
    static_assert(kSmemBytes * kCtasPerSm <= 232448 - 1024 * kCtasPerSm, "shared memory budget exceeded");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar,
                                          uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}
__device__ __forceinline__ int kv4_length(const Kv4Cache& c, int b) {
    return min(max(c.counts[b], 0), c.capacity);
}
__device__ __forceinline__ int slabs_of(int len) { return (len + kSlab - 1) / kSlab; }
// What a unit counts for in the runs: its slabs and `cost`, the slabs' worth
// of ending it.
__device__ __forceinline__ int share_of(int slabs, int cost) { return slabs > 0 ? slabs + cost : 0; }

// The shares of all units fit 31 bits (the host checks it), so positions in
// them are ints.
//
// Share per CTA: equal runs of whole groups.
__device__ __forceinline__ int slabs_per_cta(int total, int ctas) {
    return max(1, (total + ctas * kWarps - 1) / (ctas * kWarps)) * kWarps;
}

// Position in a CTA's run.
struct Cursor {
    int pos, end;       // in shares over all units
    int base;           // where sequence b begins
    int cost;
    int b, len, slabs;  // sequence, its length and the slabs of one of its units
    int unit;           // unit of sequence b
    int s0, s1;         // slabs of that unit in this run

    __device__ __forceinline__ bool valid() const { return pos < end; }
    __device__ __forceinline__ void next(const Kv4Cache& c, int units) {
        pos = slabs > 0 && s1 == slabs ? min(end, pos + share_of(slabs, cost) - s0) : end;
        if (pos >= end) return;
        s0 = 0;
        if (++unit == units) {  // the next sequence that has any slab
            unit = 0;
            base += share_of(slabs, cost) * units;
            do {
                len = kv4_length(c, ++b);
                slabs = slabs_of(len);
            } while (slabs == 0);
        }
        s1 = min(slabs, end - pos);
    }
    // Unit `cta` whole, whatever its length (an empty one is visited, too).
    __device__ __forceinline__ void start_single(const Kv4Cache& c, int units, int cta) {
        b = cta / units;
        unit = cta - b * units;
        len = kv4_length(c, b);
        slabs = slabs_of(len);
        pos = base = s0 = 0;
        s1 = slabs;
        end = max(slabs, 1);
        cost = 0;
    }
    __device__ __forceinline__ void start(const Kv4Cache& c, int units, int ctas, int cta, int unit_cost) {
        cost = unit_cost;
        const int lane = threadIdx.x % 32;
        const int len0 = lane < c.B ? kv4_length(c, lane) : 0;  // the first 32 sequences: all, mostly
        int total = share_of(slabs_of(len0), cost) * units;
        for (int x = 32 + lane; x < c.B; x += 32) total += share_of(slabs_of(kv4_length(c, x)), cost) * units;
        total = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(total)));
        const int per = slabs_per_cta(total, ctas);
        pos = static_cast<int>(min(static_cast<long long>(total), static_cast<long long>(per) * cta));
        end = min(total - pos, per) + pos;
        base = b = len = slabs = unit = s0 = s1 = 0;
        // the sequence that holds `pos`, 32 sequences at a time
        for (int b0 = 0; pos < end && b0 < c.B; b0 += 32) {
            const int mine = b0 == 0 ? len0 : b0 + lane < c.B ? kv4_length(c, b0 + lane) : 0;
            const int n = share_of(slabs_of(mine), cost) * units;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, base + incl > pos);
            if (past) {
                const int who = __ffs(static_cast<int>(past)) - 1;
                base += __shfl_sync(0xffffffffu, incl - n, who);
                len = __shfl_sync(0xffffffffu, mine, who);
                slabs = slabs_of(len);
                b = b0 + who;
                break;
            }
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (pos < end) {
            const int share = share_of(slabs, cost);
            unit = (pos - base) / share;
            s0 = pos - base - unit * share;
            s1 = min(slabs, s0 + (end - pos));
            if (s0 >= slabs) next(c, units);  // the run starts behind the unit's last slab
        }
    }
};

template <int D, int R>
__global__ void __launch_bounds__(kThreads4, Kv4Cfg<D, R>::kCtasPerSm) kv4_fwd_kernel(const __grid_constant__ Kv4FwdParams p) {
    using C = Kv4Cfg<D, R>;
    using Tile = std::conditional_t<R == 4, Paired<D>, Wide<D, R>>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = static_cast<int>(threadIdx.x) / 32, lane = static_cast<int>(threadIdx.x) % 32;
    const int g = lane / 4, t = lane % 4;
    const uint32_t sbase = smem_u32(smem);
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::kOffAbort);
    FwdParams wp;  // what a bounded wait reports to
    wp.status = p.status;
    wp.gen = p.gen;
    auto full = [&](int s) -> uint32_t { return sbase + C::kOffBar + 8u * static_cast<uint32_t>(s); };
    auto empty = [&](int s) -> uint32_t { return full(C::kStages + s); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kWarps);
        }
        *abort_flag = 0u;
        mbar_init_fence();
    }
    __syncthreads();
    grid_wait();
    grid_release();

    const int units = p.c.H_kv * p.row_blocks;
    Cursor cur;
    if (p.single)
        cur.start_single(p.c, units, static_cast<int>(blockIdx.x));
    else
        cur.start(p.c, units, p.ctas, static_cast<int>(blockIdx.x), p.unit_cost);

    // A unit's slabs go in groups of one per warp; stage i % kStages of the ring holds group i.
    if (warp == kLoadWarp) {
        if (lane == 0) {
            const uint64_t once = policy_evict_first();  // every byte is read once per block of rows
            int i = 0;
            for (; cur.valid(); cur.next(p.c, units)) {
                const long long row0 =
                    (static_cast<long long>(cur.b) * p.c.H_kv + cur.unit / p.row_blocks) * p.c.capacity;
                for (int slab = cur.s0; slab < cur.s1; slab += kWarps, ++i) {
                    const int s = i % C::kStages;
                    if (!wait_phase(empty(s), ((i / C::kStages) & 1) ^ 1, abort_flag, wp, 81)) break;
                    const int n = min(kWarps, cur.s1 - slab);
                    const long long row = row0 + static_cast<long long>(slab) * kSlab;
                    const uint32_t dst = sbase + C::kOffRing + s * C::kStageBytes;
                    const uint32_t code = n * C::kCodeBytes, scale = n * C::kScaleBytes;
                    mbar_arrive_expect_tx(full(s), 2 * (code + scale));
                    bulk_load(dst, p.c.codes[0] + row * (D / 2), code, full(s), once);
                    bulk_load(dst + 2 * kWarps * C::kCodeBytes, p.c.scales[0] + row * (D / 16), scale, full(s), once);
                    bulk_load(dst + kWarps * C::kCodeBytes, p.c.codes[1] + row * (D / 2), code, full(s), once);
                    bulk_load(dst + kWarps * (2 * C::kCodeBytes + C::kScaleBytes), p.c.scales[1] + row * (D / 16), scale,
                              full(s), once);
                }
                if (*abort_flag) break;
            }
            // every copy has landed before the block may end
            for (int k = max(0, i - C::kStages); k < i; ++k)
                wait_phase(full(k % C::kStages), (k / C::kStages) & 1, abort_flag, wp, 82, false);
        }
        return;
    }

    // q fragments: lane (g, t) holds channels (D / 4) t .. of one row per tile of 8 columns; warp nt loads tile nt
    // a unit ahead and puts it, scaled, into shared memory
    const int q_row = Tile::q_row(warp, g);
    uint4* sm_q = reinterpret_cast<uint4*>(smem + C::kOffQ);
    float* sm_c = reinterpret_cast<float*>(smem + C::kOffC);
    auto load_q = [&](const Cursor& u, uint4 (&raw)[D / 32]) {
        const int r = (u.unit % p.row_blocks) * R + q_row;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (u.valid() && r < p.rows) {
            const long long head = static_cast<long long>(u.b) * p.c.H_kv + u.unit / p.row_blocks;
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) +
                                                              (head * p.rows + r) * D + t * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) raw[i] = src[i];
        }
    };
    auto put_q = [&](const uint4 (&raw)[D / 32]) {
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            m = __vmaxu2(__vmaxu2(__vmaxu2(m, raw[i].x & 0x7FFF7FFFu), raw[i].y & 0x7FFF7FFFu),
                         __vmaxu2(raw[i].z & 0x7FFF7FFFu, raw[i].w & 0x7FFF7FFFu));
        m = max(m & 0xFFFFu, m >> 16);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t mf = __float_as_uint(p.f16 ? widen_lo16<true>(m) : widen_lo16<false>(m));
        // the row's largest magnitude is in [2^e, 2^(e+1)); zero, infinite or NaN rows stay as they are
        int e = static_cast<int>(mf >> 23) - 127;
        e = mf == 0u || e == 128 ? 14 : max(e, -100);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
        const float down = __uint_as_float(static_cast<uint32_t>(127 + e - 14) << 23);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float lo = p.f16 ? widen_lo16<true>(w[j]) : widen_lo16<false>(w[j]);
                const float hi = p.f16 ? widen_lo16<true>(w[j] >> 16) : widen_lo16<false>(w[j] >> 16);
                h[j] = pack_f16x2(lo * up, hi * up);
            }
            // words 0, 1: the two halves of step 2 i; 2, 3: of step 2 i + 1
            sm_q[(warp * (D / 32) + i) * 32 + lane] = make_uint4(h[0], h[1], h[2], h[3]);
        }
        if (t == 0) sm_c[q_row] = p.scale_log2 * down;
    };
    uint4 raw[D / 32];
    if (warp < C::kQTiles) load_q(cur, raw);

    float4* sm_o = reinterpret_cast<float4*>(smem + C::kOffO);
    float4* sm_ml = reinterpret_cast<float4*>(smem + C::kOffMl);
    int used = 0;  // groups consumed
    bool ok = true;

    while (cur.valid()) {
        const int kvh = cur.b * p.c.H_kv + cur.unit / p.row_blocks;
        const int row0 = (cur.unit % p.row_blocks) * C::kRows;  // of the head's rows
        // ---- q fragments for the block, from the rows loaded ahead
        if (warp < C::kQTiles) put_q(raw);
        sync_rows();
        Tile tile;
        tile.start(sm_c, lane);
        Slab u;
        u.q = sm_q;
        u.logits = p.logits == nullptr ? nullptr : p.logits + static_cast<long long>(kvh) * p.c.capacity * p.rows + row0;
        u.len = cur.len;
        u.rows = p.rows;
        u.row0 = row0;
        u.Nq = p.Nq;
        u.causal = p.causal;
        const int all_see = cur.len - (p.causal ? p.Nq - 1 : 0);  // slots every row sees
        for (int group = cur.s0; group < cur.s1; group += kWarps) {
            const int s = used % C::kStages;
            const int slab = group + warp;
            const bool mine = slab < cur.s1;
            if (mine) ok = ok && __all_sync(0xffffffffu, wait_phase(full(s), (used / C::kStages) & 1, abort_flag, wp, 80));
            if (mine && ok) {
                const uint8_t* stage = smem + C::kOffRing + s * C::kStageBytes;
                u.kc = stage + warp * C::kCodeBytes;
                u.vc = u.kc + kWarps * C::kCodeBytes;
                u.ks = stage + 2 * kWarps * C::kCodeBytes + warp * C::kScaleBytes;
                u.vs = u.ks + kWarps * C::kScaleBytes;
                u.key0 = slab * kSlab;
                u.masked = u.key0 + kSlab > all_see;
                u.first = group == cur.s0;
                tile.slab(u);
            }
            __syncwarp();  // the slab has been read by every lane
            if (lane == 0) mbar_arrive(empty(s));
            ++used;
        }

        // ---- the unit's result over the CTA's warps
        Target to;
        to.whole = cur.s0 == 0 && cur.s1 == cur.slabs;
        to.slot = (static_cast<long long>(blockIdx.x) * 2 + (cur.s0 > 0 ? 0 : 1)) * R;
        to.row0 = static_cast<long long>(kvh) * p.rows + row0;
        to.left = p.rows - row0;
        cur.next(p.c, units);
        tile.finish(p, to, sm_ml, sm_o, warp, [&] {
            if (warp < C::kQTiles) load_q(cur, raw);
        });
        sync_rows();
    }
}

// ------------------------------------------------------------ second kernel
// Where a unit's partial results are: CTAs first .. last of the main kernel,
// slot 1 of the first and slot 0 of the others.
struct Parts {
    int slabs, first, last;
};
// Lengths from the second-level cache: what a thread read of them ahead of its wait stays in no cache of the SM.
__device__ __forceinline__ int length_of(const Kv4Cache& c, int b) { return min(max(__ldcg(c.counts + b), 0), c.capacity); }
__device__ __forceinline__ int length_of_lane(const Kv4Cache& c) {
    const int lane = threadIdx.x % 32;
    return lane < c.B ? length_of(c, lane) : 0;
}
// Where sequence b begins, its length and slabs, a CTA's share, by a warp (every lane gets them); `mine`: the length
// of sequence `lane`.
struct Spread {
    int before, len, slabs, per, cost;
};
__device__ __forceinline__ Spread spread_of(const Kv4FwdParams& p, int b, int mine) {
    const int lane = threadIdx.x % 32, units = p.c.H_kv * p.row_blocks;
    int total = share_of(slabs_of(mine), p.unit_cost) * units;
    int before = lane < b ? total : 0;
    for (int x = 32 + lane; x < p.c.B; x += 32) {
        const int n = share_of(slabs_of(length_of(p.c, x)), p.unit_cost) * units;
        total += n;
        if (x < b) before += n;
    }
    Spread s;
    s.before = static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(before)));
    s.per = slabs_per_cta(static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(total))), p.ctas);
    s.len = b < 32 ? __shfl_sync(0xffffffffu, mine, b) : length_of(p.c, b);
    s.slabs = slabs_of(s.len);
    s.cost = p.unit_cost;
    return s;
}
__device__ __forceinline__ Parts parts_of(const Spread& s, int unit) {
    Parts r;
    r.slabs = s.slabs;
    const int hs = s.before + unit * share_of(s.slabs, s.cost);
    r.first = hs / s.per;
    r.last = s.slabs > 0 ? (hs + s.slabs - 1) / s.per : r.first;
    return r;
}
__device__ __forceinline__ long long part_row(int cta, int first, int rows, int r) {
    return (static_cast<long long>(cta) * 2 + (cta == first ? 1 : 0)) * rows + r;
}
// The sums of a row's part first + lane.
__device__ __forceinline__ float4 first_sums(const Kv4FwdParams& p, const Parts& u, int rows, int r) {
    const int c0 = u.first + static_cast<int>(threadIdx.x) % 32;
    return c0 <= u.last ? p.part_ml[part_row(c0, u.first, rows, r)] : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
}
// A row's reference, exact sum and rounded sum over its parts, by a warp, and
// the factor of the part first + lane (0 where there is none); ml0: first_sums.
__device__ __forceinline__ void row_sums(const Kv4FwdParams& p, const Parts& u, int rows, int r, const float4& ml0,
                                         float& M, float& L, float& LQ, float& f) {
    const int lane = threadIdx.x % 32, c0 = u.first + lane;
    M = ml0.x;
    for (int c = c0 + 32; c <= u.last; c += 32) M = fmaxf(M, p.part_ml[part_row(c, u.first, rows, r)].x);
#pragma unroll
    for (int o = 16; o >= 1; o /= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    f = c0 > u.last ? 0.0f : M == -INFINITY ? 1.0f : ex2(ml0.x - M);
    L = f * ml0.y;
    LQ = f * ml0.z;
    for (int c = c0 + 32; c <= u.last; c += 32) {
        const float4 ml = p.part_ml[part_row(c, u.first, rows, r)];
        const float w = M == -INFINITY ? 1.0f : ex2(ml.x - M);
        L += w * ml.y;
        LQ += w * ml.z;
    }
#pragma unroll
    for (int o = 16; o >= 1; o /= 2) {
        L += __shfl_xor_sync(0xffffffffu, L, o);
        LQ += __shfl_xor_sync(0xffffffffu, LQ, o);
    }
}

constexpr int kJoinThreads = 256;
constexpr int kJoinKeys = 1024;  // keys per block of the weights' part
constexpr int kMaxRows = 128;
constexpr int kAhead = 8;  // parts' rows loaded ahead of the factors

// Blocks 0 .. join_blocks - 1: the output rows whose unit several CTAs shared
// (or that has no slot at all), p.join_warps warps a row: one, or the whole
// block where a row has 2 kAhead parts or more.  A warp against a block, in us:
// d = 128, H = 32/8, 16384 slots, B = 1 (38 parts) 14.9 / 10.4, B = 2 (19)
// 17.5 / 16.5; 8192 slots, B = 4 (10) 15.7 / 16.1; d = 64 and 8 or 16 rows a
// head alike (16384 slots, B = 1, 16 rows 19.2 / 17.1).  The others: accumulated weight,
// kJoinKeys slots of one key/value head each.
//
// The lengths are read ahead of the wait for the main kernel, and again behind
// it: that kernel waited for whatever wrote them, but only a kernel's own wait
// makes them certain to it.  What goes by the first reading, indices within the
// workspace whatever was read and the first loads, is done again where the
// second differs.  (All behind the wait: 16384 slots, B = 8, 35.3 us instead of
// 33.9.)
template <int D, int kWays>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(const Kv4FwdParams p, int rows_per_block,
                                                                 int join_blocks) {
    grid_release();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if (static_cast<int>(blockIdx.x) < join_blocks) {
        const int way = warp % kWays;  // this warp adds parts way, way + kWays, ..
        const long long row = static_cast<long long>(blockIdx.x) * (kJoinThreads / 32 / kWays) + warp / kWays;
        if (row >= static_cast<long long>(p.c.B) * p.c.H_kv * p.rows) {
            grid_wait();
            return;
        }
        const long long kvh = row / p.rows;
        const int r = static_cast<int>(row - kvh * p.rows);
        const int b = static_cast<int>(kvh / p.c.H_kv);
        const int unit = static_cast<int>(kvh % p.c.H_kv) * p.row_blocks + r / rows_per_block;
        const int early = length_of_lane(p.c);
        Parts u = parts_of(spread_of(p, b, early), unit);
        grid_wait();
        const int mine = length_of_lane(p.c);
        constexpr int kPer = D / 32;
        const int rb = r % rows_per_block;
        int parts = 0;
        float acc[kPer] = {}, M = -INFINITY, L = 0.0f, LQ = 0.0f;
        float ahead[kAhead][kPer], x = 0.0f, f;
        float4 ml0;
        const auto load = [&](int i, float (&v)[kPer]) {
            const float* src = p.part_o + part_row(u.first + i, u.first, rows_per_block, rb) * D + lane * kPer;
#pragma unroll
            for (int j = 0; j < kPer; j += 2)
                *reinterpret_cast<float2*>(v + j) = *reinterpret_cast<const float2*>(src + j);
        };
        const auto reference = [&](int i) {
            return i < parts ? p.part_ml[part_row(u.first + i, u.first, rows_per_block, rb)].x : -INFINITY;
        };
        // the first parts' rows are on their way while the factors are formed, one per lane
        const auto begin = [&] {
            parts = u.slabs > 0 ? u.last - u.first + 1 : 0;
            if (parts == 0) return;
            if constexpr (kWays > 1) x = reference(way + kWays * lane);
            ml0 = first_sums(p, u, rows_per_block, rb);
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (way + kWays * k < parts) load(way + kWays * k, ahead[k]);
        };
        if (p.c.B <= 32) begin();
        if (p.c.B > 32 || __any_sync(0xffffffffu, mine != early)) {
            u = parts_of(spread_of(p, b, mine), unit);
            begin();
        }
        if (u.slabs > 0 && u.first == u.last) return;  // the main kernel wrote it
        if (u.slabs > 0) {
            const auto factor = [&](int i, float x) { return i >= parts ? 0.0f : M == -INFINITY ? 1.0f : ex2(x - M); };
            row_sums(p, u, rows_per_block, rb, ml0, M, L, LQ, f);
            if constexpr (kWays > 1) f = factor(way + kWays * lane, x);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const float w = __shfl_sync(0xffffffffu, f, k);
                if (way + kWays * k < parts)
#pragma unroll
                    for (int j = 0; j < kPer; ++j) acc[j] += w * ahead[k][j];
            }
            // the others: 32 factors at a time; four parts' rows in flight
            const int of_way = (parts - way + kWays - 1) / kWays;
            for (int k0 = kAhead; k0 < of_way; k0 = (k0 / 32 + 1) * 32) {
                if (k0 >= 32) f = factor(way + kWays * (k0 + lane), reference(way + kWays * (k0 + lane)));
                const int n = min((k0 / 32 + 1) * 32, of_way);
#pragma unroll 4
                for (int k = k0; k < n; ++k) {
                    const float w = __shfl_sync(0xffffffffu, f, k % 32);
                    float v[kPer];
                    load(way + kWays * k, v);
#pragma unroll
                    for (int j = 0; j < kPer; ++j) acc[j] += w * v[j];
                }
            }
        }
        if constexpr (kWays > 1) {  // a block per row: every warp is here
            __shared__ float sums[kJoinThreads / 32][D];
#pragma unroll
            for (int j = 0; j < kPer; ++j) sums[warp][lane * kPer + j] = acc[j];
            __syncthreads();
            if (warp > 0) return;
#pragma unroll
            for (int w = 1; w < kJoinThreads / 32; ++w)
#pragma unroll
                for (int j = 0; j < kPer; ++j) acc[j] += sums[w][lane * kPer + j];
        }
        const float inv = LQ == 0.0f ? 0.0f : 1.0f / LQ;
        uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + row * D + lane * kPer);
#pragma unroll
        for (int i = 0; i < kPer; i += 2)
            dst[i / 2] = p.f16 ? pack_f16x2(acc[i] * inv, acc[i + 1] * inv) : pack_bf16x2(acc[i] * inv, acc[i + 1] * inv);
        if (lane == 0 && p.lse != nullptr)
            p.lse[row] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
        return;
    }
    __shared__ float lse2[kMaxRows];
    constexpr int kMine = kJoinKeys / kJoinThreads;  // keys per thread
    const int chunks = (p.c.capacity + kJoinKeys - 1) / kJoinKeys;
    const int i = static_cast<int>(blockIdx.x) - join_blocks;
    const int kvh = i / chunks, b = kvh / p.c.H_kv;
    const int key0 = (i % chunks) * kJoinKeys;
    const int early = length_of_lane(p.c);
    Spread spread = spread_of(p, b, early);
    grid_wait();
    const int mine = length_of_lane(p.c);
    const long long slot0 = static_cast<long long>(kvh) * p.c.capacity + key0 + threadIdx.x;
    int left = 0;  // this thread's keys: 0, 256, .. below it
    // four rows (a quarter of a 16-row block, the usual group) wait in registers for the rows' sums
    float4 first4[kMine];
    float old[kMine];
    const bool four = p.rows % 4 == 0;
    const auto begin = [&] {
        left = spread.len - key0 - static_cast<int>(threadIdx.x);
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
            const long long at = slot0 + k * kJoinThreads;
            const bool in = k * kJoinThreads < left;
            old[k] = in && p.weight_in != nullptr ? p.weight_in[at] : 0.0f;
            first4[k] = in && four ? *reinterpret_cast<const float4*>(p.logits + at * p.rows)
                                   : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        }
    };
    if (p.c.B <= 32) begin();
    if (p.c.B > 32 || __any_sync(0xffffffffu, mine != early)) {
        spread = spread_of(p, b, mine);
        begin();
    }
    if (key0 >= spread.len) return;
    for (int r = warp; r < p.rows; r += kJoinThreads / 32) {
        const Parts u = parts_of(spread, (kvh % p.c.H_kv) * p.row_blocks + r / rows_per_block);
        float v;
        if (p.single || u.first == u.last) {
            v = p.row_lse2[static_cast<long long>(kvh) * p.rows + r];
        } else {
            float M, L, LQ, f;
            const float4 ml0 = first_sums(p, u, rows_per_block, r % rows_per_block);
            row_sums(p, u, rows_per_block, r % rows_per_block, ml0, M, L, LQ, f);
            v = L == 0.0f ? -INFINITY : M + log2f(L);
        }
        if (lane == 0) lse2[r] = v == -INFINITY ? INFINITY : v;  // a row that sees nothing adds nothing
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
        if (k * kJoinThreads >= left) break;
        const long long at = slot0 + k * kJoinThreads;
        const float* t = p.logits + at * p.rows;
        float s = 0.0f;
        if (four) {
            float4 y = first4[k];
            for (int r = 0;;) {
                s += (ex2(y.x - lse2[r]) + ex2(y.y - lse2[r + 1])) + (ex2(y.z - lse2[r + 2]) + ex2(y.w - lse2[r + 3]));
                if ((r += 4) >= p.rows) break;
                y = *reinterpret_cast<const float4*>(t + r);
            }
        } else {
            for (int r = 0; r < p.rows; ++r) s += ex2(t[r] - lse2[r]);
        }
        p.weight_out[at] = old[k] + s;
    }
}

template <int D, int R>
cudaError_t launch_variant(const Kv4FwdParams& p, cudaStream_t stream) {
    using C = Kv4Cfg<D, R>;
    auto kern = kv4_fwd_kernel<D, R>;
    static SmemAllowed allowed;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), C::kSmemBytes, allowed);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kern, dim3(static_cast<unsigned>(p.ctas)), kThreads4, C::kSmemBytes, stream, p);
    if (e != cudaSuccess) return e;
    const long long rows = p.single ? 0 : static_cast<long long>(p.c.B) * p.c.H_kv * p.rows;
    const int per_block = kJoinThreads / 32 / p.join_warps;
    const int join = static_cast<int>((rows + per_block - 1) / per_block);
    if (p.single && p.logits == nullptr) return cudaSuccess;
    const long long keys = p.logits == nullptr ? 0
                                               : static_cast<long long>(p.c.B) * p.c.H_kv *
                                                     ((p.c.capacity + kJoinKeys - 1) / kJoinKeys);
    auto second = p.join_warps > 1 ? kv4_join_kernel<D, kJoinThreads / 32> : kv4_join_kernel<D, 1>;
    return launch_dependent(second, dim3(static_cast<unsigned>(join + keys)), kJoinThreads, 0, stream, p, C::kRows, join);
}

}  // namespace

int kv4_rows_per_block(int64_t rows) { return rows <= 4 ? 4 : rows <= 8 ? 8 : 16; }

Kv4Plan kv4_plan(int64_t B, int64_t H_kv, int64_t rows, int64_t capacity, int sms) {
    const int64_t rpb = kv4_rows_per_block(rows);
    const int64_t units = B * H_kv * ((rows + rpb - 1) / rpb);
    Kv4Plan plan;
    plan.single = capacity <= (units >= sms ? 2 : 1) * kWholeSlots;
    if (plan.single) {
        plan.ctas = static_cast<int>(units);
    } else {
        const int64_t most = static_cast<int64_t>(sms) * (rpb <= 8 ? 2 : 1);
        const int64_t want = (units * (capacity / kSlab) + kWarps - 1) / kWarps;
        plan.ctas = static_cast<int>(want < most ? want : most);
        plan.unit_cost = want > 2 * most ? kKv4UnitCost : 0;
        if (plan.ctas >= 2 * kAhead * units) plan.join_warps = kJoinThreads / 32;
    }
    return plan;
}

cudaError_t launch_kv4_fwd(const Kv4FwdParams& p, cudaStream_t stream) {
    switch (kv4_rows_per_block(p.rows)) {
        case 4: return p.c.d == 128 ? launch_variant<128, 4>(p, stream) : launch_variant<64, 4>(p, stream);
        case 8: return p.c.d == 128 ? launch_variant<128, 8>(p, stream) : launch_variant<64, 8>(p, stream);
        default: return p.c.d == 128 ? launch_variant<128, 16>(p, stream) : launch_variant<64, 16>(p, stream);
    }
}

}  // namespace fa
