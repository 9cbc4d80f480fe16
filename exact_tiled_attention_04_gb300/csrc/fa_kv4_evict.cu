// Eviction from the 4-bit cache by accumulated weight (include/fa.h,
// fa_kv4_evict): per key/value head, the `keep` entries of largest key, where
// an entry's key orders (protected first, then weight; ties by slot).
//
// One thread-block cluster per head, every CTA holding a contiguous slice of
// the head's keys in shared memory:
//   1. radix selection, 11 + 11 + 10 bits: a histogram per CTA, summed over
//      the cluster through distributed shared memory, gives the threshold T
//      and how many entries equal to T are kept;
//   2. the entries' flags, by ballots: kept = key > T, or key == T and its
//      rank among those (in slot order) is below that count;
//   3. holes (slots below the new length whose entry leaves) and late entries
//      (kept ones at or behind it) are as many as one another; hole r takes
//      late entry r;
//   4. the moved rows are copied.  Sources lie at or behind the new length
//      and targets below it, so in place no copy reads what another writes.
#include <cstdint>

#include "fa_kv4.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvBins = 2048;
constexpr int kEvMaxCluster = 8;
constexpr int kEvMaxSlice = kKv4EvictMaxCapacity / kEvMaxCluster;  // keys per CTA

struct EvShared {
    uint32_t hist[kEvBins];
    uint32_t total[kEvBins];   // over the cluster
    uint32_t warp_sum[kEvWarps];
    uint32_t count[2];         // this CTA's counts, read by the cluster
    uint32_t pick[2];          // bin, entries above it
};

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(addr, rank)) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(addr, rank)), "r"(v) : "memory");
}

// Exclusive prefix of v over the block's threads; *sum gets the total.
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t* warp_sum, uint32_t* sum) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // warp_sum may still be read
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    uint32_t w = warp_sum[lane];  // kEvWarps == 32
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    *sum = __shfl_sync(0xffffffffu, w, 31);
    const uint32_t before = __shfl_sync(0xffffffffu, w, (warp + 31) % 32);
    return (warp > 0 ? before : 0u) + x - v;
}

// Order-preserving key: protected > NaN > numbers in order; -0 equals +0.
__device__ __forceinline__ uint32_t rank_key(float w, bool first) {
    if (first) return 0xFFFFFFFFu;
    if (w != w) return 0xFFFFFFFEu;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

// Copy one entry (8 lanes per entry, `part` = lane % 8).
template <int D>
__device__ __forceinline__ void copy_entry(const Kv4Cache& f, const Kv4Cache& t, long long at, long long to, int part) {
    constexpr int kChunks = D / 32;  // 16-byte chunks of a row's codes
    if (part < 2 * kChunks) {
        const bool value = part >= kChunks;
        const int ch = value ? part - kChunks : part;
        reinterpret_cast<uint4*>(value ? t.codes[1] : t.codes[0])[to * kChunks + ch] =
            reinterpret_cast<const uint4*>(value ? f.codes[1] : f.codes[0])[at * kChunks + ch];
    }
    const int rest = D == 128 ? part : part - 4;
    if (rest == 0 || rest == 1) {
        const uint8_t* s = rest ? f.scales[1] : f.scales[0];
        uint8_t* r = rest ? t.scales[1] : t.scales[0];
        if constexpr (D == 128)
            reinterpret_cast<uint2*>(r)[to] = reinterpret_cast<const uint2*>(s)[at];
        else
            reinterpret_cast<uint32_t*>(r)[to] = reinterpret_cast<const uint32_t*>(s)[at];
    }
    if (rest == 2 && f.pos != nullptr && t.pos != nullptr) t.pos[to] = f.pos[at];
    if (rest == 3 && f.weight != nullptr && t.weight != nullptr) t.weight[to] = f.weight[at];
}

template <int D>
__global__ void __launch_bounds__(kEvThreads, 1) kv4_evict_kernel(const Kv4EvictParams p, int slice, int advance) {
    __shared__ EvShared sh;
    extern __shared__ uint32_t keys[];  // slice, and the kept bits behind it
    const uint32_t cs = static_cast<uint32_t>(gridDim.x) / static_cast<uint32_t>(p.from.B * p.from.H_kv);
    const uint32_t rank = cluster_ctarank();
    const int head = static_cast<int>(blockIdx.x / cs);
    const int b = head / p.from.H_kv;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int n = min(max(p.from.counts[b], 0), p.from.capacity);
    const int seen = p.from.counts[p.from.B + b];
    const int nn = min(n, p.keep);  // the new length
    const bool in_place = p.to.codes[0] == p.from.codes[0];
    int32_t* src = p.src + static_cast<long long>(head) * p.keep;
    const long long row0 = static_cast<long long>(head) * p.from.capacity;
    const long long to0 = static_cast<long long>(head) * p.to.capacity;
    const int begin = static_cast<int>(min(static_cast<long long>(rank) * slice, static_cast<long long>(n)));
    const int end = min(begin + slice, n);
    uint32_t* kept = keys + slice;  // bit i % 32 of word i / 32: entry begin + i stays
    const uint32_t keys_addr = smem_u32(keys);

    if (n > nn) {
        for (int i = begin + threadIdx.x; i < end; i += kEvThreads) {
            bool first = false;
            if (p.sinks > 0 || p.recent > 0) {
                const int pos = p.from.pos[row0 + i];
                first = pos < p.sinks || static_cast<long long>(pos) >= static_cast<long long>(seen) - p.recent;
            }
            keys[i - begin] = rank_key(p.rank_by[row0 + i], first);
        }
        // 1. threshold: the entries whose upper bits equal `prefix` are still open
        uint32_t prefix = 0u, mask = 0u;
        uint32_t want = static_cast<uint32_t>(nn);  // entries to take among them
        const int shifts[3] = {21, 10, 0}, widths[3] = {11, 11, 10};
#pragma unroll
        for (int pass = 0; pass < 3; ++pass) {
            const int down = shifts[pass], bins = 1 << widths[pass];
            for (int i = threadIdx.x; i < bins; i += kEvThreads) sh.hist[i] = 0u;
            __syncthreads();
            for (int i = threadIdx.x; i < end - begin; i += kEvThreads) {
                const uint32_t k = keys[i];
                if ((k & mask) == prefix) atomicAdd(&sh.hist[(k >> down) & static_cast<uint32_t>(bins - 1)], 1u);
            }
            cluster_sync_all();
            for (int i = threadIdx.x; i < bins; i += kEvThreads) {
                uint32_t s = 0u;
                for (uint32_t r = 0; r < cs; ++r) s += ld_cluster_u32(smem_u32(&sh.hist[i]), r);
                sh.total[i] = s;
            }
            __syncthreads();
            // from the top bin down: thread t holds bins bins-1-2t and bins-2-2t
            const int hi = bins - 1 - 2 * static_cast<int>(threadIdx.x);
            const uint32_t c0 = hi >= 0 ? sh.total[hi] : 0u, c1 = hi >= 1 ? sh.total[hi - 1] : 0u;
            uint32_t all;
            const uint32_t above = block_prefix(c0 + c1, sh.warp_sum, &all);
            if (above < want && want <= above + c0) {
                sh.pick[0] = static_cast<uint32_t>(hi);
                sh.pick[1] = above;
            } else if (above + c0 < want && want <= above + c0 + c1) {
                sh.pick[0] = static_cast<uint32_t>(hi - 1);
                sh.pick[1] = above + c0;
            }
            __syncthreads();
            prefix |= sh.pick[0] << down;
            mask |= static_cast<uint32_t>(bins - 1) << down;
            want -= sh.pick[1];
            cluster_sync_all();  // every CTA has read this pass's histograms
        }
        // 2. kept flags; warps take contiguous runs of words, ranks follow slot order
        const uint32_t T = prefix;  // `want` entries equal to T are kept
        const int words = (end - begin + 31) / 32;
        const int per_warp = (words + kEvWarps - 1) / kEvWarps;
        const int w0 = min(warp * per_warp, words), w1 = min(w0 + per_warp, words);
        auto key_at = [&](int word) -> uint32_t {
            const int i = word * 32 + lane;
            return i < end - begin ? keys[i] : 0u;
        };
        uint32_t eq = 0u;
        for (int x = w0; x < w1; ++x)
            eq += __popc(__ballot_sync(0xffffffffu, x * 32 + lane < end - begin && key_at(x) == T));
        uint32_t all;
        uint32_t eq_before = __shfl_sync(0xffffffffu, block_prefix(lane == 0 ? eq : 0u, sh.warp_sum, &all), 0);
        if (threadIdx.x == 0) sh.count[0] = all;
        cluster_sync_all();
        for (uint32_t r = 0; r < rank; ++r) eq_before += ld_cluster_u32(smem_u32(&sh.count[0]), r);
        uint32_t holes = 0u, late = 0u;
        for (int x = w0; x < w1; ++x) {
            const int i = x * 32 + lane;
            const bool in = i < end - begin;
            const uint32_t k = key_at(x);
            const uint32_t eqs = __ballot_sync(0xffffffffu, in && k == T);
            const bool stay = in && (k > T || (k == T && eq_before + __popc(eqs & ((1u << lane) - 1u)) < want));
            eq_before += __popc(eqs);
            const uint32_t bits = __ballot_sync(0xffffffffu, stay);
            if (lane == 0) kept[x] = bits;
            holes += __popc(__ballot_sync(0xffffffffu, in && !stay && begin + i < nn));
            late += __popc(__ballot_sync(0xffffffffu, stay && begin + i >= nn));
        }
        // 3. ranks of holes and late entries over the cluster
        uint32_t h_all, l_all;
        uint32_t h_rank = __shfl_sync(0xffffffffu, block_prefix(lane == 0 ? holes : 0u, sh.warp_sum, &h_all), 0);
        uint32_t l_rank = __shfl_sync(0xffffffffu, block_prefix(lane == 0 ? late : 0u, sh.warp_sum, &l_all), 0);
        cluster_sync_all();  // count[0] of the previous step was read
        if (threadIdx.x == 0) {
            sh.count[0] = h_all;
            sh.count[1] = l_all;
        }
        cluster_sync_all();  // and every key: the slices now hold the list of holes
        for (uint32_t r = 0; r < rank; ++r) {
            h_rank += ld_cluster_u32(smem_u32(&sh.count[0]), r);
            l_rank += ld_cluster_u32(smem_u32(&sh.count[1]), r);
        }
        for (int x = w0; x < w1; ++x) {
            const int i = begin + x * 32 + lane;
            const bool stay = (kept[x] >> lane) & 1u;
            const bool hole = i < end && !stay && i < nn;
            const uint32_t bits = __ballot_sync(0xffffffffu, hole);
            if (hole) {
                const uint32_t r = h_rank + __popc(bits & ((1u << lane) - 1u));
                st_cluster_u32(keys_addr + 4u * (r % static_cast<uint32_t>(slice)), r / static_cast<uint32_t>(slice),
                               static_cast<uint32_t>(i));
            }
            h_rank += __popc(bits);
            if (i < nn && stay) src[i] = i;
        }
        cluster_sync_all();
        for (int x = w0; x < w1; ++x) {
            const int i = begin + x * 32 + lane;
            const bool mine = i < end && ((kept[x] >> lane) & 1u) && i >= nn;
            const uint32_t bits = __ballot_sync(0xffffffffu, mine);
            if (mine) {
                const uint32_t r = l_rank + __popc(bits & ((1u << lane) - 1u));
                src[ld_cluster_u32(keys_addr + 4u * (r % static_cast<uint32_t>(slice)),
                                   r / static_cast<uint32_t>(slice))] = i;
            }
            l_rank += __popc(bits);
        }
    } else {
        for (int i = static_cast<int>(rank) * kEvThreads + threadIdx.x; i < nn; i += static_cast<int>(cs) * kEvThreads)
            src[i] = i;
    }
    for (long long i = nn + static_cast<long long>(rank) * kEvThreads + threadIdx.x; i < p.keep;
         i += static_cast<long long>(cs) * kEvThreads)
        src[i] = -1;
    // 4. copies, 32 slots per warp and step (src was written by the whole cluster)
    cluster_sync_all();
    const int step = static_cast<int>(cs) * kEvWarps * 32;
    for (int j0 = (static_cast<int>(rank) * kEvWarps + warp) * 32; j0 < nn; j0 += step) {
        const int j = j0 + lane;
        const int from = j < nn ? __ldcg(src + j) : -1;
        uint32_t todo = __ballot_sync(0xffffffffu, from >= 0 && (!in_place || from != j));
        while (todo) {  // four entries at a time, eight lanes each
            uint32_t rest = todo;
            for (int g = 0; g < lane / 8; ++g) rest &= rest - 1u;
            const int who = rest ? __ffs(static_cast<int>(rest)) - 1 : 0;
            const int at = __shfl_sync(0xffffffffu, from, who);
            if (rest) copy_entry<D>(p.from, p.to, row0 + at, to0 + j0 + who, lane % 8);
            for (int g = 0; g < 4; ++g) todo &= todo - 1u;
        }
    }
    if (advance && head % p.from.H_kv == 0 && rank == 0 && threadIdx.x == 0) {
        p.counts_out[b] = nn;
        p.counts_out[p.from.B + b] = seen;
    }
}

// counts_out where it is the counts that the clusters of a sequence read.
__global__ void kv4_evict_counts_kernel(const Kv4EvictParams p) {
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b < p.from.B) p.counts_out[b] = min(min(max(p.from.counts[b], 0), p.from.capacity), p.keep);
}

template <int D>
cudaError_t launch_evict(const Kv4EvictParams& p, int sms, cudaStream_t stream) {
    const int heads = p.from.B * p.from.H_kv;
    // as many CTAs per head as leave no SM idle, and as its keys need
    int cs = 1;
    while (cs < kEvMaxCluster && ((p.from.capacity + cs - 1) / cs > kEvMaxSlice || 2 * cs * heads <= sms)) cs *= 2;
    const int slice = ((p.from.capacity + cs - 1) / cs + 31) / 32 * 32;
    const size_t smem = static_cast<size_t>(slice) * 4 + static_cast<size_t>(slice / 32) * 4;
    auto kern = kv4_evict_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const int advance = p.counts_out == p.from.counts ? 0 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cs) * static_cast<unsigned>(heads));
    cfg.blockDim = dim3(kEvThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cs);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, p, slice, advance);
    if (e != cudaSuccess) return e;
    if (!advance) kv4_evict_counts_kernel<<<(p.from.B + 127) / 128, 128, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_evict(const Kv4EvictParams& p, int sms, cudaStream_t stream) {
    return p.from.d == 128 ? launch_evict<128>(p, sms, stream) : launch_evict<64>(p, sms, stream);
}

}  // namespace fa
