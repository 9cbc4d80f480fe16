// Eviction from the 4-bit cache by accumulated weight (include/fa.h,
// fa_kv4_evict): per key/value head, the `keep` entries of largest key, where
// an entry's key orders (protected first, then weight; ties by slot).
//
// One block per head, or a cluster of them where heads are few or long, every
// CTA holding a contiguous slice of the head's keys in shared memory:
//   1. radix selection, 8 bits at a time, gives the threshold T and how many
//      entries equal to T are kept.  A histogram has 256 bins of 32 counters,
//      one per lane, so that no two lanes of a warp meet in a bank or on a
//      counter, however the weights are distributed (a layer's weights share a
//      few exponents, all new entries share 0);
//   2. the entries' flags, by ballots: kept = key > T, or key == T and its
//      rank among those (in slot order) is below that count;
//   3. holes (slots below the new length whose entry leaves) and late entries
//      (kept ones at or behind it) are as many as one another; hole r takes
//      late entry r;
//   4. the moved rows are copied, 32 a warp with all their loads in flight.
//      Sources lie at or behind the new length and targets below it, so in
//      place no copy reads what another writes.
// Short rows are bound by the latency of these steps, long ones that move
// many entries by their copies.
#include <cstdint>

#include "fa_kv4.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvMaxCluster = 8;
constexpr int kEvMaxSlice = kKv4EvictMaxCapacity / kEvMaxCluster;  // keys per CTA

// Shared memory: EvShared, then the slice's keys.
struct EvShared {
    uint32_t hist[256 * 32];   // [bin][lane]; after the selection a bit per key (kept)
    uint32_t bins[256];        // this CTA's sums
    uint32_t total[256];       // the cluster's
    uint32_t warp_count[2][kEvWarps];
    uint32_t count[4];         // this CTA's, read by the cluster
};

static_assert(kEvMaxSlice / 32 <= 256 * 32 && sizeof(EvShared) + kEvMaxSlice * 4 <= 232448,
              "shared memory budget exceeded");

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(addr, rank)) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(addr, rank)), "r"(v) : "memory");
}

// Order-preserving key: protected > NaN > numbers in order; -0 equals +0.
__device__ __forceinline__ uint32_t rank_key(float w, bool first) {
    if (first) return 0xFFFFFFFFu;
    if (w != w) return 0xFFFFFFFEu;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

// Entries to .. to + 31 of a head (rows `row` of the targets): lane i's entry
// comes from slot `from` of the sources, or stays out where from < 0.
template <int D>
__device__ __forceinline__ void copy_entries(const Kv4Cache& f, const Kv4Cache& t, long long from_row, int from,
                                             long long to_row) {
    constexpr int kChunks = D / 32;  // 16-byte chunks of a row's codes
    const int lane = threadIdx.x % 32;
    uint4 k[kChunks], v[kChunks];
    int src[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        src[c] = __shfl_sync(0xffffffffu, from, (c * 32 + lane) / kChunks);
        if (src[c] >= 0) {
            const long long at = (from_row + src[c]) * kChunks + lane % kChunks;
            k[c] = reinterpret_cast<const uint4*>(f.codes[0])[at];
            v[c] = reinterpret_cast<const uint4*>(f.codes[1])[at];
        }
    }
    uint2 ks{}, vs{};
    int32_t pos = 0;
    float w = 0.0f;
    const long long at = from_row + from;
    if (from >= 0) {
        if constexpr (D == 128) {
            ks = reinterpret_cast<const uint2*>(f.scales[0])[at];
            vs = reinterpret_cast<const uint2*>(f.scales[1])[at];
        } else {
            ks.x = reinterpret_cast<const uint32_t*>(f.scales[0])[at];
            vs.x = reinterpret_cast<const uint32_t*>(f.scales[1])[at];
        }
        if (f.pos != nullptr && t.pos != nullptr) pos = f.pos[at];
        if (f.weight != nullptr && t.weight != nullptr) w = f.weight[at];
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        if (src[c] >= 0) {
            const long long to = to_row * kChunks + c * 32 + lane;
            reinterpret_cast<uint4*>(t.codes[0])[to] = k[c];
            reinterpret_cast<uint4*>(t.codes[1])[to] = v[c];
        }
    }
    if (from >= 0) {
        const long long to = to_row + lane;
        if constexpr (D == 128) {
            reinterpret_cast<uint2*>(t.scales[0])[to] = ks;
            reinterpret_cast<uint2*>(t.scales[1])[to] = vs;
        } else {
            reinterpret_cast<uint32_t*>(t.scales[0])[to] = ks.x;
            reinterpret_cast<uint32_t*>(t.scales[1])[to] = vs.x;
        }
        if (f.pos != nullptr && t.pos != nullptr) t.pos[to] = pos;
        if (f.weight != nullptr && t.weight != nullptr) t.weight[to] = w;
    }
}

// kOne: a block per head (no cluster).
template <int D, bool kOne>
__global__ void __launch_bounds__(kEvThreads, 1) kv4_evict_kernel(const __grid_constant__ Kv4EvictParams p, int slice,
                                                                  int advance) {
    extern __shared__ __align__(16) uint8_t ev_smem[];
    EvShared& sh = *reinterpret_cast<EvShared*>(ev_smem);
    uint32_t* keys = reinterpret_cast<uint32_t*>(ev_smem + sizeof(EvShared));
    uint32_t* kept = sh.hist;  // bit i % 32 of word i / 32: entry begin + i stays
    const uint32_t keys_addr = smem_u32(keys);
    const uint32_t cs = kOne ? 1u : static_cast<uint32_t>(gridDim.x) / static_cast<uint32_t>(p.from.B * p.from.H_kv);
    const uint32_t rank = kOne ? 0u : cluster_ctarank();
    auto sync_all = [] {
        if constexpr (kOne) __syncthreads();
        else cluster_sync_all();
    };
    const int head = static_cast<int>(blockIdx.x / cs);
    const int b = head / p.from.H_kv;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    for (int i = threadIdx.x; i < 256 * 8; i += kEvThreads)
        reinterpret_cast<uint4*>(sh.hist)[i] = make_uint4(0u, 0u, 0u, 0u);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int n = min(max(p.from.counts[b], 0), p.from.capacity);
    const int seen = p.from.counts[p.from.B + b];
    const int nn = min(n, p.keep);  // the new length
    const bool in_place = p.to.codes[0] == p.from.codes[0];
    int32_t* src = p.src + static_cast<long long>(head) * p.keep;
    const long long row0 = static_cast<long long>(head) * p.from.capacity;
    const long long to0 = static_cast<long long>(head) * p.to.capacity;
    const int begin = static_cast<int>(min(static_cast<long long>(rank) * slice, static_cast<long long>(n)));
    const int size = min(slice, n - begin);  // this CTA's keys

    if (n > nn) {
        const float* rank_by = p.rank_by + row0 + begin;
        const int32_t* pos = p.from.pos + row0 + begin;
        const bool protect = p.sinks > 0 || p.recent > 0;
        const long long newest = static_cast<long long>(seen) - p.recent;
#pragma unroll 4
        for (int i = threadIdx.x; i < size; i += kEvThreads) {
            const float w = rank_by[i];
            const int at = protect ? pos[i] : 0;
            keys[i] = rank_key(w, protect && (at < p.sinks || at >= newest));
        }
        // 1. threshold: the entries whose upper bits equal `prefix` are still open
        uint32_t prefix = 0u;
        uint32_t want = static_cast<uint32_t>(nn), open = 0u;  // entries to take among the open ones; those of the bin
#pragma unroll 1
        for (int down = 24; down >= 0; down -= 8) {
            __syncthreads();  // keys and a zeroed histogram
#pragma unroll 4
            for (int i = threadIdx.x; i < size; i += kEvThreads) {
                const uint32_t k = keys[i];
                if (down == 24 || (k >> (down + 8)) == prefix)
                    atomicAdd(&sh.hist[((k >> down) & 255u) * 32 + lane], 1u);
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 256 / kEvWarps; ++i) {
                const int bin = warp * (256 / kEvWarps) + i;
                const uint32_t s = __reduce_add_sync(0xffffffffu, sh.hist[bin * 32 + lane]);
                sh.hist[bin * 32 + lane] = 0u;
                if (lane == 0) sh.bins[bin] = s;
            }
            sync_all();
            if constexpr (!kOne) {
                if (threadIdx.x < 256) {
                    uint32_t s = 0u;
                    for (uint32_t r = 0; r < cs; ++r) s += ld_cluster_u32(smem_u32(&sh.bins[threadIdx.x]), r);
                    sh.total[threadIdx.x] = s;
                }
                cluster_sync_all();  // and every CTA has read the others' sums
            }
            // from the top bin down: lane l holds bins 255 - 8 l .. 248 - 8 l; every warp finds the bin
            const uint4* t4 = reinterpret_cast<const uint4*>(kOne ? sh.bins : sh.total) + (31 - lane) * 2;
            const uint4 lo = t4[0], hi = t4[1];
            const uint32_t c[8] = {hi.w, hi.z, hi.y, hi.x, lo.w, lo.z, lo.y, lo.x};
            const uint32_t sum = ((c[0] + c[1]) + (c[2] + c[3])) + ((c[4] + c[5]) + (c[6] + c[7]));
            uint32_t above = sum;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, above, o);
                if (lane >= o) above += y;
            }
            above -= sum;
            const uint32_t holder = __ballot_sync(0xffffffffu, above < want && want <= above + sum);
            uint32_t bin = 0u, before = above, in_bin = 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (in_bin == 0u && before + c[i] >= want) {
                    bin = static_cast<uint32_t>(255 - 8 * lane - i);
                    in_bin = c[i];
                }
                if (in_bin == 0u) before += c[i];
            }
            const int who = __ffs(static_cast<int>(holder)) - 1;
            prefix = (prefix << 8) | __shfl_sync(0xffffffffu, bin, who);
            want -= __shfl_sync(0xffffffffu, before, who);
            open = __shfl_sync(0xffffffffu, in_bin, who);
        }
        // 2. kept flags; warps take contiguous runs of words, ranks follow slot order
        const uint32_t T = prefix;  // `want` of the `open` entries equal to T are kept
        const int words = (size + 31) / 32;
        const int per_warp = (words + kEvWarps - 1) / kEvWarps;
        const int w0 = min(warp * per_warp, words), w1 = min(w0 + per_warp, words);
        uint32_t eq_before = 0u;
        if (want < open) {  // not all of them: their ranks over the cluster
            uint32_t eq = 0u;
            for (int x = w0; x < w1; ++x)
                eq += __popc(__ballot_sync(0xffffffffu, x * 32 + lane < size && keys[x * 32 + lane] == T));
            if (lane == 0) sh.warp_count[0][warp] = eq;
            __syncthreads();
            const uint32_t mine = sh.warp_count[0][lane];
            eq_before = __reduce_add_sync(0xffffffffu, lane < warp ? mine : 0u);
            const uint32_t all = __reduce_add_sync(0xffffffffu, mine);
            if (threadIdx.x == 0) sh.count[2] = all;
            sync_all();
            for (uint32_t r = 0; r < rank; ++r) eq_before += ld_cluster_u32(smem_u32(&sh.count[2]), r);
        }
        uint32_t holes = 0u, late = 0u;
        for (int x = w0; x < w1; ++x) {
            const int i = x * 32 + lane;
            const bool in = i < size;
            const uint32_t k = in ? keys[i] : 0u;
            const uint32_t eqs = __ballot_sync(0xffffffffu, in && k == T);
            const bool stay =
                in && (k > T || (k == T && (want == open || eq_before + __popc(eqs & ((1u << lane) - 1u)) < want)));
            eq_before += __popc(eqs);
            const uint32_t bits = __ballot_sync(0xffffffffu, stay);
            if (lane == 0) kept[x] = bits;
            holes += __popc(__ballot_sync(0xffffffffu, in && !stay && begin + i < nn));
            late += __popc(__ballot_sync(0xffffffffu, stay && begin + i >= nn));
        }
        // 3. ranks of holes and late entries over the cluster
        __syncthreads();  // the counts of equal entries were read
        if (lane == 0) {
            sh.warp_count[0][warp] = holes;
            sh.warp_count[1][warp] = late;
        }
        __syncthreads();
        const uint32_t hs = sh.warp_count[0][lane], ls = sh.warp_count[1][lane];
        uint32_t h_rank = __reduce_add_sync(0xffffffffu, lane < warp ? hs : 0u);
        uint32_t l_rank = __reduce_add_sync(0xffffffffu, lane < warp ? ls : 0u);
        if constexpr (!kOne) {
            const uint32_t h_all = __reduce_add_sync(0xffffffffu, hs), l_all = __reduce_add_sync(0xffffffffu, ls);
            if (threadIdx.x == 0) {
                sh.count[0] = h_all;
                sh.count[1] = l_all;
            }
            cluster_sync_all();  // also every key was read: the slices now hold the list of holes
            for (uint32_t r = 0; r < rank; ++r) {
                h_rank += ld_cluster_u32(smem_u32(&sh.count[0]), r);
                l_rank += ld_cluster_u32(smem_u32(&sh.count[1]), r);
            }
        }
        for (int x = w0; x < w1; ++x) {
            const int i = begin + x * 32 + lane;
            const bool in = x * 32 + lane < size;
            const bool stay = (kept[x] >> lane) & 1u;
            const bool hole = in && !stay && i < nn;
            const uint32_t bits = __ballot_sync(0xffffffffu, hole);
            if (hole) {
                const uint32_t r = h_rank + __popc(bits & ((1u << lane) - 1u));
                if constexpr (kOne)
                    keys[r] = static_cast<uint32_t>(i);
                else
                    st_cluster_u32(keys_addr + 4u * (r % static_cast<uint32_t>(slice)), r / static_cast<uint32_t>(slice),
                                   static_cast<uint32_t>(i));
            }
            h_rank += __popc(bits);
            if (i < nn && stay) src[i] = i;
        }
        sync_all();
        for (int x = w0; x < w1; ++x) {
            const int i = begin + x * 32 + lane;
            const bool mine = x * 32 + lane < size && ((kept[x] >> lane) & 1u) && i >= nn;
            const uint32_t bits = __ballot_sync(0xffffffffu, mine);
            if (mine) {
                const uint32_t r = l_rank + __popc(bits & ((1u << lane) - 1u));
                uint32_t hole;
                if constexpr (kOne)
                    hole = keys[r];
                else
                    hole = ld_cluster_u32(keys_addr + 4u * (r % static_cast<uint32_t>(slice)),
                                          r / static_cast<uint32_t>(slice));
                src[hole] = i;
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
    sync_all();
    const int step = static_cast<int>(cs) * kEvWarps * 32;
    for (int j0 = (static_cast<int>(rank) * kEvWarps + warp) * 32; j0 < nn; j0 += step) {
        const int j = j0 + lane;
        int from = j < nn ? __ldcg(src + j) : -1;
        if (in_place && from == j) from = -1;
        if (__any_sync(0xffffffffu, from >= 0)) copy_entries<D>(p.from, p.to, row0, from, to0 + j0);
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
    // as many CTAs per head as leave no SM idle while each has kEvShare keys to look at, and as its keys need
    constexpr int kEvShare = 8192;
    int cs = 1;
    while (cs < kEvMaxCluster && ((p.from.capacity + cs - 1) / cs > kEvMaxSlice ||
                                  (2 * cs * heads <= sms && p.from.capacity / cs > kEvShare)))
        cs *= 2;
    const int slice = ((p.from.capacity + cs - 1) / cs + 31) / 32 * 32;
    const size_t smem = sizeof(EvShared) + static_cast<size_t>(slice) * 4;
    auto kern = cs == 1 ? kv4_evict_kernel<D, true> : kv4_evict_kernel<D, false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const int advance = p.counts_out == p.from.counts ? 0 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cs) * static_cast<unsigned>(heads));
    cfg.blockDim = dim3(kEvThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cs);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cs == 1 ? 1 : 2;
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
