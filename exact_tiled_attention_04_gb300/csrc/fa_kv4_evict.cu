// Eviction from the 4-bit cache by accumulated weight (include/fa.h,
// fa_kv4_evict): per key/value head, the `keep` entries of largest key, where
// an entry's key orders (protected first, then weight; ties by slot).
//
// One block per head, or a cluster of them where a head is long, every CTA
// holding a contiguous slice of the head's keys in shared memory:
//   1. radix selection, 8 bits at a time, gives the threshold T and how many
//      entries equal to T are kept; the first histogram is counted as the keys
//      arrive, and once at most 256 entries are open they are compared with
//      one another.  A histogram has 256 bins of 32 counters,
//      one per lane, so that no two lanes of a warp meet in a bank or on a
//      counter, however the weights are distributed (a layer's weights share a
//      few exponents, all new entries share 0);
//   2. a bit per entry: kept = key > T, or key == T and among the first of
//      those in slot order; a thread forms the word of 32 entries (a ballot
//      per entry and warp took 3000 cycles instead of 2000 for 16384 keys);
//   3. holes (slots below the new length whose entry leaves) and late entries
//      (kept ones at or behind it) are as many as one another; hole r takes
//      late entry r.  Ranks come from a scan over the words of bits, and the
//      thread of a word walks its late entries (an entry per lane: 5300 cycles
//      instead of 1500);
//   4. the moved rows are copied, 32 a warp with all their loads in flight.
//      Sources lie at or behind the new length and targets below it, so in
//      place no copy reads what another writes.
// A decode step that puts one entry too many into the cache needs no
// threshold: up to kEvFew leaving entries of a head that one block holds are
// found one by one, by a warp with the least entry of every 32nd of the head in
// a lane.  One by one against by a threshold, in us for 64 heads, d = 64: 1 entry
// of 1025 3.1 / 7.7, of 4097 4.1 / 10.8, of 16385 5.7 / 19.0; 4 more than 4096
// 5.1 / 10.8; 16 more than 4096 10.3 / 10.8, than 16384 18.0 / 19.0, than 40000
// 32.7 / 34.3.
//
// Short rows are bound by the latency of these steps (4097 slots to 4096, 64
// heads, d = 64: 4.5 us); long ones by the selection, on an SM per head, and
// then by reading scattered rows (up to 16384 slots to 2048, 64 heads,
// d = 128: 24.7 us, of them 11 for the sources and 10.5 for the 40 MB copied,
// whose 4-byte and 8-byte parts cost a 32-byte sector each).
#include <cstddef>
#include <cstdint>
#include <type_traits>

#include "fa_kv4.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvMaxCluster = 8;
constexpr int kEvMaxSlice = kKv4EvictMaxCapacity / kEvMaxCluster;  // keys per CTA

constexpr int kEvFew = 16;
constexpr uint32_t kEvList = 256;  // open entries that are compared with one another
constexpr int kEvMaxWords = (kEvMaxSlice + 31) / 32;

// Shared memory: EvShared, then the slice's keys.
struct alignas(16) EvShared {  // the keys behind it are read 16 bytes at a time
    union {
        uint32_t hist[256 * 32];  // [bin][lane]
        struct {                  // after the selection, a word per 32 entries
            uint32_t kept[kEvMaxWords];   // bit i: entry stays
            uint32_t before[kEvMaxWords]; // holes (low half) and late entries (high half) of earlier words
        };
        struct {                  // few leaving entries
            uint2 least[kEvWarps];  // a warp's least key and the highest slot that has it
            int leaving[kEvFew], hole[kEvFew], late[kEvFew];
        };
    };
    uint32_t bins[256];        // this CTA's sums
    union {
        uint32_t total[256];     // the cluster's
        uint32_t list[kEvList];  // one CTA: the open entries
    };
    uint32_t warp_count[kEvWarps];
    uint32_t pick[3];          // bin, entries above it, entries in it
    uint32_t count[2];         // this CTA's, read by the cluster
    uint32_t listed;           // open entries in the list
};

static_assert(sizeof(EvShared) % 16 == 0 && offsetof(EvShared, bins) % 16 == 0 && offsetof(EvShared, total) % 16 == 0, "16-byte reads");
static_assert(sizeof(EvShared) + kEvMaxSlice * 4 <= 232448,
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
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
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

// One entry, by a warp.
template <int D>
__device__ __forceinline__ void copy_entry(const Kv4Cache& c, long long from, long long to) {
    constexpr int kChunks = D / 32;
    const int lane = threadIdx.x % 32;
    if (lane < 2 * kChunks) {
        uint8_t* codes = lane < kChunks ? c.codes[0] : c.codes[1];
        reinterpret_cast<uint4*>(codes)[to * kChunks + lane % kChunks] =
            reinterpret_cast<const uint4*>(codes)[from * kChunks + lane % kChunks];
    } else if (lane < 10) {
        uint8_t* scales = lane == 8 ? c.scales[0] : c.scales[1];
        if (lane >= 8) {
            if constexpr (D == 128)
                reinterpret_cast<uint2*>(scales)[to] = reinterpret_cast<const uint2*>(scales)[from];
            else
                reinterpret_cast<uint32_t*>(scales)[to] = reinterpret_cast<const uint32_t*>(scales)[from];
        }
    } else if (lane == 10) {
        if (c.pos != nullptr) c.pos[to] = c.pos[from];
    } else if (lane == 11) {
        if (c.weight != nullptr) c.weight[to] = c.weight[from];
    }
}

// The bits below and above the new length nn of the word that starts at slot.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

// Exclusive prefix of v over the block's threads; *sum gets the total.
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t (&warp_count)[kEvWarps], uint32_t* sum) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_count[warp] = x;
    __syncthreads();
    const uint32_t w = warp_count[lane];
    *sum = __reduce_add_sync(0xffffffffu, w);
    const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0u);
    __syncthreads();  // warp_count may be written again
    return before + x - v;
}

// kOne: a block per head (no cluster).
template <int D, bool kOne>
__global__ void __launch_bounds__(kEvThreads, 1) kv4_evict_kernel(const __grid_constant__ Kv4EvictParams p, int slice,
                                                                  int advance) {
    extern __shared__ __align__(16) uint8_t ev_smem[];
    EvShared& sh = *reinterpret_cast<EvShared*>(ev_smem);
    uint32_t* keys = reinterpret_cast<uint32_t*>(ev_smem + sizeof(EvShared));
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
    if (threadIdx.x == 0) sh.listed = 0u;
    if (kOne && threadIdx.x < kEvList / 4)  // no key is 0
        reinterpret_cast<uint4*>(sh.list)[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = threadIdx.x; i < 256 * 8; i += kEvThreads)
        reinterpret_cast<uint4*>(sh.hist)[i] = make_uint4(0u, 0u, 0u, 0u);
    // what comes from the arguments alone is formed ahead of the wait
    grid_release();
    const bool in_place = p.to.codes[0] == p.from.codes[0];
    const bool protect = p.sinks > 0 || p.recent > 0;
    const long long row0 = static_cast<long long>(head) * p.from.capacity;
    const long long to0 = static_cast<long long>(head) * p.to.capacity;
    const float* rank_by = p.rank_by + row0 + static_cast<long long>(rank) * slice;
    const int32_t* pos = p.from.pos + row0 + static_cast<long long>(rank) * slice;
    const bool wide =
        ((reinterpret_cast<uintptr_t>(rank_by) | (protect ? reinterpret_cast<uintptr_t>(pos) : 0u)) & 15u) == 0u;
    int32_t* src = p.src + static_cast<long long>(head) * p.keep;
    const int32_t* counts = p.from.counts + b;
    bool copied = false;
    grid_wait();
    const int n = min(max(counts[0], 0), p.from.capacity);
    const int seen = counts[p.from.B];
    const int nn = min(n, p.keep);  // the new length
    const int begin = static_cast<int>(min(static_cast<long long>(rank) * slice, static_cast<long long>(n)));
    const int size = min(slice, n - begin);  // this CTA's keys

    if (n > nn) {
        // positions are ints: one below the smallest protects nothing more
        const int newest = static_cast<int>(max(static_cast<long long>(seen) - p.recent, -2147483648ll));
        auto key_of = [&](float w, int at) -> uint32_t {
            return rank_key(w, protect && (at < p.sinks || at >= newest));
        };
        const bool few = kOne && n - nn <= kEvFew;  // no threshold
        // the keys, `loads` 16-byte reads a thread in flight; where a threshold is wanted, also the histogram of
        // their first 8 bits, while others are on their way
        auto load_keys = [&](auto loads, auto counted) {
            constexpr int kLoads = decltype(loads)::value;
            auto count_key = [&](uint32_t k) {
                if constexpr (decltype(counted)::value) atomicAdd(&sh.hist[(k >> 24) * 32 + lane], 1u);
            };
            if (!wide) {
                for (int i = threadIdx.x; i < size; i += kEvThreads) {
                    keys[i] = key_of(rank_by[i], protect ? pos[i] : 0);
                    count_key(keys[i]);
                }
                return;
            }
            for (int i0 = 4 * threadIdx.x; i0 < size; i0 += kLoads * 4 * kEvThreads) {  // a row has 128 n slots
                float4 w[kLoads];
                int4 at[kLoads];
#pragma unroll
                for (int u = 0; u < kLoads; ++u) {
                    const int i = i0 + u * 4 * kEvThreads;
                    w[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    at[u] = make_int4(0, 0, 0, 0);
                    if (i < size) {
                        w[u] = *reinterpret_cast<const float4*>(rank_by + i);
                        if (protect) at[u] = *reinterpret_cast<const int4*>(pos + i);
                    }
                }
#pragma unroll
                for (int u = 0; u < kLoads; ++u) {
                    const int i = i0 + u * 4 * kEvThreads;
                    if (i >= size) break;
                    const uint4 k = make_uint4(key_of(w[u].x, at[u].x), key_of(w[u].y, at[u].y),
                                               key_of(w[u].z, at[u].z), key_of(w[u].w, at[u].w));
                    *reinterpret_cast<uint4*>(keys + i) = k;
                    count_key(k.x);
                    if (i + 1 < size) count_key(k.y);
                    if (i + 2 < size) count_key(k.z);
                    if (i + 3 < size) count_key(k.w);
                }
            }
        };
        if (few) {
            load_keys(std::integral_constant<int, 1>{}, std::false_type{});
            __syncthreads();
            // the entries in the order they leave: ascending key, descending slot.  Every warp finds the first of its
            // own (slots 128 warp + 4096 i + 0 .. 127); then one warp, with a candidate per lane, takes the first of
            // all and looks for the next one among the entries it came from, while the others begin the list
            const int e = n - nn;
            const auto earlier = [](uint32_t k, int i, uint32_t key, int slot) {
                return k < key || (k == key && i > slot);
            };
            // the first entry of `share` behind (key, slot), over the warp
            const auto first_of = [&](int share, uint32_t& key, int& slot) {
                uint32_t first = 0xFFFFFFFFu;
                int where = -1;
                for (int i = 128 * share + 4 * lane; i < n; i += 4 * kEvThreads) {
                    const uint4 k4 = *reinterpret_cast<const uint4*>(keys + i);
                    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (i + j < n && earlier(key, slot, k[j], i + j) && earlier(k[j], i + j, first, where)) {
                            first = k[j];
                            where = i + j;
                        }
                }
                key = __reduce_min_sync(0xffffffffu, first);
                slot = __reduce_max_sync(0xffffffffu, first == key ? where : -1);
            };
            uint32_t key = 0u;  // no entry's
            int slot = -1;
            first_of(warp, key, slot);
            if (lane == 0) sh.least[warp] = make_uint2(key, static_cast<uint32_t>(slot));
            __syncthreads();
            if (warp > 0)
                for (int i = threadIdx.x - 32; i < nn; i += kEvThreads - 32) src[i] = i;
            if (warp == 0) {
                const uint2 w = sh.least[lane];
                key = w.x;
                slot = static_cast<int>(w.y);
                for (int r = 0;; ++r) {
                    uint32_t least = __reduce_min_sync(0xffffffffu, key);
                    int out = __reduce_max_sync(0xffffffffu, key == least ? slot : -1);
                    if (lane == 0) sh.leaving[r] = out;
                    if (r + 1 == e) break;
                    const int share = out / 128 % kEvWarps;
                    first_of(share, least, out);
                    if (lane == share) {
                        key = least;
                        slot = out;
                    }
                }
                __syncwarp();
                const int gone = lane < e ? sh.leaving[lane] : -1, end = nn + lane;
                int hole_rank = 0, late_rank = 0;
                bool leaves = false;
                for (int i = 0; i < e; ++i) {
                    const int o = sh.leaving[i];
                    hole_rank += o < gone ? 1 : 0;
                    late_rank += o >= nn && o < end ? 1 : 0;  // leaving ones among the slots before this one
                    leaves |= o == end;
                }
                if (gone >= 0 && gone < nn) sh.hole[hole_rank] = gone;
                if (lane < e && !leaves) sh.late[lane - late_rank] = end;
            }
            const int holes = __syncthreads_count(static_cast<int>(threadIdx.x) < e && sh.leaving[threadIdx.x] < nn);
            if (in_place && warp < holes) copy_entry<D>(p.from, row0 + sh.late[warp], row0 + sh.hole[warp]);
            __syncthreads();
            if (static_cast<int>(threadIdx.x) < holes) src[sh.hole[threadIdx.x]] = sh.late[threadIdx.x];
            copied = true;
        } else {
            __syncthreads();  // the histogram is clear
            load_keys(std::integral_constant<int, 4>{}, std::true_type{});
            __syncthreads();
            // 1. threshold: the entries whose upper bits equal `prefix` are still open
            uint32_t prefix = 0u;
            uint32_t want = static_cast<uint32_t>(nn), open = 0u;  // entries to take among the open ones; those of the bin
#pragma unroll 1
            for (int down = 24; down >= 0; down -= 8) {
                if (down < 24) {
#pragma unroll 4
                    for (int i = 4 * threadIdx.x; i < size; i += 4 * kEvThreads) {
                        const uint4 k4 = *reinterpret_cast<const uint4*>(keys + i);
                        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (i + j < size && (k[j] >> (down + 8)) == prefix)
                                atomicAdd(&sh.hist[((k[j] >> down) & 255u) * 32 + lane], 1u);
                    }
                    __syncthreads();
                }
                // four threads per bin, each eight of its counters, in an order that keeps the banks apart
                const int bin = threadIdx.x / 4;
                uint32_t sum = 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += sh.hist[bin * 32 + ((threadIdx.x % 4 * 8 + i + bin) & 31)];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                if (threadIdx.x % 4 == 0) sh.bins[bin] = sum;
                sync_all();
                if constexpr (!kOne) {
                    if (threadIdx.x < 256) {
                        uint32_t t = 0u;
                        for (uint32_t r = 0; r < cs; ++r) t += ld_cluster_u32(smem_u32(&sh.bins[threadIdx.x]), r);
                        sh.total[threadIdx.x] = t;
                    }
                    cluster_sync_all();  // and every CTA has read the others' sums
                }
                if (warp == 0) {
                    // from the top bin down: lane l holds bins 255 - 8 l .. 248 - 8 l
                    const uint4* t4 = reinterpret_cast<const uint4*>(kOne ? sh.bins : sh.total) + (31 - lane) * 2;
                    const uint4 lo = t4[0], hi = t4[1];
                    const uint32_t c[8] = {hi.w, hi.z, hi.y, hi.x, lo.w, lo.z, lo.y, lo.x};
                    const uint32_t all = ((c[0] + c[1]) + (c[2] + c[3])) + ((c[4] + c[5]) + (c[6] + c[7]));
                    uint32_t above = all;
#pragma unroll
                    for (int o = 1; o < 32; o *= 2) {
                        const uint32_t y = __shfl_up_sync(0xffffffffu, above, o);
                        if (lane >= o) above += y;
                    }
                    above -= all;
                    if (above < want && want <= above + all) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (above < want && want <= above + c[i]) {
                                sh.pick[0] = static_cast<uint32_t>(255 - 8 * lane - i);
                                sh.pick[1] = above;
                                sh.pick[2] = c[i];
                            }
                            above += c[i];
                        }
                    }
                }
                __syncthreads();
                prefix = (prefix << 8) | sh.pick[0];
                want -= sh.pick[1];
                open = sh.pick[2];
                if (kOne && down > 0 && open <= kEvList) {
                    // few entries are open: each against all of them.  Those with fewer than `want` greater ones,
                    // and at least that many greater or equal, equal the threshold
#pragma unroll 4
                    for (int i = 4 * threadIdx.x; i < size; i += 4 * kEvThreads) {
                        const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
                        uint32_t match = ((k.x >> down) == prefix ? 1u : 0u) | ((k.y >> down) == prefix ? 2u : 0u) |
                                         ((k.z >> down) == prefix ? 4u : 0u) | ((k.w >> down) == prefix ? 8u : 0u);
                        for (match &= low_bits(size - i); match != 0u; match &= match - 1u)  // few have any
                            sh.list[atomicAdd(&sh.listed, 1u)] = keys[i + __ffs(static_cast<int>(match)) - 1];
                    }
                    __syncthreads();
                    // four threads per entry
                    const uint32_t mine = threadIdx.x / 4;
                    const uint32_t k = mine < open ? sh.list[mine] : 0u;
                    uint32_t more = 0u, equal = 0u;
                    for (uint32_t i = 4 * (threadIdx.x % 4); i < open; i += 16) {  // zeros behind the last
                        const uint4 o = *reinterpret_cast<const uint4*>(&sh.list[i]);
                        more += (o.x > k ? 1u : 0u) + (o.y > k ? 1u : 0u) + (o.z > k ? 1u : 0u) + (o.w > k ? 1u : 0u);
                        equal += (o.x == k ? 1u : 0u) + (o.y == k ? 1u : 0u) + (o.z == k ? 1u : 0u) + (o.w == k ? 1u : 0u);
                    }
#pragma unroll
                    for (int o = 1; o < 4; o *= 2) {
                        more += __shfl_xor_sync(0xffffffffu, more, o);
                        equal += __shfl_xor_sync(0xffffffffu, equal, o);
                    }
                    if (mine < open && more < want && want <= more + equal) {  // all that equal the threshold write the same
                        sh.pick[0] = k;
                        sh.pick[1] = more;
                        sh.pick[2] = equal;
                    }
                    __syncthreads();
                    prefix = sh.pick[0];
                    want -= sh.pick[1];
                    open = sh.pick[2];
                    break;
                }
                if (down > 0) {  // the histogram is read
                    for (int i = threadIdx.x; i < 256 * 8; i += kEvThreads)
                        reinterpret_cast<uint4*>(sh.hist)[i] = make_uint4(0u, 0u, 0u, 0u);
                    __syncthreads();
                }
            }
            // 2. a bit per entry: a word of 32 entries per thread (two in the longest slices), its eight
            // 16-byte reads begun at another one by each lane, to keep the banks apart
            const uint32_t T = prefix;  // `want` of the `open` entries equal to T are kept
            const int words = (size + 31) / 32;
            const int per = words > kEvThreads ? 2 : 1;
            const int x0 = per * static_cast<int>(threadIdx.x);
            uint32_t stay[2] = {0u, 0u}, ties[2] = {0u, 0u};
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const int x = x0 + w;
                if (w >= per || x >= words) break;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = (j + lane) & 7;
                    const uint4 k = *reinterpret_cast<const uint4*>(keys + 32 * x + 4 * c);
                    stay[w] |= ((k.x > T ? 1u : 0u) | (k.y > T ? 2u : 0u) | (k.z > T ? 4u : 0u) | (k.w > T ? 8u : 0u)) << (4 * c);
                    ties[w] |= ((k.x == T ? 1u : 0u) | (k.y == T ? 2u : 0u) | (k.z == T ? 4u : 0u) | (k.w == T ? 8u : 0u)) << (4 * c);
                }
                const uint32_t valid = low_bits(size - 32 * x);
                stay[w] &= valid;
                ties[w] &= valid;
            }
            if (want < open) {  // of the entries equal to T the first `want`, over the cluster
                uint32_t all;
                uint32_t before = block_prefix(__popc(ties[0]) + __popc(ties[1]), sh.warp_count, &all);
                if constexpr (!kOne) {
                    if (threadIdx.x == 0) sh.count[0] = all;
                    cluster_sync_all();
                    for (uint32_t r = 0; r < rank; ++r) before += ld_cluster_u32(smem_u32(&sh.count[0]), r);
                    cluster_sync_all();  // count is written again below
                }
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    uint32_t bits = ties[w];
                    const uint32_t n_bits = __popc(bits);
                    const int take = static_cast<int>(want) - static_cast<int>(before);
                    if (take < static_cast<int>(n_bits)) {
                        uint32_t some = 0u;
                        for (int j = 0; j < take; ++j) {  // the lowest `take` bits
                            some |= bits & (0u - bits);
                            bits &= bits - 1u;
                        }
                        bits = some;
                    }
                    stay[w] |= bits;
                    before += n_bits;
                }
            } else {
                stay[0] |= ties[0];
                stay[1] |= ties[1];
            }
            // 3. ranks of holes and late entries: prefixes by word
            uint32_t before[2], both[2] = {0u, 0u};
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const int x = x0 + w;
                if (w >= per || x >= words) break;
                const uint32_t below = low_bits(nn - begin - 32 * x);
                both[w] = static_cast<uint32_t>(__popc(low_bits(size - 32 * x) & below & ~stay[w])) |
                          static_cast<uint32_t>(__popc(stay[w] & ~below)) << 16;
            }
            uint32_t all;
            before[0] = block_prefix(both[0] + both[1], sh.warp_count, &all);
            before[1] = before[0] + both[0];
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                if (w >= per || x0 + w >= words) break;
                sh.kept[x0 + w] = stay[w];
                sh.before[x0 + w] = before[w];
            }
            uint32_t h_first = 0u, l_first = 0u;  // of earlier CTAs
            if constexpr (kOne) {
                __syncthreads();
            } else {
                if (threadIdx.x == 0) {
                    sh.count[0] = all & 0xFFFFu;
                    sh.count[1] = all >> 16;
                }
                cluster_sync_all();  // also every key was read: the slices now hold the list of holes
                for (uint32_t r = 0; r < rank; ++r) {
                    h_first += ld_cluster_u32(smem_u32(&sh.count[0]), r);
                    l_first += ld_cluster_u32(smem_u32(&sh.count[1]), r);
                }
            }
            const int low_words = min(words, max(0, (nn - begin + 31) / 32));  // words with slots below nn
#pragma unroll 2
            for (int x = warp; x < low_words; x += kEvWarps) {
                const int i = begin + x * 32 + lane;
                const uint32_t kept = sh.kept[x];
                const uint32_t holes = low_bits(size - x * 32) & low_bits(nn - begin - x * 32) & ~kept;
                if ((holes >> lane) & 1u) {
                    const uint32_t r = h_first + (sh.before[x] & 0xFFFFu) + __popc(holes & ((1u << lane) - 1u));
                    if constexpr (kOne)
                        keys[r] = static_cast<uint32_t>(i);
                    else
                        st_cluster_u32(keys_addr + 4u * (r % static_cast<uint32_t>(slice)),
                                       r / static_cast<uint32_t>(slice), static_cast<uint32_t>(i));
                } else if (i < nn && ((kept >> lane) & 1u)) {
                    src[i] = i;
                }
            }
            sync_all();
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const int x = x0 + w;
                if (w >= per || x >= words) break;
                uint32_t r = l_first + (before[w] >> 16);
                for (uint32_t late = stay[w] & ~low_bits(nn - begin - 32 * x); late != 0u; late &= late - 1u, ++r) {
                    uint32_t hole;
                    if constexpr (kOne)
                        hole = keys[r];
                    else
                        hole = ld_cluster_u32(keys_addr + 4u * (r % static_cast<uint32_t>(slice)),
                                              r / static_cast<uint32_t>(slice));
                    src[hole] = begin + 32 * x + __ffs(static_cast<int>(late)) - 1;
                }
            }
        }
    } else {
        for (int i = static_cast<int>(rank) * kEvThreads + threadIdx.x; i < nn; i += static_cast<int>(cs) * kEvThreads)
            src[i] = i;
    }
    for (long long i = nn + static_cast<long long>(rank) * kEvThreads + threadIdx.x; i < p.keep;
         i += static_cast<long long>(cs) * kEvThreads)
        src[i] = -1;
    // 4. copies in place, 32 slots per warp and step (src was written by the whole cluster); those into another
    // cache move every entry and have a kernel of their own, on every SM
    if (in_place && !copied) {
        sync_all();
        const int step = static_cast<int>(cs) * kEvWarps * 32;
        for (int j0 = (static_cast<int>(rank) * kEvWarps + warp) * 32; j0 < nn; j0 += step) {
            const int j = j0 + lane;
            int from = j < nn ? __ldcg(src + j) : -1;
            if (from == j) from = -1;
            if (__any_sync(0xffffffffu, from >= 0)) copy_entries<D>(p.from, p.to, row0, from, to0 + j0);
        }
    } else if (!kOne) {
        sync_all();  // no CTA leaves while its list is read
    }
    if (advance && head % p.from.H_kv == 0 && rank == 0 && threadIdx.x == 0) {
        p.counts_out[b] = nn;
        p.counts_out[p.from.B + b] = seen;
    }
}

// The entries named by src into another cache, 32 a warp; grid: heads x
// blocks of kKv4CopyRows slots.
constexpr int kCopyThreads = kKv4CopyRows;
template <int D>
__global__ void __launch_bounds__(kCopyThreads) kv4_evict_copy_kernel(const __grid_constant__ Kv4EvictParams p, int blocks) {
    const int head = static_cast<int>(blockIdx.x) / blocks;
    const int j0 = (static_cast<int>(blockIdx.x) % blocks) * kKv4CopyRows + static_cast<int>(threadIdx.x) / 32 * 32;
    grid_release();
    grid_wait();
    const int most = kv4_kept_at_most(p.keep, p.from.capacity);
    if (j0 >= most) return;
    const int j = j0 + static_cast<int>(threadIdx.x) % 32;
    const int from = j < most ? p.src[static_cast<long long>(head) * p.keep + j] : -1;
    if (__any_sync(0xffffffffu, from >= 0))
        copy_entries<D>(p.from, p.to, static_cast<long long>(head) * p.from.capacity, from,
                        static_cast<long long>(head) * p.to.capacity + j0);
}

// counts_out where it is the counts that the clusters of a sequence read.
__global__ void kv4_evict_counts_kernel(const Kv4EvictParams p) {
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    grid_release();
    grid_wait();
    if (b < p.from.B) p.counts_out[b] = min(min(max(p.from.counts[b], 0), p.from.capacity), p.keep);
}

template <int D>
cudaError_t launch_evict(const Kv4EvictParams& p, cudaStream_t stream) {
    const int heads = p.from.B * p.from.H_kv;
    // one CTA per head unless its keys need more: 64 heads of up to 16384 slots to 2048, d = 128, take 24.7 us so and
    // 32.3 by a cluster of two, which has no list of open entries and makes all four passes, two cluster barriers each
    int cs = 1;
    while (cs < kEvMaxCluster && (p.from.capacity + cs - 1) / cs > kEvMaxSlice) cs *= 2;
    const int slice = ((p.from.capacity + cs - 1) / cs + 31) / 32 * 32;
    const size_t smem = sizeof(EvShared) + static_cast<size_t>(slice) * 4;
    auto kern = cs == 1 ? kv4_evict_kernel<D, true> : kv4_evict_kernel<D, false>;
    // the limit is the kernel's, not the call's: the same for all of them, whatever other threads evict meanwhile
    static SmemAllowed allowed[2];
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), static_cast<int>(sizeof(EvShared)) + kEvMaxSlice * 4,
                               allowed[cs == 1 ? 0 : 1]);
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
    if (p.to.codes[0] != p.from.codes[0]) {
        const int blocks = kv4_copy_blocks(p.keep, p.from.capacity);
        e = launch_dependent(kv4_evict_copy_kernel<D>, dim3(static_cast<unsigned>(heads) * static_cast<unsigned>(blocks)),
                             kCopyThreads, 0, stream, p, blocks);
        if (e != cudaSuccess) return e;
    }
    if (!advance) return launch_dependent(kv4_evict_counts_kernel, dim3((p.from.B + 127) / 128), 128, 0, stream, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_evict(const Kv4EvictParams& p, cudaStream_t stream) {
    return p.from.d == 128 ? launch_evict<128>(p, stream) : launch_evict<64>(p, stream);
}

}  // namespace fa
