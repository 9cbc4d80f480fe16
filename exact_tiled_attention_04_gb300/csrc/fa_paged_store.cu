// Rows into the paged key/value cache, with the rotation by their positions
// applied on the way (include/fa.h, fa_paged_append).
//
// Mathematics.  A pair of channels (x, y) of a query or key row at position p
// becomes (x cos - y sin, x sin + y cos) with the cosine and sine of the pair's
// angle at p, read from a table the caller keeps (an angle formed here in 32
// bits would be off by 2^-24 p radians).  Products and sums in 32 bits, one
// rounding to the row's type.
//
// What bounds it: memory.  Every row is read once and written once.  A lane
// takes two 16-byte pieces of a row that hold the two sides of eight pairs, so d / 16
// lanes have a row, a warp 4 rows (d = 128) or 8; and as all heads of a token
// share its angles, a warp keeps to one token and reads the table once for all
// of them.  Two rows' loads are in flight per lane (8192 tokens: 35.0 us, with four
// 37.1, with six 38.2), the first two ahead of the lookups.  A prompt's tokens get a
// warp each; few tokens are spread over as many warps as their rows allow
// (`parts`), so that a decode step is one load and one store deep.
// Measured (H = 32 over 8, d = 128, bf16): 8192 tokens of three prompts 35 us, 5.9
// TB/s; one token of each of 32 sequences 3.1 us.
#include <cstdint>

#include "fa_paged.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kAppendWarps = 8;  // of a block, unless it has a whole sequence
constexpr int kMostWarps = 16;
constexpr int kBatch = 2;        // rows per lane whose loads are in flight

// Sequence of row t by the offsets cu[0 .. B], or -1.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, long long t) {
    if (t < cu[0] || t >= cu[B]) return -1;
    int lo = 0, hi = B;  // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int held(const PagedCache& c, int b) { return min(max(c.lengths[b], 0), c.capacity); }

__device__ __forceinline__ int advanced(const PagedAppendParams& p, int b) {
    const long long n = p.cu != nullptr ? static_cast<long long>(p.cu[b + 1]) - p.cu[b] : p.n;
    return static_cast<int>(min(held(p.c, b) + max(n, 0ll), static_cast<long long>(p.c.capacity)));
}

template <bool F16, bool kInterleaved>
__global__ void __launch_bounds__(kMostWarps * 32) paged_append_kernel(const PagedAppendParams p) {
    grid_wait();
    grid_release();
    const int warp = static_cast<int>(threadIdx.x) / 32, lane = static_cast<int>(threadIdx.x) % 32;
    const int warps = static_cast<int>(blockDim.x) / 32;
    const long long w = static_cast<long long>(blockIdx.x) * warps + warp;
    const long long t = w / p.parts;
    const int part = static_cast<int>(w % p.parts);
    const int H = p.q.data != nullptr ? p.H : 0, H_kv = p.c.H_kv;
    const int rows = H + 2 * H_kv;  // the token's query heads, key heads, value heads
    const int per_row = p.c.d / 16, u = lane % per_row;
    const int rows_per_warp = 32 / per_row, step = p.parts * rows_per_warp;
    const int pairs = p.rot / 16;
    // this lane's two pieces of a row: the sides of eight pairs, or of rows that are not turned any two
    const bool turn = u < pairs;
    const int e0 = !turn ? p.rot + 16 * (u - pairs) : kInterleaved ? 16 * u : 8 * u;
    const int e1 = !turn || kInterleaved ? e0 + 8 : e0 + p.rot / 2;
    uint4 x[kBatch], y[kBatch];
    auto load = [&](int r0) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int r = r0 + k * step;
            if (r >= rows) break;
            const bool value = r >= H + H_kv;
            const RowsView& from = r < H ? p.q : value ? p.v : p.k;
            const uint16_t* src = from.data + t * from.row + (r < H ? r : value ? r - H - H_kv : r - H) * from.head;
            x[k] = *reinterpret_cast<const uint4*>(src + (value ? 16 * u : e0));
            y[k] = *reinterpret_cast<const uint4*>(src + (value ? 16 * u + 8 : e1));
        }
    };
    // the first rows are on their way while sequence, slot, page and angles are looked up, one behind the other
    const int first = part * rows_per_warp + lane / per_row;
    if (t < p.T) load(first);
    int b = -1;
    if (t < p.T) b = p.cu != nullptr ? sequence_of(p.cu, p.c.B, t) : static_cast<int>(t / p.n);
    if (b >= 0) {
        const long long slot = held(p.c, b) + (p.cu != nullptr ? t - p.cu[b] : t % p.n);  // (64 bits: whatever cu holds)
        // where the row goes in the cache
        long long at = -1;  // its element in a head's pages
        unsigned int error = 0;
        if (slot < p.c.capacity) {
            const int page = p.c.table[static_cast<size_t>(b) * p.c.max_pages + slot / p.c.page];
            if (page >= 0 && page < p.c.num_pages)
                at = (static_cast<long long>(page) * p.c.H_kv * p.c.page + slot % p.c.page) * p.c.d;
            else
                error = kDevErrRange;
        } else {
            error = kDevErrCapacity;
        }
        float cs[8], sn[8];
        if (turn) {
            long long pos = p.positions != nullptr ? p.positions[t] : p.first_position + slot;
            if (pos < 0 || pos >= p.table_rows) {
                error |= kDevErrRange;
                pos = pos < 0 ? 0 : p.table_rows - 1;
            }
            const float4* c4 = reinterpret_cast<const float4*>(p.table + pos * p.rot + 8 * u);
            const float4* s4 = reinterpret_cast<const float4*>(p.table + pos * p.rot + p.rot / 2 + 8 * u);
            const float4 a = c4[0], c = c4[1], d = s4[0], e = s4[1];
            cs[0] = a.x, cs[1] = a.y, cs[2] = a.z, cs[3] = a.w, cs[4] = c.x, cs[5] = c.y, cs[6] = c.z, cs[7] = c.w;
            sn[0] = d.x, sn[1] = d.y, sn[2] = d.z, sn[3] = d.w, sn[4] = e.x, sn[5] = e.y, sn[6] = e.z, sn[7] = e.w;
        }
        if (error != 0 && part == 0 && lane == 0) atomicOr(&p.status->word, error);
        const size_t head_size = static_cast<size_t>(p.c.page) * p.c.d;
        for (int r0 = first; r0 < rows; r0 += kBatch * step) {
            if (r0 != first) load(r0);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int r = r0 + k * step;
                if (r >= rows) break;
                const bool value = r >= H + H_kv;
                if (turn && !value) {
                    uint32_t a[4] = {x[k].x, x[k].y, x[k].z, x[k].w}, c[4] = {y[k].x, y[k].y, y[k].z, y[k].w};
                    if (kInterleaved) {  // pair j is the two halves of word j
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            uint32_t& word = j < 4 ? a[j] : c[j - 4];
                            const float lo = widen_lo16<F16>(word), hi = widen_lo16<F16>(word >> 16);
                            word = pack_16x2<F16>(lo * cs[j] - hi * sn[j], lo * sn[j] + hi * cs[j]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float x0 = widen_lo16<F16>(a[j]), x1 = widen_lo16<F16>(a[j] >> 16);
                            const float y0 = widen_lo16<F16>(c[j]), y1 = widen_lo16<F16>(c[j] >> 16);
                            a[j] = pack_16x2<F16>(x0 * cs[2 * j] - y0 * sn[2 * j], x1 * cs[2 * j + 1] - y1 * sn[2 * j + 1]);
                            c[j] = pack_16x2<F16>(x0 * sn[2 * j] + y0 * cs[2 * j], x1 * sn[2 * j + 1] + y1 * cs[2 * j + 1]);
                        }
                    }
                    x[k] = make_uint4(a[0], a[1], a[2], a[3]);
                    y[k] = make_uint4(c[0], c[1], c[2], c[3]);
                }
                const int f0 = value ? 16 * u : e0, f1 = value ? 16 * u + 8 : e1;
                if (r < H) {
                    uint16_t* dst = p.q_out.data + t * p.q_out.row + r * p.q_out.head;
                    *reinterpret_cast<uint4*>(dst + f0) = x[k];
                    *reinterpret_cast<uint4*>(dst + f1) = y[k];
                    continue;
                }
                const int head = value ? r - H - H_kv : r - H;
                if (!value && p.k_out.data != nullptr) {
                    uint16_t* dst = p.k_out.data + t * p.k_out.row + head * p.k_out.head;
                    *reinterpret_cast<uint4*>(dst + f0) = x[k];
                    *reinterpret_cast<uint4*>(dst + f1) = y[k];
                }
                if (at >= 0) {
                    uint16_t* dst = (value ? p.c.pages[1] : p.c.pages[0]) + head * head_size + at;
                    *reinterpret_cast<uint4*>(dst + f0) = x[k];
                    *reinterpret_cast<uint4*>(dst + f1) = y[k];
                }
            }
        }
    }
    if (p.whole) {
        __syncthreads();  // every warp has read the length
        if (threadIdx.x == 0) p.lengths_out[blockIdx.x] = advanced(p, static_cast<int>(blockIdx.x));
    } else if (p.lengths_out != p.c.lengths) {
        for (long long s = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; s < p.c.B;
             s += static_cast<long long>(gridDim.x) * blockDim.x)
            p.lengths_out[s] = advanced(p, static_cast<int>(s));
    }
}

// Lengths advanced in place, behind the kernel that read them.
__global__ void __launch_bounds__(256) paged_advance_kernel(const PagedAppendParams p) {
    grid_wait();
    grid_release();
    const int b = static_cast<int>(blockIdx.x) * 256 + static_cast<int>(threadIdx.x);
    if (b < p.c.B) p.c.lengths[b] = advanced(p, b);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams& params, int sms, bool f16, bool interleaved, cudaStream_t stream) {
    PagedAppendParams p = params;
    const int per_warp = 32 / (p.c.d / 16), rows = (p.q.data != nullptr ? p.H : 0) + 2 * p.c.H_kv;
    const int most = (rows + per_warp - 1) / per_warp;  // warps a token can use
    // As many warps as fill the device about once share the tokens, 64 an SM (one token of each of 32
    // sequences, H = 32/8, d = 128: 3.1 us, by one warp a token 5.5).
    long long parts = sms * 64ll / (p.T > 0 ? p.T : 1);
    parts = parts < 1 ? 1 : parts > most ? most : parts;
    if (parts > kMostWarps) parts = kMostWarps;
    p.parts = static_cast<int>(parts);
    int warps = kAppendWarps;
    // A block per sequence, where that is a block's worth of warps: it can advance the length itself (on the device the
    // second kernel hides behind the first, but its launch takes the host 1.4 us).
    p.whole = p.cu == nullptr && p.n > 0 && static_cast<long long>(p.n) * p.parts <= kMostWarps;
    if (p.whole) warps = p.n * p.parts;
    const long long blocks = p.whole ? p.c.B : p.T > 0 ? (p.T * p.parts + warps - 1) / warps : 1;
    auto kern = f16 ? (interleaved ? paged_append_kernel<true, true> : paged_append_kernel<true, false>)
                    : (interleaved ? paged_append_kernel<false, true> : paged_append_kernel<false, false>);
    cudaError_t e = launch_dependent(kern, dim3(static_cast<unsigned>(blocks)), warps * 32, 0, stream, p);
    if (e != cudaSuccess || p.whole || p.lengths_out != p.c.lengths) return e;
    return launch_dependent(paged_advance_kernel, dim3(static_cast<unsigned>((p.c.B + 255) / 256)), 256, 0, stream, p);
}

}  // namespace fa
