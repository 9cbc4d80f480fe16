// Rows into and out of the 4-bit key/value cache (include/fa.h, "Format").
//
// Both kernels give one thread one block of 16 channels: 32 bytes of 16-bit
// values on one side, 8 bytes of codes and a scale byte on the other, all
// contiguous over a warp, so both are bound by memory traffic.
// 2 x 8192 rows of 8 heads, d = 128, stored and read back: 33.6 us for 173 MB,
// 5.1 TB/s; two 16-byte accesses a thread instead of one of 32 took 35.8.  One
// row of 8 x 8 heads: 2.2 us a kernel, the latency of a launch and of three
// reads one behind the other.
//
// Quantising is exact in fp32.  With amax and x of at most 11 significant
// bits and e4m3 midpoints of 5, amax / 6 is either a midpoint, which the
// division returns exactly, or at least 2^-11 away from it relatively, so
// the rounded quotient falls on the side the real one does.  The codes'
// quotients x / s (s of 4 bits, midpoints of 3) have the same gap; x * (1/s)
// is within 2^-22 of the quotient, and snapping it to multiples of 2^-17 (by
// adding and subtracting 96, whose ulp that is) returns a midpoint exactly
// when the quotient is one, well inside the gap of 2^-11 * 0.25.
#include <cstdint>

#include "fa_kv4.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

// e2m1 codes of two values, `lo` in bits 0-3; nearest even, saturating.
__device__ __forceinline__ uint32_t pack_e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}
// e4m3 byte of a value; nearest even, saturating.
__device__ __forceinline__ uint32_t to_e4m3(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(x));
    return r & 0xFFu;
}
// The f16x2 pair of a byte's two e2m1 codes.
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t byte) {
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(r) : "r"(byte));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t byte) {  // both halves
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(byte * 0x0101u)));
    return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 16 values of 16 bits, by one access where the rows lie on 32-byte boundaries
// (two of 16 bytes a thread leave every second one of a warp's sectors to the
// other).
__device__ __forceinline__ void load_values(const uint4* x, bool wide, uint32_t (&w)[8]) {
    if (wide) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(x));
    } else {
        const uint4 a = x[0], c = x[1];
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = c.x, w[5] = c.y, w[6] = c.z, w[7] = c.w;
    }
}
__device__ __forceinline__ void store_values(uint4* x, bool wide, const uint32_t (&w)[8]) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(x), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        x[0] = make_uint4(w[0], w[1], w[2], w[3]);
        x[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
__device__ __forceinline__ bool wide_rows(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 31u) == 0u; }

constexpr int kAppendThreads = 256;
constexpr int kAppendOneCta = 1024;  // blocks of 16 channels that a single CTA stores

// counts_out = counts advanced by n, one thread per sequence.
__device__ __forceinline__ void advance_counts(const Kv4AppendParams& p, int b) {
    const long long len = static_cast<long long>(max(p.c.counts[b], 0)) + p.n;
    const int32_t seen = p.c.counts[p.c.B + b];
    p.counts_out[b] = static_cast<int32_t>(min(len, static_cast<long long>(p.c.capacity)));
    p.counts_out[p.c.B + b] = static_cast<int32_t>(seen + p.n);
}

// Block i of 16 channels, in the order [head][key or value][row][block]; the
// host keeps their number below 2^31, so 32-bit arithmetic finds it.
template <int D, bool F16>
__device__ __forceinline__ void append_block(const Kv4AppendParams& p, uint32_t i) {
    constexpr uint32_t kBlocks = D / 16;
    const uint32_t n = static_cast<uint32_t>(p.n);
    const uint32_t blk = i % kBlocks, t = i / kBlocks;
    const uint32_t rest = t / n, row = t - rest * n;
    const bool value = (rest & 1) != 0;
    const uint32_t head = rest >> 1;  // b * H_kv + key/value head
    const uint32_t b = head / static_cast<uint32_t>(p.c.H_kv);
    const long long slot = static_cast<long long>(max(p.c.counts[b], 0)) + row;
    if (slot >= p.c.capacity) {
        if (row == n - 1 && blk == 0 && !value) atomicOr(&p.status->word, kDevErrCapacity);
        return;
    }
    const uint4* x4 = reinterpret_cast<const uint4*>(value ? p.x[1] : p.x[0]) +
                      ((static_cast<long long>(head) * n + row) * kBlocks + blk) * 2;
    uint32_t w[8];
    load_values(x4, wide_rows(x4), w);
    // magnitudes of bf16 and fp16 order as integers (NaN above infinity)
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
    m = max(m & 0xFFFFu, m >> 16);
    const bool finite = m < (F16 ? 0x7C00u : 0x7F80u);
    const uint32_t sbyte = finite ? to_e4m3(__fdiv_rn(widen_lo16<F16>(m), 6.0f)) : 0x7Fu;
    uint32_t lo = 0u, hi = 0u;
    if (finite && sbyte != 0u) {
        const float inv = 1.0f / widen_lo16<true>(e4m3_to_f16x2(sbyte));
        uint32_t byte[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x0 = __fsub_rn(__fadd_rn(__fmul_rn(widen_lo16<F16>(w[j]), inv), 96.0f), 96.0f);
            const float x1 = __fsub_rn(__fadd_rn(__fmul_rn(widen_lo16<F16>(w[j] >> 16), inv), 96.0f), 96.0f);
            byte[j] = pack_e2m1x2(x0, x1);
        }
        lo = byte[0] | byte[1] << 8 | byte[2] << 16 | byte[3] << 24;
        hi = byte[4] | byte[5] << 8 | byte[6] << 16 | byte[7] << 24;
    }
    const long long at = static_cast<long long>(head) * p.c.capacity + slot;
    reinterpret_cast<uint2*>(value ? p.c.codes[1] : p.c.codes[0])[at * kBlocks + blk] = make_uint2(lo, hi);
    (value ? p.c.scales[1] : p.c.scales[0])[at * kBlocks + blk] = static_cast<uint8_t>(sbyte);
    if (blk == 0 && !value) {
        if (p.c.pos != nullptr) p.c.pos[at] = static_cast<int32_t>(p.c.counts[p.c.B + b] + row);
        if (p.c.weight != nullptr) p.c.weight[at] = 0.0f;
    }
}

// advance: this launch also writes counts_out (a single CTA, or counts_out
// is not the counts that other CTAs still read).
template <int D, bool F16>
__global__ void kv4_append_kernel(const Kv4AppendParams p, uint32_t total, int advance) {
    const uint32_t i = blockIdx.x * blockDim.x + threadIdx.x;
    grid_release();
    grid_wait();
    if (i < total) append_block<D, F16>(p, i);
    if (advance && blockIdx.x == 0) {
        __syncthreads();
        for (int b = threadIdx.x; b < p.c.B; b += blockDim.x) advance_counts(p, b);
    }
}

__global__ void kv4_advance_kernel(const Kv4AppendParams p) {
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    grid_release();
    grid_wait();
    if (b < p.c.B) advance_counts(p, b);
}

template <int D, bool F16>
__global__ void kv4_read_kernel(const Kv4ReadParams p, uint32_t total) {
    constexpr uint32_t kBlocks = D / 16;
    const uint32_t i = blockIdx.x * blockDim.x + threadIdx.x;
    grid_release();
    grid_wait();
    if (i >= total) return;
    const bool value = blockIdx.y != 0;
    uint4* x = static_cast<uint4*>(value ? p.x[1] : p.x[0]);
    if (x == nullptr) return;
    const uint32_t count = static_cast<uint32_t>(p.count);
    const uint32_t blk = i % kBlocks, t = i / kBlocks;
    const uint32_t head = t / count, row = t - head * count;
    const uint32_t b = head / static_cast<uint32_t>(p.c.H_kv);
    const long long slot = static_cast<long long>(p.first != nullptr ? p.first[b] : 0) + row;
    uint32_t out[8] = {};
    if (slot >= 0 && slot < p.c.capacity) {
        const long long at = (static_cast<long long>(head) * p.c.capacity + slot) * kBlocks + blk;
        const uint2 codes = reinterpret_cast<const uint2*>(value ? p.c.codes[1] : p.c.codes[0])[at];
        const uint32_t s = e4m3_to_f16x2((value ? p.c.scales[1] : p.c.scales[0])[at]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t h = mul_f16x2(e2m1x2_to_f16x2(((j < 4 ? codes.x : codes.y) >> (8 * (j & 3))) & 0xFFu), s);
            out[j] = F16 ? h : pack_bf16x2(widen_lo16<true>(h), widen_lo16<true>(h >> 16));
        }
    }
    x += static_cast<long long>(i) * 2;
    store_values(x, wide_rows(x), out);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendParams& p, cudaStream_t stream) {
    const long long total = 2ll * p.c.B * p.c.H_kv * p.n * (p.c.d / 16);
    const bool in_place = p.counts_out == p.c.counts;
    const int threads = total <= kAppendOneCta ? static_cast<int>((total + 31) / 32 * 32) : kAppendThreads;
    const long long grid = (total + threads - 1) / threads;
    const int advance = (!in_place || grid == 1) ? 1 : 0;
    auto kern = p.c.d == 128 ? (p.f16 ? kv4_append_kernel<128, true> : kv4_append_kernel<128, false>)
                             : (p.f16 ? kv4_append_kernel<64, true> : kv4_append_kernel<64, false>);
    const cudaError_t e = launch_dependent(kern, dim3(static_cast<unsigned>(grid)), threads, 0, stream, p,
                                           static_cast<uint32_t>(total), advance);
    if (e != cudaSuccess || advance) return e;
    return launch_dependent(kv4_advance_kernel, dim3((p.c.B + 127) / 128), 128, 0, stream, p);
}

cudaError_t launch_kv4_read(const Kv4ReadParams& p, cudaStream_t stream) {
    const long long total = static_cast<long long>(p.c.B) * p.c.H_kv * p.count * (p.c.d / 16);
    const dim3 grid(static_cast<unsigned>((total + 255) / 256), 2);
    auto kern = p.c.d == 128 ? (p.f16 ? kv4_read_kernel<128, true> : kv4_read_kernel<128, false>)
                             : (p.f16 ? kv4_read_kernel<64, true> : kv4_read_kernel<64, false>);
    return launch_dependent(kern, grid, 256, 0, stream, p, static_cast<uint32_t>(total));
}

}  // namespace fa
