// Rows into and out of the 4-bit key/value cache (include/fa.h, "Format").
//
// Both kernels give one thread 32 channels, two blocks of 16: 64 bytes of
// 16-bit values on one side, 16 bytes of codes and two scale bytes on the
// other, contiguous over a warp.  Bound by memory traffic once the
// instructions are few: 2 x 8192 rows of 8 heads, d = 128, stored and read
// back take 27.7 us for 173 MB, 6.25 TB/s; a block of 16 a thread, divisions
// and a conversion per byte took 33.6 us at 80 and 72 % of the issue slots, and
// two 16-byte accesses instead of one of 32 took 35.8.  One row of 8 x 8
// heads: 2.2 us a kernel, a launch's latency and that of three reads one
// behind the other.
//
// Quantising is exact.  With amax and x of at most 11 significant bits and
// e4m3 midpoints of 5, amax / 6 is either a midpoint or at least 2^-11 away
// from it relatively.  amax * (1/6) in fp32 is within 2^-22 of the quotient,
// and rounding it to 16 bits (t = 257 q; t - (t - q)) returns a midpoint when
// the quotient is one and moves no other quotient past one, so the scale is
// the nearest e4m3 value of the real quotient.  The codes' quotients x / s (s
// of 4 bits, midpoints of 3) have the same gap; x * (1/s) is within 2^-22 of
// the quotient, and rounding it to multiples of 2^-17 (adding and subtracting
// 96, whose ulp that is) does the same there.
//
// Reading looks the codes up a byte at a time: four codes select four high and
// four low bytes of the 16-bit values 0, 0.5, 1, 1.5, 2, 3, 4, 6, which the
// scale multiplies; the products are exact (at most 6 significant bits).
#include <cstdint>

#include "fa_kv4.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

// e2m1 codes of eight values, the first in bits 0-3; nearest even, saturating.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&x)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}
// e4m3 byte of a value; nearest even, saturating.
__device__ __forceinline__ uint32_t to_e4m3(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(x));
    return r & 0xFFu;
}
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t byte) {  // both halves
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(byte * 0x0101u)));
    return r;
}
__device__ __forceinline__ float reciprocal(float x) {  // within 2^-23 relatively
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
template <bool F16>
__device__ __forceinline__ uint32_t mul_16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (F16)
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Codes and scale of 16 values.
template <bool F16>
__device__ __forceinline__ void quantise(const uint32_t (&w)[8], uint2& codes, uint32_t& sbyte) {
    // magnitudes of bf16 and fp16 order as integers (NaN above infinity)
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
    m = max(m & 0xFFFFu, m >> 16);
    const bool finite = m < (F16 ? 0x7C00u : 0x7F80u);
    // 8192 / 6 is past the largest scale
    const float q = __fmul_rn(fminf(widen_lo16<F16>(m), 8192.0f), 1.0f / 6.0f), t = __fmul_rn(q, 257.0f);
    sbyte = finite ? to_e4m3(__fsub_rn(t, __fsub_rn(t, q))) : 0x7Fu;
    const float inv = reciprocal(widen_lo16<true>(e4m3_to_f16x2(sbyte)));
    const uint64_t inv2 = f2_pack(inv, inv), up = f2_pack(96.0f, 96.0f), down = f2_pack(-96.0f, -96.0f);
    uint32_t c[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t v = w[4 * half + j];
            const float hi = F16 ? widen_lo16<true>(v >> 16) : __uint_as_float(v & 0xFFFF0000u);
            f2_unpack(f2_add(f2_fma(f2_pack(widen_lo16<F16>(v), hi), inv2, up), down), x[2 * j], x[2 * j + 1]);
        }
        c[half] = pack_e2m1x8(x);
    }
    const bool some = finite && sbyte != 0u;
    codes = make_uint2(some ? c[0] : 0u, some ? c[1] : 0u);
}

// The values of four codes (the low 16 bits of `sel`, without their signs)
// times the scale; `sign` holds each code's sign in the top bit of its byte.
template <bool F16>
__device__ __forceinline__ void values_of_four(uint32_t sel, uint32_t sign, uint32_t scale, uint32_t& v01, uint32_t& v23) {
    // high and low bytes of 0, 0.5, 1, 1.5 | 2, 3, 4, 6
    const uint32_t high = (F16 ? __byte_perm(0x3E3C3800u, 0x46444240u, sel) : __byte_perm(0x3F3F3F00u, 0x40404040u, sel)) |
                          (sign & 0x80808080u);
    const uint32_t low = F16 ? 0u : __byte_perm(0xC0800000u, 0xC0804000u, sel);
    v01 = mul_16x2<F16>(__byte_perm(low, high, 0x5140), scale);
    v23 = mul_16x2<F16>(__byte_perm(low, high, 0x7362), scale);
}
template <bool F16>
__device__ __forceinline__ void dequantise(uint2 codes, uint32_t sbyte, uint32_t (&out)[8]) {
    const uint32_t s = e4m3_to_f16x2(sbyte);
    const float f = widen_lo16<true>(s);
    const uint32_t scale = F16 ? s : pack_bf16x2(f, f);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const uint32_t c = half == 0 ? codes.x : codes.y, even = c << 4, sel = c & 0x77777777u;
        // byte i of each: the sign of code i (even codes sit in the low halves of c's bytes)
        values_of_four<F16>(sel, __byte_perm(even, c, 0x5140), scale, out[4 * half], out[4 * half + 1]);
        values_of_four<F16>(sel >> 16, __byte_perm(even, c, 0x7362), scale, out[4 * half + 2], out[4 * half + 3]);
    }
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
constexpr int kAppendOneCta = 512;  // pairs of blocks that a single CTA stores

// counts_out = counts advanced by n, one thread per sequence.
__device__ __forceinline__ void advance_counts(const Kv4AppendParams& p, int b) {
    const long long len = static_cast<long long>(max(p.c.counts[b], 0)) + p.n;
    const int32_t seen = p.c.counts[p.c.B + b];
    p.counts_out[b] = static_cast<int32_t>(min(len, static_cast<long long>(p.c.capacity)));
    p.counts_out[p.c.B + b] = static_cast<int32_t>(seen + p.n);
}

// Blocks 2 i and 2 i + 1 of 16 channels, in the order [head][key or value][row][block];
// the host keeps their number below 2^31, so 32-bit arithmetic finds them.
template <int D, bool F16>
__device__ __forceinline__ void append_pair(const Kv4AppendParams& p, uint32_t i) {
    constexpr uint32_t kPairs = D / 32;
    const uint32_t n = static_cast<uint32_t>(p.n);
    const uint32_t pair = i % kPairs, t = i / kPairs;
    const uint32_t rest = t / n, row = t - rest * n;
    const bool value = (rest & 1) != 0;
    const uint32_t head = rest >> 1;  // b * H_kv + key/value head
    const uint32_t b = head / static_cast<uint32_t>(p.c.H_kv);
    const uint4* x4 = reinterpret_cast<const uint4*>(value ? p.x[1] : p.x[0]) +
                      ((static_cast<long long>(head) * n + row) * kPairs + pair) * 4;
    const bool wide = wide_rows(x4);
    uint32_t w[2][8];
    load_values(x4, wide, w[0]);
    load_values(x4 + 2, wide, w[1]);
    const long long slot = static_cast<long long>(max(p.c.counts[b], 0)) + row;
    if (slot >= p.c.capacity) {
        if (row == n - 1 && pair == 0 && !value) atomicOr(&p.status->word, kDevErrCapacity);
        return;
    }
    uint2 c[2];
    uint32_t s[2];
    quantise<F16>(w[0], c[0], s[0]);
    quantise<F16>(w[1], c[1], s[1]);
    const long long at = static_cast<long long>(head) * p.c.capacity + slot;
    reinterpret_cast<uint4*>(value ? p.c.codes[1] : p.c.codes[0])[at * kPairs + pair] =
        make_uint4(c[0].x, c[0].y, c[1].x, c[1].y);
    reinterpret_cast<uint16_t*>(value ? p.c.scales[1] : p.c.scales[0])[at * kPairs + pair] =
        static_cast<uint16_t>(s[0] | s[1] << 8);
    if (pair == 0 && !value) {
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
    if (i < total) append_pair<D, F16>(p, i);
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
    constexpr uint32_t kPairs = D / 32;
    const uint32_t i = blockIdx.x * blockDim.x + threadIdx.x;
    grid_release();
    grid_wait();
    if (i >= total) return;
    const bool value = blockIdx.y != 0;
    uint4* x = static_cast<uint4*>(value ? p.x[1] : p.x[0]);
    if (x == nullptr) return;
    const uint32_t count = static_cast<uint32_t>(p.count);
    const uint32_t pair = i % kPairs, t = i / kPairs;
    const uint32_t head = t / count, row = t - head * count;
    const uint32_t b = head / static_cast<uint32_t>(p.c.H_kv);
    const long long slot = static_cast<long long>(p.first != nullptr ? p.first[b] : 0) + row;
    uint32_t out[2][8] = {};
    if (slot >= 0 && slot < p.c.capacity) {
        const long long at = (static_cast<long long>(head) * p.c.capacity + slot) * kPairs + pair;
        const uint4 codes = reinterpret_cast<const uint4*>(value ? p.c.codes[1] : p.c.codes[0])[at];
        const uint32_t s = reinterpret_cast<const uint16_t*>(value ? p.c.scales[1] : p.c.scales[0])[at];
        dequantise<F16>(make_uint2(codes.x, codes.y), s & 0xFFu, out[0]);
        dequantise<F16>(make_uint2(codes.z, codes.w), s >> 8, out[1]);
    }
    x += static_cast<long long>(i) * 4;
    store_values(x, wide_rows(x), out[0]);
    store_values(x + 2, wide_rows(x), out[1]);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendParams& p, cudaStream_t stream) {
    const long long total = 2ll * p.c.B * p.c.H_kv * p.n * (p.c.d / 32);
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
    const long long total = static_cast<long long>(p.c.B) * p.c.H_kv * p.count * (p.c.d / 32);
    const dim3 grid(static_cast<unsigned>((total + 255) / 256), 2);
    auto kern = p.c.d == 128 ? (p.f16 ? kv4_read_kernel<128, true> : kv4_read_kernel<128, false>)
                             : (p.f16 ? kv4_read_kernel<64, true> : kv4_read_kernel<64, false>);
    return launch_dependent(kern, grid, 256, 0, stream, p, static_cast<uint32_t>(total));
}

}  // namespace fa
