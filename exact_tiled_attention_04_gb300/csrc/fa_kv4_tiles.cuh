// Register layouts of the attention over the 4-bit cache (fa_kv4_fwd.cu): how
// a warp holds one block of query rows and works through a slab of 32 slots.
//
// Both compute S^T = K Q^T and O^T = V^T P^T with m16n8k16, keys (or channels)
// on the 16-row side, and read a slab's bytes straight in fragment order: the
// contraction index of S and the rows of O^T are permuted so that lane (g, t)
// (g = lane / 4, t = lane % 4) reads consecutive bytes of a key's codes
// (channels (D / 4) t ..) and of a value's (channels (D / 8) g ..).  A stored
// value is e2m1 x e4m3: two conversions and a product, exact in fp16.
//
// Wide<D, R>: 8 or 16 rows, one column of Q^T each.  The second product's A
// operand holds, per channel, the values of two keys side by side, while a
// byte holds two channels of one key: nibbles of two keys are interleaved
// (24 bit operations per 16 keys at D = 128) before they are widened.
//
// Paired<D>: up to 4 rows (the usual group of query heads of a decode step),
// which leave half of the 8 columns free.  The contraction runs over (key,
// channel parity) instead of keys, so that a byte's two channels are
// neighbours in the A operand as they are; the result's columns are (row,
// parity) and P^T has zeros where the parities differ.  It takes as many
// products as Wide, but no interleaving, half the exponentials (each row's
// scores are spread over all lanes) and half the accumulators.  4 rows by
// Paired instead of Wide<D, 8>: 36.3 against 39.7 us at B = 8, H = 32/8, 16384
// slots, d = 128; 29.5 against 33.9 for 16 ragged sequences with weights.
#pragma once

#include <cmath>
#include <cstdint>

#include "fa_kv4.h"
#include "fa_ptx.cuh"

namespace fa {
namespace kv4 {

constexpr int kWarps = 8;
constexpr int kSlab = 32;          // keys per slab
constexpr float kRefShift = 7.0f;  // weights are 2^7 at the row's reference maximum: fp16 then
                                   // holds weights down to 2^-31 of it
constexpr float kGrow = 15.0f;     // and up to 2^8 times it before the reference moves
constexpr uint32_t kOnes = 0x3C003C00u;  // fp16 1, 1

// The four f16x2 pairs of a word's eight e2m1 codes.
__device__ __forceinline__ void widen_codes(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
    return r;
}
__device__ __forceinline__ uint32_t mul16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
template <typename T>
__device__ __forceinline__ T lds(const uint8_t* p) {
    return *reinterpret_cast<const T*>(p);
}


// Barrier of the warps that hold rows.
__device__ __forceinline__ void sync_rows() { named_barrier_sync(1, kWarps * 32); }

// One slab and what is needed to work through it.
struct Slab {
    const uint8_t *kc, *vc, *ks, *vs;  // its codes and scales in shared memory
    const uint4* q;                    // the block's q fragments
    float* logits;                     // scores of the head's slot 0 from this block's first row on, or nullptr
    int key0, len;                     // first slot, slots of the sequence
    int rows, row0;                    // rows of the head, first row of the block
    int Nq, causal;
    bool masked;                       // some row does not see all of it
    bool first;                        // the warp's first of the unit
};
// Slots that row r of the head sees (rows behind the last: all).
__device__ __forceinline__ int slots_seen(const Slab& u, int r) {
    return u.len - (u.causal && r < u.rows ? u.Nq - 1 - r % u.Nq : 0);
}
// Slots behind the length hold anything: their values count 0.
__device__ __forceinline__ uint32_t held_scale(uint32_t byte, bool held) { return held ? byte : 0u; }
__device__ __forceinline__ bool is_nan_scale(uint32_t byte) { return (byte & 0x7Fu) == 0x7Fu; }

__device__ __forceinline__ void write_row(const Kv4FwdParams& p, long long row, float M, float L) {
    const float lse2 = L == 0.0f ? -INFINITY : M + log2f(L);
    if (p.lse != nullptr) p.lse[row] = lse2 * 0.69314718055994531f;
    p.row_lse2[row] = lse2;
}
// Where a unit's result goes.
struct Target {
    bool whole;            // the output, else the partial rows from `slot` on
    long long slot, row0;  // row0: output row of the block's first row
    int left;              // rows of the block that exist
};

template <int D, int R>
struct Wide {
    static constexpr int NT = R / 8;
    static constexpr int kMt = D / 16;  // 16-row tiles of O^T
    int g, t, lane;
    float c[NT][2];                     // score factor of rows 8 nt + 2 t, + 1
    float ref[NT][2];                   // the exponent's reference (base 2), set by the first slab
    float l[NT][2], lq[NT][4], o[NT][kMt][4];

    // row of the block whose channels lane g of q tile nt loads
    static __device__ __forceinline__ int q_row(int nt, int g) { return 8 * nt + g; }

    __device__ __forceinline__ void start(const float* factors, int lane_) {
        lane = lane_, g = lane / 4, t = lane % 4;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                c[nt][i] = factors[8 * nt + 2 * t + i];
                ref[nt][i] = l[nt][i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lq[nt][i] = 0.0f;
#pragma unroll
                for (int mt = 0; mt < kMt; ++mt) o[nt][mt][i] = 0.0f;
            }
        }
    }
    __device__ __forceinline__ int limit(const Slab& u, int nt, int i) const {
        return slots_seen(u, u.row0 + 8 * nt + 2 * t + i);
    }

    __device__ __forceinline__ void slab(const Slab& u) {
                const int kg = (g >> 1) + 4 * (g & 1);  // key of fragment row g (and 8 more of row g + 8)

        // ---- S^T of both halves of 16 keys
        float x[2][NT][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[h][nt][i] = 0.0f;
            const int ka = 16 * h + kg, kb = ka + 8;
            uint32_t wa[D / 32], wb[D / 32], sa[D / 64], sb[D / 64];
            if constexpr (D == 128) {
                const uint4 a = lds<uint4>(u.kc + ka * 64 + t * 16), b = lds<uint4>(u.kc + kb * 64 + t * 16);
                wa[0] = a.x, wa[1] = a.y, wa[2] = a.z, wa[3] = a.w;
                wb[0] = b.x, wb[1] = b.y, wb[2] = b.z, wb[3] = b.w;
                const uint32_t s2a = e4m3x2_to_f16x2(lds<uint16_t>(u.ks + ka * 8 + t * 2));
                const uint32_t s2b = e4m3x2_to_f16x2(lds<uint16_t>(u.ks + kb * 8 + t * 2));
                sa[0] = __byte_perm(s2a, 0, 0x1010), sa[1] = __byte_perm(s2a, 0, 0x3232);
                sb[0] = __byte_perm(s2b, 0, 0x1010), sb[1] = __byte_perm(s2b, 0, 0x3232);
            } else {
                const uint2 a = lds<uint2>(u.kc + ka * 32 + t * 8), b = lds<uint2>(u.kc + kb * 32 + t * 8);
                wa[0] = a.x, wa[1] = a.y;
                wb[0] = b.x, wb[1] = b.y;
                sa[0] = e4m3x2_to_f16x2(lds<uint8_t>(u.ks + ka * 4 + t) * 0x0101u);
                sb[0] = e4m3x2_to_f16x2(lds<uint8_t>(u.ks + kb * 4 + t) * 0x0101u);
            }
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                uint32_t ha[4], hb[4];
                widen_codes(wa[w], ha);
                widen_codes(wb[w], hb);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ha[i] = mul16x2(ha[i], sa[w / 2]);
                    hb[i] = mul16x2(hb[i], sb[w / 2]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint4 q = u.q[(nt * (D / 32) + w) * 32 + lane];
                    mma_f16(x[h][nt], ha[0], hb[0], ha[1], hb[1], q.x, q.y);
                    mma_f16(x[h][nt], ha[2], hb[2], ha[3], hb[3], q.z, q.w);
                }
            }
        }
        // ---- exponents (base 2) against the reference; hidden slots are -inf whatever is stored there
        float top = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[h][nt][i] = fmaf(x[h][nt][i], c[nt][i & 1], -ref[nt][i & 1]);
        if (u.masked) {
            asm volatile("");  // a branch: few slabs are masked
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int lim = limit(u, nt, i) - u.key0 - kg;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (16 * h >= lim) x[h][nt][i] = -INFINITY;
                        if (16 * h + 8 >= lim) x[h][nt][i + 2] = -INFINITY;
                    }
                }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmax3(top, x[0][nt][i], x[1][nt][i]);
        // the first slab sets the reference (nothing to rescale); later ones move it when a weight would
        // pass fp16's range
        if (u.first || __any_sync(0xffffffffu, top > kGrow)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float m = fmaxf(fmaxf(x[0][nt][i], x[0][nt][i + 2]), fmaxf(x[1][nt][i], x[1][nt][i + 2]));
#pragma unroll
                    for (int off = 4; off < 32; off *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
                    // a row that sees none of a first slab sees none of the warp's later ones either
                    float shift = m == -INFINITY ? 0.0f : m - kRefShift;
                    if (!u.first) {
                        shift = fmaxf(shift, 0.0f);
                        const float alpha = ex2(-shift);
                        l[nt][i] *= alpha;
                        lq[nt][i] *= alpha;
#pragma unroll
                        for (int mt = 0; mt < kMt; ++mt) {
                            o[nt][mt][i] *= alpha;
                            o[nt][mt][i + 2] *= alpha;
                        }
                    }
                    ref[nt][i] += shift;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        x[h][nt][i] -= shift;
                        x[h][nt][i + 2] -= shift;
                    }
                }
        }
        if (u.logits != nullptr) {
            float* dst = u.logits + static_cast<long long>(u.key0 + kg) * u.rows + 2 * t;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i2 = 0; i2 < 2; ++i2) {
                    if (!u.masked || u.key0 + kg + 16 * h + 8 * i2 < u.len) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const int left = u.rows - u.row0 - 8 * nt - 2 * t;  // rows from 2t on
                            const float y0 = x[h][nt][2 * i2] + ref[nt][0], y1 = x[h][nt][2 * i2 + 1] + ref[nt][1];
                            if (u.rows % 2 == 0 && left > 0) {  // both rows exist, 8-byte aligned
                                *reinterpret_cast<float2*>(dst + 8 * nt) = make_float2(y0, y1);
                            } else {
                                if (left > 0) dst[8 * nt] = y0;
                                if (left > 1) dst[8 * nt + 1] = y1;
                            }
                        }
                    }
                    dst += 8 * u.rows;
                }
        }
        // ---- weights, O^T += V^T P^T
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t pb[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[i] = ex2(x[h][nt][i]);
                    l[nt][i & 1] += w[i];
                }
                pb[nt][0] = transpose8x8(pack_f16x2(w[0], w[1]));
                pb[nt][1] = transpose8x8(pack_f16x2(w[2], w[3]));
                mma_f16(lq[nt], kOnes, kOnes, kOnes, kOnes, pb[nt][0], pb[nt][1]);
            }
            uint32_t sc[4], v[4][D / 64];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = 16 * h + 4 * i + t;
                if constexpr (D == 128) {
                    const uint2 a = lds<uint2>(u.vc + key * 64 + g * 8);
                    v[i][0] = a.x, v[i][1] = a.y;
                    sc[i] = lds<uint8_t>(u.vs + key * 8 + g);
                } else {
                    v[i][0] = lds<uint32_t>(u.vc + key * 32 + g * 4);
                    sc[i] = lds<uint8_t>(u.vs + key * 4 + g / 2);
                }
            }
            if (u.masked) {
                // slots behind the length hold anything: values 0.  A NaN in a slot that only some
                // rows see must not reach the others (0 * NaN): it is taken out of the product and
                // set in the rows that see it.
                bool nan = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (u.key0 + 16 * h + 4 * i + t >= u.len) sc[i] = 0u;
                    nan |= (sc[i] & 0x7Fu) == 0x7Fu;
                }
                if (__any_sync(0xffffffffu, nan)) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t su = __shfl_sync(0xffffffffu, sc[i], (lane & ~3) | k);
                            if ((su & 0x7Fu) == 0x7Fu) {
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                    for (int j = 0; j < 2; ++j)
                                        if (u.key0 + 16 * h + 4 * i + k < limit(u, nt, j)) {
#pragma unroll
                                            for (int mt = 0; mt < kMt; ++mt)
                                                o[nt][mt][j] = o[nt][mt][j + 2] = __int_as_float(0x7FC00000);
                                        }
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if ((sc[i] & 0x7Fu) == 0x7Fu) sc[i] = 0u;
                }
            }
            const uint32_t s01 = e4m3x2_to_f16x2(sc[0] | sc[1] << 8), s23 = e4m3x2_to_f16x2(sc[2] | sc[3] << 8);
#pragma unroll
            for (int w = 0; w < D / 64; ++w) {
                constexpr uint32_t kLow = 0x0F0F0F0Fu;
                uint32_t a0[4], a1[4], a2[4], a3[4];
                widen_codes((v[0][w] & kLow) | ((v[1][w] << 4) & ~kLow), a0);
                widen_codes(((v[0][w] >> 4) & kLow) | (v[1][w] & ~kLow), a1);
                widen_codes((v[2][w] & kLow) | ((v[3][w] << 4) & ~kLow), a2);
                widen_codes(((v[2][w] >> 4) & kLow) | (v[3][w] & ~kLow), a3);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a0[i] = mul16x2(a0[i], s01);
                    a1[i] = mul16x2(a1[i], s01);
                    a2[i] = mul16x2(a2[i], s23);
                    a3[i] = mul16x2(a3[i], s23);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16(o[nt][4 * w + i], a0[i], a1[i], a2[i], a3[i], pb[nt][0], pb[nt][1]);
                }
            }
        }
    }

    // The block's rows over the CTA's warps.  ahead(): work to do while the sums are on their way.
    template <class Ahead>
    __device__ __forceinline__ void finish(const Kv4FwdParams& p, const Target& to, float4* sm_ml, float4* sm_o, int warp,
                                           Ahead ahead) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float s = l[nt][i];
#pragma unroll
                for (int off = 4; off < 32; off *= 2) s += __shfl_xor_sync(0xffffffffu, s, off);
                if (g == 0)
                    sm_ml[warp * R + 8 * nt + 2 * t + i] =
                        make_float4(s == 0.0f ? -INFINITY : ref[nt][i], s, lq[nt][i], 0.0f);
            }
        sync_rows();
        // lane (g, t): row g of each block of 8, warps t and t + 4; then the quad's M, L, LQ of that row
        float M[NT], L[NT], LQ[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float4 ma = sm_ml[t * R + 8 * nt + g], mb = sm_ml[(t + 4) * R + 8 * nt + g];
            float m = fmaxf(ma.x, mb.x);
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            // a warp that saw nothing counts 0 (a NaN sum stays one)
            const float fa = m == -INFINITY ? 1.0f : ex2(ma.x - m), fb = m == -INFINITY ? 1.0f : ex2(mb.x - m);
            M[nt] = m;
            L[nt] = fa * ma.y + fb * mb.y;
            LQ[nt] = fa * ma.z + fb * mb.z;
#pragma unroll
            for (int off = 1; off < 4; off *= 2) {
                L[nt] += __shfl_xor_sync(0xffffffffu, L[nt], off);
                LQ[nt] += __shfl_xor_sync(0xffffffffu, LQ[nt], off);
            }
            // this warp's weight in row g, then in rows 2t, 2t + 1
            const float f = __shfl_sync(0xffffffffu, warp < 4 ? fa : fb, (lane & ~3) | (warp & 3));
            const float f0 = __shfl_sync(0xffffffffu, f, 8 * t), f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt)
                sm_o[((warp * kMt + mt) * NT + nt) * 32 + lane] =
                    make_float4(o[nt][mt][0] * f0, o[nt][mt][1] * f1, o[nt][mt][2] * f0, o[nt][mt][3] * f1);
        }
        ahead();
        sync_rows();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = 8 * nt + 2 * t;
            if (warp < kMt) {  // each of the first D / 16 warps adds up one 16-channel tile
                float4 acc = sm_o[(warp * NT + nt) * 32 + lane];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) {
                    const float4 v = sm_o[((w * kMt + warp) * NT + nt) * 32 + lane];
                    acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
                }
                const int ch = (D / 8) * g + 2 * warp;  // channels ch, ch + 1 of rows r (x, z) and r + 1 (y, w)
                const float q0 = __shfl_sync(0xffffffffu, LQ[nt], 8 * t), q1 = __shfl_sync(0xffffffffu, LQ[nt], 8 * t + 4);
                if (to.whole) {
                    const float i0 = q0 == 0.0f ? 0.0f : 1.0f / q0, i1 = q1 == 0.0f ? 0.0f : 1.0f / q1;
                    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + (to.row0 + r) * D + ch);
                    if (r < to.left)
                        out[0] = p.f16 ? pack_f16x2(acc.x * i0, acc.z * i0) : pack_bf16x2(acc.x * i0, acc.z * i0);
                    if (r + 1 < to.left)
                        out[D / 2] = p.f16 ? pack_f16x2(acc.y * i1, acc.w * i1) : pack_bf16x2(acc.y * i1, acc.w * i1);
                } else {
                    float* out = p.part_o + (to.slot + r) * D + ch;
                    *reinterpret_cast<float2*>(out) = make_float2(acc.x, acc.z);
                    *reinterpret_cast<float2*>(out + D) = make_float2(acc.y, acc.w);
                }
            }
            if (warp == 0 && t == 0) {
                const int rg = 8 * nt + g;
                if (!to.whole)
                    p.part_ml[to.slot + rg] = make_float4(M[nt], L[nt], LQ[nt], 0.0f);
                else if (rg < to.left)
                    write_row(p, to.row0 + rg, M[nt], L[nt]);
            }
        }
    }
};

template <int D>
struct Paired {
    static constexpr int kMt = D / 32;  // tiles of 16 channel pairs
    int g, t, lane;
    float c, ref, l, lq[4], o[kMt][4];  // of row t; o: channels (D / 8) g + 4 mt ..

    // the column pair (row, parity) of the first product is the same row twice
    static __device__ __forceinline__ int q_row(int, int g) { return g >> 1; }

    __device__ __forceinline__ void start(const float* factors, int lane_) {
        lane = lane_, g = lane / 4, t = lane % 4;
        c = factors[t];
        ref = l = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lq[i] = 0.0f;
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt) o[mt][i] = 0.0f;
        }
    }

    __device__ __forceinline__ void slab(const Slab& u) {
        // ---- S^T of both halves of 16 keys: row t's scores of keys 16 h + g and + 8
        float x[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // columns 2t, 2t + 1 are equal
            const int ka = 16 * h + g, kb = ka + 8;
            uint32_t wa[D / 32], wb[D / 32], sa[D / 64], sb[D / 64];
            if constexpr (D == 128) {
                const uint4 a = lds<uint4>(u.kc + ka * 64 + t * 16), b = lds<uint4>(u.kc + kb * 64 + t * 16);
                wa[0] = a.x, wa[1] = a.y, wa[2] = a.z, wa[3] = a.w;
                wb[0] = b.x, wb[1] = b.y, wb[2] = b.z, wb[3] = b.w;
                const uint32_t s2a = e4m3x2_to_f16x2(lds<uint16_t>(u.ks + ka * 8 + t * 2));
                const uint32_t s2b = e4m3x2_to_f16x2(lds<uint16_t>(u.ks + kb * 8 + t * 2));
                sa[0] = __byte_perm(s2a, 0, 0x1010), sa[1] = __byte_perm(s2a, 0, 0x3232);
                sb[0] = __byte_perm(s2b, 0, 0x1010), sb[1] = __byte_perm(s2b, 0, 0x3232);
            } else {
                const uint2 a = lds<uint2>(u.kc + ka * 32 + t * 8), b = lds<uint2>(u.kc + kb * 32 + t * 8);
                wa[0] = a.x, wa[1] = a.y;
                wb[0] = b.x, wb[1] = b.y;
                sa[0] = e4m3x2_to_f16x2(lds<uint8_t>(u.ks + ka * 4 + t) * 0x0101u);
                sb[0] = e4m3x2_to_f16x2(lds<uint8_t>(u.ks + kb * 4 + t) * 0x0101u);
            }
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                uint32_t ha[4], hb[4];
                widen_codes(wa[w], ha);
                widen_codes(wb[w], hb);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ha[i] = mul16x2(ha[i], sa[w / 2]);
                    hb[i] = mul16x2(hb[i], sb[w / 2]);
                }
                const uint4 q = u.q[w * 32 + lane];
                mma_f16(s, ha[0], hb[0], ha[1], hb[1], q.x, q.y);
                mma_f16(s, ha[2], hb[2], ha[3], hb[3], q.z, q.w);
            }
            x[h][0] = s[0];
            x[h][1] = s[2];
        }
        // ---- exponents (base 2) against the reference; hidden slots are -inf whatever is stored there
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) x[h][i] = fmaf(x[h][i], c, -ref);
        if (u.masked) {
            asm volatile("");  // a branch: few slabs are masked
            const int lim = slots_seen(u, u.row0 + t) - u.key0 - g;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (16 * h + 8 * i >= lim) x[h][i] = -INFINITY;
        }
        float top = fmaxf(fmax3(x[0][0], x[0][1], x[1][0]), x[1][1]);
        // the first slab sets the reference (nothing to rescale); later ones move it when a weight would
        // pass fp16's range
        if (u.first || __any_sync(0xffffffffu, top > kGrow)) {
#pragma unroll
            for (int off = 4; off < 32; off *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            // a row that sees none of a first slab sees none of the warp's later ones either
            float shift = top == -INFINITY ? 0.0f : top - kRefShift;
            if (!u.first) {
                shift = fmaxf(shift, 0.0f);
                const float alpha = ex2(-shift);
                l *= alpha;
                lq[0] *= alpha;
#pragma unroll
                for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[mt][i] *= alpha;
            }
            ref += shift;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) x[h][i] -= shift;
        }
        if (u.logits != nullptr && u.row0 + t < u.rows) {
            float* dst = u.logits + static_cast<long long>(u.key0 + g) * u.rows + t;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (!u.masked || u.key0 + g + 16 * h + 8 * i < u.len) *dst = x[h][i] + ref;
                    dst += 8 * u.rows;
                }
        }
        // ---- weights, O^T += V^T P^T
        const uint32_t low = g & 1 ? 0x1044u : 0x4410u, high = g & 1 ? 0x3244u : 0x4432u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float w0 = ex2(x[h][0]), w1 = ex2(x[h][1]);
            l += w0 + w1;
            // weights of keys g (low half) and g + 8 of row t; B wants keys t, 4 + t, 8 + t, 12 + t of row g / 2,
            // in the half of the column's parity
            const uint32_t w = pack_f16x2(w0, w1);
            const uint32_t wa = __shfl_sync(0xffffffffu, w, 4 * t + (g >> 1));
            const uint32_t wb = __shfl_sync(0xffffffffu, w, 16 + 4 * t + (g >> 1));
            const uint32_t b0 = __byte_perm(wa, 0, low), b1 = __byte_perm(wb, 0, low);    // keys t, 4 + t
            const uint32_t b2 = __byte_perm(wa, 0, high), b3 = __byte_perm(wb, 0, high);  // keys 8 + t, 12 + t
            mma_f16(lq, kOnes, kOnes, kOnes, kOnes, b0, b1);
            mma_f16(lq, kOnes, kOnes, kOnes, kOnes, b2, b3);
            uint32_t sc[4], v[4][D / 64];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = 16 * h + 4 * i + t;
                if constexpr (D == 128) {
                    const uint2 a = lds<uint2>(u.vc + key * 64 + g * 8);
                    v[i][0] = a.x, v[i][1] = a.y;
                    sc[i] = lds<uint8_t>(u.vs + key * 8 + g);
                } else {
                    v[i][0] = lds<uint32_t>(u.vc + key * 32 + g * 4);
                    sc[i] = lds<uint8_t>(u.vs + key * 4 + g / 2);
                }
            }
            if (u.masked) {
                // A NaN in a slot that only some rows see must not reach the others (0 * NaN): it is taken out of
                // the product and set in the rows that see it.
                bool nan = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sc[i] = held_scale(sc[i], u.key0 + 16 * h + 4 * i + t < u.len);
                    nan |= is_nan_scale(sc[i]);
                }
                if (__any_sync(0xffffffffu, nan)) {
                    const int lim = slots_seen(u, u.row0 + t);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (is_nan_scale(__shfl_sync(0xffffffffu, sc[i], (lane & ~3) | k)) &&
                                u.key0 + 16 * h + 4 * i + k < lim) {
#pragma unroll
                                for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
                                    for (int j = 0; j < 4; ++j) o[mt][j] = __int_as_float(0x7FC00000);
                            }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (is_nan_scale(sc[i])) sc[i] = 0u;
                }
            }
            uint32_t s2[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) s2[i] = e4m3x2_to_f16x2(sc[i] * 0x0101u);
#pragma unroll
            for (int w4 = 0; w4 < D / 64; ++w4) {
                uint32_t a[4][4];  // [key][byte]
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    widen_codes(v[i][w4], a[i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) a[i][j] = mul16x2(a[i][j], s2[i]);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    mma_f16(o[2 * w4 + j], a[0][2 * j], a[0][2 * j + 1], a[1][2 * j], a[1][2 * j + 1], b0, b1);
                    mma_f16(o[2 * w4 + j], a[2][2 * j], a[2][2 * j + 1], a[3][2 * j], a[3][2 * j + 1], b2, b3);
                }
            }
        }
    }

    template <class Ahead>
    __device__ __forceinline__ void finish(const Kv4FwdParams& p, const Target& to, float4* sm_ml, float4* sm_o, int warp,
                                           Ahead ahead) {
        float s = l;
#pragma unroll
        for (int off = 4; off < 32; off *= 2) s += __shfl_xor_sync(0xffffffffu, s, off);
        if (g == 0) sm_ml[warp * 4 + t] = make_float4(s == 0.0f ? -INFINITY : ref, s, lq[0], 0.0f);
        sync_rows();
        // lane (g, t): row t of warp g; then every lane has M, L, LQ of row t
        const float4 ml = sm_ml[g * 4 + t];
        float M = ml.x;
#pragma unroll
        for (int off = 4; off < 32; off *= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        const float f = M == -INFINITY ? 1.0f : ex2(ml.x - M);  // a warp that saw nothing counts 0
        float L = f * ml.y, LQ = f * ml.z;
#pragma unroll
        for (int off = 4; off < 32; off *= 2) {
            L += __shfl_xor_sync(0xffffffffu, L, off);
            LQ += __shfl_xor_sync(0xffffffffu, LQ, off);
        }
        const float mine = __shfl_sync(0xffffffffu, f, 4 * warp + t);
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt)
            sm_o[(warp * kMt + mt) * 32 + lane] =
                make_float4(o[mt][0] * mine, o[mt][1] * mine, o[mt][2] * mine, o[mt][3] * mine);
        ahead();
        sync_rows();
        if (warp < kMt) {
            float4 acc = sm_o[warp * 32 + lane];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
                const float4 v = sm_o[(w * kMt + warp) * 32 + lane];
                acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
            }
            const int ch = (D / 8) * g + 4 * warp;
            if (!to.whole) {
                *reinterpret_cast<float4*>(p.part_o + (to.slot + t) * D + ch) = acc;
            } else if (t < to.left) {
                const float inv = LQ == 0.0f ? 0.0f : 1.0f / LQ;
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + (to.row0 + t) * D + ch) =
                    p.f16 ? make_uint2(pack_f16x2(acc.x * inv, acc.y * inv), pack_f16x2(acc.z * inv, acc.w * inv))
                          : make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
            }
        }
        if (warp == 0 && g == 0) {
            if (!to.whole)
                p.part_ml[to.slot + t] = make_float4(M, L, LQ, 0.0f);
            else if (t < to.left)
                write_row(p, to.row0 + t, M, L);
        }
    }
};

}  // namespace kv4
}  // namespace fa
