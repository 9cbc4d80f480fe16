// C-ABI entry points of the 4-bit key/value cache and of the attention weight
// of a prompt (declared in include/fa.h): argument checks, workspace layout
// and launches on the caller's stream.
#include <cmath>
#include <cstddef>
#include <cstdint>

#include <cudaTypedefs.h>

#include "fa.h"
#include "fa_host.h"
#include "fa_kv4.h"

using namespace fa::host;

namespace {

constexpr int64_t kInt32Max = 2147483647;
constexpr int64_t kMaxRowsPerHead = 128;  // fa_kv4_fwd: N_q * H / H_kv
constexpr float kLog2e = 1.4426950408889634f;

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// a * b, or -1 past 2^62 (-1 passes through)
int64_t mul(int64_t a, int64_t b) {
    if (a < 0 || b < 0) return -1;
    if (b != 0 && a > (int64_t(1) << 62) / b) return -1;
    return a * b;
}

struct Span {
    const void* p;
    size_t n;
};
bool meet(const Span& a, const Span& b) { return a.p != nullptr && b.p != nullptr && overlaps(a.p, a.n, b.p, b.n); }

// The arrays of a cache: k_codes, k_scales, v_codes, v_scales, weight, pos, counts.
constexpr int kArrays = 7, kWeightArray = 4;
void cache_spans(const fa_kv4_cache_t& c, Span (&s)[kArrays]) {
    const size_t slots = static_cast<size_t>(c.B * c.H_kv * c.capacity);
    const size_t codes = slots * static_cast<size_t>(c.d / 2), scales = slots * static_cast<size_t>(c.d / 16);
    s[0] = {c.k_codes, codes};
    s[1] = {c.k_scales, scales};
    s[2] = {c.v_codes, codes};
    s[3] = {c.v_scales, scales};
    s[4] = {c.weight, slots * 4};
    s[5] = {c.pos, slots * 4};
    s[6] = {c.counts, static_cast<size_t>(c.B) * 8};
}

int check_cache(const fa_kv4_cache_t* c) {
    if (c == nullptr || !c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales || !c->counts)
        return FA_ERR_INVALID_ARG;
    if (c->B < 1 || c->H_kv < 1 || c->d < 1 || c->capacity < 1 || c->capacity % 128 != 0) return FA_ERR_INVALID_ARG;
    if (c->d != 64 && c->d != 128) return FA_ERR_UNSUPPORTED;
    if (mul(mul(mul(c->B, c->H_kv), c->capacity), c->d) < 0) return FA_ERR_INVALID_ARG;
    if (c->B > kInt32Max / c->H_kv || c->capacity > kInt32Max - 128) return FA_ERR_UNSUPPORTED;
    if (misaligned(c->k_codes, 16) || misaligned(c->k_scales, 16) || misaligned(c->v_codes, 16) ||
        misaligned(c->v_scales, 16) || misaligned(c->weight, 4) || misaligned(c->pos, 4) || misaligned(c->counts, 4))
        return FA_ERR_ALIGNMENT;
    Span s[kArrays];
    cache_spans(*c, s);
    for (int i = 0; i < kArrays; ++i)
        for (int j = i + 1; j < kArrays; ++j)
            if (meet(s[i], s[j])) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

fa::Kv4Cache device_cache(const fa_kv4_cache_t& c) {
    fa::Kv4Cache k{};
    k.codes[0] = c.k_codes;
    k.codes[1] = c.v_codes;
    k.scales[0] = c.k_scales;
    k.scales[1] = c.v_scales;
    k.weight = c.weight;
    k.pos = c.pos;
    k.counts = c.counts;
    k.B = static_cast<int>(c.B);
    k.H_kv = static_cast<int>(c.H_kv);
    k.capacity = static_cast<int>(c.capacity);
    k.d = static_cast<int>(c.d);
    return k;
}

bool meets_cache(const Span& x, const fa_kv4_cache_t& c, int except = -1) {
    Span s[kArrays];
    cache_spans(c, s);
    for (int i = 0; i < kArrays; ++i)
        if (i != except && meet(x, s[i])) return true;
    return false;
}

int check_dtype16(int dtype) {
    if (dtype == FA_DTYPE_BF16 || dtype == FA_DTYPE_F16) return FA_OK;
    return dtype >= 0 && dtype < 0x100 ? FA_ERR_UNSUPPORTED : FA_ERR_INVALID_ARG;
}

int sm_count() {
    static std::atomic<int> counts[64];  // 0: not asked yet
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) == cudaSuccess) {
        if (dev < 64 && (n = counts[dev].load(std::memory_order_relaxed)) > 0) return n;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0) {
            if (dev < 64) counts[dev].store(n, std::memory_order_relaxed);
            return n;
        }
    }
    cudaGetLastError();
    return 0;
}

int launched(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return FA_OK;
    set_error(what, static_cast<int>(e), cudaGetErrorString(e));
    return FA_ERR_CUDA;
}

// ------------------------------------------------------------------- append
int validate_append(const fa_kv4_cache_t* c, const void* k, const void* v, int64_t n, int dtype,
                    const int32_t* counts_out) {
    int st = check_cache(c);
    if (st != FA_OK) return st;
    if (!k || !v || !counts_out || n < 1) return FA_ERR_INVALID_ARG;
    if ((st = check_dtype16(dtype)) != FA_OK) return st;
    const int64_t elems = mul(mul(mul(c->B, c->H_kv), n), c->d);
    if (elems < 0) return FA_ERR_INVALID_ARG;
    if (n > kInt32Max || elems / 8 > kInt32Max) return FA_ERR_UNSUPPORTED;  // the grid
    if (misaligned(k, 16) || misaligned(v, 16) || misaligned(counts_out, 4)) return FA_ERR_ALIGNMENT;
    const Span sk{k, static_cast<size_t>(elems) * 2}, sv{v, static_cast<size_t>(elems) * 2};
    const Span co{counts_out, static_cast<size_t>(c->B) * 8};
    if (meets_cache(sk, *c) || meets_cache(sv, *c) || meet(co, sk) || meet(co, sv)) return FA_ERR_INVALID_ARG;
    if (counts_out != c->counts && meets_cache(co, *c)) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

// --------------------------------------------------------------------- read
int validate_read(const fa_kv4_cache_t* c, const int32_t* first, int64_t count, const void* k, const void* v,
                  int dtype) {
    int st = check_cache(c);
    if (st != FA_OK) return st;
    if ((!k && !v) || count < 1) return FA_ERR_INVALID_ARG;
    if ((st = check_dtype16(dtype)) != FA_OK) return st;
    const int64_t elems = mul(mul(mul(c->B, c->H_kv), count), c->d);
    if (elems < 0) return FA_ERR_INVALID_ARG;
    if (count > kInt32Max || elems / 16 > kInt32Max) return FA_ERR_UNSUPPORTED;
    if (misaligned(k, 16) || misaligned(v, 16) || misaligned(first, 4)) return FA_ERR_ALIGNMENT;
    const Span sk{k, static_cast<size_t>(elems) * 2}, sv{v, static_cast<size_t>(elems) * 2};
    const Span sf{first, static_cast<size_t>(c->B) * 4};
    if (meets_cache(sk, *c) || meets_cache(sv, *c) || meet(sk, sv) || meet(sk, sf) || meet(sv, sf))
        return FA_ERR_INVALID_ARG;
    return FA_OK;
}

// ---------------------------------------------------------------- attention
struct FwdLayout {
    fa::Kv4Plan plan;
    size_t part_ml, part_o, logits, bytes;  // offsets (row_lse2 is first), total
};

// false: sizes the call does not take
bool fwd_layout(int64_t B, int64_t H, int64_t H_kv, int64_t N_q, int64_t capacity, int64_t d, bool weight, int sms,
                FwdLayout* l) {
    if (B < 1 || H < 1 || H_kv < 1 || N_q < 1 || capacity < 1 || capacity % 128 != 0 || H % H_kv != 0) return false;
    if (d != 64 && d != 128) return false;
    if (mul(mul(mul(B, H_kv), capacity), d) < 0 || B > kInt32Max / H_kv || capacity > kInt32Max - 128) return false;
    const int64_t group = H / H_kv;
    if (N_q > kMaxRowsPerHead || group > kMaxRowsPerHead || N_q * group > kMaxRowsPerHead) return false;
    const int64_t rows = N_q * group, all = mul(mul(B, H_kv), rows);
    const int64_t logits = mul(mul(B, H_kv), mul(capacity, rows * 4));
    const int64_t chunks = mul(B * H_kv, (capacity + 1023) / 1024);
    // the slabs of 32 slots over all blocks of 8 rows; the second kernel's grid: a warp per row, a block per 1024 slots
    const int64_t slabs = mul(mul(B * H_kv, (rows + 7) / 8), capacity / 32 + fa::kKv4UnitCost);
    if (slabs < 0 || slabs > kInt32Max / 2) return false;
    if (all < 0 || all > kInt32Max || logits < 0 || chunks < 0 || chunks > kInt32Max / 2) return false;
    l->plan = fa::kv4_plan(B, H_kv, rows, capacity, sms > 0 ? sms : 1024);
    const size_t parts = l->plan.single ? 0 : static_cast<size_t>(l->plan.ctas) * 2 *
                                                  static_cast<size_t>(fa::kv4_rows_per_block(rows));
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    l->part_ml = up(static_cast<size_t>(all) * 4);
    l->part_o = l->part_ml + up(parts * 16);
    l->logits = l->part_o + up(parts * static_cast<size_t>(d) * 4);
    l->bytes = l->logits + (weight ? up(static_cast<size_t>(logits)) : 0);
    return true;
}

int validate_fwd(const fa_kv4_cache_t* c, const void* q, const void* o, const float* lse, const float* weight_out,
                 int64_t H, int64_t N_q, float scale, int dtype_arg, const void* ws, size_t ws_bytes, int sms,
                 FwdLayout* l) {
    int st = check_cache(c);
    if (st != FA_OK) return st;
    if (!q || !o || !ws || H < 1 || N_q < 1 || H % c->H_kv != 0) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || (dtype_arg & ~(0xFF | FA_FLAG_CAUSAL))) return FA_ERR_INVALID_ARG;
    if ((st = check_dtype16(dtype_arg & 0xFF)) != FA_OK) return st;
    if (!fwd_layout(c->B, H, c->H_kv, N_q, c->capacity, c->d, weight_out != nullptr, sms, l))
        return FA_ERR_UNSUPPORTED;
    if (misaligned(q, 16) || misaligned(o, 16) || misaligned(ws, 16) || misaligned(lse, 4) || misaligned(weight_out, 4))
        return FA_ERR_ALIGNMENT;
    if (ws_bytes < l->bytes) return FA_ERR_INVALID_ARG;
    const size_t rows = static_cast<size_t>(c->B * H * N_q);
    const Span in{q, rows * static_cast<size_t>(c->d) * 2}, out{o, in.n}, sl{lse, rows * 4};
    const Span sw{weight_out, static_cast<size_t>(c->B * c->H_kv * c->capacity) * 4}, work{ws, l->bytes};
    const Span written[4] = {out, sl, sw, work};
    for (int i = 0; i < 4; ++i) {
        if (meet(written[i], in)) return FA_ERR_INVALID_ARG;
        // the weights may be added in place
        if (meets_cache(written[i], *c, i == 2 && weight_out == c->weight ? kWeightArray : -1))
            return FA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 4; ++j)
            if (meet(written[i], written[j])) return FA_ERR_INVALID_ARG;
    }
    return FA_OK;
}

// ----------------------------------------------------------------- eviction
int validate_evict(const fa_kv4_cache_t* c, int64_t keep, int64_t sinks, int64_t recent, const float* rank_by,
                   const fa_kv4_cache_t* to, const int32_t* src, const int32_t* counts_out) {
    int st = check_cache(c);
    if (st != FA_OK) return st;
    if (keep < 1 || sinks < 0 || recent < 0 || !src || !counts_out) return FA_ERR_INVALID_ARG;
    if (!rank_by && !c->weight) return FA_ERR_INVALID_ARG;
    if ((sinks > 0 || recent > 0) && !c->pos) return FA_ERR_INVALID_ARG;
    if (c->capacity > fa::kKv4EvictMaxCapacity || keep > kInt32Max || sinks > kInt32Max || recent > kInt32Max)
        return FA_ERR_UNSUPPORTED;
    const int64_t entries = mul(mul(c->B, c->H_kv), keep);
    if (mul(entries, 4) < 0) return FA_ERR_INVALID_ARG;
    if (mul(c->B * c->H_kv, fa::kv4_copy_blocks(keep, c->capacity)) > kInt32Max || c->B * c->H_kv > kInt32Max / 8) return FA_ERR_UNSUPPORTED;
    if (misaligned(rank_by, 4) || misaligned(src, 4) || misaligned(counts_out, 4)) return FA_ERR_ALIGNMENT;
    const Span rank{rank_by, static_cast<size_t>(c->B * c->H_kv * c->capacity) * 4};
    const Span list{src, static_cast<size_t>(entries) * 4}, co{counts_out, static_cast<size_t>(c->B) * 8};
    if (meets_cache(list, *c) || meet(list, rank) || meet(list, co) || meet(co, rank)) return FA_ERR_INVALID_ARG;
    if (counts_out != c->counts && meets_cache(co, *c)) return FA_ERR_INVALID_ARG;
    // the ranking weights are the cache's own (which move along) or apart from it
    if (meets_cache(rank, *c, rank_by == c->weight ? kWeightArray : -1)) return FA_ERR_INVALID_ARG;
    if (to != nullptr) {
        if ((st = check_cache(to)) != FA_OK) return st;
        if (to->B != c->B || to->H_kv != c->H_kv || to->d != c->d || to->capacity < keep) return FA_ERR_INVALID_ARG;
        Span s[kArrays];
        cache_spans(*to, s);
        for (int i = 0; i < kArrays; ++i)
            if (meets_cache(s[i], *c) || meet(s[i], rank) || meet(s[i], list)) return FA_ERR_INVALID_ARG;
        if (counts_out != to->counts && meets_cache(co, *to)) return FA_ERR_INVALID_ARG;
    }
    return FA_OK;
}

// ------------------------------------------------------------------ weights
int validate_weights(const void* q, const void* k, const float* lse, const float* weight_in, const float* weight_out,
                     int64_t stride, int64_t B, int64_t H, int64_t H_kv, int64_t N_q, int64_t N_kv, int64_t d,
                     int64_t first_query, float scale, int dtype_arg) {
    if (!q || !k || !lse || !weight_out) return FA_ERR_INVALID_ARG;
    if (B < 1 || H < 1 || H_kv < 1 || N_q < 1 || N_kv < 1 || d < 1 || H % H_kv != 0) return FA_ERR_INVALID_ARG;
    if (first_query < 0 || first_query >= N_q || stride < N_kv) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || (dtype_arg & ~(0xFF | FA_FLAG_CAUSAL))) return FA_ERR_INVALID_ARG;
    const int st = check_dtype16(dtype_arg & 0xFF);
    if (st != FA_OK) return st;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    const int64_t qn = mul(mul(mul(B, H), N_q), d), kn = mul(mul(mul(B, H_kv), N_kv), d);
    const int64_t wn = mul(mul(B, H_kv), stride);
    if (qn < 0 || kn < 0 || mul(wn, 4) < 0) return FA_ERR_INVALID_ARG;
    if (B > kInt32Max / H || N_q > kInt32Max - 512 || N_kv > kInt32Max - 512) return FA_ERR_UNSUPPORTED;
    const int64_t blocks = mul(B * H_kv, (N_kv + 255) / 256), steps = mul(H / H_kv, (N_q + 127) / 128);
    if (blocks < 0 || blocks > kInt32Max / 8 || steps < 0 || steps > kInt32Max / 8) return FA_ERR_UNSUPPORTED;
    if (misaligned(q, 16) || misaligned(k, 16) || misaligned(lse, 4) || misaligned(weight_in, 4) ||
        misaligned(weight_out, 4))
        return FA_ERR_ALIGNMENT;
    const Span out{weight_out, static_cast<size_t>((B * H_kv - 1) * stride + N_kv) * 4}, in{weight_in, out.n};
    const Span sq{q, static_cast<size_t>(qn) * 2}, sk{k, static_cast<size_t>(kn) * 2};
    const Span sl{lse, static_cast<size_t>(B * H * N_q) * 4};
    if (meet(out, sq) || meet(out, sk) || meet(out, sl)) return FA_ERR_INVALID_ARG;
    if (weight_in != weight_out && meet(in, out)) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

}  // namespace

extern "C" {

int fa_kv4_append_validate(const fa_kv4_cache_t* cache, const void* k, const void* v, int64_t n, int dtype,
                           const int32_t* counts_out) {
    return validate_append(cache, k, v, n, dtype, counts_out);
}

int fa_kv4_append(const fa_kv4_cache_t* cache, const void* k, const void* v, int64_t n, int dtype,
                  int32_t* counts_out, void* stream) {
    int st = validate_append(cache, k, v, n, dtype, counts_out);
    if (st != FA_OK) return st;
    fa::Kv4AppendParams p{};
    p.status = device_status_words(&st);
    if (st != FA_OK) return st;
    p.c = device_cache(*cache);
    p.x[0] = k;
    p.x[1] = v;
    p.counts_out = counts_out;
    p.n = n;
    p.f16 = dtype == FA_DTYPE_F16;
    return launched(fa::launch_kv4_append(p, static_cast<cudaStream_t>(stream)), "fa_kv4_append launch");
}

int fa_kv4_read_validate(const fa_kv4_cache_t* cache, const int32_t* first, int64_t count, const void* k,
                         const void* v, int dtype) {
    return validate_read(cache, first, count, k, v, dtype);
}

int fa_kv4_read(const fa_kv4_cache_t* cache, const int32_t* first, int64_t count, void* k, void* v, int dtype,
                void* stream) {
    const int st = validate_read(cache, first, count, k, v, dtype);
    if (st != FA_OK) return st;
    fa::Kv4ReadParams p{};
    p.c = device_cache(*cache);
    p.first = first;
    p.x[0] = k;
    p.x[1] = v;
    p.count = count;
    p.f16 = dtype == FA_DTYPE_F16;
    return launched(fa::launch_kv4_read(p, static_cast<cudaStream_t>(stream)), "fa_kv4_read launch");
}

size_t fa_kv4_fwd_workspace_size(int64_t B, int64_t H, int64_t H_kv, int64_t N_q, int64_t capacity, int64_t d,
                                 int with_weight) {
    FwdLayout l;
    return fwd_layout(B, H, H_kv, N_q, capacity, d, with_weight != 0, sm_count(), &l) ? l.bytes : 0;
}

int fa_kv4_fwd_validate(const fa_kv4_cache_t* cache, const void* q, const void* o, const float* lse,
                        const float* weight_out, int64_t H, int64_t N_q, float scale, int dtype,
                        const void* workspace, size_t workspace_bytes) {
    FwdLayout l;
    return validate_fwd(cache, q, o, lse, weight_out, H, N_q, scale, dtype, workspace, workspace_bytes, sm_count(), &l);
}

int fa_kv4_fwd(const fa_kv4_cache_t* cache, const void* q, void* o, float* lse, float* weight_out, int64_t H,
               int64_t N_q, float scale, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    FwdLayout l;
    int st = validate_fwd(cache, q, o, lse, weight_out, H, N_q, scale, dtype, workspace, workspace_bytes, sm_count(),
                          &l);
    if (st != FA_OK) return st;
    fa::Kv4FwdParams p{};
    p.status = device_status_words(&st);
    if (st != FA_OK) return st;
    p.gen = next_generation();
    p.c = device_cache(*cache);
    p.q = q;
    p.o = o;
    p.lse = lse;
    p.weight_in = cache->weight;
    p.weight_out = weight_out;
    p.Nq = static_cast<int>(N_q);
    p.group = static_cast<int>(H / cache->H_kv);
    p.rows = p.Nq * p.group;
    const int rpb = fa::kv4_rows_per_block(p.rows);
    p.row_blocks = (p.rows + rpb - 1) / rpb;
    p.causal = (dtype & FA_FLAG_CAUSAL) != 0;
    p.f16 = (dtype & 0xFF) == FA_DTYPE_F16;
    p.scale_log2 = scale * kLog2e;
    p.ctas = l.plan.ctas;
    p.single = l.plan.single ? 1 : 0;
    p.unit_cost = l.plan.unit_cost;
    p.join_warps = l.plan.join_warps;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.row_lse2 = reinterpret_cast<float*>(ws);
    p.part_ml = reinterpret_cast<float4*>(ws + l.part_ml);
    p.part_o = reinterpret_cast<float*>(ws + l.part_o);
    p.logits = weight_out != nullptr ? reinterpret_cast<float*>(ws + l.logits) : nullptr;
    return launched(fa::launch_kv4_fwd(p, static_cast<cudaStream_t>(stream)), "fa_kv4_fwd launch");
}

int fa_kv4_evict_validate(const fa_kv4_cache_t* cache, int64_t keep, int64_t sinks, int64_t recent,
                          const float* rank_by, const fa_kv4_cache_t* to, const int32_t* src,
                          const int32_t* counts_out) {
    return validate_evict(cache, keep, sinks, recent, rank_by, to, src, counts_out);
}

int fa_kv4_evict(const fa_kv4_cache_t* cache, int64_t keep, int64_t sinks, int64_t recent, const float* rank_by,
                 const fa_kv4_cache_t* to, int32_t* src, int32_t* counts_out, void* stream) {
    const int st = validate_evict(cache, keep, sinks, recent, rank_by, to, src, counts_out);
    if (st != FA_OK) return st;
    fa::Kv4EvictParams p{};
    p.from = device_cache(*cache);
    p.to = to != nullptr ? device_cache(*to) : p.from;
    p.rank_by = rank_by != nullptr ? rank_by : cache->weight;
    p.src = src;
    p.counts_out = counts_out;
    p.keep = static_cast<int>(keep);
    p.sinks = static_cast<int>(sinks);
    p.recent = static_cast<int>(recent);
    return launched(fa::launch_kv4_evict(p, static_cast<cudaStream_t>(stream)), "fa_kv4_evict launch");
}

int fa_fwd_weights_validate(const void* q, const void* k, const float* lse, const float* weight_in,
                            const float* weight_out, int64_t weight_stride, int64_t B, int64_t H, int64_t H_kv,
                            int64_t N_q, int64_t N_kv, int64_t d, int64_t first_query, float scale, int dtype) {
    return validate_weights(q, k, lse, weight_in, weight_out, weight_stride, B, H, H_kv, N_q, N_kv, d, first_query,
                            scale, dtype);
}

int fa_fwd_weights(const void* q, const void* k, const float* lse, const float* weight_in, float* weight_out,
                   int64_t weight_stride, int64_t B, int64_t H, int64_t H_kv, int64_t N_q, int64_t N_kv, int64_t d,
                   int64_t first_query, float scale, int dtype_arg, void* stream) {
    int st = validate_weights(q, k, lse, weight_in, weight_out, weight_stride, B, H, H_kv, N_q, N_kv, d, first_query,
                              scale, dtype_arg);
    if (st != FA_OK) return st;
    const int dtype = dtype_arg & 0xFF;
    CUtensorMap mq, mk;
    if ((st = encode_map(&mq, q, dtype, B * H, N_q, d)) != FA_OK) return st;
    if ((st = encode_map(&mk, k, dtype, B * H_kv, N_kv, d)) != FA_OK) return st;
    fa::WeightsParams p{};
    p.status = device_status_words(&st);
    if (st != FA_OK) return st;
    p.gen = next_generation();
    p.lse = lse;
    p.weight_in = weight_in;
    p.weight_out = weight_out;
    p.weight_stride = weight_stride;
    p.Nq = static_cast<int>(N_q);
    p.Nkv = static_cast<int>(N_kv);
    p.H = static_cast<int>(H);
    p.H_kv = static_cast<int>(H_kv);
    p.group = static_cast<int>(H / H_kv);
    p.first_query = static_cast<int>(first_query);
    p.causal = (dtype_arg & FA_FLAG_CAUSAL) != 0;
    p.causal_offset = static_cast<int>(N_kv - N_q);
    p.scale_log2 = scale * kLog2e;
    const int64_t items = B * H_kv * ((N_kv + 255) / 256);
    const int64_t steps = (H / H_kv) * ((N_q - first_query + 127) / 128);
    // CTAs that share a key block: as many as leave no SM idle, two steps each
    p.splits = 1;
    const int sms = sm_count();
    while (p.splits < 8 && 2 * p.splits * items <= sms && 4 * p.splits <= steps) p.splits *= 2;
    return launched(fa::launch_weights(static_cast<int>(d), dtype == FA_DTYPE_F16, mq, mk, p,
                                       static_cast<unsigned int>(items * p.splits), static_cast<cudaStream_t>(stream)),
                    "fa_fwd_weights launch");
}

}  // extern "C"
