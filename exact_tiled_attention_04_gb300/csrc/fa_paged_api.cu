// C-ABI entry points of the paged key/value cache (declared in include/fa.h):
// argument checks, tensor maps, workspace layout and launches.
#include <atomic>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "fa.h"
#include "fa_host.h"
#include "fa_paged.h"
#include "fa_views.h"

using namespace fa::host;

namespace {

constexpr int64_t kInt32Max = 2147483647;
constexpr int64_t kMaxRowsPerHead = 128;  // fa_paged_fwd: N_q * H / H_kv
constexpr int kMaxPrefixSplits = 64;

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// a * b, or -1 past 2^62 (-1 passes through)
int64_t mul(int64_t a, int64_t b) {
    if (a < 0 || b < 0) return -1;
    if (b != 0 && a > (int64_t(1) << 62) / b) return -1;
    return a * b;
}

size_t pool_bytes(const fa_paged_cache_t& c) {
    return static_cast<size_t>(c.num_pages * c.H_kv * c.page_size * c.d) * 2;
}

struct Span {
    const void* p;
    size_t n;
};
bool meet(const Span& a, const Span& b) {
    return a.p != nullptr && b.p != nullptr && a.n > 0 && b.n > 0 && overlaps(a.p, a.n, b.p, b.n);
}
// The arrays of a cache: k_pages, v_pages, block_table, lengths.
constexpr int kArrays = 4;
void cache_spans(const fa_paged_cache_t& c, Span (&s)[kArrays]) {
    s[0] = {c.k_pages, pool_bytes(c)};
    s[1] = {c.v_pages, pool_bytes(c)};
    s[2] = {c.block_table, static_cast<size_t>(c.B * c.max_pages) * 4};
    s[3] = {c.lengths, static_cast<size_t>(c.B) * 4};
}
bool meets_cache(const Span& x, const fa_paged_cache_t& c, int arrays = kArrays) {
    Span s[kArrays];
    cache_spans(c, s);
    for (int i = 0; i < arrays; ++i)
        if (meet(x, s[i])) return true;
    return false;
}

int check_cache(const fa_paged_cache_t* c) {
    if (c == nullptr || !c->k_pages || !c->v_pages || !c->block_table || !c->lengths) return FA_ERR_INVALID_ARG;
    if (c->B < 1 || c->H_kv < 1 || c->d < 1 || c->num_pages < 1 || c->max_pages < 1 || c->page_size < 1)
        return FA_ERR_INVALID_ARG;
    if (c->d != 64 && c->d != 128) return FA_ERR_UNSUPPORTED;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return FA_ERR_UNSUPPORTED;
    if (mul(mul(mul(c->num_pages, c->H_kv), c->page_size), 2 * c->d) < 0 || mul(c->B, mul(c->max_pages, 4)) < 0)
        return FA_ERR_INVALID_ARG;
    if (c->num_pages > kInt32Max || c->max_pages > (kInt32Max - 128) / c->page_size || c->B > kInt32Max / 256 ||
        c->H_kv > 65535 || c->H_kv > kInt32Max / c->page_size)
        return FA_ERR_UNSUPPORTED;
    if (misaligned(c->k_pages, 16) || misaligned(c->v_pages, 16) || misaligned(c->block_table, 4) || misaligned(c->lengths, 4))
        return FA_ERR_ALIGNMENT;
    Span s[kArrays];
    cache_spans(*c, s);
    for (int i = 0; i < kArrays; ++i)
        for (int j = i + 1; j < kArrays; ++j)
            if (meet(s[i], s[j])) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

fa::PagedCache device_cache(const fa_paged_cache_t& c) {
    fa::PagedCache k{};
    k.pages[0] = static_cast<uint16_t*>(c.k_pages);
    k.pages[1] = static_cast<uint16_t*>(c.v_pages);
    k.table = c.block_table;
    k.lengths = c.lengths;
    k.num_pages = static_cast<int>(c.num_pages);
    k.page = static_cast<int>(c.page_size);
    k.B = static_cast<int>(c.B);
    k.max_pages = static_cast<int>(c.max_pages);
    k.H_kv = static_cast<int>(c.H_kv);
    k.d = static_cast<int>(c.d);
    k.capacity = static_cast<int>(c.max_pages * c.page_size);
    return k;
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

int cuda_failed(const char* what, cudaError_t e) {
    set_error(what, static_cast<int>(e), cudaGetErrorString(e));
    return FA_ERR_CUDA;
}

// --------------------------------------------------------------- append
struct AppendArgs {
    const fa_paged_cache_t* cache;
    const fa_rows_t *k, *v;
    const int32_t* cu;
    int64_t T;
    const fa_rows_t *q, *q_out;
    int64_t H;
    const fa_rows_t* k_out;
    const float* table;
    int64_t table_rows, rot;
    const int32_t* positions;
    int64_t first_position;
    int32_t* lengths_out;
    int dtype;
};
struct AppendViews {
    View k{}, v{}, q{}, q_out{}, k_out{};
};

bool same_view(const View& a, const View& b) { return a.data == b.data && a.row == b.row && a.head == b.head; }

int check_append(const AppendArgs& a, AppendViews* w) {
    int st = check_cache(a.cache);
    if (st != FA_OK) return st;
    const fa_paged_cache_t& c = *a.cache;
    if (a.lengths_out == nullptr || a.T < 0) return FA_ERR_INVALID_ARG;
    if ((a.q == nullptr) != (a.q_out == nullptr)) return FA_ERR_INVALID_ARG;
    if (a.dtype & ~(0xFF | FA_FLAG_INTERLEAVED)) return FA_ERR_INVALID_ARG;
    if ((st = check_dtype16(a.dtype & 0xFF)) != FA_OK) return st;
    if (a.T > kInt32Max - 256) return FA_ERR_UNSUPPORTED;
    if (a.cu == nullptr && a.T % c.B != 0) return FA_ERR_INVALID_ARG;
    if (a.q != nullptr && (a.H < 1 || a.H > 65535)) return FA_ERR_INVALID_ARG;
    if ((st = make_view(a.k, a.T, c.H_kv, c.d, &w->k)) != FA_OK) return st;
    if ((st = make_view(a.v, a.T, c.H_kv, c.d, &w->v)) != FA_OK) return st;
    if (a.q != nullptr) {
        if ((st = make_view(a.q, a.T, a.H, c.d, &w->q)) != FA_OK) return st;
        if ((st = make_view(a.q_out, a.T, a.H, c.d, &w->q_out)) != FA_OK) return st;
    }
    if (a.k_out != nullptr && (st = make_view(a.k_out, a.T, c.H_kv, c.d, &w->k_out)) != FA_OK) return st;
    if (a.table != nullptr) {
        if (a.table_rows < 1 || a.rot < 16 || a.rot > c.d || a.rot % 16 != 0) return FA_ERR_INVALID_ARG;
        if (mul(a.table_rows, a.rot * 4) < 0) return FA_ERR_INVALID_ARG;
        if (misaligned(a.table, 16)) return FA_ERR_ALIGNMENT;
        // positions are sums with slots in 64 bits
        if (a.first_position < -(int64_t{1} << 40) || a.first_position > (int64_t{1} << 40)) return FA_ERR_INVALID_ARG;
    } else if (a.positions != nullptr) {
        return FA_ERR_INVALID_ARG;  // nothing to turn by them
    }
    if (misaligned(a.cu, 4) || misaligned(a.positions, 4) || misaligned(a.lengths_out, 4)) return FA_ERR_ALIGNMENT;
    const Span lengths{a.lengths_out, static_cast<size_t>(c.B) * 4};
    const Span plain[3] = {{a.cu, static_cast<size_t>(c.B + 1) * 4},
                           {a.table, static_cast<size_t>(a.table_rows * a.rot) * 4},
                           {a.positions, static_cast<size_t>(a.T) * 4}};
    // what is written (pages, q_out, k_out, lengths) meets nothing else, but q_out may be q and k_out k
    const View* in[3] = {&w->k, &w->v, &w->q};
    const View* out[2] = {&w->q_out, &w->k_out};
    for (const View* x : in)
        if (x->rows > 0 && (meets_cache({x->data, x->span()}, c, 2) || meets(*x, lengths.p, lengths.n))) return FA_ERR_INVALID_ARG;
    for (int i = 0; i < 2; ++i) {
        if (out[i]->rows == 0) continue;
        if (meets_cache({out[i]->data, out[i]->span()}, c) || meets(*out[i], lengths.p, lengths.n)) return FA_ERR_INVALID_ARG;
        for (const View* x : in)
            if (!disjoint(*out[i], *x) && !(x == (i == 0 ? &w->q : &w->k) && same_view(*out[i], *x))) return FA_ERR_INVALID_ARG;
        for (const Span& s : plain)
            if (meets(*out[i], s.p, s.n)) return FA_ERR_INVALID_ARG;
    }
    if (!disjoint(w->q_out, w->k_out)) return FA_ERR_INVALID_ARG;
    for (const Span& s : plain)
        if (meets_cache(s, c, 2) || meet(s, lengths)) return FA_ERR_INVALID_ARG;
    if (meets_cache(lengths, c, 3)) return FA_ERR_INVALID_ARG;
    if (a.lengths_out != c.lengths && meet(lengths, {c.lengths, static_cast<size_t>(c.B) * 4})) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

fa::RowsView device_view(const View& v) { return {reinterpret_cast<uint16_t*>(v.data), v.row, v.head}; }

// -------------------------------------------------------------- attention
struct FwdSizes {
    int64_t B, H, H_kv, N_q, capacity, d, prefix;
};

bool sizes_fit(const FwdSizes& z) {
    if (z.B < 1 || z.H < 1 || z.H_kv < 1 || z.N_q < 1 || z.capacity < 1 || z.prefix < 0) return false;
    if (z.H % z.H_kv != 0 || (z.d != 64 && z.d != 128)) return false;
    if (z.N_q > kMaxRowsPerHead || z.H / z.H_kv > kMaxRowsPerHead || z.N_q * (z.H / z.H_kv) > kMaxRowsPerHead) return false;
    if (z.B > kInt32Max / 256 || z.H > (1 << 24) || z.capacity > kInt32Max - 128 || z.prefix > kInt32Max - 128) return false;
    // tiles of all units, and rows of all heads, in 31 bits
    const int64_t blocks = (z.N_q * (z.H / z.H_kv) + 31) / 32;
    const int64_t units = mul(z.B, z.H_kv * blocks);
    const int64_t tiles = mul(units, (z.capacity + 127) / 128 + 1);
    return tiles >= 0 && tiles < kInt32Max - 65536 && mul(mul(z.B, z.H), z.N_q) < kInt32Max;
}

// The launches of a call and where their workspace lies.
struct FwdPlan {
    int rows, row_blocks, rows_per_block, ctas;
    int prefix_seqs, prefix_blocks, prefix_splits, prefix_tiles;  // tiles per partition
    size_t part_ml, unit_o, prefix_ml, prefix_o, total;           // bytes
};

FwdPlan plan_fwd(const FwdSizes& z, int sms) {
    FwdPlan p{};
    p.rows = static_cast<int>(z.N_q * (z.H / z.H_kv));
    p.rows_per_block = fa::paged_rows_per_block(p.rows);
    p.row_blocks = (p.rows + p.rows_per_block - 1) / p.rows_per_block;
    const int64_t units = z.B * z.H_kv * p.row_blocks;
    const int64_t most = units * ((z.capacity + 127) / 128);
    p.ctas = static_cast<int>(most < sms ? most : sms);
    size_t slots = static_cast<size_t>(2 * p.ctas), rows = 0;
    if (z.prefix > 0) {
        slots += static_cast<size_t>(units);
        // Two tiles of sequences a CTA where there are more than one holds (64 sequences behind a prefix of 8192 slots,
        // H = 32/8, d = 128: 42.3 us, with one 44.8), and one wave of partitions (half as many 47.2, twice 49.8).
        p.prefix_seqs = static_cast<int>(128 / p.rows);
        const int64_t per_cta = z.B <= p.prefix_seqs ? p.prefix_seqs : 2 * p.prefix_seqs;
        p.prefix_blocks = static_cast<int>((z.B + per_cta - 1) / per_cta);
        const int64_t tiles = (z.prefix + 127) / 128;
        int64_t splits = sms / (z.H_kv * p.prefix_blocks);
        splits = splits < 1 ? 1 : splits > tiles ? tiles : splits;
        if (splits > kMaxPrefixSplits) splits = kMaxPrefixSplits;
        p.prefix_tiles = static_cast<int>((tiles + splits - 1) / splits);
        p.prefix_splits = static_cast<int>((tiles + p.prefix_tiles - 1) / p.prefix_tiles);
        rows = static_cast<size_t>(p.prefix_splits) * static_cast<size_t>(z.B * z.H * z.N_q);
    }
    p.part_ml = 0;
    p.prefix_ml = slots * p.rows_per_block * 16;
    p.unit_o = p.prefix_ml + rows * 16;
    p.prefix_o = p.unit_o + slots * p.rows_per_block * static_cast<size_t>(z.d) * 4;
    p.total = p.prefix_o + rows * static_cast<size_t>(z.d) * 4;
    return p;
}

int check_fwd(const fa_paged_cache_t* cache, const void* q, const void* o, const float* lse, int64_t H, int64_t N_q,
              const int32_t* prefix_pages, int64_t prefix_length, float scale, int dtype, const void* workspace,
              size_t workspace_bytes, int sms, FwdPlan* plan) {
    int st = check_cache(cache);
    if (st != FA_OK) return st;
    const fa_paged_cache_t& c = *cache;
    if (!q || !o || !workspace || H < 1 || N_q < 1 || H % c.H_kv != 0 || prefix_length < 0) return FA_ERR_INVALID_ARG;
    if ((prefix_length > 0) != (prefix_pages != nullptr)) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || (dtype & ~(0xFF | FA_FLAG_CAUSAL))) return FA_ERR_INVALID_ARG;
    if ((st = check_dtype16(dtype & 0xFF)) != FA_OK) return st;
    const FwdSizes z{c.B, H, c.H_kv, N_q, c.max_pages * c.page_size, c.d, prefix_length};
    if (!sizes_fit(z)) return FA_ERR_UNSUPPORTED;
    if (misaligned(q, 16) || misaligned(o, 16) || misaligned(workspace, 16) || misaligned(lse, 4) || misaligned(prefix_pages, 4))
        return FA_ERR_ALIGNMENT;
    *plan = plan_fwd(z, sms);
    if (workspace_bytes < plan->total) return FA_ERR_INVALID_ARG;
    const size_t rows = static_cast<size_t>(c.B * H * N_q);
    const Span s[5] = {{q, rows * static_cast<size_t>(c.d) * 2},
                       {prefix_pages, static_cast<size_t>((prefix_length + c.page_size - 1) / c.page_size) * 4},
                       {o, rows * static_cast<size_t>(c.d) * 2},
                       {lse, rows * 4},
                       {workspace, plan->total}};
    for (int i = 2; i < 5; ++i) {  // what is written
        if (meets_cache(s[i], c)) return FA_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (meet(s[i], s[j])) return FA_ERR_INVALID_ARG;
    }
    return FA_OK;
}

}  // namespace

extern "C" {

int fa_paged_append_validate(const fa_paged_cache_t* cache, const fa_rows_t* k, const fa_rows_t* v, const int32_t* cu,
                             int64_t T, const fa_rows_t* q, const fa_rows_t* q_out, int64_t H, const fa_rows_t* k_out,
                             const float* table, int64_t table_rows, int64_t rot, const int32_t* positions,
                             int64_t first_position, const int32_t* lengths_out, int dtype) {
    AppendViews w;
    return check_append({cache, k, v, cu, T, q, q_out, H, k_out, table, table_rows, rot, positions, first_position,
                         const_cast<int32_t*>(lengths_out), dtype}, &w);
}

int fa_paged_append(const fa_paged_cache_t* cache, const fa_rows_t* k, const fa_rows_t* v, const int32_t* cu, int64_t T,
                    const fa_rows_t* q, const fa_rows_t* q_out, int64_t H, const fa_rows_t* k_out, const float* table,
                    int64_t table_rows, int64_t rot, const int32_t* positions, int64_t first_position,
                    int32_t* lengths_out, int dtype, void* stream) {
    AppendViews w;
    int st = check_append({cache, k, v, cu, T, q, q_out, H, k_out, table, table_rows, rot, positions, first_position,
                           lengths_out, dtype}, &w);
    if (st != FA_OK) return st;
    fa::PagedAppendParams p{};
    p.status = device_status_words(&st);
    if (st != FA_OK) return st;
    p.c = device_cache(*cache);
    p.k = device_view(w.k);
    p.v = device_view(w.v);
    p.q = device_view(w.q);
    p.q_out = device_view(w.q_out);
    p.k_out = device_view(w.k_out);
    p.cu = cu;
    p.table = table;
    p.rot = table != nullptr ? static_cast<int>(rot) : 0;
    p.table_rows = table_rows;
    p.positions = positions;
    p.first_position = first_position;
    p.lengths_out = lengths_out;
    p.T = T;
    p.n = cu == nullptr ? static_cast<int>(T / cache->B) : 0;
    p.H = static_cast<int>(H);
    const cudaError_t e = fa::launch_paged_append(p, sm_count(), (dtype & 0xFF) == FA_DTYPE_F16,
                                                  (dtype & FA_FLAG_INTERLEAVED) != 0, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : cuda_failed("paged append launch", e);
}

size_t fa_paged_fwd_workspace_size(int64_t B, int64_t H, int64_t H_kv, int64_t N_q, int64_t capacity, int64_t d,
                                   int64_t prefix_length) {
    const FwdSizes z{B, H, H_kv, N_q, capacity, d, prefix_length};
    if (!sizes_fit(z)) return 0;
    const int sms = sm_count();
    return plan_fwd(z, sms > 0 ? sms : 1024).total;
}

int fa_paged_fwd_validate(const fa_paged_cache_t* cache, const void* q, const void* o, const float* lse, int64_t H,
                          int64_t N_q, const int32_t* prefix_pages, int64_t prefix_length, float scale, int dtype,
                          const void* workspace, size_t workspace_bytes) {
    FwdPlan plan;
    const int sms = sm_count();
    return check_fwd(cache, q, o, lse, H, N_q, prefix_pages, prefix_length, scale, dtype, workspace, workspace_bytes,
                     sms > 0 ? sms : 1024, &plan);
}

int fa_paged_fwd(const fa_paged_cache_t* cache, const void* q, void* o, float* lse, int64_t H, int64_t N_q,
                 const int32_t* prefix_pages, int64_t prefix_length, float scale, int dtype_arg, void* workspace,
                 size_t workspace_bytes, void* stream) {
    FwdPlan plan;
    const int sms = sm_count();
    int st = check_fwd(cache, q, o, lse, H, N_q, prefix_pages, prefix_length, scale, dtype_arg, workspace, workspace_bytes,
                       sms > 0 ? sms : 1024, &plan);
    if (st != FA_OK) return st;
    if (sms <= 0) {
        set_error("cudaDevAttrMultiProcessorCount", 0, "no device answered");
        return FA_ERR_CUDA;
    }
    const fa_paged_cache_t& c = *cache;
    const int dtype = dtype_arg & 0xFF, d = static_cast<int>(c.d);
    const bool f16 = dtype == FA_DTYPE_F16;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    CUtensorMap mk, mv, mq;
    const int64_t dims[4] = {c.d, c.page_size, c.H_kv, c.num_pages};
    const int64_t strides[4] = {1, c.d, c.page_size * c.d, c.H_kv * c.page_size * c.d};
    const uint32_t box[4] = {64, static_cast<uint32_t>(c.page_size), 1, 1};
    if ((st = encode_strided(&mk, c.k_pages, dtype, 4, dims, strides, box)) != FA_OK) return st;
    if ((st = encode_strided(&mv, c.v_pages, dtype, 4, dims, strides, box)) != FA_OK) return st;
    char* ws = static_cast<char*>(workspace);
    fa::PagedFwdParams p{};
    p.status = device_status_words(&st);
    if (st != FA_OK) return st;
    p.c = device_cache(c);
    p.rows = plan.rows;
    p.row_blocks = plan.row_blocks;
    p.ctas = plan.ctas;
    p.parts_always = prefix_length > 0 ? 1 : 0;
    p.c.unwaited = p.parts_always;
    p.part_ml = reinterpret_cast<float4*>(ws + plan.part_ml);
    p.unit_o = reinterpret_cast<float*>(ws + plan.unit_o);
    p.ml_part = reinterpret_cast<float*>(ws + plan.prefix_ml);
    p.o_part = reinterpret_cast<float*>(ws + plan.prefix_o);
    p.splits = plan.prefix_splits;
    p.out = o;
    p.lse = lse;
    p.Nq = static_cast<int>(N_q);
    p.H = static_cast<int>(H);
    p.H_kv = static_cast<int>(c.H_kv);
    p.group = static_cast<int>(H / c.H_kv);
    p.causal = (dtype_arg & FA_FLAG_CAUSAL) && N_q > 1 ? 1 : 0;  // a single query sees every slot
    p.scale_log2 = scale * 1.4426950408889634f;
    if (prefix_length > 0) {
        fa::PrefixFwdParams f{};
        f.status = p.status;
        f.gen = next_generation();
        f.ml_part = p.ml_part;
        f.o_part = p.o_part;
        f.part_rows = c.B * H * N_q;
        f.Nkv = static_cast<int>(prefix_length);
        f.n_kv_tiles = static_cast<int>((prefix_length + 127) / 128);
        f.H = p.H;
        f.H_kv = p.H_kv;
        f.group = p.group;
        f.splits = plan.prefix_splits;
        f.tiles_per_split = plan.prefix_tiles;
        f.scale_log2 = std::fmax(std::fabs(p.scale_log2), 1.17549435e-38f);  // as fa_packed_fwd's
        f.negate = scale < 0.0f ? 1 : 0;
        f.pages = prefix_pages;
        f.page = p.c.page;
        f.n_pages = static_cast<int>((prefix_length + c.page_size - 1) / c.page_size);
        f.B = p.c.B;
        f.rows = plan.rows;
        f.seqs = plan.prefix_seqs;
        f.blocks = plan.prefix_blocks;
        f.pair = c.B > plan.prefix_seqs ? 1 : 0;
        const int64_t qdims[4] = {c.d, plan.rows, c.H_kv, c.B};
        const int64_t qstrides[4] = {1, c.d, plan.rows * c.d, H * N_q * c.d};
        const uint32_t qbox[4] = {64, static_cast<uint32_t>(plan.rows), 1, static_cast<uint32_t>(plan.prefix_seqs)};
        if ((st = encode_strided(&mq, q, dtype, 4, qdims, qstrides, qbox)) != FA_OK) return st;
        const cudaError_t e = f16 ? fa::launch_prefix_fwd_f16(d, mq, mk, mv, f, s) : fa::launch_prefix_fwd_bf16(d, mq, mk, mv, f, s);
        if (e != cudaSuccess) return cuda_failed("prefix launch", e);
    }
    p.gen = next_generation();
    const int64_t qdims[3] = {c.d, plan.rows, c.B * c.H_kv};
    const int64_t qstrides[3] = {1, c.d, plan.rows * c.d};
    const uint32_t qbox[3] = {64, plan.rows_per_block < 16 ? 16u : static_cast<uint32_t>(plan.rows_per_block), 1};
    if ((st = encode_strided(&mq, q, dtype, 3, qdims, qstrides, qbox)) != FA_OK) return st;
    const cudaError_t e = f16 ? fa::launch_paged_fwd_f16(mq, mk, mv, p, s) : fa::launch_paged_fwd_bf16(mq, mk, mv, p, s);
    return e == cudaSuccess ? FA_OK : cuda_failed("paged attention launch", e);
}

}  // extern "C"
