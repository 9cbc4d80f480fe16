// C-ABI entry points of attention over packed sequences (declared in
// include/fa.h): argument checks, tensor maps, workspace layout and launches.
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <utility>

#include "fa.h"
#include "fa_host.h"
#include "fa_packed.cuh"
#include "fa_packed.h"
#include "fa_views.h"

using namespace fa::host;

namespace {

constexpr int64_t kInt32Max = 2147483647;

struct Sizes {
    int64_t B, Tq, Tk, H, H_kv, d;
};

int check_sizes(const Sizes& z, float scale, int dtype_arg) {
    if (z.B < 1 || z.Tq < 0 || z.Tk < 0 || z.H < 1 || z.H_kv < 1 || z.d < 1 || z.H % z.H_kv != 0) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || (dtype_arg & ~(0xFF | FA_FLAG_CAUSAL))) return FA_ERR_INVALID_ARG;
    const int dtype = dtype_arg & 0xFF;
    if (dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_F16) return FA_ERR_UNSUPPORTED;
    if (z.d != 64 && z.d != 128) return FA_ERR_UNSUPPORTED;
    if (z.B > kInt32Max / 256 || z.Tq > kInt32Max || z.Tk > kInt32Max || z.Tq + 128 * z.B + 256 > kInt32Max || z.Tk + 128 * z.B + 256 > kInt32Max)
        return FA_ERR_UNSUPPORTED;
    // grids: a block of rows per head (blockIdx.y is a head in the backward's small kernels)
    if (z.H > 65535 || z.H * ((z.Tq + z.Tk) / 128 + z.B + 2) > kInt32Max) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

int check_offsets(const int32_t* cu_q, const int32_t* cu_k, const float* lse, bool need_lse) {
    if (cu_q == nullptr || cu_k == nullptr || (need_lse && lse == nullptr)) return FA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(cu_q) | reinterpret_cast<uintptr_t>(cu_k) | reinterpret_cast<uintptr_t>(lse)) & 3u)
        return FA_ERR_ALIGNMENT;
    return FA_OK;
}

// Views of a call: q, o, dout, dq by queries and k, v, dk, dv by keys.
struct Fwd {
    View q, k, v, o;
};
struct Bwd {
    View q, k, v, o, dout, dq, dk, dv;
};

int check_fwd(const fa_rows_t* q, const fa_rows_t* k, const fa_rows_t* v, const fa_rows_t* o, const float* lse,
              const int32_t* cu_q, const int32_t* cu_k, const Sizes& z, float scale, int dtype, Fwd* out) {
    int st = check_sizes(z, scale, dtype);
    if (st == FA_OK) st = check_offsets(cu_q, cu_k, lse, false);
    if (st == FA_OK) st = make_view(q, z.Tq, z.H, z.d, &out->q);
    if (st == FA_OK) st = make_view(k, z.Tk, z.H_kv, z.d, &out->k);
    if (st == FA_OK) st = make_view(v, z.Tk, z.H_kv, z.d, &out->v);
    if (st == FA_OK) st = make_view(o, z.Tq, z.H, z.d, &out->o);
    if (st != FA_OK) return st;
    const size_t lse_bytes = static_cast<size_t>(z.H) * static_cast<size_t>(z.Tq) * 4;
    const size_t cu_bytes = static_cast<size_t>(z.B + 1) * 4;
    for (const View* in : {&out->q, &out->k, &out->v})
        if (!disjoint(out->o, *in) || meets(*in, lse, lse_bytes)) return FA_ERR_INVALID_ARG;
    if (meets(out->o, lse, lse_bytes) || meets(out->o, cu_q, cu_bytes) || meets(out->o, cu_k, cu_bytes))
        return FA_ERR_INVALID_ARG;
    if (lse != nullptr && lse_bytes > 0 && (overlaps(lse, lse_bytes, cu_q, cu_bytes) || overlaps(lse, lse_bytes, cu_k, cu_bytes)))
        return FA_ERR_INVALID_ARG;
    return FA_OK;
}

int64_t pad_tiles(const Sizes& z) { return z.Tq / 128 + z.B; }

// Workspace: 128 bytes to align by, the row statistics, the dQ accumulator.
struct Layout {
    size_t stats, acc, total;
};
Layout layout(const Sizes& z) {
    Layout l;
    const size_t tiles = static_cast<size_t>(z.H) * static_cast<size_t>(pad_tiles(z));
    l.stats = 0;
    l.acc = l.stats + tiles * fa::kStatFloatsPerTile * sizeof(float);
    l.total = l.acc + tiles * 128 * static_cast<size_t>(z.d) * sizeof(float) + 128;
    return l;
}

int check_bwd(const fa_rows_t* q, const fa_rows_t* k, const fa_rows_t* v, const fa_rows_t* o, const fa_rows_t* dout,
              const float* lse, const fa_rows_t* dq, const fa_rows_t* dk, const fa_rows_t* dv, const int32_t* cu_q,
              const int32_t* cu_k, const Sizes& z, float scale, int dtype, const void* ws, size_t ws_bytes, Bwd* out) {
    int st = check_sizes(z, scale, dtype);
    if (st == FA_OK) st = check_offsets(cu_q, cu_k, lse, z.Tq > 0);
    const struct {
        const fa_rows_t* in;
        View* out;
        bool of_q;
    } views[8] = {{q, &out->q, true},       {k, &out->k, false},   {v, &out->v, false},   {o, &out->o, true},
                  {dout, &out->dout, true}, {dq, &out->dq, true}, {dk, &out->dk, false}, {dv, &out->dv, false}};
    for (const auto& w : views)
        if (st == FA_OK) st = make_view(w.in, w.of_q ? z.Tq : z.Tk, w.of_q ? z.H : z.H_kv, z.d, w.out);
    if (st != FA_OK) return st;
    if (ws == nullptr) return FA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(ws) & 15u) return FA_ERR_ALIGNMENT;
    const size_t need = layout(z).total;
    if (ws_bytes < need) return FA_ERR_INVALID_ARG;
    const size_t lse_bytes = static_cast<size_t>(z.H) * static_cast<size_t>(z.Tq) * 4;
    const size_t cu_bytes = static_cast<size_t>(z.B + 1) * 4;
    for (int i = 0; i < 8; ++i) {
        if (meets(*views[i].out, ws, need)) return FA_ERR_INVALID_ARG;
        if (i < 5) continue;
        for (int j = 0; j < i; ++j)
            if (!disjoint(*views[i].out, *views[j].out)) return FA_ERR_INVALID_ARG;
        if (meets(*views[i].out, lse, lse_bytes) || meets(*views[i].out, cu_q, cu_bytes) ||
            meets(*views[i].out, cu_k, cu_bytes))
            return FA_ERR_INVALID_ARG;
    }
    if ((lse_bytes > 0 && overlaps(ws, need, lse, lse_bytes)) || overlaps(ws, need, cu_q, cu_bytes) ||
        overlaps(ws, need, cu_k, cu_bytes))
        return FA_ERR_INVALID_ARG;
    return FA_OK;
}

int map_of(CUtensorMap* m, const View& v, int dtype) {
    const int64_t dims[3] = {v.d, v.rows, v.heads}, strides[3] = {1, v.row, v.head};
    const uint32_t box[3] = {64, 128, 1};
    return encode_strided(m, v.data, dtype, 3, dims, strides, box);
}

fa::PackedSeqs seqs_of(const Sizes& z, const int32_t* cu_q, const int32_t* cu_k, int dtype_arg) {
    fa::PackedSeqs s{};
    s.cu_q = cu_q;
    s.cu_k = cu_k;
    s.B = static_cast<int>(z.B);
    s.Tq = static_cast<int>(z.Tq);
    s.Tk = static_cast<int>(z.Tk);
    s.causal = (dtype_arg & FA_FLAG_CAUSAL) ? 1 : 0;
    s.max_level = static_cast<int>(((z.Tq > z.Tk ? z.Tq : z.Tk) + 127) / 128 + 2);
    return s;
}

int cuda_failed(const char* what, cudaError_t e) {
    set_error(what, static_cast<int>(e), cudaGetErrorString(e));
    return FA_ERR_CUDA;
}

}  // namespace

extern "C" {

int fa_packed_fwd_validate(const fa_rows_t* q, const fa_rows_t* k, const fa_rows_t* v, const fa_rows_t* o,
                           const float* lse, const int32_t* cu_q, const int32_t* cu_k, int64_t B, int64_t T_q,
                           int64_t T_k, int64_t H, int64_t H_kv, int64_t d, float scale, int dtype) {
    Fwd w;
    return check_fwd(q, k, v, o, lse, cu_q, cu_k, Sizes{B, T_q, T_k, H, H_kv, d}, scale, dtype, &w);
}

int fa_packed_fwd(const fa_rows_t* q, const fa_rows_t* k, const fa_rows_t* v, const fa_rows_t* o, float* lse,
                  const int32_t* cu_q, const int32_t* cu_k, int64_t B, int64_t T_q, int64_t T_k, int64_t H,
                  int64_t H_kv, int64_t d, float scale, int dtype_arg, void* stream) {
    const Sizes z{B, T_q, T_k, H, H_kv, d};
    Fwd w;
    int st = check_fwd(q, k, v, o, lse, cu_q, cu_k, z, scale, dtype_arg, &w);
    if (st != FA_OK || T_q == 0) return st;
    const int dtype = dtype_arg & 0xFF;
    CUtensorMap mq, mk, mv;
    if ((st = map_of(&mq, w.q, dtype)) != FA_OK) return st;
    mk = mv = mq;  // (no keys: not used)
    if (T_k > 0 && ((st = map_of(&mk, w.k, dtype)) != FA_OK || (st = map_of(&mv, w.v, dtype)) != FA_OK)) return st;
    fa::PackedFwdParams p{};
    p.status = device_status_words(&st);
    if (st != FA_OK) return st;
    p.gen = next_generation();
    p.lse = lse;
    p.out = w.o.data;
    p.o_row = w.o.row;
    p.o_head = w.o.head;
    p.seqs = seqs_of(z, cu_q, cu_k, dtype_arg);
    p.H = static_cast<int>(H);
    p.H_kv = static_cast<int>(H_kv);
    p.group = static_cast<int>(H / H_kv);
    p.splits = 1;
    p.n_q_blocks = 1;
    p.causal = p.seqs.causal;
    // masked scores are -inf, so a scale of 0 becomes one that makes every other score 0
    p.scale_log2 = std::fmax(std::fabs(scale) * 1.4426950408889634f, 1.17549435e-38f);
    p.negate = scale < 0.0f ? 1 : 0;
    // Groups of an even number of heads: the CTA's two tiles are the same rows of two heads, which see the same keys
    // (a block of 256 rows runs its first tile through keys only the second sees) and leave fewer rows empty: 16 ragged
    // prompts (H = 32/8, causal) 143 us against 169 at d = 128 and 98 against 114 at d = 64, up to 16384 rows 2036
    // against 2056 and 1282 against 1293, 16 of 512 without the mask 74 against 74 and 51 against 51, 64 of 128 54
    // against 82 and 42 against 74; slower only for 100 of 240 rows, causal, d = 128 (200 against 167; 122, 137 at d = 64).
    const bool pairs = p.group % 2 == 0;
    p.head_step = pairs ? 1 : 0;
    p.tile_step = pairs ? 0 : 128;
    p.units = static_cast<int>(pairs ? H / 2 : H);
    const int64_t rows = pairs ? 128 : 256;
    const unsigned int grid = static_cast<unsigned int>((T_q / rows + B) * p.units);
    const cudaError_t e = dtype == FA_DTYPE_BF16
                              ? fa::launch_packed_fwd_bf16(static_cast<int>(d), mq, mk, mv, p, grid, static_cast<cudaStream_t>(stream))
                              : fa::launch_packed_fwd_f16(static_cast<int>(d), mq, mk, mv, p, grid, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? FA_OK : cuda_failed("packed forward launch", e);
}

size_t fa_packed_bwd_workspace_size(int64_t B, int64_t T_q, int64_t H, int64_t d) {
    const Sizes z{B, T_q, 0, H, 1, d};
    return check_sizes(z, 1.0f, FA_DTYPE_BF16) == FA_OK ? layout(z).total : 0;
}

int fa_packed_bwd_validate(const fa_rows_t* q, const fa_rows_t* k, const fa_rows_t* v, const fa_rows_t* o,
                           const fa_rows_t* dout, const float* lse, const fa_rows_t* dq, const fa_rows_t* dk,
                           const fa_rows_t* dv, const int32_t* cu_q, const int32_t* cu_k, int64_t B, int64_t T_q,
                           int64_t T_k, int64_t H, int64_t H_kv, int64_t d, float scale, int dtype,
                           const void* workspace, size_t workspace_bytes) {
    Bwd w;
    return check_bwd(q, k, v, o, dout, lse, dq, dk, dv, cu_q, cu_k, Sizes{B, T_q, T_k, H, H_kv, d}, scale, dtype,
                     workspace, workspace_bytes, &w);
}

int fa_packed_bwd(const fa_rows_t* q, const fa_rows_t* k, const fa_rows_t* v, const fa_rows_t* o,
                  const fa_rows_t* dout, const float* lse, const fa_rows_t* dq, const fa_rows_t* dk,
                  const fa_rows_t* dv, const int32_t* cu_q, const int32_t* cu_k, int64_t B, int64_t T_q,
                  int64_t T_k, int64_t H, int64_t H_kv, int64_t d, float scale, int dtype_arg, void* workspace,
                  size_t workspace_bytes, void* stream) {
    const Sizes z{B, T_q, T_k, H, H_kv, d};
    Bwd w;
    int st = check_bwd(q, k, v, o, dout, lse, dq, dk, dv, cu_q, cu_k, z, scale, dtype_arg, workspace, workspace_bytes, &w);
    if (st != FA_OK || (T_q == 0 && T_k == 0)) return st;
    const int dtype = dtype_arg & 0xFF;
    const bool f16 = dtype == FA_DTYPE_F16;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Layout l = layout(z);
    char* ws = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(workspace) + 127) & ~uintptr_t{127});
    fa::PackedAuxParams a{};
    a.seqs = seqs_of(z, cu_q, cu_k, dtype_arg);
    a.H = static_cast<int>(H);
    a.tiles = static_cast<int>(pad_tiles(z));
    a.o = reinterpret_cast<const uint16_t*>(w.o.data);
    a.dout = reinterpret_cast<const uint16_t*>(w.dout.data);
    a.o_row = w.o.row;
    a.o_head = w.o.head;
    a.dout_row = w.dout.row;
    a.dout_head = w.dout.head;
    a.lse = lse;
    a.stats = reinterpret_cast<float*>(ws + l.stats);
    a.dq_acc = reinterpret_cast<float*>(ws + l.acc);
    a.dq = reinterpret_cast<uint16_t*>(w.dq.data);
    a.dq_row = w.dq.row;
    a.dq_head = w.dq.head;
    a.scale = scale;
    cudaError_t e = cudaSuccess;
    if (T_q > 0) e = fa::launch_packed_prep(a, static_cast<int>(d), f16, s);
    if (e != cudaSuccess) return cuda_failed("packed backward prep launch", e);
    if (T_k > 0) {
        fa::PackedMaps m{};
        if ((st = encode_map(&m.dq, a.dq_acc, FA_DTYPE_F32, H, int64_t{128} * a.tiles, d)) != FA_OK) return st;
        const std::pair<CUtensorMap*, const View*> maps[6] = {{&m.k, &w.k},   {&m.v, &w.v}, {&m.dk, &w.dk},
                                                              {&m.dv, &w.dv}, {&m.q, &w.q}, {&m.dout, &w.dout}};
        for (const auto& x : maps) {
            if (x.second->rows > 0) st = map_of(x.first, *x.second, dtype);
            else *x.first = m.k;  // (no queries: not used)
            if (st != FA_OK) return st;
        }
        fa::PackedBwdParams p{};
        p.status = device_status_words(&st);
        if (st != FA_OK) return st;
        p.gen = next_generation();
        p.stats = a.stats;
        p.Nq_pad = 128 * a.tiles;
        p.n_kv_blocks = 1;
        p.H = static_cast<int>(H);
        p.H_kv = static_cast<int>(H_kv);
        p.group = static_cast<int>(H / H_kv);
        p.causal = a.seqs.causal;
        p.scale_log2 = scale * 1.4426950408889634f;
        p.scale = scale;
        p.seqs = a.seqs;
        p.tiles = a.tiles;
        p.dk = reinterpret_cast<uint16_t*>(w.dk.data);
        p.dv = reinterpret_cast<uint16_t*>(w.dv.data);
        p.dk_row = w.dk.row;
        p.dk_head = w.dk.head;
        p.dv_row = w.dv.row;
        p.dv_head = w.dv.head;
        const unsigned int grid = static_cast<unsigned int>((T_k / 128 + B) * H_kv);
        e = f16 ? fa::launch_packed_bwd_f16(static_cast<int>(d), m, p, grid, s)
                : fa::launch_packed_bwd_bf16(static_cast<int>(d), m, p, grid, s);
        if (e != cudaSuccess) return cuda_failed("packed backward launch", e);
    }
    if (T_q > 0) {
        e = fa::launch_packed_dq(a, static_cast<int>(d), f16, s);
        if (e != cudaSuccess) return cuda_failed("packed backward dQ conversion launch", e);
    }
    return FA_OK;
}

}  // extern "C"
