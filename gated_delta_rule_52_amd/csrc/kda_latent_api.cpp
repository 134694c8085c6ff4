// kda_latent_api.cpp - host entry points of latent attention in include/kda.h: rotary positions, the paged cache, attention
// of prompts with its gradients, and of single tokens.  As in kda_api.cpp every argument is validated before anything
// is enqueued.
#include <cmath>

#include "kda_checks.h"
#include "kda_latent.h"

namespace {

constexpr int64_t kMostRows = int64_t{1} << 30;
constexpr int64_t kAttendStride = int64_t{1} << 22;  // a tile of up to 64 rows lies within 2^30 bytes

// A [rows, heads, width] tensor.
struct Tensor {
    const char *name;
    const void *p;
    int64_t rows, heads, width, stride, head_stride;
    kda_dtype dtype;
    bool heads_inside() const { return heads <= 1 || rows <= 1 || head_stride <= stride; }
    // the memory of one row's heads, or of one head's rows
    int64_t inner() const { return heads_inside() ? (heads - 1) * head_stride + width : (rows - 1) * stride + width; }
};

kda_status check_tensor(const Tensor &t, int64_t below) {
    if (!t.p || t.rows <= 0 || t.heads <= 0) return KDA_OK;
    if (t.rows > 1) KDA_TRY(check_stride(t.name, t.p, t.stride, t.width, t.rows, below));
    if (t.heads > 1) KDA_TRY(check_stride(t.name, t.p, t.head_stride, t.width, t.heads, kAnyStride));
    if (t.rows > 1 && t.heads > 1 && t.inner() > (t.heads_inside() ? t.stride : t.head_stride))
        return fail(KDA_ERR_BAD_SHAPE, "%s: rows %lld and heads %lld apart overlap", t.name, static_cast<long long>(t.stride),
                    static_cast<long long>(t.head_stride));
    return KDA_OK;
}
kda_status check_aligned(const Tensor &t) {
    if (!t.p || t.rows <= 0) return KDA_OK;
    const int64_t e = dsize(t.dtype);
    if (reinterpret_cast<uintptr_t>(t.p) % 16 || (t.rows > 1 && t.stride * e % 16) || (t.heads > 1 && t.head_stride * e % 16))
        return fail(KDA_ERR_UNSUPPORTED, "%s: base and strides have to be multiples of 16 bytes", t.name);
    return KDA_OK;
}
// A stride that is not looked at (of one row, or one head) may hold anything: the width takes its place, as the kernels' tiles reach
// behind the last row and count on the zeros that a buffer gives past its end.
kda::Heads heads_of(const Tensor &t) {
    return {const_cast<void *>(t.p), t.rows > 1 ? t.stride : t.width, t.heads > 1 ? t.head_stride : t.width};
}
Span span(const Tensor &t) {
    const kda::Heads at = heads_of(t);
    Span s = t.heads_inside() ? strided(t.name, t.p, t.rows, t.width, at.stride, t.dtype) : strided(t.name, t.p, t.heads, t.width, at.head_stride, t.dtype);
    s.parts = t.heads_inside() ? t.heads : t.rows;
    s.part_stride = (t.heads_inside() ? at.head_stride : at.stride) * dsize(t.dtype);
    return s;
}

kda_status check_scale(float scale) {
    if (!(std::isfinite(scale) && scale > 0.f)) return fail(KDA_ERR_BAD_SHAPE, "scale must be finite and positive");
    return KDA_OK;
}
kda_status check_width(const char *name, int32_t d, int32_t most) {
    if (d < 1) return fail(KDA_ERR_BAD_SHAPE, "%s=%d", name, d);
    if (d > most || d % 8) return fail(KDA_ERR_UNSUPPORTED, "%s=%d (a multiple of 8, at most %d)", name, d, most);
    return KDA_OK;
}

// ---- rotary positions and the cache --------------------------------------------------------------------

kda_status rotary(const kda_rotary_args *a, bool inverse, const char *what) {
    kda::set_last_error("");
    KDA_TRY(check_struct(a));
    if (a->rows < 0 || a->heads < 0 || a->dim < 1 || a->rot < 2 || a->rot % 2 || a->offset < 0 || a->rot > a->dim ||
        a->offset > a->dim - a->rot)
        return fail(KDA_ERR_BAD_SHAPE, "rows=%lld heads=%d dim=%d rot=%d offset=%d", static_cast<long long>(a->rows), a->heads,
                    a->dim, a->rot, a->offset);
    if (a->rows > INT32_MAX || a->rot > 4096 || a->dim > 1 << 15 || a->heads > 1 << 20)
        return fail(KDA_ERR_UNSUPPORTED, "rows=%lld heads=%d dim=%d rot=%d", static_cast<long long>(a->rows), a->heads, a->dim, a->rot);
    if (!valid_dtype(a->dtype)) return fail(KDA_ERR_UNSUPPORTED, "dtype=%d", a->dtype);
    if (a->flags & ~KDA_ROTARY_INTERLEAVED) return fail(KDA_ERR_UNSUPPORTED, "unknown flags 0x%x", a->flags);
    if (!std::isfinite(a->scale)) return fail(KDA_ERR_BAD_SHAPE, "scale must be finite");
    if (a->rows == 0 || a->heads == 0) return KDA_OK;
    if (!a->x || !a->y || !a->positions || !a->inv_freq)
        return fail(KDA_ERR_NULL_POINTER, "x, y, positions and inv_freq are required");
    const Tensor x{"x", a->x, a->rows, a->heads, a->dim, a->x_stride, a->x_head_stride, a->dtype};
    const Tensor y{"y", a->y, a->rows, a->heads, a->dim, a->y_stride, a->y_head_stride, a->dtype};
    KDA_TRY(check_tensor(x, kAnyStride));
    KDA_TRY(check_tensor(y, kAnyStride));
    kda::RotaryLaunch L{};
    L.x = heads_of(x); L.y = heads_of(y);
    L.positions = a->positions; L.inv_freq = a->inv_freq;
    L.rows = a->rows; L.heads = a->heads; L.dim = a->dim; L.rot = a->rot; L.offset = a->offset;
    L.scale = a->scale;
    L.interleaved = (a->flags & KDA_ROTARY_INTERLEAVED) != 0;
    L.inverse = inverse;
    L.bf16 = a->dtype == KDA_DTYPE_BF16;
    L.stream = static_cast<hipStream_t>(a->stream);
    KDA_TRY(check_grid(kda::rotary_threads(L)));
    const bool in_place = a->x == a->y && (a->rows == 1 || a->x_stride == a->y_stride) &&
                          (a->heads == 1 || a->x_head_stride == a->y_head_stride);
    const Span ins[] = {in_place ? flat("x", nullptr, 0) : span(x), flat("positions", a->positions, a->rows * 4),
                        flat("inv_freq", a->inv_freq, a->rot * 2)};
    const Span outs[] = {span(y)};
    KDA_TRY(check_overlaps(ins, outs));
    return hip_status(kda::launch_rotary(L), what);
}

// ---- attention -----------------------------------------------------------------------------------------

template <class A>
kda_status check_attend_sizes(const A *a) {
    KDA_TRY(check_struct(a));
    if (a->batch < 0 || a->Tq < 0 || a->Tk < 0 || a->H < 1 || a->num_seqs < 0)
        return fail(KDA_ERR_BAD_SHAPE, "batch=%d Tq=%d Tk=%d H=%d num_seqs=%d", a->batch, a->Tq, a->Tk, a->H, a->num_seqs);
    if ((a->cu_seqlens_q == nullptr) != (a->cu_seqlens_k == nullptr))
        return fail(KDA_ERR_NULL_POINTER, "cu_seqlens_q and cu_seqlens_k are given together");
    if (a->cu_seqlens_q ? a->batch != 1 : a->num_seqs != a->batch)
        return fail(KDA_ERR_BAD_SHAPE, "num_seqs=%d with batch=%d (%s)", a->num_seqs, a->batch,
                    a->cu_seqlens_q ? "packed input needs batch = 1" : "num_seqs must equal batch");
    KDA_TRY(check_width("dn", a->dn, 128));
    KDA_TRY(check_width("dr", a->dr, 64));
    KDA_TRY(check_width("dv", a->dv, 128));
    KDA_TRY(check_scale(a->scale));
    if (!valid_dtype(a->in_dtype)) return fail(KDA_ERR_UNSUPPORTED, "in_dtype=%d", a->in_dtype);
    if (a->flags & ~KDA_ATTENTION_CAUSAL) return fail(KDA_ERR_UNSUPPORTED, "unknown flags 0x%x", a->flags);
    const int64_t rows_q = static_cast<int64_t>(a->batch) * a->Tq, rows_k = static_cast<int64_t>(a->batch) * a->Tk;
    if (rows_q > kMostRows || rows_k > kMostRows) return fail(KDA_ERR_UNSUPPORTED, "more than 2^30 rows");
    if (a->num_seqs > 65535 || a->H > 65535) return fail(KDA_ERR_UNSUPPORTED, "num_seqs=%d H=%d (at most 65535)", a->num_seqs, a->H);
    return KDA_OK;
}
template <class A>
kda::AttendLaunch attend_launch(const A *a) {
    kda::AttendLaunch L{};
    L.q_seq = {a->cu_seqlens_q, a->num_seqs, a->Tq, 128};
    L.k_seq = {a->cu_seqlens_k, a->num_seqs, a->Tk, 128};
    L.H = a->H; L.dn = a->dn; L.dr = a->dr; L.dv = a->dv;
    L.scale = a->scale;
    L.causal = (a->flags & KDA_ATTENTION_CAUSAL) != 0;
    L.bf16 = a->in_dtype == KDA_DTYPE_BF16;
    L.stream = static_cast<hipStream_t>(a->stream);
    return L;
}
// The tensors that both directions take.
template <class A>
struct AttendTensors {
    int64_t rows_q, rows_k;
    Tensor q, k, kr, v;
    explicit AttendTensors(const A *a)
        : rows_q(static_cast<int64_t>(a->batch) * a->Tq), rows_k(static_cast<int64_t>(a->batch) * a->Tk),
          q{"q", a->q, rows_q, a->H, a->dn + a->dr, a->q_stride, a->q_head_stride, a->in_dtype},
          k{"k", a->k, rows_k, a->H, a->dn, a->k_stride, a->k_head_stride, a->in_dtype},
          kr{"k_rope", a->k_rope, rows_k, 1, a->dr, a->k_rope_stride, 0, a->in_dtype},
          v{"v", a->v, rows_k, a->H, a->dv, a->v_stride, a->v_head_stride, a->in_dtype} {}
};
kda_status check_attend_tensor(const Tensor &t) {
    KDA_TRY(check_tensor(t, kAttendStride));
    return check_aligned(t);
}
size_t delta_bytes(int64_t rows_q, int H) { return (static_cast<size_t>(rows_q) * H * 4 + 15) / 16 * 16; }
template <class A>
size_t attend_bwd_bytes(const A *a) {
    return (a->in_dtype == KDA_DTYPE_BF16 ? 2 : 1) * delta_bytes(static_cast<int64_t>(a->batch) * a->Tq, a->H) + static_cast<size_t>(a->batch) * a->Tk * a->H * a->dr * 4;
}

int step_splits(const kda_latent_step_args *a) {
    return kda::latent_step_splits(a->N, a->H, static_cast<int64_t>(a->max_blocks) * a->page, a->in_dtype == KDA_DTYPE_BF16);
}
kda_status check_step_sizes(const kda_latent_step_args *a) {
    KDA_TRY(check_struct(a));
    if (a->N < 0 || a->H < 1 || a->page < 1 || a->num_blocks < 0 || a->max_blocks < 0)
        return fail(KDA_ERR_BAD_SHAPE, "N=%d H=%d page=%d num_blocks=%d max_blocks=%d", a->N, a->H, a->page, a->num_blocks, a->max_blocks);
    KDA_TRY(check_width("dl", a->dl, 512));
    KDA_TRY(check_width("dr", a->dr, 64));
    KDA_TRY(check_scale(a->scale));
    if (!valid_dtype(a->in_dtype) || !valid_dtype(a->out_dtype))
        return fail(KDA_ERR_UNSUPPORTED, "in_dtype=%d out_dtype=%d", a->in_dtype, a->out_dtype);
    if (a->N > 65535 || a->H > 65535) return fail(KDA_ERR_UNSUPPORTED, "N=%d H=%d (at most 65535)", a->N, a->H);
    if (static_cast<int64_t>(a->max_blocks) * a->page > kMostRows || static_cast<int64_t>(a->num_blocks) * a->page > INT32_MAX)
        return fail(KDA_ERR_UNSUPPORTED, "more than 2^30 rows per sequence or 2^31 - 1 in the cache");
    // the sequences' tiles, of 16 rows or more, are counted in 32 bits
    if (((static_cast<int64_t>(a->max_blocks) * a->page + 15) / 16) * a->N > INT32_MAX)
        return fail(KDA_ERR_UNSUPPORTED, "N * max_blocks * page is 2^35 rows or more");
    return check_grid(kda::latent_step_threads(a->N, a->H, a->in_dtype == KDA_DTYPE_BF16, step_splits(a)));
}

}  // namespace

extern "C" {

kda_status kda_rotary_fwd(const kda_rotary_args *a) { return rotary(a, false, "kda_rotary_fwd launch"); }
kda_status kda_rotary_bwd(const kda_rotary_args *a) { return rotary(a, true, "kda_rotary_bwd launch"); }

kda_status kda_latent_cache_append(const kda_latent_append_args *a) {
    kda::set_last_error("");
    KDA_TRY(check_struct(a));
    if (a->rows < 0 || a->num_blocks < 0 || a->page < 1 || a->dl < 1 || a->dr < 1)
        return fail(KDA_ERR_BAD_SHAPE, "rows=%lld num_blocks=%d page=%d dl=%d dr=%d", static_cast<long long>(a->rows),
                    a->num_blocks, a->page, a->dl, a->dr);
    if (a->dl > 1 << 16 || a->dr > 1 << 16) return fail(KDA_ERR_UNSUPPORTED, "dl=%d dr=%d (at most 2^16)", a->dl, a->dr);
    const int64_t cache_rows = static_cast<int64_t>(a->num_blocks) * a->page;
    if (a->rows > kMostRows || cache_rows > INT32_MAX)
        return fail(KDA_ERR_UNSUPPORTED, "more than 2^30 rows, or 2^31 - 1 in the cache");
    if (!valid_dtype(a->dtype)) return fail(KDA_ERR_UNSUPPORTED, "dtype=%d", a->dtype);
    if (a->flags & ~KDA_ROTARY_INTERLEAVED) return fail(KDA_ERR_UNSUPPORTED, "unknown flags 0x%x", a->flags);
    if (!std::isfinite(a->scale)) return fail(KDA_ERR_BAD_SHAPE, "scale must be finite");
    KDA_TRY(check_grid((a->rows + 3) / 4 * 256));
    if ((a->inv_freq == nullptr) != (a->positions == nullptr))
        return fail(KDA_ERR_NULL_POINTER, "positions and inv_freq are given together");
    if (a->inv_freq && a->dr % 2) return fail(KDA_ERR_BAD_SHAPE, "dr=%d is rotated and has to be even", a->dr);
    if (a->rows == 0 || cache_rows == 0) return KDA_OK;
    if (!a->latent || !a->rope || !a->cache || !a->slots)
        return fail(KDA_ERR_NULL_POINTER, "latent, rope, cache and slots are required");
    const Tensor latent{"latent", a->latent, a->rows, 1, a->dl, a->latent_stride, 0, a->dtype};
    const Tensor rope{"rope", a->rope, a->rows, 1, a->dr, a->rope_stride, 0, a->dtype};
    KDA_TRY(check_tensor(latent, kAnyStride));
    KDA_TRY(check_tensor(rope, kAnyStride));
    const Span ins[] = {span(latent), span(rope), flat("slots", a->slots, a->rows * 4),
                        flat("positions", a->positions, a->rows * 4), flat("inv_freq", a->inv_freq, static_cast<int64_t>(a->dr) * 2)};
    const Span outs[] = {flat("cache", a->cache, cache_rows * (a->dl + a->dr) * dsize(a->dtype))};
    KDA_TRY(check_overlaps(ins, outs));
    kda::AppendLaunch L{};
    L.latent = heads_of(latent); L.rope = heads_of(rope);
    L.cache = a->cache; L.slots = a->slots; L.positions = a->positions; L.inv_freq = a->inv_freq;
    L.rows = a->rows; L.cache_rows = cache_rows; L.dl = a->dl; L.dr = a->dr;
    L.scale = a->scale;
    L.interleaved = (a->flags & KDA_ROTARY_INTERLEAVED) != 0;
    L.bf16 = a->dtype == KDA_DTYPE_BF16;
    L.stream = static_cast<hipStream_t>(a->stream);
    return hip_status(kda::launch_append(L), "kda_latent_cache_append launch");
}

size_t kda_latent_attention_step_workspace_bytes(const kda_latent_step_args *a) {
    if (check_step_sizes(a) != KDA_OK) return static_cast<size_t>(-1);
    return kda::latent_step_workspace_bytes(a->N, a->H, a->dl, step_splits(a), a->in_dtype == KDA_DTYPE_BF16);
}

kda_status kda_latent_attention_step(const kda_latent_step_args *a) {
    kda::set_last_error("");
    KDA_TRY(check_step_sizes(a));
    if (a->N == 0) return KDA_OK;
    if (!a->q_latent || !a->q_rope || !a->lengths || !a->o)
        return fail(KDA_ERR_NULL_POINTER, "q_latent, q_rope, lengths and o are required");
    if (a->num_blocks > 0 && a->max_blocks > 0 && (!a->cache || !a->block_table))
        return fail(KDA_ERR_NULL_POINTER, "cache and block_table are required");
    const Tensor ql{"q_latent", a->q_latent, a->N, a->H, a->dl, a->q_latent_stride, a->q_latent_head_stride, a->in_dtype};
    const Tensor qr{"q_rope", a->q_rope, a->N, a->H, a->dr, a->q_rope_stride, a->q_rope_head_stride, a->in_dtype};
    const Tensor o{"o", a->o, a->N, a->H, a->dl, a->o_stride, a->o_head_stride, a->out_dtype};
    const int64_t cache_rows = static_cast<int64_t>(a->num_blocks) * a->page, head = static_cast<int64_t>(a->N) * a->H;
    const Tensor cache{"cache", a->cache, cache_rows, 1, a->dl + a->dr, a->dl + a->dr, 0, a->in_dtype};
    for (const Tensor *t : {&ql, &qr, &o}) KDA_TRY(check_tensor(*t, kAnyStride));
    for (const Tensor *t : {&ql, &qr, &o, &cache}) KDA_TRY(check_aligned(*t));
    if (a->N > 1) KDA_TRY(check_stride("block_table", a->block_table, a->block_table_stride, a->max_blocks, a->N, kAnyStride));
    const int splits = step_splits(a);
    const size_t need = kda::latent_step_workspace_bytes(a->N, a->H, a->dl, splits, a->in_dtype == KDA_DTYPE_BF16);
    if (a->workspace_bytes < need || (need > 0 && !a->workspace))
        return fail(KDA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu < %zu bytes", a->workspace_bytes, need);
    if (need && reinterpret_cast<uintptr_t>(a->workspace) % 16) return fail(KDA_ERR_UNSUPPORTED, "workspace has to be aligned to 16 bytes");
    const Span ins[] = {span(ql), span(qr), span(cache), flat("lengths", a->lengths, static_cast<int64_t>(a->N) * 4),
                        flat("block_table", a->max_blocks ? a->block_table : nullptr,
                             ((a->N > 1 ? (a->N - 1) * a->block_table_stride : 0) + a->max_blocks) * 4)};
    const Span outs[] = {span(o), flat("lse", a->lse, head * 4), flat("workspace", a->workspace, static_cast<int64_t>(a->workspace_bytes))};
    KDA_TRY(check_overlaps(ins, outs));
    kda::LatentStepLaunch L{};
    L.ql = heads_of(ql); L.qr = heads_of(qr); L.o = heads_of(o);
    L.cache = a->cache; L.lengths = a->lengths; L.lse = a->lse;
    L.pages = {a->block_table, a->block_table_stride, a->page, a->num_blocks, a->num_blocks > 0 ? a->max_blocks : 0};
    L.N = a->N; L.H = a->H; L.dl = a->dl; L.dr = a->dr;
    L.scale = a->scale;
    L.bf16 = a->in_dtype == KDA_DTYPE_BF16; L.out_bf16 = a->out_dtype == KDA_DTYPE_BF16;
    L.splits = splits;
    L.ws = static_cast<float *>(a->workspace);
    L.stream = static_cast<hipStream_t>(a->stream);
    return hip_status(kda::launch_latent_step(L), "kda_latent_attention_step launch");
}

kda_status kda_latent_attention_fwd(const kda_latent_attention_args *a) {
    kda::set_last_error("");
    KDA_TRY(check_attend_sizes(a));
    if (!valid_dtype(a->out_dtype)) return fail(KDA_ERR_UNSUPPORTED, "out_dtype=%d", a->out_dtype);
    const AttendTensors<kda_latent_attention_args> t(a);
    kda::AttendLaunch L = attend_launch(a);
    KDA_TRY(check_grid(kda::attend_threads(L.q_seq, L.k_seq, a->H, a->dr, L.bf16, false)));
    if (t.rows_q == 0 || a->num_seqs == 0) return KDA_OK;
    if (!a->q || !a->o) return fail(KDA_ERR_NULL_POINTER, "q and o are required");
    if (t.rows_k > 0 && (!a->k || !a->k_rope || !a->v)) return fail(KDA_ERR_NULL_POINTER, "k, k_rope and v are required");
    const Tensor o{"o", a->o, t.rows_q, a->H, a->dv, a->o_stride, a->o_head_stride, a->out_dtype};
    for (const Tensor *x : {&t.q, &t.k, &t.kr, &t.v, &o}) KDA_TRY(check_attend_tensor(*x));
    const int64_t cu = (static_cast<int64_t>(a->num_seqs) + 1) * 4;
    const Span ins[] = {span(t.q), span(t.k), span(t.kr), span(t.v), flat("cu_seqlens_q", a->cu_seqlens_q, cu),
                        flat("cu_seqlens_k", a->cu_seqlens_k, cu)};
    const Span outs[] = {span(o), flat("lse", a->lse, t.rows_q * a->H * 4)};
    KDA_TRY(check_overlaps(ins, outs));
    L.q = heads_of(t.q); L.k = heads_of(t.k); L.kr = heads_of(t.kr); L.v = heads_of(t.v); L.o = heads_of(o);
    L.lse = a->lse;
    L.out_bf16 = a->out_dtype == KDA_DTYPE_BF16;
    return hip_status(kda::launch_attend_fwd(L), "kda_latent_attention_fwd launch");
}

size_t kda_latent_attention_bwd_workspace_bytes(const kda_latent_attention_bwd_args *a) {
    if (check_attend_sizes(a) != KDA_OK) return static_cast<size_t>(-1);
    return attend_bwd_bytes(a);
}

kda_status kda_latent_attention_bwd(const kda_latent_attention_bwd_args *a) {
    kda::set_last_error("");
    KDA_TRY(check_attend_sizes(a));
    if (!valid_dtype(a->grad_dtype)) return fail(KDA_ERR_UNSUPPORTED, "grad_dtype=%d", a->grad_dtype);
    const AttendTensors<kda_latent_attention_bwd_args> t(a);
    kda::AttendLaunch L = attend_launch(a);
    KDA_TRY(check_grid(kda::attend_threads(L.q_seq, L.k_seq, a->H, a->dr, L.bf16, true)));
    if (t.rows_q + t.rows_k == 0 || a->num_seqs == 0) return KDA_OK;
    if (t.rows_q > 0 && (!a->q || !a->o || !a->lse || !a->grad_o || !a->grad_q))
        return fail(KDA_ERR_NULL_POINTER, "q, o, lse, grad_o and grad_q are required");
    if (t.rows_k > 0 && (!a->k || !a->k_rope || !a->v || !a->grad_k || !a->grad_k_rope || !a->grad_v))
        return fail(KDA_ERR_NULL_POINTER, "k, k_rope, v and their gradients are required");
    const kda_dtype g = a->grad_dtype;
    const Tensor o{"o", a->o, t.rows_q, a->H, a->dv, a->o_stride, a->o_head_stride, a->in_dtype};
    const Tensor go{"grad_o", a->grad_o, t.rows_q, a->H, a->dv, a->grad_o_stride, a->grad_o_head_stride, a->in_dtype};
    const Tensor dq{"grad_q", a->grad_q, t.rows_q, a->H, a->dn + a->dr, a->grad_q_stride, a->grad_q_head_stride, g};
    const Tensor dk{"grad_k", a->grad_k, t.rows_k, a->H, a->dn, a->grad_k_stride, a->grad_k_head_stride, g};
    const Tensor dkr{"grad_k_rope", a->grad_k_rope, t.rows_k, 1, a->dr, a->grad_k_rope_stride, 0, g};
    const Tensor dv{"grad_v", a->grad_v, t.rows_k, a->H, a->dv, a->grad_v_stride, a->grad_v_head_stride, g};
    for (const Tensor *x : {&t.q, &t.k, &t.kr, &t.v, &o, &go, &dq, &dk, &dkr, &dv}) KDA_TRY(check_attend_tensor(*x));
    const size_t need = attend_bwd_bytes(a);
    if (a->workspace_bytes < need || (need > 0 && !a->workspace))
        return fail(KDA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu < %zu bytes", a->workspace_bytes, need);
    if (reinterpret_cast<uintptr_t>(a->workspace) % 16) return fail(KDA_ERR_UNSUPPORTED, "workspace has to be aligned to 16 bytes");
    const int64_t cu = (static_cast<int64_t>(a->num_seqs) + 1) * 4;
    const Span ins[] = {span(t.q), span(t.k), span(t.kr), span(t.v), span(o), span(go), flat("lse", a->lse, t.rows_q * a->H * 4),
                        flat("cu_seqlens_q", a->cu_seqlens_q, cu), flat("cu_seqlens_k", a->cu_seqlens_k, cu)};
    const Span outs[] = {span(dq), span(dk), span(dkr), span(dv),
                         flat("workspace", a->workspace, static_cast<int64_t>(a->workspace_bytes))};
    KDA_TRY(check_overlaps(ins, outs));
    L.q = heads_of(t.q); L.k = heads_of(t.k); L.kr = heads_of(t.kr); L.v = heads_of(t.v); L.o = heads_of(o);
    L.lse = const_cast<float *>(a->lse);
    L.go = heads_of(go); L.dq = heads_of(dq); L.dk = heads_of(dk); L.dkr = heads_of(dkr); L.dvg = heads_of(dv);
    L.grad_bf16 = g == KDA_DTYPE_BF16;
    L.delta = static_cast<float *>(a->workspace);
    const size_t stats = delta_bytes(t.rows_q, a->H);
    L.lse2 = reinterpret_cast<float *>(static_cast<char *>(a->workspace) + stats);
    L.dkr_part = reinterpret_cast<float *>(static_cast<char *>(a->workspace) + (L.bf16 ? 2 : 1) * stats);
    return hip_status(kda::launch_attend_bwd(L), "kda_latent_attention_bwd launch");
}

}  // extern "C"
