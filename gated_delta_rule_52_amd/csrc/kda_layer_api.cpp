// kda_layer_api.cpp - host entry points of the layer operators in include/kda.h: selective scan, short
// convolution, layer norm.  As in kda_api.cpp every argument is validated before anything is enqueued.
#include <cmath>
#include <cstdarg>
#include <cstddef>
#include <cstdio>

#include "kda.h"
#include "kda_internal.h"
#include "kda_layer.h"

namespace {

kda_status fail(kda_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
kda_status fail(kda_status s, const char *fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    kda::set_last_error(buf);
    return s;
}

kda_status hip_status(hipError_t e, const char *what) {
    if (e == hipSuccess) return KDA_OK;
    return fail(KDA_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool valid_dtype(kda_dtype d) { return d == KDA_DTYPE_BF16 || d == KDA_DTYPE_FP32; }
int64_t dsize(kda_dtype d) { return d == KDA_DTYPE_BF16 ? 2 : 4; }

// The memory of a tensor: `rows` rows of `width` bytes, `stride` bytes apart.
struct Span {
    const char *name;
    uintptr_t at;
    int64_t rows, width, stride;
    bool empty() const { return !at || rows <= 0 || width <= 0; }
    uintptr_t end() const { return at + static_cast<uintptr_t>((rows - 1) * stride + width); }
};
Span flat(const char *name, const void *p, int64_t bytes) {
    return {name, reinterpret_cast<uintptr_t>(p), 1, bytes, bytes};
}
Span strided(const char *name, const void *p, int64_t rows, int64_t width, int64_t stride, kda_dtype d) {
    return {name, reinterpret_cast<uintptr_t>(p), rows, width * dsize(d), stride * dsize(d)};
}
bool overlap(const Span &a, const Span &b) {
    if (a.empty() || b.empty() || a.at >= b.end() || b.at >= a.end()) return false;
    if (a.stride == b.stride && a.rows > 1 && b.rows > 1) {  // column slices of one buffer may interleave
        const int64_t m = a.stride, d = ((static_cast<int64_t>(b.at - a.at) % m) + m) % m;
        if (d >= a.width && d + b.width <= m) return false;
    }
    return true;
}
// Every output against every input and the other outputs.
template <size_t NI, size_t NO>
kda_status check_overlaps(const Span (&ins)[NI], const Span (&outs)[NO]) {
    for (size_t i = 0; i < NO; ++i) {
        for (const Span &s : ins)
            if (overlap(outs[i], s)) return fail(KDA_ERR_ALIAS, "%s overlaps %s", outs[i].name, s.name);
        for (size_t j = i + 1; j < NO; ++j)
            if (overlap(outs[i], outs[j])) return fail(KDA_ERR_ALIAS, "%s overlaps %s", outs[i].name, outs[j].name);
    }
    return KDA_OK;
}

// Row strides below which an operator's address arithmetic holds; the others form every row's address in 64 bits.
constexpr int64_t kAnyStride = int64_t{1} << 40;
constexpr int64_t kScanStride = int64_t{1} << 22;  // the walk over tokens: a row's bytes in a 24-bit multiply
constexpr int64_t kNormStride = int64_t{1} << 26;  // rows that share a workgroup, up to 16: 32-bit distances within it

kda_status check_stride(const char *name, const void *p, int64_t stride, int64_t width, int64_t rows, int64_t below) {
    if (p && (stride < width || stride >= below || stride > (int64_t{1} << 40) / (rows > 0 ? rows : 1)))
        return fail(KDA_ERR_BAD_SHAPE, "%s: stride %lld for rows of %lld", name, static_cast<long long>(stride),
                    static_cast<long long>(width));
    return KDA_OK;
}
#define KDA_TRY(x)                          \
    do {                                    \
        const kda_status st_ = (x);         \
        if (st_ != KDA_OK) return st_;      \
    } while (0)

kda::Rows rows_of(const void *p, int64_t stride, kda_dtype d) {
    return {const_cast<void *>(p), stride, d == KDA_DTYPE_BF16 ? 1 : 0};
}

// Checks the batch of sequences that the scan and the convolution share.
template <class A>
kda_status check_batch(const A *a) {
    if (a->batch < 0 || a->T < 0 || a->dim <= 0 || a->num_seqs < 0)
        return fail(KDA_ERR_BAD_SHAPE, "batch=%d T=%d dim=%d num_seqs=%d", a->batch, a->T, a->dim, a->num_seqs);
    if (a->cu_seqlens ? a->batch != 1 : a->num_seqs != a->batch)
        return fail(KDA_ERR_BAD_SHAPE, "num_seqs=%d with batch=%d (%s)", a->num_seqs, a->batch,
                    a->cu_seqlens ? "packed input needs batch = 1" : "num_seqs must equal batch");
    const int64_t rows = static_cast<int64_t>(a->batch) * a->T;
    if (rows > INT32_MAX) return fail(KDA_ERR_BAD_SHAPE, "%lld rows (at most %d)", static_cast<long long>(rows), INT32_MAX);
    if (rows * a->dim > (int64_t{1} << 40) || static_cast<int64_t>(a->num_seqs) * a->dim > (int64_t{1} << 32))
        return fail(KDA_ERR_BAD_SHAPE, "problem too large");
    if (a->dim >= 1 << 22) return fail(KDA_ERR_UNSUPPORTED, "dim=%d (below 2^22)", a->dim);
    if (a->num_seqs > 65535) return fail(KDA_ERR_UNSUPPORTED, "num_seqs=%d (at most 65535)", a->num_seqs);
    return KDA_OK;
}
// Threads of one launch stay below 2^32.
kda_status check_grid(int64_t threads) {
    if (threads < 0 || threads >= (int64_t{1} << 32)) return fail(KDA_ERR_UNSUPPORTED, "problem too large for one launch");
    return KDA_OK;
}

template <class A>
kda_status check_struct(const A *a) {
    if (!a) return fail(KDA_ERR_NULL_POINTER, "args is NULL");
    if (a->struct_size != sizeof(A))
        return fail(KDA_ERR_BAD_STRUCT, "struct_size %u (expected %zu)", a->struct_size, sizeof(A));
    return KDA_OK;
}

// ---- selective scan ------------------------------------------------------------------------------------

kda_status check_scan_sizes(const kda_selective_scan_args *a) {
    KDA_TRY(check_struct(a));
    KDA_TRY(check_batch(a));
    if (a->ds < 1 || a->ds > 64) return fail(KDA_ERR_UNSUPPORTED, "ds=%d (supported: 1 to 64)", a->ds);
    if (!valid_dtype(a->in_dtype) || !valid_dtype(a->out_dtype))
        return fail(KDA_ERR_UNSUPPORTED, "in_dtype=%d out_dtype=%d", a->in_dtype, a->out_dtype);
    if (a->flags & ~KDA_SCAN_DT_SOFTPLUS) return fail(KDA_ERR_UNSUPPORTED, "unknown flags 0x%x", a->flags);
    const kda::SeqTiles s = kda::scan_fwd_tiles(a->cu_seqlens, a->num_seqs, a->T, a->dim, a->ds);
    return check_grid(s.slots() * ((a->dim + 63) / 64) * 256);
}

// One token per sequence is the first row of a tile of its own, at no distance from it.
template <class A>
int64_t scan_stride(const A *a) {
    return a->cu_seqlens || a->T > 1 ? kScanStride : kAnyStride;
}

kda_status check_scan(const kda_selective_scan_args *a) {
    KDA_TRY(check_scan_sizes(a));
    const int64_t rows = static_cast<int64_t>(a->batch) * a->T;
    if (rows > 0 && (!a->u || !a->dt || !a->B || !a->C || !a->y))
        return fail(KDA_ERR_NULL_POINTER, "u, dt, B, C and y are required");
    if (!a->A) return fail(KDA_ERR_NULL_POINTER, "A is required");
    const int64_t below = scan_stride(a);
    KDA_TRY(check_stride("u", a->u, a->u_stride, a->dim, rows, below));
    KDA_TRY(check_stride("dt", a->dt, a->dt_stride, a->dim, rows, below));
    KDA_TRY(check_stride("B", a->B, a->B_stride, a->ds, rows, below));
    KDA_TRY(check_stride("C", a->C, a->C_stride, a->ds, rows, below));
    KDA_TRY(check_stride("z", a->z, a->z_stride, a->dim, rows, below));
    KDA_TRY(check_stride("y", a->y, a->y_stride, a->dim, rows, below));
    const int64_t state = static_cast<int64_t>(a->num_seqs) * a->dim * a->ds * 4, param = static_cast<int64_t>(a->dim) * 4;
    const bool in_place = a->initial_state == a->final_state;
    const Span ins[] = {strided("u", a->u, rows, a->dim, a->u_stride, a->in_dtype),
                        strided("dt", a->dt, rows, a->dim, a->dt_stride, a->in_dtype),
                        strided("B", a->B, rows, a->ds, a->B_stride, a->in_dtype),
                        strided("C", a->C, rows, a->ds, a->C_stride, a->in_dtype),
                        strided("z", a->z, rows, a->dim, a->z_stride, a->in_dtype),
                        flat("A", a->A, param * a->ds), flat("D", a->D, param), flat("dt_bias", a->dt_bias, param),
                        flat("initial_state", in_place ? nullptr : a->initial_state, state),
                        flat("cu_seqlens", a->cu_seqlens, (static_cast<int64_t>(a->num_seqs) + 1) * 4)};
    const Span outs[] = {strided("y", a->y, rows, a->dim, a->y_stride, a->out_dtype),
                         flat("final_state", a->final_state, state),
                         flat("workspace", a->workspace, static_cast<int64_t>(a->workspace_bytes))};
    return check_overlaps(ins, outs);
}

kda::ScanFwdLaunch scan_launch(const kda_selective_scan_args *a) {
    kda::ScanFwdLaunch L{};
    L.u = rows_of(a->u, a->u_stride, a->in_dtype);
    L.dt = rows_of(a->dt, a->dt_stride, a->in_dtype);
    L.B = rows_of(a->B, a->B_stride, a->in_dtype);
    L.C = rows_of(a->C, a->C_stride, a->in_dtype);
    L.z = rows_of(a->z, a->z_stride, a->in_dtype);
    L.y = rows_of(a->y, a->y_stride, a->out_dtype);
    L.A = a->A; L.D = a->D; L.dt_bias = a->dt_bias;
    L.h0 = a->initial_state; L.hT = a->final_state;
    L.seq = kda::scan_fwd_tiles(a->cu_seqlens, a->num_seqs, a->T, a->dim, a->ds);
    L.dim = a->dim; L.ds = a->ds;
    L.softplus = (a->flags & KDA_SCAN_DT_SOFTPLUS) != 0;
    L.ws = static_cast<float *>(a->workspace);
    L.stream = static_cast<hipStream_t>(a->stream);
    return L;
}

kda_status check_scan_bwd_sizes(const kda_selective_scan_bwd_args *a) {
    KDA_TRY(check_struct(a));
    KDA_TRY(check_batch(a));
    if (a->ds < 1 || a->ds > 64) return fail(KDA_ERR_UNSUPPORTED, "ds=%d (supported: 1 to 64)", a->ds);
    if (!valid_dtype(a->in_dtype) || !valid_dtype(a->grad_dtype))
        return fail(KDA_ERR_UNSUPPORTED, "in_dtype=%d grad_dtype=%d", a->in_dtype, a->grad_dtype);
    if (a->flags & ~KDA_SCAN_DT_SOFTPLUS) return fail(KDA_ERR_UNSUPPORTED, "unknown flags 0x%x", a->flags);
    const kda::SeqTiles s = kda::scan_bwd_tiles(a->cu_seqlens, a->num_seqs, a->T, a->dim, a->ds);
    return check_grid(kda::scan_bwd_threads(s, a->dim, a->ds));
}

// ---- short convolution ---------------------------------------------------------------------------------

template <class A>
kda_status check_conv_sizes(const A *a) {
    KDA_TRY(check_struct(a));
    KDA_TRY(check_batch(a));
    if (a->width < 2 || a->width > 4) return fail(KDA_ERR_UNSUPPORTED, "width=%d (supported: 2 to 4)", a->width);
    if (!valid_dtype(a->in_dtype) || !valid_dtype(a->w_dtype))
        return fail(KDA_ERR_UNSUPPORTED, "in_dtype=%d w_dtype=%d", a->in_dtype, a->w_dtype);
    if (a->flags & ~KDA_CONV_SILU) return fail(KDA_ERR_UNSUPPORTED, "unknown flags 0x%x", a->flags);
    return check_grid(static_cast<int64_t>(a->num_seqs) * ((a->dim + 255) / 256) * 256);  // the states', at least the step's
}

kda_status check_conv(const kda_short_conv_args *a) {
    KDA_TRY(check_conv_sizes(a));
    if (!valid_dtype(a->out_dtype)) return fail(KDA_ERR_UNSUPPORTED, "out_dtype=%d", a->out_dtype);
    const int64_t rows = static_cast<int64_t>(a->batch) * a->T;
    KDA_TRY(check_grid(kda::conv_fwd_threads(rows, a->dim)));
    if (rows > 0 && (!a->x || !a->y)) return fail(KDA_ERR_NULL_POINTER, "x and y are required");
    if (!a->weight) return fail(KDA_ERR_NULL_POINTER, "weight is required");
    KDA_TRY(check_stride("x", a->x, a->x_stride, a->dim, rows, kAnyStride));
    KDA_TRY(check_stride("y", a->y, a->y_stride, a->dim, rows, kAnyStride));
    const int64_t state = static_cast<int64_t>(a->num_seqs) * (a->width - 1) * a->dim * dsize(a->in_dtype);
    const int64_t param = a->dim * dsize(a->w_dtype);
    const bool in_place = a->initial_state == a->final_state;
    const Span ins[] = {strided("x", a->x, rows, a->dim, a->x_stride, a->in_dtype),
                        flat("weight", a->weight, param * a->width), flat("bias", a->bias, param),
                        flat("initial_state", in_place ? nullptr : a->initial_state, state),
                        flat("cu_seqlens", a->cu_seqlens, (static_cast<int64_t>(a->num_seqs) + 1) * 4)};
    const Span outs[] = {strided("y", a->y, rows, a->dim, a->y_stride, a->out_dtype),
                         flat("final_state", a->final_state, state)};
    return check_overlaps(ins, outs);
}

kda_status check_conv_bwd_sizes(const kda_short_conv_bwd_args *a) {
    KDA_TRY(check_conv_sizes(a));
    return check_grid(kda::conv_bwd_threads(static_cast<int64_t>(a->batch) * a->T, a->dim, a->in_dtype == KDA_DTYPE_BF16));
}

kda::ConvLaunch conv_launch(const kda_short_conv_args *a) {
    kda::ConvLaunch L{};
    L.x = rows_of(a->x, a->x_stride, a->in_dtype);
    L.y = rows_of(a->y, a->y_stride, a->out_dtype);
    L.w = a->weight; L.bias = a->bias; L.w_bf16 = a->w_dtype == KDA_DTYPE_BF16;
    L.h0 = a->initial_state; L.hT = a->final_state;
    L.cu = a->cu_seqlens;
    L.N = a->num_seqs; L.T = a->T; L.dim = a->dim; L.width = a->width;
    L.silu = (a->flags & KDA_CONV_SILU) != 0;
    L.stream = static_cast<hipStream_t>(a->stream);
    return L;
}

// ---- layer norm ----------------------------------------------------------------------------------------

// Up to 2048 elements several rows share a workgroup.
int64_t norm_stride(int32_t dim) { return dim > 2048 ? kAnyStride : kNormStride; }

kda_status check_norm_sizes(int64_t rows, int32_t dim, float eps) {
    if (rows < 0 || dim < 1) return fail(KDA_ERR_BAD_SHAPE, "rows=%lld dim=%d", static_cast<long long>(rows), dim);
    if (dim > 16384) return fail(KDA_ERR_UNSUPPORTED, "dim=%d (at most 16384)", dim);
    if (!(std::isfinite(eps) && eps >= 0.f)) return fail(KDA_ERR_BAD_SHAPE, "eps must be finite and >= 0");
    if (rows > (int64_t{1} << 40) / dim) return fail(KDA_ERR_BAD_SHAPE, "problem too large");
    return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_selective_scan_fwd_workspace_bytes(const kda_selective_scan_args *a) {
    if (check_scan_sizes(a) != KDA_OK) return static_cast<size_t>(-1);
    return kda::scan_fwd_workspace_bytes(kda::scan_fwd_tiles(a->cu_seqlens, a->num_seqs, a->T, a->dim, a->ds), a->dim, a->ds);
}

kda_status kda_selective_scan_fwd(const kda_selective_scan_args *a) {
    kda::set_last_error("");
    KDA_TRY(check_scan(a));
    if (a->num_seqs == 0 || (static_cast<int64_t>(a->batch) * a->T == 0 && !a->final_state)) return KDA_OK;
    if (!a->cu_seqlens && a->T == 1 && a->final_state) return kda_selective_scan_step(a);
    const kda::ScanFwdLaunch L = scan_launch(a);
    const size_t need = kda::scan_fwd_workspace_bytes(L.seq, a->dim, a->ds);
    if (a->workspace_bytes < need || (need > 0 && !a->workspace))
        return fail(KDA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu < %zu bytes", a->workspace_bytes, need);
    return hip_status(kda::launch_scan_fwd(L), "kda_selective_scan_fwd launch");
}

kda_status kda_selective_scan_step(const kda_selective_scan_args *a) {
    kda::set_last_error("");
    KDA_TRY(check_scan(a));
    if (a->cu_seqlens || a->T != 1) return fail(KDA_ERR_BAD_SHAPE, "a step takes T = 1 and no cu_seqlens (T=%d)", a->T);
    if (a->num_seqs == 0) return KDA_OK;
    if (!a->final_state) return fail(KDA_ERR_NULL_POINTER, "final_state is required");
    return hip_status(kda::launch_scan_step(scan_launch(a)), "kda_selective_scan_step launch");
}

size_t kda_selective_scan_bwd_workspace_bytes(const kda_selective_scan_bwd_args *a) {
    if (check_scan_bwd_sizes(a) != KDA_OK) return static_cast<size_t>(-1);
    return kda::scan_bwd_workspace_bytes(kda::scan_bwd_tiles(a->cu_seqlens, a->num_seqs, a->T, a->dim, a->ds), a->dim, a->ds);
}

kda_status kda_selective_scan_bwd(const kda_selective_scan_bwd_args *a) {
    kda::set_last_error("");
    KDA_TRY(check_scan_bwd_sizes(a));
    const int64_t rows = static_cast<int64_t>(a->batch) * a->T;
    if (rows > 0 && (!a->u || !a->dt || !a->B || !a->C || !a->grad_y || !a->grad_u || !a->grad_dt || !a->grad_B || !a->grad_C))
        return fail(KDA_ERR_NULL_POINTER, "u, dt, B, C, grad_y and their gradients are required");
    if (!a->A || !a->grad_A) return fail(KDA_ERR_NULL_POINTER, "A and grad_A are required");
    if (rows > 0 && (a->z == nullptr) != (a->grad_z == nullptr))
        return fail(KDA_ERR_NULL_POINTER, "grad_z is given exactly where z is");
    if (a->grad_dt_bias && !a->dt_bias) return fail(KDA_ERR_NULL_POINTER, "grad_dt_bias without dt_bias");
    if (a->grad_D && !a->D) return fail(KDA_ERR_NULL_POINTER, "grad_D without D");
    const int64_t below = scan_stride(a);
    KDA_TRY(check_stride("u", a->u, a->u_stride, a->dim, rows, below));
    KDA_TRY(check_stride("dt", a->dt, a->dt_stride, a->dim, rows, below));
    KDA_TRY(check_stride("B", a->B, a->B_stride, a->ds, rows, below));
    KDA_TRY(check_stride("C", a->C, a->C_stride, a->ds, rows, below));
    KDA_TRY(check_stride("z", a->z, a->z_stride, a->dim, rows, below));
    KDA_TRY(check_stride("grad_y", a->grad_y, a->grad_y_stride, a->dim, rows, below));
    KDA_TRY(check_stride("grad_u", a->grad_u, a->grad_u_stride, a->dim, rows, below));
    KDA_TRY(check_stride("grad_dt", a->grad_dt, a->grad_dt_stride, a->dim, rows, below));
    KDA_TRY(check_stride("grad_B", a->grad_B, a->grad_B_stride, a->ds, rows, below));
    KDA_TRY(check_stride("grad_C", a->grad_C, a->grad_C_stride, a->ds, rows, below));
    KDA_TRY(check_stride("grad_z", a->grad_z, a->grad_z_stride, a->dim, rows, below));
    const kda::SeqTiles seq = kda::scan_bwd_tiles(a->cu_seqlens, a->num_seqs, a->T, a->dim, a->ds);
    const size_t need = kda::scan_bwd_workspace_bytes(seq, a->dim, a->ds);
    if (a->workspace_bytes < need || (need > 0 && !a->workspace))
        return fail(KDA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu < %zu bytes", a->workspace_bytes, need);
    const int64_t state = static_cast<int64_t>(a->num_seqs) * a->dim * a->ds * 4, param = static_cast<int64_t>(a->dim) * 4;
    const kda_dtype g = a->grad_dtype;
    const Span ins[] = {strided("u", a->u, rows, a->dim, a->u_stride, a->in_dtype),
                        strided("dt", a->dt, rows, a->dim, a->dt_stride, a->in_dtype),
                        strided("B", a->B, rows, a->ds, a->B_stride, a->in_dtype),
                        strided("C", a->C, rows, a->ds, a->C_stride, a->in_dtype),
                        strided("z", a->z, rows, a->dim, a->z_stride, a->in_dtype),
                        strided("grad_y", a->grad_y, rows, a->dim, a->grad_y_stride, a->in_dtype),
                        flat("A", a->A, param * a->ds), flat("D", a->D, param), flat("dt_bias", a->dt_bias, param),
                        flat("initial_state", a->initial_state == a->grad_initial_state ? nullptr : a->initial_state, state),
                        flat("grad_final_state",
                             a->grad_final_state == a->grad_initial_state ? nullptr : a->grad_final_state, state),
                        flat("cu_seqlens", a->cu_seqlens, (static_cast<int64_t>(a->num_seqs) + 1) * 4)};
    const Span outs[] = {strided("grad_u", a->grad_u, rows, a->dim, a->grad_u_stride, g),
                         strided("grad_dt", a->grad_dt, rows, a->dim, a->grad_dt_stride, g),
                         strided("grad_z", a->grad_z, rows, a->dim, a->grad_z_stride, g),
                         strided("grad_B", a->grad_B, rows, a->ds, a->grad_B_stride, g),
                         strided("grad_C", a->grad_C, rows, a->ds, a->grad_C_stride, g),
                         flat("grad_A", a->grad_A, param * a->ds), flat("grad_D", a->grad_D, param),
                         flat("grad_dt_bias", a->grad_dt_bias, param),
                         flat("grad_initial_state", a->grad_initial_state, state),
                         flat("workspace", a->workspace, static_cast<int64_t>(need))};
    KDA_TRY(check_overlaps(ins, outs));

    kda::ScanBwdLaunch L{};
    L.u = rows_of(a->u, a->u_stride, a->in_dtype);
    L.dt = rows_of(a->dt, a->dt_stride, a->in_dtype);
    L.B = rows_of(a->B, a->B_stride, a->in_dtype);
    L.C = rows_of(a->C, a->C_stride, a->in_dtype);
    L.z = rows_of(a->z, a->z_stride, a->in_dtype);
    L.gy = rows_of(a->grad_y, a->grad_y_stride, a->in_dtype);
    L.du = rows_of(a->grad_u, a->grad_u_stride, g);
    L.ddt = rows_of(a->grad_dt, a->grad_dt_stride, g);
    L.dB = rows_of(a->grad_B, a->grad_B_stride, g);
    L.dC = rows_of(a->grad_C, a->grad_C_stride, g);
    L.dz = rows_of(a->grad_z, a->grad_z_stride, g);
    L.A = a->A; L.D = a->D; L.dt_bias = a->dt_bias; L.h0 = a->initial_state; L.dhT = a->grad_final_state;
    L.dA = a->grad_A; L.dD = a->grad_D; L.ddt_bias = a->grad_dt_bias; L.dh0 = a->grad_initial_state;
    L.seq = seq;
    L.dim = a->dim; L.ds = a->ds;
    L.softplus = (a->flags & KDA_SCAN_DT_SOFTPLUS) != 0;
    L.ws = static_cast<float *>(a->workspace);
    L.stream = static_cast<hipStream_t>(a->stream);
    return hip_status(kda::launch_scan_bwd(L), "kda_selective_scan_bwd launch");
}

kda_status kda_short_conv_fwd(const kda_short_conv_args *a) {
    kda::set_last_error("");
    KDA_TRY(check_conv(a));
    if (a->num_seqs == 0 || (static_cast<int64_t>(a->batch) * a->T == 0 && !a->final_state)) return KDA_OK;
    const kda::ConvLaunch L = conv_launch(a);
    const bool step = !a->cu_seqlens && a->T == 1;
    return hip_status(step ? kda::launch_conv_step(L) : kda::launch_conv_fwd(L), "kda_short_conv_fwd launch");
}

kda_status kda_short_conv_step(const kda_short_conv_args *a) {
    kda::set_last_error("");
    KDA_TRY(check_conv(a));
    if (a->cu_seqlens || a->T != 1) return fail(KDA_ERR_BAD_SHAPE, "a step takes T = 1 and no cu_seqlens (T=%d)", a->T);
    if (a->num_seqs == 0) return KDA_OK;
    if (!a->final_state) return fail(KDA_ERR_NULL_POINTER, "final_state is required");
    return hip_status(kda::launch_conv_step(conv_launch(a)), "kda_short_conv_step launch");
}

size_t kda_short_conv_bwd_workspace_bytes(const kda_short_conv_bwd_args *a) {
    if (check_conv_bwd_sizes(a) != KDA_OK) return static_cast<size_t>(-1);
    return kda::conv_bwd_workspace_bytes(static_cast<int64_t>(a->batch) * a->T, a->dim, a->width, a->in_dtype == KDA_DTYPE_BF16);
}

kda_status kda_short_conv_bwd(const kda_short_conv_bwd_args *a) {
    kda::set_last_error("");
    KDA_TRY(check_conv_bwd_sizes(a));
    if (!valid_dtype(a->grad_dtype)) return fail(KDA_ERR_UNSUPPORTED, "grad_dtype=%d", a->grad_dtype);
    const int64_t rows = static_cast<int64_t>(a->batch) * a->T;
    if (rows > 0 && (!a->x || !a->grad_y || !a->grad_x)) return fail(KDA_ERR_NULL_POINTER, "x, grad_y and grad_x are required");
    if (!a->weight || !a->grad_weight) return fail(KDA_ERR_NULL_POINTER, "weight and grad_weight are required");
    KDA_TRY(check_stride("x", a->x, a->x_stride, a->dim, rows, kAnyStride));
    KDA_TRY(check_stride("grad_y", a->grad_y, a->grad_y_stride, a->dim, rows, kAnyStride));
    KDA_TRY(check_stride("grad_x", a->grad_x, a->grad_x_stride, a->dim, rows, kAnyStride));
    const size_t need = kda::conv_bwd_workspace_bytes(rows, a->dim, a->width, a->in_dtype == KDA_DTYPE_BF16);
    if (a->workspace_bytes < need || (need > 0 && !a->workspace))
        return fail(KDA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu < %zu bytes", a->workspace_bytes, need);
    const int64_t states = static_cast<int64_t>(a->num_seqs) * (a->width - 1) * a->dim;
    const int64_t param = a->dim * dsize(a->w_dtype), grad = static_cast<int64_t>(a->dim) * 4;
    const Span ins[] = {strided("x", a->x, rows, a->dim, a->x_stride, a->in_dtype),
                        strided("grad_y", a->grad_y, rows, a->dim, a->grad_y_stride, a->in_dtype),
                        flat("weight", a->weight, param * a->width), flat("bias", a->bias, param),
                        flat("initial_state", a->initial_state, states * dsize(a->in_dtype)),
                        flat("grad_final_state",
                             a->grad_final_state == a->grad_initial_state ? nullptr : a->grad_final_state, states * 4),
                        flat("cu_seqlens", a->cu_seqlens, (static_cast<int64_t>(a->num_seqs) + 1) * 4)};
    const Span outs[] = {strided("grad_x", a->grad_x, rows, a->dim, a->grad_x_stride, a->grad_dtype),
                         flat("grad_weight", a->grad_weight, grad * a->width), flat("grad_bias", a->grad_bias, grad),
                         flat("grad_initial_state", a->grad_initial_state, states * 4),
                         flat("workspace", a->workspace, static_cast<int64_t>(need))};
    KDA_TRY(check_overlaps(ins, outs));

    kda::ConvBwdLaunch L{};
    L.x = rows_of(a->x, a->x_stride, a->in_dtype);
    L.gy = rows_of(a->grad_y, a->grad_y_stride, a->in_dtype);
    L.dx = rows_of(a->grad_x, a->grad_x_stride, a->grad_dtype);
    L.w = a->weight; L.bias = a->bias; L.w_bf16 = a->w_dtype == KDA_DTYPE_BF16;
    L.h0 = a->initial_state; L.dhT = a->grad_final_state;
    L.dw = a->grad_weight; L.db = a->grad_bias; L.dh0 = a->grad_initial_state;
    L.cu = a->cu_seqlens;
    L.N = a->num_seqs; L.T = a->T; L.dim = a->dim; L.width = a->width;
    L.silu = (a->flags & KDA_CONV_SILU) != 0;
    L.ws = static_cast<float *>(a->workspace);
    L.stream = static_cast<hipStream_t>(a->stream);
    return hip_status(kda::launch_conv_bwd(L), "kda_short_conv_bwd launch");
}

kda_status kda_layer_norm_fwd(const kda_layer_norm_args *a) {
    kda::set_last_error("");
    KDA_TRY(check_struct(a));
    KDA_TRY(check_norm_sizes(a->rows, a->dim, a->eps));
    if (!valid_dtype(a->x_dtype) || !valid_dtype(a->out_dtype) || !valid_dtype(a->w_dtype) || !valid_dtype(a->res_dtype))
        return fail(KDA_ERR_UNSUPPORTED, "x_dtype=%d res_dtype=%d w_dtype=%d out_dtype=%d", a->x_dtype, a->res_dtype,
                    a->w_dtype, a->out_dtype);
    if (a->rows == 0) return KDA_OK;
    if (!a->x || !a->y) return fail(KDA_ERR_NULL_POINTER, "x and y are required");
    if ((a->residual == nullptr) != (a->residual_out == nullptr))
        return fail(KDA_ERR_NULL_POINTER, "residual and residual_out come together");
    const int64_t below = norm_stride(a->dim);
    KDA_TRY(check_stride("x", a->x, a->x_stride, a->dim, a->rows, below));
    KDA_TRY(check_stride("y", a->y, a->y_stride, a->dim, a->rows, below));
    KDA_TRY(check_stride("residual", a->residual, a->residual_stride, a->dim, a->rows, below));
    KDA_TRY(check_stride("residual_out", a->residual_out, a->residual_out_stride, a->dim, a->rows, below));
    KDA_TRY(check_grid(kda::norm_fwd_threads(a->rows, a->dim)));
    const int64_t param = a->dim * dsize(a->w_dtype);
    const bool in_place = a->residual == a->residual_out && a->residual_stride == a->residual_out_stride;
    const Span ins[] = {strided("x", a->x, a->rows, a->dim, a->x_stride, a->x_dtype),
                        strided("residual", in_place ? nullptr : a->residual, a->rows, a->dim, a->residual_stride, a->res_dtype),
                        flat("weight", a->weight, param), flat("bias", a->bias, param)};
    const Span outs[] = {strided("y", a->y, a->rows, a->dim, a->y_stride, a->out_dtype),
                         strided("residual_out", a->residual_out, a->rows, a->dim, a->residual_out_stride, a->res_dtype)};
    KDA_TRY(check_overlaps(ins, outs));

    kda::NormFwdLaunch L{};
    L.x = rows_of(a->x, a->x_stride, a->x_dtype);
    L.res = rows_of(a->residual, a->residual_stride, a->res_dtype);
    L.y = rows_of(a->y, a->y_stride, a->out_dtype);
    L.res_out = rows_of(a->residual_out, a->residual_out_stride, a->res_dtype);
    L.w = a->weight; L.b = a->bias; L.w_bf16 = a->w_dtype == KDA_DTYPE_BF16;
    L.rows = a->rows; L.dim = a->dim; L.eps = a->eps;
    L.stream = static_cast<hipStream_t>(a->stream);
    return hip_status(kda::launch_norm_fwd(L), "kda_layer_norm_fwd launch");
}

size_t kda_layer_norm_bwd_workspace_bytes(const kda_layer_norm_bwd_args *a) {
    if (check_struct(a) != KDA_OK || check_norm_sizes(a->rows, a->dim, a->eps) != KDA_OK) return static_cast<size_t>(-1);
    return a->grad_weight || a->grad_bias ? kda::norm_bwd_workspace_bytes(a->rows, a->dim) : 0;
}

kda_status kda_layer_norm_bwd(const kda_layer_norm_bwd_args *a) {
    kda::set_last_error("");
    KDA_TRY(check_struct(a));
    KDA_TRY(check_norm_sizes(a->rows, a->dim, a->eps));
    if (!valid_dtype(a->x_dtype) || !valid_dtype(a->gy_dtype) || !valid_dtype(a->w_dtype) || !valid_dtype(a->res_dtype) ||
        !valid_dtype(a->grad_dtype))
        return fail(KDA_ERR_UNSUPPORTED, "x_dtype=%d gy_dtype=%d res_dtype=%d w_dtype=%d grad_dtype=%d", a->x_dtype,
                    a->gy_dtype, a->res_dtype, a->w_dtype, a->grad_dtype);
    if (a->rows > 0 && (!a->x || !a->grad_y || !a->grad_x))
        return fail(KDA_ERR_NULL_POINTER, "x, grad_y and grad_x are required");
    const int64_t below = norm_stride(a->dim);
    KDA_TRY(check_stride("x", a->x, a->x_stride, a->dim, a->rows, below));
    KDA_TRY(check_stride("grad_y", a->grad_y, a->grad_y_stride, a->dim, a->rows, below));
    KDA_TRY(check_stride("grad_residual", a->grad_residual, a->grad_residual_stride, a->dim, a->rows, below));
    KDA_TRY(check_stride("grad_x", a->grad_x, a->grad_x_stride, a->dim, a->rows, below));
    const size_t need = kda_layer_norm_bwd_workspace_bytes(a);
    if (a->workspace_bytes < need || (need > 0 && !a->workspace))
        return fail(KDA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu < %zu bytes", a->workspace_bytes, need);
    const int64_t param = a->dim * dsize(a->w_dtype), grad = static_cast<int64_t>(a->dim) * 4;
    const Span ins[] = {strided("x", a->x, a->rows, a->dim, a->x_stride, a->x_dtype),
                        strided("grad_y", a->grad_y, a->rows, a->dim, a->grad_y_stride, a->gy_dtype),
                        strided("grad_residual", a->grad_residual, a->rows, a->dim, a->grad_residual_stride, a->res_dtype),
                        flat("weight", a->weight, param)};
    const Span outs[] = {strided("grad_x", a->grad_x, a->rows, a->dim, a->grad_x_stride, a->grad_dtype),
                         flat("grad_weight", a->grad_weight, grad), flat("grad_bias", a->grad_bias, grad),
                         flat("workspace", a->workspace, static_cast<int64_t>(need))};
    KDA_TRY(check_overlaps(ins, outs));

    kda::NormBwdLaunch L{};
    L.x = rows_of(a->x, a->x_stride, a->x_dtype);
    L.gy = rows_of(a->grad_y, a->grad_y_stride, a->gy_dtype);
    L.gres = rows_of(a->grad_residual, a->grad_residual_stride, a->res_dtype);
    L.dx = rows_of(a->grad_x, a->grad_x_stride, a->grad_dtype);
    L.w = a->weight; L.w_bf16 = a->w_dtype == KDA_DTYPE_BF16;
    L.dw = a->grad_weight; L.db = a->grad_bias;
    L.rows = a->rows; L.dim = a->dim; L.eps = a->eps;
    L.ws = need > 0 ? static_cast<float *>(a->workspace) : nullptr;
    L.stream = static_cast<hipStream_t>(a->stream);
    return hip_status(kda::launch_norm_bwd(L), "kda_layer_norm_bwd launch");
}

}  // extern "C"
