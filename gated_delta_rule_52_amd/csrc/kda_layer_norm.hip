// kda_layer_norm.hip - layer norm, forward and gradients, and the column sum of parameter gradients, gfx950.
//
//     y = (s - mean) rstd w + b, s = x + residual;      with g = dy w, xh = (s - mean) rstd:
//     dx = rstd (g - mean(g) - xh mean(g xh)) + dres,   dw = sum dy xh,   db = sum dy
//
// Bound by HBM.  A row stays in registers between its one read and its one write, so the deviations are summed
// around a mean already known and cost no memory.  A row is held by LANES lanes of a wave (short rows:
// several per wave) or by a workgroup of WAVES waves; a lane holds U units of 8 elements.  The backward pass
// gives each workgroup a share of the rows and keeps its part of dw and db in registers over all of them:
// one partial row per workgroup, summed by the column sum in a fixed order.
#include "kda_layer.h"

namespace kda {

namespace {

// A lane's row of a tensor: the address of the workgroup's first one, which is uniform, and the byte offset from there.
struct Walk {
    char *at;
    uint32_t off;
    int bf16;
    __device__ __forceinline__ Walk(const Rows &r, int64_t row, int sub) {
        const int e = r.bf16 ? 2 : 4;
        at = static_cast<char *>(r.p) + row * r.stride * e;
        off = static_cast<uint32_t>(sub) * static_cast<uint32_t>(r.stride * e);
        bf16 = r.bf16;
    }
    __device__ __forceinline__ char *unit(int col) const { return at + (off + static_cast<uint32_t>(col) * (bf16 ? 2 : 4)); }
};
// 8 elements, 16 bytes at a time wherever the row starts (the hardware takes these accesses at any element's
// alignment); of a row that has only `left` elements these, singly, and zeros.
typedef uint32_t any4 __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ void load8(const char *p, int bf16, int left, float (&x)[8]) {
    if (left < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = i >= left ? 0.f : bf16 ? bf16_to_f32(reinterpret_cast<const uint16_t *>(p)[i]) : reinterpret_cast<const float *>(p)[i];
    } else if (bf16) {
        const any4 v = *reinterpret_cast<const any4 *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(v[i] << 16);
            x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
        }
    } else {
        const any4 a = reinterpret_cast<const any4 *>(p)[0], b = reinterpret_cast<const any4 *>(p)[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = __uint_as_float(a[i]);
            x[4 + i] = __uint_as_float(b[i]);
        }
    }
}
__device__ __forceinline__ void store8(char *p, int bf16, int left, const float (&x)[8]) {
    if (left < 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= left) break;
            if (bf16) reinterpret_cast<uint16_t *>(p)[i] = to_bf16(x[i]);
            else reinterpret_cast<float *>(p)[i] = x[i];
        }
    } else if (bf16) {
        any4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = to_bf16(x[2 * i]) | static_cast<uint32_t>(to_bf16(x[2 * i + 1])) << 16;
        *reinterpret_cast<any4 *>(p) = v;
    } else {
        any4 a, b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = __float_as_uint(x[i]);
            b[i] = __float_as_uint(x[4 + i]);
        }
        reinterpret_cast<any4 *>(p)[0] = a;
        reinterpret_cast<any4 *>(p)[1] = b;
    }
}
__device__ __forceinline__ void load_param(const void *p, int bf16, int col, int left, float (&x)[8]) {
    load8(static_cast<const char *>(p) + static_cast<int64_t>(col) * (bf16 ? 2 : 4), bf16, left, x);
}

// First column of unit u of a lane among the SPAN that share a row.
template <int SPAN>
__device__ __forceinline__ int first_col(int lane, int u) {
    return (u * SPAN + lane) * 8;
}

// The sum over each LANES neighbouring lanes, in all of them: lane moves only, no LDS.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float x) {
    x += dpp_mov<0xB1>(x);   // quad permute [1, 0, 3, 2]
    x += dpp_mov<0x4E>(x);   // quad permute [2, 3, 0, 1]
    x += dpp_mov<0x141>(x);  // mirror in 8 lanes
    x += dpp_mov<0x140>(x);  // mirror in 16
    if constexpr (LANES >= 32) x = swap_add(x, x, true);
    if constexpr (LANES >= 64) x = swap_add(x, x, false);
    return x;
}

// What a row's lanes need of the whole row.  Each wave takes its own mean as pivot and sums the squared
// deviations from it and g times the deviations; one exchange then moves every sum to the row's mean,
//     sum (x - m)^2 = sum_w [M2_w + n_w (p_w - m)^2],   sum g (x - m) = sum_w [S_w + (p_w - m) G_w],
// which loses nothing to a mean far above the spread and needs one barrier per row instead of five.
struct RowSums {
    float mean, rstd, g, gx;  // g: sum of g, gx: sum of g times the normalised x (0 without g)
};
// BACK: a row's last unit was moved back inside the row, and its first elements are the neighbour's; otherwise the
// values past the row are zeros.
template <int LANES, int WAVES, int U, bool GRAD, bool BACK>
__device__ __forceinline__ RowSums row_sums(const float (&x)[U][8], const float (&g)[U][8], const float (&w)[U][8], int lane,
                                            int dim, float inv_n, float n, float inv_dim, float eps, float (*shared)[4]) {
    constexpr int SPAN = LANES * WAVES;
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int left = dim - first_col<SPAN>(lane, u);
        if (!BACK || left >= 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) s += x[u][i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) s += i >= 8 - left ? x[u][i] : 0.f;
        }
    }
    const float p = lanes_sum<LANES>(s) * inv_n;
    float m2 = 0.f, sg = 0.f, sx = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int left = dim - first_col<SPAN>(lane, u);
        if (left >= 8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = x[u][i] - p;
                m2 = fmaf(d, d, m2);
                if (GRAD) sx = fmaf(g[u][i] * w[u][i], d, sx);
                if (GRAD && BACK) sg = fmaf(g[u][i], w[u][i], sg);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool in = BACK ? i >= 8 - left : i < left;
                const float d = in ? x[u][i] - p : 0.f;
                m2 = fmaf(d, d, m2);
                if (GRAD) sx = fmaf(g[u][i] * w[u][i], d, sx);
                if (GRAD && BACK) sg = fmaf(in ? g[u][i] : 0.f, w[u][i], sg);
            }
        }
        if (GRAD && !BACK) {
#pragma unroll
            for (int i = 0; i < 8; ++i) sg = fmaf(g[u][i], w[u][i], sg);
        }
    }
    m2 = lanes_sum<LANES>(m2);
    if (GRAD) {
        sg = lanes_sum<LANES>(sg);
        sx = lanes_sum<LANES>(sx);
    }
    RowSums r{p, 0.f, sg, sx};
    if constexpr (WAVES > 1) {
        const int wave = lane >> 6;
        if ((lane & 63) == 0) {
            shared[2 * wave][0] = n;
            shared[2 * wave][1] = p;
            shared[2 * wave][2] = m2;
            shared[2 * wave][3] = sg;
            shared[2 * wave + 1][0] = sx;
        }
        __syncthreads();
        float total = 0.f;
#pragma unroll 4
        for (int w = 0; w < WAVES; ++w) total = fmaf(shared[2 * w][0], shared[2 * w][1], total);
        r.mean = total * inv_dim;
        m2 = sg = sx = 0.f;
#pragma unroll 4
        for (int w = 0; w < WAVES; ++w) {
            const float off = shared[2 * w][1] - r.mean;
            m2 += fmaf(shared[2 * w][0] * off, off, shared[2 * w][2]);
            if (GRAD) {
                sg += shared[2 * w][3];
                sx += fmaf(off, shared[2 * w][3], shared[2 * w + 1][0]);
            }
        }
        r.g = sg;
        r.gx = sx;
    }
    const float var = fmaf(m2, inv_dim, eps);  // the instruction takes a denormal (eps of 0, tiny values) as 0
    r.rstd = var < 0x1p-120f ? __builtin_amdgcn_rsqf(var * 0x1p60f) * 0x1p30f : __builtin_amdgcn_rsqf(var);
    r.gx *= r.rstd;
    return r;
}

// Elements of a row that a wave holds (all of them where a row is one wave's), and its inverse.
template <int LANES, int WAVES, int U>
__device__ __forceinline__ float wave_count(int lane, int dim) {
    if constexpr (WAVES == 1) return static_cast<float>(dim);
    float n = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int left = dim - first_col<LANES * WAVES>(lane, u);
        n += static_cast<float>(left < 0 ? 0 : left > 8 ? 8 : left);
    }
    return lanes_sum<LANES>(n);
}

template <int LANES, int WAVES>
constexpr int norm_threads() { return WAVES <= 4 ? 256 : 64 * WAVES; }
template <int LANES, int WAVES>
constexpr int rows_per_group() { return norm_threads<LANES, WAVES>() / (LANES * WAVES); }

// As the gradients below, a row's last unit is moved back inside the row; TINY rows, of fewer than 8 elements, are read
// singly.  residual_out is written behind the sums, when every lane of the row has read what it may replace.
template <int LANES, int WAVES, int U, bool TINY>
__global__ void __launch_bounds__((norm_threads<LANES, WAVES>())) norm_fwd_kernel(NormFwdLaunch P) {
    constexpr int SPAN = LANES * WAVES, ROWS = rows_per_group<LANES, WAVES>();
    __shared__ float shared[2 * WAVES][4];
    const int lane = threadIdx.x % SPAN;
    int sub = threadIdx.x / SPAN;
    const int64_t base = static_cast<int64_t>(blockIdx.x) * ROWS;
    const bool live = base + sub < P.rows;
    if (!live) sub = static_cast<int>(P.rows - 1 - base);  // keeps the wave whole for the sums; stores nothing
    const Walk wx(P.x, base, sub), wr(P.res, base, sub), wo(P.res_out, base, sub), wy(P.y, base, sub);
    const float n = wave_count<LANES, WAVES, U>(lane, P.dim), inv_dim = 1.f / static_cast<float>(P.dim);
    float x[U][8];
    int col[U], left[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = first_col<SPAN>(lane, u);
        col[u] = TINY ? 0 : c + 8 > P.dim ? P.dim - 8 : c;
        left[u] = c >= P.dim ? 0 : TINY ? P.dim : 8;
        const int all = TINY ? left[u] : 8;
        load8(wx.unit(col[u]), P.x.bf16, all, x[u]);
        if (P.res.p) {
            float r[8];
            load8(wr.unit(col[u]), P.res.bf16, all, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[u][i] += r[i];
        }
    }
    const RowSums s = row_sums<LANES, WAVES, U, false, !TINY>(x, x, x, lane, P.dim, n > 0.f ? 1.f / n : 0.f, n, inv_dim, P.eps, shared);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (left[u] == 0 || !live) continue;
        const int all = TINY ? left[u] : 8;
        if (P.res_out.p) store8(wo.unit(col[u]), P.res_out.bf16, all, x[u]);
        float w[8], b[8] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.f;
        if (P.w) load_param(P.w, P.w_bf16, col[u], all, w);
        if (P.b) load_param(P.b, P.w_bf16, col[u], all, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[u][i] = fmaf((x[u][i] - s.mean) * s.rstd, w[i], b[i]);
        store8(wy.unit(col[u]), P.y.bf16, all, x[u]);
    }
}

// The next rows' loads are issued before a row's sums and wait in registers behind its stores, so that the exchange
// and its barrier leave HBM busy.  Loads carry no branch: the unit that a row's end cuts is moved back inside,
// computes some of its neighbour's elements again and stores the same values; only the sums leave them out.  That
// takes rows of 8 elements; TINY ones are read singly, by one lane each.
template <int U, bool Bf16, bool TINY>
struct RawRow {
    any4 v[U][Bf16 && !TINY ? 1 : 2];
    // lanes with nothing to read (left <= 0) read what their neighbour does
    __device__ __forceinline__ void load(const char *at, uint32_t off, const uint32_t (&col)[U], int left) {
        if constexpr (TINY) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[0][i / 4][i % 4] = 0;
                if (i >= left) continue;
                if (Bf16) v[0][i / 4][i % 4] = static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(at + off)[i]) << 16;
                else v[0][i / 4][i % 4] = reinterpret_cast<const uint32_t *>(at + off)[i];
            }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < (Bf16 ? 1 : 2); ++k)
                    v[u][k] = reinterpret_cast<const any4 *>(at + (off + col[u] * (Bf16 ? 2 : 4)))[k];
        }
    }
    __device__ __forceinline__ void widen(float (&x)[U][8]) const {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if constexpr (Bf16 && !TINY) x[u][i] = __uint_as_float(i & 1 ? v[u][0][i / 2] & 0xffff0000u : v[u][0][i / 2] << 16);
                else x[u][i] = __uint_as_float(v[u][i / 4][i % 4]);
    }
};
template <int LANES, int WAVES, int U, bool XBf16, bool GBf16, bool TINY>
__global__ void __launch_bounds__((norm_threads<LANES, WAVES>())) norm_bwd_kernel(NormBwdLaunch P) {
    constexpr int SPAN = LANES * WAVES, ROWS = rows_per_group<LANES, WAVES>();
    constexpr bool AHEAD = U == 1 || WAVES <= 8 || (XBf16 && GBf16);  // 16 waves leave the others no registers for it
    // the residual's gradient too is loaded before the sums where registers allow (8,192 x 4,096 bf16 with one: 61 us
    // against 69; one unit per lane: 58 against 55, as fewer waves are resident)
    constexpr bool EARLY = U == 2 && WAVES <= 8;
    __shared__ float shared[2][ROWS][2 * WAVES][4];     // two rows' exchanges: one barrier each
    __shared__ float fold[ROWS > 1 ? 256 * 8 : 1];
    const int lane = threadIdx.x % SPAN, sub = ROWS > 1 ? threadIdx.x / SPAN : 0;
    float w[U][8], dw[U][8], db[U][8], x[U][8], g[U][8];
    uint32_t col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int c = first_col<SPAN>(lane, u);
        col[u] = TINY ? 0 : c + 8 > P.dim ? P.dim - 8 : c;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[u][i] = 1.f;
            dw[u][i] = db[u][i] = 0.f;
        }
        if (P.w) load_param(P.w, P.w_bf16, col[u], TINY ? P.dim : 8, w[u]);
    }
    const int tiny = lane == 0 ? P.dim : 0;  // elements of a TINY row
    const float n = wave_count<LANES, WAVES, U>(lane, P.dim), inv_n = n > 0.f ? 1.f / n : 0.f;
    const float inv_dim = 1.f / static_cast<float>(P.dim);
    auto row_at = [](const Rows &r, int64_t row) { return static_cast<char *>(r.p) + row * r.stride * (r.bf16 ? 2 : 4); };
    auto step = [](const Rows &r) { return static_cast<uint32_t>(r.stride) * (r.bf16 ? 2 : 4); };
    RawRow<U, XBf16, TINY> nx;
    RawRow<U, GBf16, TINY> ng;
    // of the rows from `base` on this lane's, or the last one there is
    auto load = [&](int64_t base) {
        const int last = P.rows - 1 - base < ROWS ? static_cast<int>(P.rows - 1 - base) : ROWS - 1;
        const uint32_t k = sub < last ? sub : last;
        nx.load(row_at(P.x, base), k * step(P.x), col, tiny);
        ng.load(row_at(P.gy, base), k * step(P.gy), col, tiny);
    };
    const int64_t stride = static_cast<int64_t>(gridDim.x) * ROWS;
    int64_t base = static_cast<int64_t>(blockIdx.x) * ROWS;
    if (AHEAD) load(base);
    // whole rounds for every lane of the workgroup: lanes past the last row store and count nothing
    for (int round = 0; base < P.rows; base += stride, round ^= 1) {
        if (!AHEAD) load(base);
        nx.widen(x);
        ng.widen(g);
        const bool live = ROWS == 1 || base + sub < P.rows;
        const char *res = row_at(P.gres, base) + (live ? sub : 0) * step(P.gres);
        any4 rv[U][2];
        if (EARLY && P.gres.p) {
#pragma unroll
            for (int u = 0; u < U; ++u) {  // both halves of a bf16 unit are its one
                const char *p = res + col[u] * (P.gres.bf16 ? 2 : 4);
                rv[u][0] = *reinterpret_cast<const any4 *>(p);
                rv[u][1] = *reinterpret_cast<const any4 *>(p + (P.gres.bf16 ? 0 : 16));
            }
        }
        if (AHEAD) load(base + stride < P.rows ? base + stride : base);
        const RowSums s = row_sums<LANES, WAVES, U, true, !TINY>(x, g, w, lane, P.dim, inv_n, n, inv_dim, P.eps, shared[round][sub]);
        const float m1 = s.g * inv_dim, m2 = s.gx * inv_dim;
        if (live) {
            char *dx = row_at(P.dx, base) + sub * step(P.dx);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int left = TINY ? tiny : first_col<SPAN>(lane, u) < P.dim ? 8 : 0;
                float r[8] = {};
                if (!EARLY && P.gres.p) {
                    load8(res + col[u] * (P.gres.bf16 ? 2 : 4), P.gres.bf16, TINY ? tiny : 8, r);
                } else if (P.gres.p) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t h = i & 1 ? rv[u][0][i / 2] & 0xffff0000u : rv[u][0][i / 2] << 16;
                        r[i] = __uint_as_float(P.gres.bf16 ? h : rv[u][i / 4][i % 4]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float xh = (x[u][i] - s.mean) * s.rstd;  // past a TINY row g is 0
                    dw[u][i] = fmaf(g[u][i], xh, dw[u][i]);
                    db[u][i] += g[u][i];
                    r[i] = fmaf(s.rstd, fmaf(g[u][i], w[u][i], -fmaf(xh, m2, m1)), r[i]);
                }
                if (left > 0) store8(dx + col[u] * (P.dx.bf16 ? 2 : 4), P.dx.bf16, TINY ? tiny : 8, r);
            }
        }
    }
    if (!P.ws) return;
    // one partial row of dw and of db per workgroup
    float *pw = P.ws + static_cast<int64_t>(blockIdx.x) * 2 * P.dim, *pb = pw + P.dim;
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float (&v)[8] = half ? db[u] : dw[u];
            if constexpr (ROWS > 1) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < 8; ++i) fold[i * 256 + threadIdx.x] = v[i];
                __syncthreads();
                if (sub == 0) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float s = 0.f;
                        for (int k = 0; k < ROWS; ++k) s += fold[i * 256 + k * SPAN + lane];
                        v[i] = s;
                    }
                }
            }
            if (sub == 0 && first_col<SPAN>(lane, u) < P.dim)
                store8(reinterpret_cast<char *>((half ? pb : pw) + col[u]), 0, TINY ? P.dim : 8, v);
        }
    }
}

// 16 columns by 64 slices of the parts per workgroup: rows of 64 bytes, slices joined in LDS.  Eight loads in flight
// per thread (1,024 parts of 256 columns: 4.3 us, one by one 7.9).
__global__ void __launch_bounds__(1024) column_sum_kernel(const float *in, int64_t ld, int parts, ColumnSums to) {
    __shared__ float s[64][17];
    const int c = threadIdx.x & 15, k = threadIdx.x >> 4;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 16 + c, all = to.cols[0] + to.cols[1] + to.cols[2];
    float a = 0.f;
    if (col < all) {
        const float *at = in + col;
        int p = k;
        for (; p + 448 < parts; p += 512) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = at[(p + 64 * i) * ld];
#pragma unroll
            for (int i = 0; i < 8; ++i) a += v[i];
        }
        for (; p + 64 < parts; p += 128) {
            const float v = at[p * ld], w = at[(p + 64) * ld];
            a += v;
            a += w;
        }
        if (p < parts) a += at[p * ld];
    }
    s[k][c] = a;
    __syncthreads();
#pragma unroll
    for (int h = 32; h >= 1; h >>= 1) {
        if (k < h) s[k][c] += s[k + h][c];
        __syncthreads();
    }
    if (k > 0) return;
    int64_t at = col;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if (at >= 0 && at < to.cols[i] && to.out[i]) to.out[i][at] = s[0][c];
        at -= to.cols[i];
    }
}

// Rows per workgroup of the backward pass, as its launch arranges them.
int rows_of(int dim) {
    return dim <= 128 ? 16 : dim <= 256 ? 8 : dim <= 1024 ? 4 : dim <= 2048 ? 2 : 1;
}
// The backward pass's workgroups: no more than are resident at once, and of these as few as keep HBM busy, as each
// adds a partial row to sum (32,768 x 1,024 bf16: 45 us with 768, 47 with 512, 52 with 1,024; 262,144 x 128: 45
// with 1,024, 46 with 768, 54 with 512; 8,192 x 4,096: 53 with 512, 61 with 256).
int64_t bwd_groups(int64_t rows, int dim) {
    const int64_t whole = (rows + rows_of(dim) - 1) / rows_of(dim);
    const int64_t most = dim <= 512 ? 1024 : dim <= 2048 ? 768 : dim <= 4096 ? 512 : 256;
    return whole < most ? whole : most;
}

}  // namespace

void launch_column_sum(const float *in, int64_t ld, int parts, const ColumnSums &to, hipStream_t stream) {
    const int64_t cols = to.cols[0] + to.cols[1] + to.cols[2];
    if (cols > 0) column_sum_kernel<<<static_cast<unsigned>((cols + 15) / 16), 1024, 0, stream>>>(in, ld, parts, to);
}
int64_t column_sum_threads(int64_t cols) { return (cols + 15) / 16 * 1024; }

template <int LANES, int WAVES, int U, bool TINY = false>
static void launch_fwd(const NormFwdLaunch &P) {
    constexpr int ROWS = rows_per_group<LANES, WAVES>();
    norm_fwd_kernel<LANES, WAVES, U, TINY>
        <<<static_cast<unsigned>((P.rows + ROWS - 1) / ROWS), norm_threads<LANES, WAVES>(), 0, P.stream>>>(P);
}

// The smallest arrangement that holds a row: 16 lanes (to 128 elements), 32, a wave (to 1,024), then several.
hipError_t launch_norm_fwd(const NormFwdLaunch &P) {
    if (P.dim < 8) launch_fwd<16, 1, 1, true>(P);
    else if (P.dim <= 128) launch_fwd<16, 1, 1>(P);
    else if (P.dim <= 256) launch_fwd<32, 1, 1>(P);
    else if (P.dim <= 512) launch_fwd<64, 1, 1>(P);
    else if (P.dim <= 1024) launch_fwd<64, 1, 2>(P);
    else if (P.dim <= 2048) launch_fwd<64, 4, 1>(P);
    else if (P.dim <= 4096) launch_fwd<64, 4, 2>(P);
    else if (P.dim <= 8192) launch_fwd<64, 8, 2>(P);
    else launch_fwd<64, 16, 2>(P);
    return hipGetLastError();
}
int64_t norm_fwd_threads(int64_t rows, int dim) {
    const int lanes = dim <= 128 ? 16 : dim <= 256 ? 32 : dim <= 1024 ? 64 : dim <= 4096 ? 256 : dim <= 8192 ? 512 : 1024;
    const int group = lanes < 256 ? 256 : lanes;
    return (rows + group / lanes - 1) / (group / lanes) * group;
}

size_t norm_bwd_workspace_bytes(int64_t rows, int dim) {
    return static_cast<size_t>(bwd_groups(rows, dim)) * 2 * dim * 4;
}

template <int LANES, int WAVES, int U, bool TINY = false>
static void launch_bwd(const NormBwdLaunch &P, int64_t groups) {
    const unsigned grid = static_cast<unsigned>(groups);
    constexpr int threads = norm_threads<LANES, WAVES>();
    if (P.x.bf16 && P.gy.bf16) norm_bwd_kernel<LANES, WAVES, U, true, true, TINY><<<grid, threads, 0, P.stream>>>(P);
    else if (P.x.bf16) norm_bwd_kernel<LANES, WAVES, U, true, false, TINY><<<grid, threads, 0, P.stream>>>(P);
    else if (P.gy.bf16) norm_bwd_kernel<LANES, WAVES, U, false, true, TINY><<<grid, threads, 0, P.stream>>>(P);
    else norm_bwd_kernel<LANES, WAVES, U, false, false, TINY><<<grid, threads, 0, P.stream>>>(P);
}

hipError_t launch_norm_bwd(const NormBwdLaunch &P) {
    const int64_t groups = bwd_groups(P.rows, P.dim);
    // As many units per lane as registers hold the next row's loads beside: rows in fewer waves spend less on the
    // exchange (8,192 x 8,192 bf16: 94 us with 8 waves of two units, 124 with 16 of one).
    if (groups > 0) {
        if (P.dim < 8) launch_bwd<16, 1, 1, true>(P, groups);
        else if (P.dim <= 128) launch_bwd<16, 1, 1>(P, groups);
        else if (P.dim <= 256) launch_bwd<32, 1, 1>(P, groups);
        else if (P.dim <= 512) launch_bwd<64, 1, 1>(P, groups);
        else if (P.dim <= 1024) launch_bwd<64, 1, 2>(P, groups);
        else if (P.dim <= 2048) launch_bwd<64, 2, 2>(P, groups);
        else if (P.dim <= 4096) launch_bwd<64, 4, 2>(P, groups);
        else if (P.dim <= 8192) launch_bwd<64, 8, 2>(P, groups);
        else launch_bwd<64, 16, 2>(P, groups);
    }
    if (P.dw || P.db)
        launch_column_sum(P.ws, 2 * P.dim, static_cast<int>(groups), {{P.dw, P.db, nullptr}, {P.dim, P.dim, 0}}, P.stream);
    return hipGetLastError();
}

}  // namespace kda
