// kda_layer_norm.hip - layer norm, forward and gradients, and the column sum of parameter gradients, gfx950.
//
//     y = (s - mean) rstd w + b, s = x + residual;      with g = dy w, xh = (s - mean) rstd:
//     dx = rstd (g - mean(g) - xh mean(g xh)) + dres,   dw = sum dy xh,   db = sum dy
//
// Bound by HBM.  A row stays in registers between its one read and its one write, so mean and variance take
// two exact passes over registers and cost no memory.  A row is held by LANES lanes of a wave (short rows:
// several per wave) or by a workgroup of WAVES waves; a lane holds U units of 8 elements.  The backward pass
// gives each workgroup a share of the rows and keeps its part of dw and db in registers over all of them:
// one partial row per workgroup, summed by the column sum in a fixed order.
#include "kda_layer.h"

namespace kda {

namespace {

// 8 elements of a row from `col` on, 16 bytes at a time wherever the row starts (the hardware takes these accesses
// at any element's alignment); the row's last elements singly.
typedef uint32_t any4 __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ void load8(const Rows &r, int64_t row, int col, int dim, float (&x)[8]) {
    const int64_t at = row * r.stride + col;
    if (col + 8 > dim) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = col + i < dim ? r.get(row, col + i) : 0.f;
    } else if (r.bf16) {
        const any4 v = *reinterpret_cast<const any4 *>(static_cast<const uint16_t *>(r.p) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(v[i] << 16);
            x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
        }
    } else {
        const any4 *p = reinterpret_cast<const any4 *>(static_cast<const float *>(r.p) + at);
        const any4 a = p[0], b = p[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = __uint_as_float(a[i]);
            x[4 + i] = __uint_as_float(b[i]);
        }
    }
}
__device__ __forceinline__ void store8(const Rows &r, int64_t row, int col, int dim, const float (&x)[8]) {
    const int64_t at = row * r.stride + col;
    if (col + 8 > dim) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < dim) r.put(row, col + i, x[i]);
    } else if (r.bf16) {
        any4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = to_bf16(x[2 * i]) | static_cast<uint32_t>(to_bf16(x[2 * i + 1])) << 16;
        *reinterpret_cast<any4 *>(static_cast<uint16_t *>(r.p) + at) = v;
    } else {
        any4 *p = reinterpret_cast<any4 *>(static_cast<float *>(r.p) + at);
        any4 a, b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = __float_as_uint(x[i]);
            b[i] = __float_as_uint(x[4 + i]);
        }
        p[0] = a;
        p[1] = b;
    }
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
template <int LANES, int WAVES, int U, bool GRAD>
__device__ __forceinline__ RowSums row_sums(const float (&x)[U][8], const float (&g)[U][8], int lane, int dim, float eps,
                                            float (*shared)[4]) {
    constexpr int SPAN = LANES * WAVES;
    float s = 0.f, n = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int in = dim - first_col<SPAN>(lane, u);  // elements of the unit that the row has
        n += static_cast<float>(in < 0 ? 0 : in > 8 ? 8 : in);
#pragma unroll
        for (int i = 0; i < 8; ++i) s += x[u][i];  // zeros past the row
    }
    s = lanes_sum<LANES>(s);
    if constexpr (WAVES > 1) n = lanes_sum<LANES>(n);
    else n = static_cast<float>(dim);
    const float p = n > 0.f ? s / n : 0.f;
    float m2 = 0.f, sg = 0.f, sx = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = first_col<SPAN>(lane, u) + i < dim ? x[u][i] - p : 0.f;
            m2 = fmaf(d, d, m2);
            if (GRAD) {
                sg += g[u][i];
                sx = fmaf(g[u][i], d, sx);
            }
        }
    m2 = lanes_sum<LANES>(m2);
    if (GRAD) {
        sg = lanes_sum<LANES>(sg);
        sx = lanes_sum<LANES>(sx);
    }
    RowSums r{p, 0.f, sg, sx};
    if constexpr (WAVES > 1) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
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
        r.mean = total / static_cast<float>(dim);
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
    r.rstd = 1.f / sqrtf(m2 / static_cast<float>(dim) + eps);
    r.gx *= r.rstd;
    return r;
}

template <int LANES, int WAVES>
constexpr int norm_threads() { return WAVES == 1 ? 256 : 64 * WAVES; }
template <int LANES, int WAVES>
constexpr int rows_per_group() { return WAVES == 1 ? 256 / LANES : 1; }

template <int LANES, int WAVES, int U>
__global__ void __launch_bounds__((norm_threads<LANES, WAVES>())) norm_fwd_kernel(NormFwdLaunch P) {
    constexpr int SPAN = LANES * WAVES;
    __shared__ float shared[2 * WAVES][4];
    const int lane = threadIdx.x % SPAN;
    int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_group<LANES, WAVES>() + threadIdx.x / SPAN;
    const bool live = row < P.rows;
    if (WAVES == 1 && !live) row = P.rows - 1;  // keeps the wave whole for the sums; stores nothing
    float x[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int col = first_col<SPAN>(lane, u);
        if (col < P.dim) {
            load8(P.x, row, col, P.dim, x[u]);
            if (P.res.p) {
                float r[8];
                load8(P.res, row, col, P.dim, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[u][i] += r[i];
                if (live) store8(P.res_out, row, col, P.dim, x[u]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[u][i] = 0.f;
        }
    }
    const RowSums s = row_sums<LANES, WAVES, U, false>(x, x, lane, P.dim, P.eps, shared);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int col = first_col<SPAN>(lane, u);
        if (col >= P.dim || !live) continue;
        float w[8], b[8];
        const Rows wr{const_cast<void *>(P.w), 0, P.w_bf16}, br{const_cast<void *>(P.b), 0, P.w_bf16};
        if (P.w) load8(wr, 0, col, P.dim, w);
        if (P.b) load8(br, 0, col, P.dim, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float n = (x[u][i] - s.mean) * s.rstd;
            x[u][i] = fmaf(n, P.w ? w[i] : 1.f, P.b ? b[i] : 0.f);
        }
        store8(P.y, row, col, P.dim, x[u]);
    }
}

template <int LANES, int WAVES, int U>
__global__ void __launch_bounds__((norm_threads<LANES, WAVES>())) norm_bwd_kernel(NormBwdLaunch P) {
    constexpr int SPAN = LANES * WAVES, ROWS = rows_per_group<LANES, WAVES>();
    __shared__ float shared[2][2 * WAVES][4];  // two rows' exchanges: one barrier each
    __shared__ float fold[ROWS > 1 ? 256 * 8 : 1];
    const int lane = threadIdx.x % SPAN, sub = threadIdx.x / SPAN;
    float w[U][8], dw[U][8], db[U][8], x[U][8], g[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int col = first_col<SPAN>(lane, u);
        const Rows wr{const_cast<void *>(P.w), 0, P.w_bf16};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[u][i] = 1.f;
            x[u][i] = g[u][i] = dw[u][i] = db[u][i] = 0.f;
        }
        if (P.w && col < P.dim) load8(wr, 0, col, P.dim, w[u]);
    }
    const int64_t stride = static_cast<int64_t>(gridDim.x) * ROWS;
    int64_t base = static_cast<int64_t>(blockIdx.x) * ROWS;
    // whole rounds for every lane of the workgroup: rows past the end are computed from the last and dropped
    for (int round = 0; base < P.rows; base += stride, round ^= 1) {
        const bool live = base + sub < P.rows;
        const int64_t row = live ? base + sub : P.rows - 1;
        float gy[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int col = first_col<SPAN>(lane, u);
            if (col < P.dim) {
                load8(P.x, row, col, P.dim, x[u]);
                load8(P.gy, row, col, P.dim, gy[u]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) gy[u][i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) g[u][i] = gy[u][i] * w[u][i];
        }
        const RowSums s = row_sums<LANES, WAVES, U, true>(x, g, lane, P.dim, P.eps, shared[round]);
        const float m1 = s.g / static_cast<float>(P.dim), m2 = s.gx / static_cast<float>(P.dim);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int col = first_col<SPAN>(lane, u);
            float r[8] = {}, xh[8];
            if (P.gres.p && live && col < P.dim) load8(P.gres, row, col, P.dim, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                xh[i] = (x[u][i] - s.mean) * s.rstd;  // past the row gy is 0
                if (live) {
                    dw[u][i] = fmaf(gy[u][i], xh[i], dw[u][i]);
                    db[u][i] += gy[u][i];
                }
                r[i] = fmaf(s.rstd, g[u][i] - fmaf(xh[i], m2, m1), r[i]);
            }
            if (live && col < P.dim) store8(P.dx, row, col, P.dim, r);
        }
    }
    if (!P.ws) return;
    // one partial row of dw and of db per workgroup
    float *pw = P.ws + static_cast<int64_t>(blockIdx.x) * 2 * P.dim, *pb = pw + P.dim;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int col = first_col<SPAN>(lane, u);
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
            if (sub == 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (col + i < P.dim) (half ? pb : pw)[col + i] = v[i];
            }
        }
    }
}

// 16 columns by 64 slices of the parts per workgroup: rows of 64 bytes, slices joined in LDS.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float *in, int64_t ld, int parts, ColumnSums to) {
    __shared__ float s[64][17];
    const int c = threadIdx.x & 15, k = threadIdx.x >> 4;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 16 + c, all = to.cols[0] + to.cols[1] + to.cols[2];
    float a = 0.f;
    if (col < all)
        for (int p = k; p < parts; p += 64) a += in[p * ld + col];
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

// The smallest arrangement that holds a row with at most two units per lane, which is what leaves the backward
// pass three waves per SIMD: 16 lanes (to 128 elements), 32, a wave (to 1,024), four, eight and sixteen waves.
#define KDA_NORM_PICK(CALL)                        \
    do {                                           \
        if (P.dim <= 128) CALL(16, 1, 1);          \
        else if (P.dim <= 256) CALL(32, 1, 1);     \
        else if (P.dim <= 512) CALL(64, 1, 1);     \
        else if (P.dim <= 1024) CALL(64, 1, 2);    \
        else if (P.dim <= 2048) CALL(64, 4, 1);    \
        else if (P.dim <= 4096) CALL(64, 4, 2);    \
        else if (P.dim <= 8192) CALL(64, 8, 2);    \
        else CALL(64, 16, 2);                      \
    } while (0)

int rows_of(int dim) {
    return dim <= 128 ? 16 : dim <= 256 ? 8 : dim <= 1024 ? 4 : 1;
}
int64_t bwd_groups(int64_t rows, int dim) {
    const int64_t whole = (rows + rows_of(dim) - 1) / rows_of(dim), most = dim <= 1024 ? 1024 : dim <= 4096 ? 512 : 256;
    return whole < most ? whole : most;
}

}  // namespace

void launch_column_sum(const float *in, int64_t ld, int parts, const ColumnSums &to, hipStream_t stream) {
    const int64_t cols = to.cols[0] + to.cols[1] + to.cols[2];
    if (cols > 0) column_sum_kernel<<<static_cast<unsigned>((cols + 15) / 16), 1024, 0, stream>>>(in, ld, parts, to);
}

hipError_t launch_norm_fwd(const NormFwdLaunch &P) {
#define KDA_NORM_FWD(L, W, U)                                                                                    \
    norm_fwd_kernel<L, W, U><<<static_cast<unsigned>((P.rows + rows_per_group<L, W>() - 1) / rows_per_group<L, W>()), \
                               norm_threads<L, W>(), 0, P.stream>>>(P)
    KDA_NORM_PICK(KDA_NORM_FWD);
#undef KDA_NORM_FWD
    return hipGetLastError();
}

size_t norm_bwd_workspace_bytes(int64_t rows, int dim) {
    return static_cast<size_t>(bwd_groups(rows, dim)) * 2 * dim * 4;
}

hipError_t launch_norm_bwd(const NormBwdLaunch &P) {
    const int64_t groups = bwd_groups(P.rows, P.dim);
#define KDA_NORM_BWD(L, W, U) \
    norm_bwd_kernel<L, W, U><<<static_cast<unsigned>(groups), norm_threads<L, W>(), 0, P.stream>>>(P)
    if (groups > 0) KDA_NORM_PICK(KDA_NORM_BWD);
#undef KDA_NORM_BWD
    if (P.dw || P.db)
        launch_column_sum(P.ws, 2 * P.dim, static_cast<int>(groups), {{P.dw, P.db, nullptr}, {P.dim, P.dim, 0}}, P.stream);
    return hipGetLastError();
}

}  // namespace kda
