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

// 8 elements of a row from `col` on: VEC for aligned units, else single elements `step` apart.
template <bool VEC>
__device__ __forceinline__ void load8(const Rows &r, int64_t row, int col, int step, int dim, float *x) {
    if constexpr (VEC) {
        const int64_t at = row * r.stride + col;
        if (r.bf16) {
            const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(r.p) + at);
            const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(v[i] << 16);
                x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
            }
        } else {
            const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(r.p) + at);
            const float4 a = p[0], b = p[1];
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = col + i * step < dim ? r.get(row, col + i * step) : 0.f;
    }
}
template <bool VEC>
__device__ __forceinline__ void store8(const Rows &r, int64_t row, int col, int step, int dim, const float *x) {
    if constexpr (VEC) {
        const int64_t at = row * r.stride + col;
        if (r.bf16) {
            uint32_t v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = static_cast<uint32_t>(f32_to_bf16(x[2 * i])) | static_cast<uint32_t>(f32_to_bf16(x[2 * i + 1])) << 16;
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(r.p) + at) = make_uint4(v[0], v[1], v[2], v[3]);
        } else {
            float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(r.p) + at);
            p[0] = make_float4(x[0], x[1], x[2], x[3]);
            p[1] = make_float4(x[4], x[5], x[6], x[7]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i * step < dim) r.put(row, col + i * step, x[i]);
    }
}

// Column of element i of unit u of a lane, and whether the row has it.
template <int SPAN, bool VEC>  // SPAN: lanes that share a row
struct Cols {
    static constexpr int kStep = VEC ? 1 : SPAN;
    static __device__ __forceinline__ int first(int lane, int u) {
        return VEC ? (u * SPAN + lane) * 8 : u * 8 * SPAN + lane;
    }
};

// Sums over the lanes of a row.
template <int LANES, int WAVES>
__device__ __forceinline__ void row_sum2(float &a, float &b, float *shared) {
#pragma unroll
    for (int m = LANES / 2; m >= 1; m >>= 1) {
        a += __shfl_xor(a, m, kWave);
        b += __shfl_xor(b, m, kWave);
    }
    if constexpr (WAVES > 1) {
        const int wave = threadIdx.x >> 6;
        __syncthreads();
        if ((threadIdx.x & 63) == 0) {
            shared[2 * wave] = a;
            shared[2 * wave + 1] = b;
        }
        __syncthreads();
        a = b = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            a += shared[2 * w];
            b += shared[2 * w + 1];
        }
    }
}

// mean and 1 / sqrt(var + eps) of a row in registers (elements past the row are 0 and left out of var)
template <int LANES, int WAVES, int U, bool VEC>
__device__ __forceinline__ void row_stats(const float (&x)[U][8], int lane, int dim, float eps, float *shared,
                                          float &mean, float &rstd) {
    using C = Cols<LANES * WAVES, VEC>;
    float s = 0.f, v = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) s += x[u][i];
    row_sum2<LANES, WAVES>(s, v, shared);
    mean = s / static_cast<float>(dim);
    float z = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = x[u][i] - mean;
            if (C::first(lane, u) + i * C::kStep < dim) v = fmaf(d, d, v);
        }
    row_sum2<LANES, WAVES>(v, z, shared);
    rstd = 1.f / sqrtf(v / static_cast<float>(dim) + eps);
}

template <int LANES, int WAVES>
constexpr int norm_threads() { return WAVES == 1 ? 256 : 64 * WAVES; }
template <int LANES, int WAVES>
constexpr int rows_per_group() { return WAVES == 1 ? 256 / LANES : 1; }

template <int LANES, int WAVES, int U, bool VEC>
__global__ void __launch_bounds__((norm_threads<LANES, WAVES>())) norm_fwd_kernel(NormFwdLaunch P) {
    constexpr int SPAN = LANES * WAVES;
    using C = Cols<SPAN, VEC>;
    __shared__ float shared[2 * WAVES];
    const int lane = threadIdx.x % SPAN;
    int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_group<LANES, WAVES>() + threadIdx.x / SPAN;
    const bool live = row < P.rows;
    if (WAVES == 1 && !live) row = P.rows - 1;  // keeps the wave whole for the sums; stores nothing
    float x[U][8], mean, rstd;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int col = C::first(lane, u);
        if (col < P.dim) {
            load8<VEC>(P.x, row, col, C::kStep, P.dim, x[u]);
            if (P.res.p) {
                float r[8];
                load8<VEC>(P.res, row, col, C::kStep, P.dim, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[u][i] += r[i];
                if (live) store8<VEC>(P.res_out, row, col, C::kStep, P.dim, x[u]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[u][i] = 0.f;
        }
    }
    row_stats<LANES, WAVES, U, VEC>(x, lane, P.dim, P.eps, shared, mean, rstd);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int col = C::first(lane, u);
        if (col >= P.dim || !live) continue;
        float w[8], b[8];
        const Rows wr{const_cast<void *>(P.w), 0, P.w_bf16}, br{const_cast<void *>(P.b), 0, P.w_bf16};
        if (P.w) load8<VEC>(wr, 0, col, C::kStep, P.dim, w);
        if (P.b) load8<VEC>(br, 0, col, C::kStep, P.dim, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float n = (x[u][i] - mean) * rstd;
            x[u][i] = fmaf(n, P.w ? w[i] : 1.f, P.b ? b[i] : 0.f);
        }
        store8<VEC>(P.y, row, col, C::kStep, P.dim, x[u]);
    }
}

template <int LANES, int WAVES, int U, bool VEC>
__global__ void __launch_bounds__((norm_threads<LANES, WAVES>())) norm_bwd_kernel(NormBwdLaunch P) {
    constexpr int SPAN = LANES * WAVES, ROWS = rows_per_group<LANES, WAVES>();
    using C = Cols<SPAN, VEC>;
    __shared__ float shared[2 * WAVES];
    __shared__ float fold[ROWS > 1 ? 256 * 8 : 1];
    const int lane = threadIdx.x % SPAN, sub = threadIdx.x / SPAN;
    float w[U][8], dw[U][8], db[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int col = C::first(lane, u);
        const Rows wr{const_cast<void *>(P.w), 0, P.w_bf16};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[u][i] = 1.f;
            dw[u][i] = db[u][i] = 0.f;
        }
        if (P.w && col < P.dim) load8<VEC>(wr, 0, col, C::kStep, P.dim, w[u]);
    }
    // whole rounds for every lane of the workgroup: rows past the end are computed from the last and dropped
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * ROWS; base < P.rows; base += static_cast<int64_t>(gridDim.x) * ROWS) {
        const bool live = base + sub < P.rows;
        const int64_t row = live ? base + sub : P.rows - 1;
        float x[U][8], g[U][8], mean, rstd;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int col = C::first(lane, u);
            if (col < P.dim) {
                load8<VEC>(P.x, row, col, C::kStep, P.dim, x[u]);
                load8<VEC>(P.gy, row, col, C::kStep, P.dim, g[u]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[u][i] = g[u][i] = 0.f;
            }
        }
        row_stats<LANES, WAVES, U, VEC>(x, lane, P.dim, P.eps, shared, mean, rstd);
        float m1 = 0.f, m2 = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float xh = (x[u][i] - mean) * rstd;  // past the row g is 0
                if (live) {
                    dw[u][i] = fmaf(g[u][i], xh, dw[u][i]);
                    db[u][i] += g[u][i];
                }
                g[u][i] *= w[u][i];
                x[u][i] = xh;
                m1 += g[u][i];
                m2 = fmaf(g[u][i], xh, m2);
            }
        row_sum2<LANES, WAVES>(m1, m2, shared);
        m1 /= static_cast<float>(P.dim);
        m2 /= static_cast<float>(P.dim);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int col = C::first(lane, u);
            if (col >= P.dim || !live) continue;
            float r[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] = 0.f;
            if (P.gres.p) load8<VEC>(P.gres, row, col, C::kStep, P.dim, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[u][i] = fmaf(rstd, g[u][i] - fmaf(x[u][i], m2, m1), r[i]);
            store8<VEC>(P.dx, row, col, C::kStep, P.dim, x[u]);
        }
    }
    if (!P.ws) return;
    // one partial row of dw and of db per workgroup
    float *pw = P.ws + static_cast<int64_t>(blockIdx.x) * 2 * P.dim, *pb = pw + P.dim;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int col = C::first(lane, u);
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
                    if (col + i * C::kStep < P.dim) (half ? pb : pw)[col + i * C::kStep] = v[i];
            }
        }
    }
}

// 16 columns by 64 slices of the parts per workgroup: rows of 64 bytes, slices joined in LDS.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float *in, int64_t ld, int parts, int64_t cols, float *out) {
    __shared__ float s[64][17];
    const int c = threadIdx.x & 15, k = threadIdx.x >> 4;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 16 + c;
    float a = 0.f;
    if (col < cols)
        for (int p = k; p < parts; p += 64) a += in[p * ld + col];
    s[k][c] = a;
    __syncthreads();
#pragma unroll
    for (int h = 32; h >= 1; h >>= 1) {
        if (k < h) s[k][c] += s[k + h][c];
        __syncthreads();
    }
    if (k == 0 && col < cols) out[col] = s[0][c];
}

bool aligned16(const Rows &r) {
    const int64_t e = r.bf16 ? 2 : 4;
    return !r.p || (reinterpret_cast<uintptr_t>(r.p) % 16 == 0 && (r.stride * e) % 16 == 0);
}
bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// The smallest arrangement that holds a row: 16 lanes (to 128 elements), 32, a wave with 1, 2 or 4 units per
// lane (to 2,048), four waves (to 8,192), sixteen (to 16,384).
#define KDA_NORM_PICK(CALL)                        \
    do {                                           \
        if (P.dim <= 128) CALL(16, 1, 1);          \
        else if (P.dim <= 256) CALL(32, 1, 1);     \
        else if (P.dim <= 512) CALL(64, 1, 1);     \
        else if (P.dim <= 1024) CALL(64, 1, 2);    \
        else if (P.dim <= 2048) CALL(64, 1, 4);    \
        else if (P.dim <= 4096) CALL(64, 4, 2);    \
        else if (P.dim <= 8192) CALL(64, 4, 4);    \
        else CALL(64, 16, 2);                      \
    } while (0)

int rows_of(int dim) {
    return dim <= 128 ? 16 : dim <= 256 ? 8 : dim <= 2048 ? 4 : 1;
}
int64_t bwd_groups(int64_t rows, int dim) {
    const int64_t whole = (rows + rows_of(dim) - 1) / rows_of(dim), most = dim <= 8192 ? 1024 : 512;
    return whole < most ? whole : most;
}

}  // namespace

void launch_column_sum(const float *in, int64_t ld, int parts, int64_t cols, float *out, hipStream_t stream) {
    if (cols > 0) column_sum_kernel<<<static_cast<unsigned>((cols + 15) / 16), 1024, 0, stream>>>(in, ld, parts, cols, out);
}

hipError_t launch_norm_fwd(const NormFwdLaunch &P) {
    const bool vec = P.dim % 8 == 0 && aligned16(P.x) && aligned16(P.res) && aligned16(P.y) && aligned16(P.res_out) &&
                     aligned16(P.w) && aligned16(P.b);
#define KDA_NORM_FWD(L, W, U)                                                                              \
    do {                                                                                                   \
        const unsigned grid = static_cast<unsigned>((P.rows + rows_per_group<L, W>() - 1) / rows_per_group<L, W>()); \
        if (vec) norm_fwd_kernel<L, W, U, true><<<grid, norm_threads<L, W>(), 0, P.stream>>>(P);           \
        else norm_fwd_kernel<L, W, U, false><<<grid, norm_threads<L, W>(), 0, P.stream>>>(P);              \
    } while (0)
    KDA_NORM_PICK(KDA_NORM_FWD);
#undef KDA_NORM_FWD
    return hipGetLastError();
}

size_t norm_bwd_workspace_bytes(int64_t rows, int dim) {
    return static_cast<size_t>(bwd_groups(rows, dim)) * 2 * dim * 4;
}

hipError_t launch_norm_bwd(const NormBwdLaunch &P) {
    const bool vec = P.dim % 8 == 0 && aligned16(P.x) && aligned16(P.gy) && aligned16(P.gres) && aligned16(P.dx) &&
                     aligned16(P.w);
    const int64_t groups = bwd_groups(P.rows, P.dim);
#define KDA_NORM_BWD(L, W, U)                                                                              \
    do {                                                                                                   \
        const unsigned grid = static_cast<unsigned>(groups);                                               \
        if (vec) norm_bwd_kernel<L, W, U, true><<<grid, norm_threads<L, W>(), 0, P.stream>>>(P);           \
        else norm_bwd_kernel<L, W, U, false><<<grid, norm_threads<L, W>(), 0, P.stream>>>(P);              \
    } while (0)
    if (groups > 0) KDA_NORM_PICK(KDA_NORM_BWD);
#undef KDA_NORM_BWD
    if (P.dw) launch_column_sum(P.ws, 2 * P.dim, static_cast<int>(groups), P.dim, P.dw, P.stream);
    if (P.db) launch_column_sum(P.ws + P.dim, 2 * P.dim, static_cast<int>(groups), P.dim, P.db, P.stream);
    return hipGetLastError();
}

}  // namespace kda
