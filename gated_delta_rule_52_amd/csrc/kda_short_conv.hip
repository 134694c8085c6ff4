// kda_short_conv.hip - the short causal depthwise convolution, forward, step and gradients, for gfx950.
//
//     p_t = bias + sum_j w[j] x_{t-W+1+j},   y = p or p sigmoid(p)
//
// Bound by HBM: x read and y written once (plus W - 1 rows of each tile's past, which the neighbour tile has
// just read).  A thread holds V adjacent channels (one 16-byte access) and walks a tile of tokens with the
// last W - 1 inputs in registers, so every input is loaded once.  A sequence's first W - 1 outputs take
// their past from its state; tiles cut the rows without regard to sequences, and the walk reloads the window
// where a sequence starts.
#include "kda_layer.h"

namespace kda {

namespace {

// The sequence that row t lies in (an empty one has no rows); N: behind the last.
__device__ __forceinline__ int sequence_of(const int32_t *cu, int N, int T, int64_t t) {
    if (!cu) return static_cast<int>(t / T);
    int lo = 0, hi = N;  // the first sequence that ends behind t
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}
__device__ __forceinline__ void bounds_of(const int32_t *cu, int N, int T, int n, int64_t &s, int64_t &e) {
    SeqTiles q{cu, N, T, 1};
    int len;
    q.sequence(n, s, len);
    e = s + len;
}

template <int V, bool InBf16>
__device__ __forceinline__ void load_v(const void *p, int64_t at, float *x) {
    if constexpr (V == 1) {
        x[0] = Elem<InBf16>::load(static_cast<const typename Elem<InBf16>::T *>(p), at);
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 f = Elem<InBf16>::load4(static_cast<const typename Elem<InBf16>::T *>(p), at + i);
            x[i] = f.x; x[i + 1] = f.y; x[i + 2] = f.z; x[i + 3] = f.w;
        }
    }
}
template <int V>
__device__ __forceinline__ void store_v(const Rows &r, int64_t row, int col, const float *x) {
    if constexpr (V == 1) {
        r.put(row, col, x[0]);
    } else {
        const int64_t at = row * r.stride + col;
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 f = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
            if (r.bf16) Elem<true>::store4(static_cast<uint16_t *>(r.p), at + i, f);
            else Elem<false>::store4(static_cast<float *>(r.p), at + i, f);
        }
    }
}

template <int W, int V>
struct Taps {
    float w[W][V], b[V];
    __device__ __forceinline__ Taps(const void *wp, const void *bp, int bf16, int c0) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][v] = param(wp, bf16, static_cast<int64_t>(c0 + v) * W + j);
            b[v] = bp ? param(bp, bf16, c0 + v) : 0.f;
        }
    }
};

// Fills win (the W - 1 inputs before row t of the sequence from row `s` on, oldest first).
template <int W, int V, bool InBf16>
__device__ __forceinline__ void window(const Rows &x, const void *h0, int dim, int n, int64_t s, int64_t t, int c0,
                                       float (&win)[W - 1][V]) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int64_t from = t - (W - 1) + j;
        if (from >= s) {
            load_v<V, InBf16>(x.p, from * x.stride + c0, win[j]);
        } else if (h0) {  // state row i is W - 1 - i tokens before the start
            const int64_t i = W - 1 + from - s;
            load_v<V, InBf16>(h0, (static_cast<int64_t>(n) * (W - 1) + i) * dim + c0, win[j]);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) win[j][v] = 0.f;
        }
    }
}

constexpr int kConvTile = 32;  // rows per thread

template <int W, int V, bool InBf16>
__global__ void __launch_bounds__(256) conv_kernel(ConvLaunch P, int64_t rows, int cblocks) {
    const int c0 = (static_cast<int>(blockIdx.x % cblocks) * 256 + threadIdx.x) * V;
    int64_t t = static_cast<int64_t>(blockIdx.x / cblocks) * kConvTile;
    const int64_t end = t + kConvTile < rows ? t + kConvTile : rows;
    int n = sequence_of(P.cu, P.N, P.T, t);
    if (c0 >= P.dim || n >= P.N) return;
    const Taps<W, V> k(P.w, P.bias, P.w_bf16, c0);
    while (t < end) {  // the part of one sequence that lies in the tile
        int64_t s, e;
        bounds_of(P.cu, P.N, P.T, n, s, e);
        if (e <= t) {  // an empty sequence
            if (++n >= P.N) return;
            continue;
        }
        if (s > t) t = s;
        float win[W - 1][V], x[V], y[V];
        window<W, V, InBf16>(P.x, P.h0, P.dim, n, s, t, c0, win);
        const int64_t stop = e < end ? e : end;
        for (; t < stop; ++t) {
            load_v<V, InBf16>(P.x.p, t * P.x.stride + c0, x);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float p = k.b[v];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) p = fmaf(k.w[j][v], win[j][v], p);
                p = fmaf(k.w[W - 1][v], x[v], p);
                y[v] = P.silu ? p * sigmoid_f(p) : p;
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) win[j][v] = win[j + 1][v];
                win[W - 2][v] = x[v];
            }
            store_v<V>(P.y, t, c0, y);
        }
        if (++n >= P.N) return;
    }
}

// The state each sequence leaves: the last W - 1 of its inputs with its old state in front.  A launch of its
// own behind the outputs, so that the new state may take the old one's place.  One thread per sequence and
// channel reads all its rows before it writes one.
template <int W, typename T>
__global__ void __launch_bounds__(256) conv_state_kernel(ConvLaunch P, int cblocks) {
    const int c = static_cast<int>(blockIdx.x % cblocks) * 256 + threadIdx.x, n = blockIdx.x / cblocks;
    if (c >= P.dim) return;
    int64_t s, e;
    bounds_of(P.cu, P.N, P.T, n, s, e);
    T v[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int64_t from = e - (W - 1) + j;
        if (from >= s) v[j] = static_cast<const T *>(P.x.p)[from * P.x.stride + c];
        else v[j] = P.h0 ? static_cast<const T *>(P.h0)[(static_cast<int64_t>(n) * (W - 1) + W - 1 + from - s) * P.dim + c]
                         : static_cast<T>(0);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) static_cast<T *>(P.hT)[(static_cast<int64_t>(n) * (W - 1) + j) * P.dim + c] = v[j];
}

// One token per sequence: output and shifted state in one pass.
template <int W, int V, bool InBf16>
__global__ void __launch_bounds__(256) conv_step_kernel(ConvLaunch P, int cblocks) {
    const int c0 = (static_cast<int>(blockIdx.x % cblocks) * 256 + threadIdx.x) * V, n = blockIdx.x / cblocks;
    if (c0 >= P.dim) return;
    const Taps<W, V> k(P.w, P.bias, P.w_bf16, c0);
    float win[W - 1][V], x[V], y[V];
    window<W, V, InBf16>(P.x, P.h0, P.dim, n, n, n, c0, win);
    load_v<V, InBf16>(P.x.p, n * P.x.stride + c0, x);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float p = k.b[v];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) p = fmaf(k.w[j][v], win[j][v], p);
        p = fmaf(k.w[W - 1][v], x[v], p);
        y[v] = P.silu ? p * sigmoid_f(p) : p;
    }
    store_v<V>(P.y, n, c0, y);
    if (P.hT) {
        const Rows out{P.hT, P.dim, InBf16};
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            store_v<V>(out, static_cast<int64_t>(n) * (W - 1) + j, c0, j + 1 < W - 1 ? win[j + 1] : x);
    }
}

// ---- gradients -----------------------------------------------------------------------------------------

constexpr int kGradTile = 64;

// d silu(p) / dp times g.
__device__ __forceinline__ float silu_grad(float g, float p) {
    const float s = sigmoid_f(p);
    return g * (s * fmaf(p, 1.f - s, 1.f));
}

// dx of a tile's rows and the tile's share of dweight and dbias.  dx_t needs gp of the W - 1 rows behind it,
// so the walk runs W - 1 rows past the tile's end (inside the sequence) and those rows' gp is computed twice.
template <int W, int V, bool InBf16>
__global__ void __launch_bounds__(256) conv_grad_kernel(ConvBwdLaunch P, int64_t rows, int cblocks) {
    const int c0 = (static_cast<int>(blockIdx.x % cblocks) * 256 + threadIdx.x) * V;
    const int64_t tile = blockIdx.x / cblocks;
    int64_t t = tile * kGradTile;
    const int64_t end = t + kGradTile < rows ? t + kGradTile : rows;
    if (c0 >= P.dim) return;
    const Taps<W, V> k(P.w, P.bias, P.w_bf16, c0);
    float dw[W][V], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][v] = 0.f;
    }
    for (int n = sequence_of(P.cu, P.N, P.T, t); n < P.N && t < end; ++n) {
        int64_t s, e;
        bounds_of(P.cu, P.N, P.T, n, s, e);
        if (e <= t) continue;
        if (s > t) t = s;
        if (t >= end) break;
        float win[W - 1][V], x[V], g[V], gp[W][V];  // gp[j]: of row i - (W - 1) + j
        window<W, V, InBf16>(P.x, P.h0, P.dim, n, s, t, c0, win);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < W; ++j) gp[j][v] = 0.f;
        const int64_t stop = e < end ? e : end, first = t;
        for (int64_t i = t; i < stop + W - 1; ++i) {
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int j = 0; j < W - 1; ++j) gp[j][v] = gp[j + 1][v];
            if (i < e) {
                load_v<V, InBf16>(P.x.p, i * P.x.stride + c0, x);
                load_v<V, InBf16>(P.gy.p, i * P.gy.stride + c0, g);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (P.silu) {
                        float p = k.b[v];
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) p = fmaf(k.w[j][v], win[j][v], p);
                        p = fmaf(k.w[W - 1][v], x[v], p);
                        g[v] = silu_grad(g[v], p);
                    }
                    gp[W - 1][v] = g[v];
                    if (i < stop) {
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) dw[j][v] = fmaf(g[v], win[j][v], dw[j][v]);
                        dw[W - 1][v] = fmaf(g[v], x[v], dw[W - 1][v]);
                        db[v] += g[v];
                    }
#pragma unroll
                    for (int j = 0; j + 1 < W - 1; ++j) win[j][v] = win[j + 1][v];
                    win[W - 2][v] = x[v];
                }
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) gp[W - 1][v] = 0.f;
            }
            const int64_t o = i - (W - 1);  // the row whose gradient is complete
            if (o >= first) {
                float d[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    d[v] = 0.f;
#pragma unroll
                    for (int j = 0; j < W; ++j) d[v] = fmaf(k.w[W - 1 - j][v], gp[j][v], d[v]);
                }
                const int64_t back = e - o;  // the row is also row W - 1 - back of the final state
                if (P.dhT && back <= W - 1) {
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        d[v] += P.dhT[(static_cast<int64_t>(n) * (W - 1) + W - 1 - back) * P.dim + c0 + v];
                }
                store_v<V>(P.dx, o, c0, d);
            }
        }
        t = stop;
    }
    float *part = P.ws + tile * static_cast<int64_t>(W + 1) * P.dim;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) part[static_cast<int64_t>(c0 + v) * W + j] = dw[j][v];
        part[static_cast<int64_t>(W) * P.dim + c0 + v] = db[v];
    }
}

// The initial state's gradient: row i of it is the input W - 1 - i tokens before the start, which the first
// outputs' taps reach, and which a sequence shorter than W - 1 hands on to its final state.
template <int W, bool InBf16>
__global__ void __launch_bounds__(256) conv_state_grad_kernel(ConvBwdLaunch P, int cblocks) {
    const int c = static_cast<int>(blockIdx.x % cblocks) * 256 + threadIdx.x, n = blockIdx.x / cblocks;
    if (c >= P.dim) return;
    int64_t s, e;
    bounds_of(P.cu, P.N, P.T, n, s, e);
    const Taps<W, 1> k(P.w, P.bias, P.w_bf16, c);
    float win[W - 1][1], d[W - 1], x[1];
    window<W, 1, InBf16>(P.x, P.h0, P.dim, n, s, s, c, win);
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        d[i] = 0.f;
        const int64_t f = i - (e - s);  // the final state's row that holds this one
        if (P.dhT && f >= 0) d[i] = P.dhT[(static_cast<int64_t>(n) * (W - 1) + f) * P.dim + c];
    }
#pragma unroll
    for (int o = 0; o < W - 1; ++o) {  // output s + o meets state row i with tap i - o
        if (s + o >= e) break;
        load_v<1, InBf16>(P.x.p, (s + o) * P.x.stride + c, x);
        float g = P.gy.get(s + o, c);
        if (P.silu) {
            float p = k.b[0];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) p = fmaf(k.w[j][0], win[j][0], p);
            g = silu_grad(g, fmaf(k.w[W - 1][0], x[0], p));
        }
#pragma unroll
        for (int i = o; i < W - 1; ++i) d[i] = fmaf(k.w[i - o][0], g, d[i]);
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) win[j][0] = win[j + 1][0];
        win[W - 2][0] = x[0];
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i) P.dh0[(static_cast<int64_t>(n) * (W - 1) + i) * P.dim + c] = d[i];
}

bool aligned(const Rows &r, int V) {
    const int64_t e = r.bf16 ? 2 : 4, a = V * e < 16 ? V * e : 16;
    return !r.p || (reinterpret_cast<uintptr_t>(r.p) % a == 0 && (r.stride * e) % a == 0);
}

// Channels per thread: 4 where every access of 4 is aligned, else 1.
int vector_of(int dim, const Rows *r, int count, const void *h0, const void *hT, bool in_bf16) {
    bool ok = dim % 4 == 0;
    for (int i = 0; i < count; ++i) ok = ok && aligned(r[i], 4);
    const Rows s0{const_cast<void *>(h0), dim, in_bf16}, s1{const_cast<void *>(hT), dim, in_bf16};
    return ok && aligned(s0, 4) && aligned(s1, 4) ? 4 : 1;
}

#define KDA_CONV_PICK(KERNEL, GRID, ...)                                                          \
    do {                                                                                          \
        if (P.x.bf16) KDA_CONV_W(KERNEL, true, GRID, __VA_ARGS__);                                \
        else KDA_CONV_W(KERNEL, false, GRID, __VA_ARGS__);                                        \
    } while (0)
#define KDA_CONV_W(KERNEL, BF, GRID, ...)                                                         \
    do {                                                                                          \
        if (P.width == 2) KDA_CONV_V(KERNEL, 2, BF, GRID, __VA_ARGS__);                           \
        else if (P.width == 3) KDA_CONV_V(KERNEL, 3, BF, GRID, __VA_ARGS__);                      \
        else KDA_CONV_V(KERNEL, 4, BF, GRID, __VA_ARGS__);                                        \
    } while (0)
#define KDA_CONV_V(KERNEL, W, BF, GRID, ...)                                                      \
    do {                                                                                          \
        if (V == 4) KERNEL<W, 4, BF><<<GRID, 256, 0, P.stream>>>(__VA_ARGS__);                    \
        else KERNEL<W, 1, BF><<<GRID, 256, 0, P.stream>>>(__VA_ARGS__);                           \
    } while (0)

template <typename T>
void launch_state(const ConvLaunch &P) {
    const int cb = (P.dim + 255) / 256;
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(P.N) * cb);
    if (P.width == 2) conv_state_kernel<2, T><<<grid, 256, 0, P.stream>>>(P, cb);
    else if (P.width == 3) conv_state_kernel<3, T><<<grid, 256, 0, P.stream>>>(P, cb);
    else conv_state_kernel<4, T><<<grid, 256, 0, P.stream>>>(P, cb);
}

template <bool InBf16>
void launch_state_grad(const ConvBwdLaunch &P) {
    const int cb = (P.dim + 255) / 256;
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(P.N) * cb);
    if (P.width == 2) conv_state_grad_kernel<2, InBf16><<<grid, 256, 0, P.stream>>>(P, cb);
    else if (P.width == 3) conv_state_grad_kernel<3, InBf16><<<grid, 256, 0, P.stream>>>(P, cb);
    else conv_state_grad_kernel<4, InBf16><<<grid, 256, 0, P.stream>>>(P, cb);
}

int64_t conv_rows(const int32_t *cu, int N, int T) { return cu ? T : static_cast<int64_t>(N) * T; }

}  // namespace

hipError_t launch_conv_fwd(const ConvLaunch &P) {
    const int64_t rows = conv_rows(P.cu, P.N, P.T);
    const Rows r[] = {P.x, P.y};
    const int V = vector_of(P.dim, r, 2, P.h0, nullptr, P.x.bf16);
    const int cb = (P.dim + 256 * V - 1) / (256 * V);
    const unsigned grid = static_cast<unsigned>((rows + kConvTile - 1) / kConvTile * cb);
    if (rows > 0) KDA_CONV_PICK(conv_kernel, grid, P, rows, cb);
    if (P.hT) {
        if (P.x.bf16) launch_state<uint16_t>(P);
        else launch_state<float>(P);
    }
    return hipGetLastError();
}

hipError_t launch_conv_step(const ConvLaunch &P) {
    const Rows r[] = {P.x, P.y};
    const int V = vector_of(P.dim, r, 2, P.h0, P.hT, P.x.bf16);
    const int cb = (P.dim + 256 * V - 1) / (256 * V);
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(P.N) * cb);
    KDA_CONV_PICK(conv_step_kernel, grid, P, cb);
    return hipGetLastError();
}

size_t conv_bwd_workspace_bytes(int64_t rows, int dim, int width) {
    return static_cast<size_t>((rows + kGradTile - 1) / kGradTile) * (width + 1) * dim * 4;
}

hipError_t launch_conv_bwd(const ConvBwdLaunch &P) {
    const int64_t rows = conv_rows(P.cu, P.N, P.T), tiles = (rows + kGradTile - 1) / kGradTile;
    const Rows r[] = {P.x, P.gy, P.dx};
    const int V = vector_of(P.dim, r, 3, P.h0, nullptr, P.x.bf16);
    const int cb = (P.dim + 256 * V - 1) / (256 * V);
    if (rows > 0) KDA_CONV_PICK(conv_grad_kernel, static_cast<unsigned>(tiles * cb), P, rows, cb);
    const int64_t ld = static_cast<int64_t>(P.width + 1) * P.dim;
    launch_column_sum(P.ws, ld, static_cast<int>(tiles), static_cast<int64_t>(P.width) * P.dim, P.dw, P.stream);
    if (P.db)
        launch_column_sum(P.ws + static_cast<int64_t>(P.width) * P.dim, ld, static_cast<int>(tiles), P.dim, P.db, P.stream);
    if (P.dh0) {
        if (P.x.bf16) launch_state_grad<true>(P);
        else launch_state_grad<false>(P);
    }
    return hipGetLastError();
}

}  // namespace kda
