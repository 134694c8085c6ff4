// kda_short_conv.hip - the short causal depthwise convolution, forward, step and gradients, for gfx950.
//
//     p_t = bias + sum_j w[j] x_{t-W+1+j},   y = p or p sigmoid(p)
//
// Bound by HBM: x read and y written once (plus W - 1 rows of each tile's past, which the neighbour tile has
// just read).  A thread holds V adjacent channels and walks a tile of tokens with the last W - 1 inputs in
// registers, so every input is loaded once, four rows in flight.  A sequence's first W - 1 outputs take
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

// V adjacent channels: one, or 4 or 8 in accesses of up to 16 bytes, which the hardware takes at any element's
// alignment.  Where the width is no multiple of V the last thread's channels are moved back inside: it computes
// some of its neighbour's again and stores the same values.
typedef uint32_t any4 __attribute__((ext_vector_type(4), aligned(2)));
template <int V, bool InBf16>
struct Raw {
    static constexpr int kWords = V == 1 ? 1 : V * (InBf16 ? 2 : 4) / 4;
    typedef uint32_t some __attribute__((ext_vector_type(kWords), aligned(2)));
    some v;
    __device__ __forceinline__ void load(const void *p, int64_t at) {
        const typename Elem<InBf16>::T *e = static_cast<const typename Elem<InBf16>::T *>(p) + at;
        if constexpr (V == 1) v[0] = InBf16 ? *reinterpret_cast<const uint16_t *>(e) : *reinterpret_cast<const uint32_t *>(e);
        else v = *reinterpret_cast<const some *>(e);
    }
    __device__ __forceinline__ void widen(float *x) const {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if constexpr (!InBf16) x[i] = __uint_as_float(v[i]);
            else x[i] = __uint_as_float(V > 1 && (i & 1) ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
    }
};
template <int V, bool InBf16>
__device__ __forceinline__ void load_v(const void *p, int64_t at, float *x) {
    Raw<V, InBf16> r;
    r.load(p, at);
    r.widen(x);
}
template <int V>
__device__ __forceinline__ void store_v(const Rows &r, int64_t row, int col, const float *x) {
    if constexpr (V == 1) {
        r.put(row, col, x[0]);
    } else {
        const int64_t at = row * r.stride + col;
        if (r.bf16) {
            typedef uint32_t some __attribute__((ext_vector_type(V / 2), aligned(2)));
            some v;
#pragma unroll
            for (int i = 0; i < V / 2; ++i) v[i] = to_bf16(x[2 * i]) | static_cast<uint32_t>(to_bf16(x[2 * i + 1])) << 16;
            *reinterpret_cast<some *>(static_cast<uint16_t *>(r.p) + at) = v;
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                any4 v;
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = __float_as_uint(x[i + k]);
                *reinterpret_cast<any4 *>(static_cast<float *>(r.p) + at + i) = v;
            }
        }
    }
}
template <int V>
__device__ __forceinline__ int first_channel(int thread, int dim) {
    const int c = thread * V;
    return c + V > dim && c < dim ? dim - V : c;
}

template <int W, int V>
struct Taps {
    float w[W][V], b[V];
    __device__ __forceinline__ Taps(const void *wp, const void *bp, int bf16, int c0) {
        auto all = [&](auto bf) {
            using E = Elem<decltype(bf)::value>;
            const auto *p = static_cast<const typename E::T *>(wp) + static_cast<int64_t>(c0) * W;
            const auto *q = static_cast<const typename E::T *>(bp) + c0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
                for (int j = 0; j < W; ++j) w[j][v] = E::load(p, v * W + j);
                b[v] = bp ? E::load(q, v) : 0.f;
            }
        };
        if (bf16) all(std::true_type{});
        else all(std::false_type{});
    }
    __device__ __forceinline__ float at(int v, const float (&win)[W - 1][V], const float *x) const {
        float p = b[v];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) p = fmaf(w[j][v], win[j][v], p);
        return fmaf(w[W - 1][v], x[v], p);
    }
};
template <int W, int V>
__device__ __forceinline__ void shift(float (&win)[W - 1][V], const float *x) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) win[j][v] = win[j + 1][v];
        win[W - 2][v] = x[v];
    }
}

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

constexpr int kAhead = 4;      // rows loaded together
// Tiles per workgroup, one to a wave of 64 threads across: 32,768 x 1,536 bf16 take 45 us, with one tile and 256 across,
// a quarter of them idle, 56.  Tiles of 16 rows: 8,192 x 2,048 19 us, of 32 20.
constexpr int kWaves = 4;

template <int W, int V, bool InBf16>
__global__ void __launch_bounds__(256) conv_kernel(ConvLaunch P, int64_t rows, int cblocks, int tile) {
    const int c0 = first_channel<V>(static_cast<int>(blockIdx.x % cblocks) * 64 + (threadIdx.x & 63), P.dim);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t t = (static_cast<int64_t>(blockIdx.x / cblocks) * kWaves + wave) * tile;
    if (t >= rows) return;
    const int64_t end = t + tile < rows ? t + tile : rows;
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
        if (t >= end) return;
        float win[W - 1][V], x[kAhead][V];
        window<W, V, InBf16>(P.x, P.h0, P.dim, n, s, t, c0, win);
        const int64_t stop = e < end ? e : end;
        auto output = [&](int64_t row, const float (&x)[V]) {
            float y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float p = k.at(v, win, x);
                y[v] = P.silu ? p * sigmoid_f(p) : p;
            }
            shift<W, V>(win, x);
            store_v<V>(P.y, row, c0, y);
        };
        for (; t + kAhead <= stop; t += kAhead) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) load_v<V, InBf16>(P.x.p, (t + i) * P.x.stride + c0, x[i]);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) output(t + i, x[i]);
        }
        for (; t < stop; ++t) {
            load_v<V, InBf16>(P.x.p, t * P.x.stride + c0, x[0]);
            output(t, x[0]);
        }
        t = stop;
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
    const int c0 = first_channel<V>(static_cast<int>(blockIdx.x % cblocks) * 256 + threadIdx.x, P.dim), n = blockIdx.x / cblocks;
    if (c0 >= P.dim) return;
    const Taps<W, V> k(P.w, P.bias, P.w_bf16, c0);
    float win[W - 1][V], x[V], y[V];
    window<W, V, InBf16>(P.x, P.h0, P.dim, n, n, n, c0, win);
    load_v<V, InBf16>(P.x.p, n * P.x.stride + c0, x);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float p = k.at(v, win, x);
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

constexpr int kGradSubs = 8;   // tiles per workgroup, of 256 / kGradSubs threads each
constexpr int kGradAhead = 2;  // rows loaded together, a round ahead (4 x 4,096 x 4,096 bf16 105 us, on the spot 115)

// d silu(p) / dp times g.
__device__ __forceinline__ float silu_grad(float g, float p) {
    const float s = sigmoid_f(p);
    return g * (s * fmaf(p, 1.f - s, 1.f));
}

// dx of a tile's rows and the workgroup's share of dweight and dbias.  dx_t needs gp of the W - 1 rows behind it,
// so the walk runs W - 1 rows past the tile's end (inside the sequence) and those rows' gp is computed twice.
template <int W, int V, bool InBf16>
__global__ void __launch_bounds__(256) conv_grad_kernel(ConvBwdLaunch P, int64_t rows, int cblocks, int tile) {
    constexpr int LANES = 256 / kGradSubs;
    __shared__ float fold[kGradSubs][V][LANES];
    const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    int c0 = first_channel<V>(static_cast<int>(blockIdx.x % cblocks) * LANES + lane, P.dim);
    const bool live = c0 < P.dim;
    if (!live) c0 = 0;  // walks no rows, but stays for the barriers
    const int64_t part = blockIdx.x / cblocks;
    int64_t t = (part * kGradSubs + sub) * tile;
    const int64_t end = !live ? t : t + tile < rows ? t + tile : rows;
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
        float win[W - 1][V], gp[W - 1][V];  // gp[j]: of the row W - 1 - j behind the next
        window<W, V, InBf16>(P.x, P.h0, P.dim, n, s, t, c0, win);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < W - 1; ++j) gp[j][v] = 0.f;
        const int64_t stop = e < end ? e : end, first = t, over = stop + W - 1;
        // row i's pre-activation gradient in g's place, and its share of dweight and dbias if it is the tile's
        auto gradient = [&](const float (&x)[V], float (&g)[V], bool own) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (P.silu) g[v] = silu_grad(g[v], k.at(v, win, x));
                if (!own) continue;
#pragma unroll
                for (int j = 0; j < W - 1; ++j) dw[j][v] = fmaf(g[v], win[j][v], dw[j][v]);
                dw[W - 1][v] = fmaf(g[v], x[v], dw[W - 1][v]);
                db[v] += g[v];
            }
            shift<W, V>(win, x);
        };
        // the gradient of row i - (W - 1), complete with row i's g
        auto finish = [&](int64_t i, const float (&g)[V], bool last) {
            const int64_t o = i - (W - 1);
            float d[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                d[v] = k.w[0][v] * g[v];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) d[v] = fmaf(k.w[W - 1 - j][v], gp[j][v], d[v]);
            }
            if (last && P.dhT && e - o <= W - 1) {  // the row is also row W - 1 - (e - o) of the final state
#pragma unroll
                for (int v = 0; v < V; ++v)
                    d[v] += P.dhT[(static_cast<int64_t>(n) * (W - 1) + W - 1 - (e - o)) * P.dim + c0 + v];
            }
            store_v<V>(P.dx, o, c0, d);
            shift<W, V>(gp, g);
        };
        float x[kGradAhead][V], g[kGradAhead][V];
        auto load = [&](int64_t i, float (&x)[V], float (&g)[V]) {
            load_v<V, InBf16>(P.x.p, i * P.x.stride + c0, x);
            load_v<V, InBf16>(P.gy.p, i * P.gy.stride + c0, g);
        };
        int64_t i = t;
        for (; i < stop && i < first + W - 1; ++i) {
            load(i, x[0], g[0]);
            gradient(x[0], g[0], true);
            shift<W, V>(gp, g[0]);
        }
        // nothing to ask here; the next rows' loads are in flight behind a pair's work
        Raw<V, InBf16> nx[kGradAhead], ng[kGradAhead];
        auto ahead = [&](int64_t i) {
#pragma unroll
            for (int a = 0; a < kGradAhead; ++a) {
                const int64_t row = i + a < stop ? i + a : stop - 1;
                nx[a].load(P.x.p, row * P.x.stride + c0);
                ng[a].load(P.gy.p, row * P.gy.stride + c0);
            }
        };
        ahead(i);
        for (; i + kGradAhead <= stop; i += kGradAhead) {
#pragma unroll
            for (int a = 0; a < kGradAhead; ++a) {
                nx[a].widen(x[a]);
                ng[a].widen(g[a]);
            }
            ahead(i + kGradAhead);
#pragma unroll
            for (int a = 0; a < kGradAhead; ++a) {
                gradient(x[a], g[a], true);
                finish(i + a, g[a], false);
            }
        }
        for (; i < stop; ++i) {
            load(i, x[0], g[0]);
            gradient(x[0], g[0], true);
            finish(i, g[0], false);
        }
        for (; i < over; ++i) {
            if (i < e) {
                load(i, x[0], g[0]);
                gradient(x[0], g[0], false);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) g[0][v] = 0.f;
            }
            if (i - (W - 1) >= first) finish(i, g[0], true);
            else shift<W, V>(gp, g[0]);
        }
        t = stop;
    }
    float *out = P.ws + part * static_cast<int64_t>(W + 1) * P.dim;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) fold[sub][v][lane] = j < W ? dw[j < W ? j : 0][v] : db[v];
        __syncthreads();
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < V / kGradSubs + (V % kGradSubs != 0); ++i) {
            const int v = i * kGradSubs + sub;
            if (v >= V) break;
            float sum = fold[0][v][lane];
#pragma unroll
            for (int f = 1; f < kGradSubs; ++f) sum += fold[f][v][lane];
            out[j < W ? static_cast<int64_t>(c0 + v) * W + j : static_cast<int64_t>(W) * P.dim + c0 + v] = sum;
        }
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
        if (P.silu) g = silu_grad(g, k.at(0, win, x));
#pragma unroll
        for (int i = o; i < W - 1; ++i) d[i] = fmaf(k.w[i - o][0], g, d[i]);
        shift<W, 1>(win, x);
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i) P.dh0[(static_cast<int64_t>(n) * (W - 1) + i) * P.dim + c] = d[i];
}

// Rows per thread: `most`, or down to 8 where that leaves fewer than 512 workgroups of `lanes` threads across the
// channels, whose walks would then be what the call waits for.
int tile_of(int64_t rows, int dim, int V, int lanes, int most) {
    const int64_t across = (dim + lanes * V - 1) / (lanes * V), tiles = 256 / lanes;
    int tile = most;
    while (tile > 8 && (rows + tile * tiles - 1) / (tile * tiles) * across < 512) tile /= 2;
    return tile;
}

// Channels per thread where the width has as many.  Forward 4, as 8 channels' taps cost waves: 32,768 x 4,096 bf16
// 114 us against 117 with 8, x 1,536 44 against 51.  Gradients 8 for bf16, which wide layers gain by: 4 x 4,096 x 4,096
// 101 us against 126 with 4; 32,768 x 1,536, where 8 give 384 workgroups for 256 CUs, 93 against 77.
int vector_of(int dim, int most) { return dim >= most ? most : 1; }

// KERNEL<W, V, bf16> for the call's width, VB or VF channels per thread (bf16, fp32) or one, and type.
#define KDA_CONV_PICK(KERNEL, VB, VF, GRID, ...)                                                  \
    do {                                                                                          \
        if (P.width == 2) KDA_CONV_W(KERNEL, 2, VB, VF, GRID, __VA_ARGS__);                       \
        else if (P.width == 3) KDA_CONV_W(KERNEL, 3, VB, VF, GRID, __VA_ARGS__);                  \
        else KDA_CONV_W(KERNEL, 4, VB, VF, GRID, __VA_ARGS__);                                    \
    } while (0)
#define KDA_CONV_W(KERNEL, W, VB, VF, GRID, ...)                                                  \
    do {                                                                                          \
        if (P.x.bf16 && V > 1) KERNEL<W, VB, true><<<GRID, 256, 0, P.stream>>>(__VA_ARGS__);      \
        else if (P.x.bf16) KERNEL<W, 1, true><<<GRID, 256, 0, P.stream>>>(__VA_ARGS__);           \
        else if (V > 1) KERNEL<W, VF, false><<<GRID, 256, 0, P.stream>>>(__VA_ARGS__);            \
        else KERNEL<W, 1, false><<<GRID, 256, 0, P.stream>>>(__VA_ARGS__);                        \
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

// How the forward kernel cuts its rows.
struct ConvFwdCut {
    int V, tile, cb;
    int64_t grid;
};
static ConvFwdCut conv_fwd_cut(int64_t rows, int dim) {
    const int V = vector_of(dim, 4), cb = (dim + 64 * V - 1) / (64 * V), tile = tile_of(rows, dim, V, 64, 16);
    return {V, tile, cb, (rows + tile * kWaves - 1) / (tile * kWaves) * cb};
}
int64_t conv_fwd_threads(int64_t rows, int dim) { return conv_fwd_cut(rows, dim).grid * 256; }

hipError_t launch_conv_fwd(const ConvLaunch &P) {
    const int64_t rows = conv_rows(P.cu, P.N, P.T);
    const ConvFwdCut cut = conv_fwd_cut(rows, P.dim);
    const int V = cut.V;
    if (rows > 0) KDA_CONV_PICK(conv_kernel, 4, 4, static_cast<unsigned>(cut.grid), P, rows, cut.cb, cut.tile);
    if (P.hT) {
        if (P.x.bf16) launch_state<uint16_t>(P);
        else launch_state<float>(P);
    }
    return hipGetLastError();
}

hipError_t launch_conv_step(const ConvLaunch &P) {
    // whole vectors only: a thread moved back over its neighbour's channels could read a state that the neighbour
    // has already shifted in place
    const int V = P.dim % 4 == 0 ? 4 : 1, cb = (P.dim + 256 * V - 1) / (256 * V);
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(P.N) * cb);
    KDA_CONV_PICK(conv_step_kernel, 4, 4, grid, P, cb);
    return hipGetLastError();
}

// How the gradient kernel cuts its rows: 64 to a thread (bf16, 8 channels wide, 4 x 4,096 x 4,096: 101 us, 32 rows 108,
// 128 rows 101).
struct ConvCut {
    int V, tile, cb;  // cb: workgroups across the channels
    int64_t parts;    // and along the rows
};
static ConvCut conv_cut(int64_t rows, int dim, bool bf16) {
    const int V = vector_of(dim, bf16 ? 8 : 4), tile = tile_of(rows, dim, V, 256 / kGradSubs, 64);
    const int cb = (dim + 256 / kGradSubs * V - 1) / (256 / kGradSubs * V);
    return {V, tile, cb, (rows + tile * kGradSubs - 1) / (tile * kGradSubs)};
}
int64_t conv_bwd_threads(int64_t rows, int dim, bool bf16) {
    const ConvCut cut = conv_cut(rows, dim, bf16);
    return cut.parts * cut.cb * 256;
}

size_t conv_bwd_workspace_bytes(int64_t rows, int dim, int width, bool bf16) {
    return static_cast<size_t>(conv_cut(rows, dim, bf16).parts) * (width + 1) * dim * 4;
}

hipError_t launch_conv_bwd(const ConvBwdLaunch &P) {
    const int64_t rows = conv_rows(P.cu, P.N, P.T);
    const ConvCut cut = conv_cut(rows, P.dim, P.x.bf16);
    const int V = cut.V;
    if (rows > 0)
        KDA_CONV_PICK(conv_grad_kernel, 8, 4, static_cast<unsigned>(cut.parts * cut.cb), P, rows, cut.cb, cut.tile);
    const int64_t ld = static_cast<int64_t>(P.width + 1) * P.dim;
    launch_column_sum(P.ws, ld, static_cast<int>(cut.parts), {{P.dw, P.db, nullptr}, {static_cast<int64_t>(P.width) * P.dim, P.dim, 0}},
                      P.stream);
    if (P.dh0 && P.N > 0) {
        if (P.x.bf16) launch_state_grad<true>(P);
        else launch_state_grad<false>(P);
    }
    return hipGetLastError();
}

}  // namespace kda
