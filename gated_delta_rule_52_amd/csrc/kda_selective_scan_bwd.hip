// kda_selective_scan_bwd.hip - gradients of the selective state space scan, for gfx950.
//
// With gp = grad_y silu(z) and G_t = C_t gp_t + exp(delta_{t+1} A) G_{t+1} going backwards,
//     dC = sum_d gp h,  dB = sum_d G delta u,  P = sum_n G B,  du = D gp + delta P,
//     ddelta = u P + sum_n A G c,  dA = sum_t delta G c,       c_t = exp(delta_t A) h_{t-1}
// (c is kept from the recomputed forward step; taking it as h - delta u B would cancel).
//
// Passes: scan_states_kernel walks each tile forwards and stores the state every kCkpt tokens; the gradient
// kernel takes the blocks of kCkpt tokens in reverse, recomputes a block's states from its stored one into
// registers and walks it backwards.  dB and dC sum over channels: in the wave, then over the workgroup's
// waves in LDS, then over workgroups by a last kernel, always in the same order.  Parameter gradients leave
// one partial per tile, summed by the column sum.
#include <type_traits>

#include "kda_layer.h"

namespace kda {

namespace {

// Tokens between stored states: what a block's decays and states take of the registers.
constexpr int ckpt_of(int R) { return R > 8 ? 4 : 8; }
constexpr int kBlock = 16;  // tokens per LDS block of the forward walk

template <bool InBf16>
struct Raw {
    using T = typename Elem<InBf16>::T;
    static __device__ __forceinline__ float f(T x) { return Elem<InBf16>::load(&x, 0); }
};

// Workspace, in floats.
struct BwdSpace {
    float *ck;  // [block][dim][ds] states entering each block of tokens; block = row / ckpt + slot + index
    float *pA;  // [slot][dim][ds]
    float *pD;  // [slot][dim]
    float *pb;  // [slot][dim]
    float *pBC; // [channel group][rows][2][ds]
    int64_t bytes;
};

// First stored block of a tile: tiles are disjoint in rows, so these ranges do not meet.
template <int R>
__device__ __forceinline__ int64_t first_block(const Tile &t, int64_t slot) {
    return t.begin / ckpt_of(R) + slot;
}

template <int R, bool InBf16>
__global__ void __launch_bounds__(256) scan_states_kernel(ScanBwdLaunch P, BwdSpace W) {
    using E = typename Raw<InBf16>::T;
    constexpr int NS = 4 * R, kSt = kBlock * NS / 256, kCkpt = ckpt_of(R);
    __shared__ __attribute__((aligned(16))) float sB[2][kBlock][NS];
    const int groups = (P.dim + 63) / 64;
    const int64_t slot = blockIdx.x / groups;
    const Tile tl = find_tile(P.seq, slot);
    if (!tl.valid || tl.len <= 0) return;
    const int q = threadIdx.x & 3;
    const int ch = static_cast<int>(blockIdx.x % groups) * 64 + (threadIdx.x >> 2);
    const bool live = ch < P.dim;
    const int chc = live ? ch : P.dim - 1;
    float A2[R], h[R];
    const int64_t sbase = (static_cast<int64_t>(tl.n) * P.dim + chc) * P.ds + q * R;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool in = q * R + r < P.ds;
        A2[r] = in ? kLog2e * P.A[static_cast<int64_t>(chc) * P.ds + q * R + r] : 0.f;
        h[r] = in && P.h0 ? P.h0[sbase + r] : 0.f;
    }
    const float bias = P.dt_bias ? P.dt_bias[chc] : 0.f;
    const E *u = static_cast<const E *>(P.u.p), *dt = static_cast<const E *>(P.dt.p);
    const E *Bp = static_cast<const E *>(P.B.p);
    E ru[4], rdt[4], rB[kSt];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = t0 + 4 * j + q;
            const int64_t row = tl.begin + (t < tl.len ? t : tl.len - 1);
            rdt[j] = dt[row * P.dt.stride + chc];
            ru[j] = u[row * P.u.stride + chc];
        }
#pragma unroll
        for (int i = 0; i < kSt; ++i) {
            const int e = i * 256 + threadIdx.x, t = t0 + e / NS, n = e % NS;
            rB[i] = t < tl.len && n < P.ds ? Bp[(tl.begin + t) * P.B.stride + n] : static_cast<E>(0);
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kSt; ++i) (&sB[buf][0][0])[i * 256 + threadIdx.x] = Raw<InBf16>::f(rB[i]);
    };
    fetch(0);
    stage(0);
    __syncthreads();
    float *ck = W.ck + (first_block<R>(tl, slot) * P.dim + chc) * P.ds + q * R;
    for (int t0 = 0, buf = 0; t0 < tl.len; t0 += kBlock, buf ^= 1) {
        float de[4], xs[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = t0 + 4 * j + q < tl.len;
            const float d = Raw<InBf16>::f(rdt[j]) + bias;
            de[j] = in ? (P.softplus ? softplus_f(d) : d) : 0.f;
            xs[j] = in ? de[j] * Raw<InBf16>::f(ru[j]) : 0.f;
        }
        const bool more = t0 + kBlock < tl.len;
        if (more) fetch(t0 + kBlock);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (t0 + 4 * j >= tl.len) break;
            if (j % (kCkpt / 4) == 0) {
                if (live) {
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        if (q * R + r < P.ds) ck[r] = h[r];
                }
                ck += static_cast<int64_t>(P.dim) * P.ds;
            }
            auto token = [&](float dl, float xl, int i) {
                const float *bt = &sB[buf][4 * j + i][q * R];
#pragma unroll
                for (int r = 0; r < R; ++r)
                    h[r] = fmaf(__builtin_amdgcn_exp2f(dl * A2[r]), h[r], xl * bt[r]);
            };
            token(quad_bcast<0>(de[j]), quad_bcast<0>(xs[j]), 0);
            token(quad_bcast<1>(de[j]), quad_bcast<1>(xs[j]), 1);
            token(quad_bcast<2>(de[j]), quad_bcast<2>(xs[j]), 2);
            token(quad_bcast<3>(de[j]), quad_bcast<3>(xs[j]), 3);
        }
        if (more) stage(buf ^ 1);
        __syncthreads();
    }
}

// Sum over the 16 lanes of a wave that hold the same states of different channels (lane = 4 c + q).
__device__ __forceinline__ float channel_sum(float x) {
    x += dpp_mov<0x124>(x);  // row rotate by 4
    x += dpp_mov<0x128>(x);  // row rotate by 8
    x += __shfl_xor(x, 16, kWave);
    return x + __shfl_xor(x, 32, kWave);
}

// M channels per quad: a wave holds 16 M channels (c, c + 16, ...), a workgroup 64 M.
template <int R, int M, bool InBf16>
__global__ void __launch_bounds__(256) scan_grad_kernel(ScanBwdLaunch P, BwdSpace W) {
    using E = typename Raw<InBf16>::T;
    constexpr int kCkpt = ckpt_of(R), NS = 4 * R, J = kCkpt / 4, kSt = (kCkpt * NS + 255) / 256;
    __shared__ __attribute__((aligned(16))) float sB[2][kCkpt][NS], sC[2][kCkpt][NS];
    __shared__ float sR[2][4][kCkpt][2 * NS];  // per wave: dB, dC of each token
    const int groups = (P.dim + 64 * M - 1) / (64 * M);
    const int64_t slot = blockIdx.x / groups;
    const int group = static_cast<int>(blockIdx.x % groups);
    const Tile tl = find_tile(P.seq, slot);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, q = lane & 3;
    int chn[M], chc[M];
    bool live[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        chn[m] = group * 64 * M + wave * 16 * M + 16 * m + (lane >> 2);
        live[m] = chn[m] < P.dim;
        chc[m] = live[m] ? chn[m] : P.dim - 1;
    }
    float A2[M][R], G[M][R], dA[M][R], skip[M], bias[M], dD[M], db[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        skip[m] = P.D ? P.D[chc[m]] : 0.f;
        bias[m] = P.dt_bias ? P.dt_bias[chc[m]] : 0.f;
        dD[m] = db[m] = 0.f;
        const int64_t sb = (static_cast<int64_t>(tl.n) * P.dim + chc[m]) * P.ds + q * R;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = q * R + r < P.ds;
            A2[m][r] = in ? kLog2e * P.A[static_cast<int64_t>(chc[m]) * P.ds + q * R + r] : 0.f;
            G[m][r] = in && tl.valid && P.dhT ? P.dhT[sb + r] : 0.f;
            dA[m][r] = 0.f;
        }
    }
    if (tl.valid && tl.len > 0) {
        const E *u = static_cast<const E *>(P.u.p), *dt = static_cast<const E *>(P.dt.p);
        const E *z = static_cast<const E *>(P.z.p), *gy = static_cast<const E *>(P.gy.p);
        const E *Bp = static_cast<const E *>(P.B.p), *Cp = static_cast<const E *>(P.C.p);
        E ru[M][J], rdt[M][J], rz[M][J], rg[M][J], rB[kSt], rC[kSt];
        float ck[M][R];
        const int blocks = (tl.len + kCkpt - 1) / kCkpt;
        auto fetch = [&](int b) {
#pragma unroll
            for (int m = 0; m < M; ++m) {
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int t = b * kCkpt + 4 * j + q;
                    const int64_t row = tl.begin + (t < tl.len ? t : tl.len - 1);
                    rdt[m][j] = dt[row * P.dt.stride + chc[m]];
                    ru[m][j] = u[row * P.u.stride + chc[m]];
                    rg[m][j] = gy[row * P.gy.stride + chc[m]];
                    if (z) rz[m][j] = z[row * P.z.stride + chc[m]];
                }
                const float *c = W.ck + ((first_block<R>(tl, slot) + b) * P.dim + chc[m]) * P.ds + q * R;
#pragma unroll
                for (int r = 0; r < R; ++r) ck[m][r] = q * R + r < P.ds ? c[r] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < kSt; ++i) {
                const int e = i * 256 + threadIdx.x, t = b * kCkpt + e / NS, n = e % NS;
                rB[i] = rC[i] = 0;
                if (e < kCkpt * NS && t < tl.len && n < P.ds) {
                    rB[i] = Bp[(tl.begin + t) * P.B.stride + n];
                    rC[i] = Cp[(tl.begin + t) * P.C.stride + n];
                }
            }
        };
        auto stage = [&](int buf) {
#pragma unroll
            for (int i = 0; i < kSt; ++i) {
                const int e = i * 256 + threadIdx.x;
                if (e < kCkpt * NS) {
                    (&sB[buf][0][0])[e] = Raw<InBf16>::f(rB[i]);
                    (&sC[buf][0][0])[e] = Raw<InBf16>::f(rC[i]);
                }
            }
        };
        fetch(blocks - 1);
        stage(0);
        __syncthreads();
        int buf = 0;
        for (int b = blocks - 1; b >= 0; --b, buf ^= 1) {
            float de[M][J], sl[M][J], us[M][J], xs[M][J], gp[M][J], gv[M][J], zs[M][J], h[M][R];
#pragma unroll
            for (int m = 0; m < M; ++m) {
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const bool in = live[m] && b * kCkpt + 4 * j + q < tl.len;
                    const float d = Raw<InBf16>::f(rdt[m][j]) + bias[m];
                    de[m][j] = in ? (P.softplus ? softplus_f(d) : d) : 0.f;
                    sl[m][j] = P.softplus ? sigmoid_f(d) : 1.f;
                    us[m][j] = in ? Raw<InBf16>::f(ru[m][j]) : 0.f;
                    xs[m][j] = de[m][j] * us[m][j];
                    gv[m][j] = in ? Raw<InBf16>::f(rg[m][j]) : 0.f;
                    zs[m][j] = in && z ? Raw<InBf16>::f(rz[m][j]) : 0.f;
                    gp[m][j] = z ? gv[m][j] * (zs[m][j] * sigmoid_f(zs[m][j])) : gv[m][j];
                }
#pragma unroll
                for (int r = 0; r < R; ++r) h[m][r] = ck[m][r];
            }
            if (b > 0) fetch(b - 1);
            // forwards: decay a, carried state c = a h and the output sum of every token of the block
            float ha[kCkpt][M][R], hc[kCkpt][M][R], yp[M][kCkpt], dA8[M][R];
            auto ahead = [&](auto jc, auto ic) {
                constexpr int j = decltype(jc)::value, i = decltype(ic)::value, t = 4 * j + i;
                const float *bt = &sB[buf][t][q * R], *ct = &sC[buf][t][q * R];
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const float dl = quad_bcast<i>(de[m][j]), xl = quad_bcast<i>(xs[m][j]);
                    float acc = 0.f;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float a = __builtin_amdgcn_exp2f(dl * A2[m][r]), c = a * h[m][r];
                        h[m][r] = fmaf(xl, bt[r], c);
                        ha[t][m][r] = a;
                        hc[t][m][r] = c;
                        acc = fmaf(ct[r], h[m][r], acc);
                    }
                    yp[m][t] = acc;
                }
            };
            // backwards
            float Pn[M][kCkpt], Sn[M][kCkpt];
            auto back = [&](auto jc, auto ic) {
                constexpr int j = decltype(jc)::value, i = decltype(ic)::value, t = 4 * j + i;
                const float *bt = &sB[buf][t][q * R], *ct = &sC[buf][t][q * R];
                float dB[R], dC[R];
#pragma unroll
                for (int r = 0; r < R; ++r) dB[r] = dC[r] = 0.f;
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const float dl = quad_bcast<i>(de[m][j]), xl = quad_bcast<i>(xs[m][j]), g = quad_bcast<i>(gp[m][j]);
                    float pn = 0.f, sn = 0.f;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float gg = fmaf(ct[r], g, G[m][r]), c = hc[t][m][r];
                        dC[r] = fmaf(fmaf(xl, bt[r], c), g, dC[r]);
                        dB[r] = fmaf(gg, xl, dB[r]);
                        pn = fmaf(gg, bt[r], pn);
                        const float e = gg * c;
                        sn = fmaf(e, A2[m][r], sn);
                        dA8[m][r] = fmaf(e, dl, dA8[m][r]);
                        G[m][r] = ha[t][m][r] * gg;
                    }
                    Pn[m][t] = pn;
                    Sn[m][t] = sn;
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float sb = channel_sum(dB[r]), sc = channel_sum(dC[r]);
                    if (lane < 4) {
                        sR[buf][wave][t][q * R + r] = sb;
                        sR[buf][wave][t][NS + q * R + r] = sc;
                    }
                }
            };
#define KDA_I(v) std::integral_constant<int, v>{}
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int r = 0; r < R; ++r) dA8[m][r] = 0.f;
            ahead(KDA_I(0), KDA_I(0)); ahead(KDA_I(0), KDA_I(1)); ahead(KDA_I(0), KDA_I(2)); ahead(KDA_I(0), KDA_I(3));
            if constexpr (J > 1) {
                ahead(KDA_I(1), KDA_I(0)); ahead(KDA_I(1), KDA_I(1)); ahead(KDA_I(1), KDA_I(2)); ahead(KDA_I(1), KDA_I(3));
                back(KDA_I(1), KDA_I(3)); back(KDA_I(1), KDA_I(2)); back(KDA_I(1), KDA_I(1)); back(KDA_I(1), KDA_I(0));
            }
            back(KDA_I(0), KDA_I(3)); back(KDA_I(0), KDA_I(2)); back(KDA_I(0), KDA_I(1)); back(KDA_I(0), KDA_I(0));
#undef KDA_I
#pragma unroll
            for (int m = 0; m < M; ++m) {
#pragma unroll
                for (int r = 0; r < R; ++r) dA[m][r] += dA8[m][r];
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int t = b * kCkpt + 4 * j + q;
                    const int64_t row = tl.begin + t;
                    const float pn = quad_transpose_sum(Pn[m][4 * j], Pn[m][4 * j + 1], Pn[m][4 * j + 2], Pn[m][4 * j + 3], q);
                    const float sn = quad_transpose_sum(Sn[m][4 * j], Sn[m][4 * j + 1], Sn[m][4 * j + 2], Sn[m][4 * j + 3], q);
                    // sn carries A log2(e)
                    const float dd = sl[m][j] * fmaf(us[m][j], pn, 0.6931471805599453f * sn);
                    const float du = fmaf(skip[m], gp[m][j], de[m][j] * pn);
                    if (z) {
                        const float yv = fmaf(skip[m], us[m][j],
                                              quad_transpose_sum(yp[m][4 * j], yp[m][4 * j + 1], yp[m][4 * j + 2], yp[m][4 * j + 3], q));
                        const float sg = sigmoid_f(zs[m][j]);
                        if (live[m] && t < tl.len)
                            P.dz.put(row, chn[m], gv[m][j] * yv * (sg * fmaf(zs[m][j], 1.f - sg, 1.f)));
                    }
                    dD[m] = fmaf(gp[m][j], us[m][j], dD[m]);
                    if (live[m] && t < tl.len) {
                        db[m] += dd;
                        P.du.put(row, chn[m], du);
                        P.ddt.put(row, chn[m], dd);
                    }
                }
            }
            if (b > 0) stage(buf ^ 1);
            __syncthreads();
            for (int e = threadIdx.x; e < kCkpt * 2 * NS; e += 256) {
                const int t = e / (2 * NS), n = e % (2 * NS), half = n / NS, s = n % NS;
                if (b * kCkpt + t < tl.len && s < P.ds)
                    W.pBC[((static_cast<int64_t>(group) * P.seq.rows() + tl.begin + b * kCkpt + t) * 2 + half) * P.ds + s] =
                        (sR[buf][0][t][n] + sR[buf][1][t][n]) + (sR[buf][2][t][n] + sR[buf][3][t][n]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const float d = quad_sum(dD[m]), bsum = quad_sum(db[m]);
        if (!live[m]) continue;
        const int64_t pb = slot * P.dim + chn[m];
        if (q == 0) {
            W.pD[pb] = d;
            W.pb[pb] = bsum;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (q * R + r >= P.ds) continue;
            W.pA[pb * P.ds + q * R + r] = dA[m][r];
            if (P.dh0 && tl.valid && tl.k == 0)
                P.dh0[(static_cast<int64_t>(tl.n) * P.dim + chn[m]) * P.ds + q * R + r] = G[m][r];
        }
    }
}

// dB, dC: the channel groups' partials summed and rounded.  Rows behind the last sequence stay as they are.
__global__ void __launch_bounds__(256) scan_bc_sum_kernel(ScanBwdLaunch P, const float *pBC, int groups) {
    const int64_t rows = P.seq.rows(), per = 2 * P.ds, e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (e >= rows * per) return;
    const int64_t row = e / per;
    const int half = static_cast<int>(e % per) / P.ds, s = static_cast<int>(e % per) % P.ds;
    if (P.seq.cu && (row < P.seq.offset(0) || row >= P.seq.offset(P.seq.N))) return;
    float a = 0.f;
    for (int g = 0; g < groups; ++g) a += pBC[static_cast<int64_t>(g) * rows * per + e];
    (half ? P.dC : P.dB).put(row, s, a);
}

int channels_per_quad(int ds) { return ds <= 16 ? 2 : 1; }

BwdSpace space(float *ws, const SeqTiles &seq, int dim, int ds) {
    const int64_t slots = seq.slots(), rows = seq.rows(), wide = 64 * channels_per_quad(ds);
    const int64_t groups = (dim + wide - 1) / wide, blocks = rows / (ds <= 32 ? 8 : 4) + slots + 1;
    BwdSpace w{};
    int64_t at = 0;
    auto take = [&](int64_t n) {
        float *p = ws ? ws + at : nullptr;
        at += (n + 3) & ~int64_t{3};
        return p;
    };
    w.ck = take(blocks * dim * ds);
    w.pA = take(slots * dim * ds);
    w.pD = take(slots * dim);
    w.pb = take(slots * dim);
    w.pBC = take(groups * rows * 2 * ds);
    w.bytes = at * 4;
    return w;
}

template <int R, int M, bool InBf16>
void launch_grad(const ScanBwdLaunch &P, const BwdSpace &w) {
    const int64_t slots = P.seq.slots();
    if (slots == 0) return;
    const int g1 = (P.dim + 63) / 64, g2 = (P.dim + 64 * M - 1) / (64 * M);
    scan_states_kernel<R, InBf16><<<static_cast<unsigned>(slots * g1), 256, 0, P.stream>>>(P, w);
    scan_grad_kernel<R, M, InBf16><<<static_cast<unsigned>(slots * g2), 256, 0, P.stream>>>(P, w);
    const int64_t n = P.seq.rows() * 2 * P.ds;
    if (n > 0) scan_bc_sum_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, P.stream>>>(P, w.pBC, g2);
}

template <bool InBf16>
void launch_any(const ScanBwdLaunch &P, const BwdSpace &w) {
    if (P.ds <= 16) launch_grad<4, 2, InBf16>(P, w);
    else if (P.ds <= 32) launch_grad<8, 1, InBf16>(P, w);
    else launch_grad<16, 1, InBf16>(P, w);
}

}  // namespace

SeqTiles scan_bwd_tiles(const int32_t *cu, int N, int T, int dim, int ds) {
    SeqTiles s{cu, N, T, T > 0 ? T : 1};
    return s;
}

size_t scan_bwd_workspace_bytes(const SeqTiles &seq, int dim, int ds) { return space(nullptr, seq, dim, ds).bytes; }

hipError_t launch_scan_bwd(const ScanBwdLaunch &P) {
    const BwdSpace w = space(P.ws, P.seq, P.dim, P.ds);
    if (P.u.bf16) launch_any<true>(P, w);
    else launch_any<false>(P, w);
    const int slots = static_cast<int>(P.seq.slots());
    launch_column_sum(w.pA, static_cast<int64_t>(P.dim) * P.ds, slots, static_cast<int64_t>(P.dim) * P.ds, P.dA, P.stream);
    if (P.dD) launch_column_sum(w.pD, P.dim, slots, P.dim, P.dD, P.stream);
    if (P.ddt_bias) launch_column_sum(w.pb, P.dim, slots, P.dim, P.ddt_bias, P.stream);
    return hipGetLastError();
}

}  // namespace kda
