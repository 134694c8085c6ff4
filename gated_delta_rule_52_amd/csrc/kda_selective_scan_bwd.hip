// kda_selective_scan_bwd.hip - gradients of the selective state space scan, for gfx950.
//
// With gp = grad_y silu(z) and G_t = C_t gp_t + exp(delta_{t+1} A) G_{t+1} going backwards,
//     dC = sum_d gp h,  dB = sum_d G delta u,  P = sum_n G B,  du = D gp + delta P,
//     ddelta = u P + sum_n A G c,  dA = sum_t delta G c,       c_t = exp(delta_t A) h_{t-1}
// (c is kept from the recomputed forward step; taking it as h - delta u B would cancel).
//
// Passes: scan_states_kernel walks each tile forwards and stores the state every 8 tokens (4 beyond 16 states); the
// gradient kernel takes these blocks in reverse, recomputes a block's states from its stored one into
// registers and walks it backwards.  Sequences too few to fill the chip are cut into tiles, which a combine
// chains both ways.  dB and dC sum over channels: in the wave, then over the workgroup's
// waves in LDS, then over workgroups by a last kernel, always in the same order.  Parameter gradients leave
// one partial per tile, summed by the column sum.
#include <type_traits>

#include "kda_layer.h"

namespace kda {

namespace {

// Tokens between stored states: what a block's decays and states take of the registers.  8 states per lane with 4
// tokens leave two waves per SIMD, with 8 one (4 x 2,048 x 2,048 x 24 bf16: 715 us against 820).
constexpr int ckpt_of(int R) { return R > 4 ? 4 : 8; }
constexpr int kBlock = 16;  // tokens per LDS block of the forward walk

template <bool InBf16>
struct Raw {
    using T = typename Elem<InBf16>::T;
    static __device__ __forceinline__ float f(T x) { return Elem<InBf16>::load(&x, 0); }
};

// Workspace, in floats.
struct BwdSpace {
    float *ck;   // [block][dim][4 R] states entering each block of tokens, from the tile's start; block = row / ckpt + slot + index
    float *cum;  // [block][dim] sum of delta from the tile's start to the block
    float *H;    // [slot][dim][ds] state a tile reaches from zero, then the one it starts from
    float *G;    // [slot][dim][ds] state gradient at a tile's start from its own outputs, then the one behind its end
    float *sum;  // [slot][dim] sum of delta over a tile
    float *par;  // [slot][dim ds + 2 dim] partial gradients of A, D and the bias
    float *pBC;  // [channel group][rows][2][ds]
    int64_t bytes;
};

// First stored block of a tile: tiles are disjoint in rows, so these ranges do not meet.
template <int R>
__device__ __forceinline__ int64_t first_block(const Tile &t, int64_t slot) {
    return t.begin / ckpt_of(R) + slot;
}

// One walk over a tile: states at every block, and for sequences of several tiles what the two chains need,
// the state reached from zero and the gradient that the tile's outputs send to its start,
//     sum_t (prod_{s <= t} a_s) C_t gp_t,
// which the forward order gives with a running product.
template <int R, bool InBf16, bool TILED, bool GATED>
__global__ void __launch_bounds__(256) scan_states_kernel(ScanBwdLaunch P, BwdSpace W) {
    using E = typename Raw<InBf16>::T;
    constexpr int NS = 4 * R, kSt = kBlock * NS / 256, kCkpt = ckpt_of(R);
    __shared__ __attribute__((aligned(16))) float sB[2][kBlock][NS], sC[TILED ? 2 : 1][kBlock][NS];
    const int groups = (P.dim + 63) / 64;
    const int64_t slot = blockIdx.x / groups;
    const Tile tl = find_tile(P.seq, slot);
    if (!tl.valid || tl.len <= 0) return;
    const int q = threadIdx.x & 3;
    const int ch = static_cast<int>(blockIdx.x % groups) * 64 + (threadIdx.x >> 2);
    const bool live = ch < P.dim, chained = TILED && tl.count > 1;
    const int chc = live ? ch : P.dim - 1;
    float A2[R], h[R], prod[R], acc[R];
    const int64_t sbase = (static_cast<int64_t>(tl.n) * P.dim + chc) * P.ds + q * R;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool in = q * R + r < P.ds;
        A2[r] = in ? kLog2e * P.A[static_cast<int64_t>(chc) * P.ds + q * R + r] : 0.f;
        h[r] = in && P.h0 && !chained ? P.h0[sbase + r] : 0.f;
        prod[r] = 1.f;
        acc[r] = 0.f;
    }
    const float bias = P.dt_bias ? P.dt_bias[chc] : 0.f;
    const Column cu(P.u, tl.begin, chc), cd(P.dt, tl.begin, chc), cz(P.z, tl.begin, chc), cg(P.gy, tl.begin, chc);
    const E *Bp = static_cast<const E *>(P.B.p) + tl.begin * P.B.stride;
    const E *Cp = static_cast<const E *>(P.C.p) + tl.begin * P.C.stride;
    E ru[4], rdt[4], rz[4], rg[4], rB[kSt], rC[kSt];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const Group g(t0 + 4 * j, tl.len, q);
            rdt[j] = cd.get<E>(g);
            ru[j] = cu.get<E>(g);
            if (TILED) rg[j] = cg.get<E>(g);
            if (TILED && GATED) rz[j] = cz.get<E>(g);
        }
#pragma unroll
        for (int i = 0; i < kSt; ++i) {
            const int e = i * 256 + threadIdx.x, n = e % NS < P.ds ? e % NS : P.ds - 1;
            const int left = tl.len - 1 - t0, t = e / NS < left ? e / NS : left;
            rB[i] = (Bp + t0 * P.B.stride)[static_cast<uint32_t>(t) * static_cast<uint32_t>(P.B.stride) + n];
            if (TILED) rC[i] = (Cp + t0 * P.C.stride)[static_cast<uint32_t>(t) * static_cast<uint32_t>(P.C.stride) + n];
        }
    };
    auto stage = [&](int t0, int buf) {
#pragma unroll
        for (int i = 0; i < kSt; ++i) {
            const int e = i * 256 + threadIdx.x;
            const bool in = t0 + e / NS < tl.len && e % NS < P.ds;
            (&sB[buf][0][0])[e] = in ? Raw<InBf16>::f(rB[i]) : 0.f;
            if (TILED) (&sC[buf][0][0])[e] = in ? Raw<InBf16>::f(rC[i]) : 0.f;
        }
    };
    fetch(0);
    stage(0, 0);
    __syncthreads();
    int64_t at = first_block<R>(tl, slot) * P.dim + chc;
    float total = 0.f;
    for (int t0 = 0, buf = 0; t0 < tl.len; t0 += kBlock, buf ^= 1) {
        float de[4], xs[4], gp[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) de[j] = Raw<InBf16>::f(rdt[j]) + bias;
        if (P.softplus) {
#pragma unroll
            for (int j = 0; j < 4; ++j) de[j] = softplus_f(de[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = t0 + 4 * j + q < tl.len;
            de[j] = in ? de[j] : 0.f;
            xs[j] = in ? de[j] * Raw<InBf16>::f(ru[j]) : 0.f;
            if (TILED) {
                gp[j] = Raw<InBf16>::f(rg[j]);
                if (GATED) {
                    const float z = Raw<InBf16>::f(rz[j]);
                    gp[j] *= z * sigmoid_f(z);
                }
                gp[j] = in ? gp[j] : 0.f;
            }
        }
        const bool more = t0 + kBlock < tl.len;
        if (more) fetch(t0 + kBlock);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (t0 + 4 * j >= tl.len) break;
            if (j % (kCkpt / 4) == 0) {
                if (live) {
                    float4 *c = reinterpret_cast<float4 *>(W.ck + at * NS + q * R);
#pragma unroll
                    for (int r = 0; r < R; r += 4) c[r / 4] = make_float4(h[r], h[r + 1], h[r + 2], h[r + 3]);
                }
                if (TILED) {
                    const float before = quad_sum(total);
                    if (live && q == 0) W.cum[at] = before;
                }
                at += P.dim;
            }
            if (TILED) total += de[j];
            auto token = [&](float dl, float xl, float g, int i) {
                const float *bt = &sB[buf][4 * j + i][q * R], *ct = &sC[TILED ? buf : 0][4 * j + i][q * R];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float a = __builtin_amdgcn_exp2f(dl * A2[r]);
                    h[r] = fmaf(a, h[r], xl * bt[r]);
                    if (TILED) {
                        prod[r] *= a;
                        acc[r] = fmaf(prod[r], ct[r] * g, acc[r]);
                    }
                }
            };
            token(lane_bcast<0>(de[j]), lane_bcast<0>(xs[j]), lane_bcast<0>(TILED ? gp[j] : 0.f), 0);
            token(lane_bcast<1>(de[j]), lane_bcast<1>(xs[j]), lane_bcast<1>(TILED ? gp[j] : 0.f), 1);
            token(lane_bcast<2>(de[j]), lane_bcast<2>(xs[j]), lane_bcast<2>(TILED ? gp[j] : 0.f), 2);
            token(lane_bcast<3>(de[j]), lane_bcast<3>(xs[j]), lane_bcast<3>(TILED ? gp[j] : 0.f), 3);
        }
        if (more) stage(t0 + kBlock, buf ^ 1);
        __syncthreads();
    }
    if (chained) {
        total = quad_sum(total);
        const int64_t w = slot * P.dim + chc;
        if (live) {
            if (q == 0) W.sum[w] = total;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (q * R + r < P.ds) {
                    W.H[w * P.ds + q * R + r] = h[r];
                    W.G[w * P.ds + q * R + r] = acc[r];
                }
        }
    }
}

// Chains the tiles of every sequence that has several, both ways: H becomes the state each tile starts from,
// G the gradient of the state each tile leaves.
__global__ void __launch_bounds__(256) scan_bwd_combine_kernel(ScanBwdLaunch P, BwdSpace W) {
    const int n = blockIdx.y;
    const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, states = static_cast<int64_t>(P.dim) * P.ds;
    int64_t start;
    int len;
    P.seq.sequence(n, start, len);
    const int count = P.seq.tiles(len);
    if (e >= states || count <= 1) return;
    const int64_t first = P.seq.first_slot(n, start);
    const float A2 = kLog2e * P.A[e];
    float ahead = P.h0 ? P.h0[n * states + e] : 0.f, back = P.dhT ? P.dhT[n * states + e] : 0.f;
    float *H = W.H + first * states + e, *G = W.G + first * states + e;
    const float *sum = W.sum + first * P.dim + static_cast<int>(e / P.ds);
    constexpr int U = 4;  // tiles in flight: their loads do not wait for the chains
    for (int k = 0; k < count; k += U) {
        float h[U], g[U], dh[U], dg[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const bool in = k + i < count;
            const int64_t f = k + i, b = count - 1 - f;
            h[i] = in ? H[f * states] : 0.f;
            g[i] = in ? G[b * states] : 0.f;
            dh[i] = in ? sum[f * P.dim] : 0.f;
            dg[i] = in ? sum[b * P.dim] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (k + i >= count) break;
            H[(k + i) * states] = ahead;
            ahead = fmaf(__builtin_amdgcn_exp2f(A2 * dh[i]), ahead, h[i]);
            G[(count - 1 - k - i) * states] = back;
            back = fmaf(__builtin_amdgcn_exp2f(A2 * dg[i]), back, g[i]);
        }
    }
}

template <int R, bool InBf16, bool TILED, bool GATED>
__global__ void __launch_bounds__(256) scan_grad_kernel(ScanBwdLaunch P, BwdSpace W) {
    using E = typename Raw<InBf16>::T;
    constexpr int kCkpt = ckpt_of(R), NS = 4 * R, J = kCkpt / 4, kSt = 2 * kCkpt * NS / 256;
    static_assert(R % 4 == 0, "the channel sums take four states at a time");
    static_assert(2 * kCkpt * NS % 256 == 0, "staging");
    __shared__ __attribute__((aligned(16))) float sBC[2][2][kCkpt][NS];
    __shared__ float sR[2][4][kCkpt][2 * NS];  // per wave: dB, dC of each token
    // A block's decays wait in LDS, each lane's own, not in registers: with them there three waves fit a SIMD.
    constexpr bool kStash = R <= 4;
    __shared__ float4 sA[kStash ? kCkpt : 1][kStash ? 256 : 1];
    const int groups = (P.dim + 63) / 64;
    const int64_t slot = blockIdx.x / groups;
    const int group = static_cast<int>(blockIdx.x % groups);
    const Tile tl = find_tile(P.seq, slot);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, q = lane & 3;
    const int ch = group * 64 + (threadIdx.x >> 2);
    const bool chained = TILED && tl.count > 1, live = ch < P.dim;
    const int chc = live ? ch : P.dim - 1;
    float A2[R], G[R], from[R], dA[R], dD = 0.f, db = 0.f;
    const float skip = P.D ? P.D[chc] : 0.f, bias = P.dt_bias ? P.dt_bias[chc] : 0.f;
    {
        const int64_t sb = (static_cast<int64_t>(tl.n) * P.dim + chc) * P.ds + q * R;
        const int64_t wb = (slot * P.dim + chc) * P.ds + q * R;
        const float *g = !tl.valid ? nullptr : chained ? W.G + wb : P.dhT ? P.dhT + sb : nullptr;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = q * R + r < P.ds;
            A2[r] = in ? kLog2e * P.A[static_cast<int64_t>(chc) * P.ds + q * R + r] : 0.f;
            G[r] = in && g ? g[r] : 0.f;
            from[r] = in && chained && tl.valid ? W.H[wb + r] : 0.f;
            dA[r] = 0.f;
        }
    }
    if (tl.valid && tl.len > 0) {
        const int blocks = (tl.len + kCkpt - 1) / kCkpt;
        const Column cu(P.u, tl.begin, chc), cd(P.dt, tl.begin, chc), cz(P.z, tl.begin, chc), cg(P.gy, tl.begin, chc);
        const Column ou(P.du, tl.begin, chc), od(P.ddt, tl.begin, chc), oz(P.dz, tl.begin, chc);
        const E *Bp = static_cast<const E *>(P.B.p) + tl.begin * P.B.stride;
        const E *Cp = static_cast<const E *>(P.C.p) + tl.begin * P.C.stride;
        E ru[J], rdt[J], rz[J], rg[J], rBC[kSt];
        float4 ck[R / 4];
        float cum = 0.f;
        // a thread stages B or C of one token and state
        const E *half[kSt];
        uint32_t halfstep[kSt];
#pragma unroll
        for (int i = 0; i < kSt; ++i) {
            const bool second = i * 256 + threadIdx.x >= kCkpt * NS;
            const int n = (i * 256 + threadIdx.x) % NS;
            half[i] = (second ? Cp : Bp) + (n < P.ds ? n : P.ds - 1);
            halfstep[i] = static_cast<uint32_t>(second ? P.C.stride : P.B.stride);
        }
        auto fetch = [&](int b) {
            const int t0 = b * kCkpt;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const Group g(t0 + 4 * j, tl.len, q);
                rdt[j] = cd.get<E>(g);
                ru[j] = cu.get<E>(g);
                rg[j] = cg.get<E>(g);
                if (GATED) rz[j] = cz.get<E>(g);
            }
            const int64_t at = (first_block<R>(tl, slot) + b) * P.dim;
            const float4 *c = reinterpret_cast<const float4 *>(W.ck + at * NS) + (static_cast<uint32_t>(chc) * NS + q * R) / 4;
#pragma unroll
            for (int r = 0; r < R / 4; ++r) ck[r] = c[r];
            if (TILED) cum = (W.cum + at)[static_cast<uint32_t>(chc)];
#pragma unroll
            for (int i = 0; i < kSt; ++i) {
                const int left = tl.len - 1, row = t0 + (i * 256 + static_cast<int>(threadIdx.x)) / NS % kCkpt;
                rBC[i] = half[i][static_cast<int64_t>(row < left ? row : left) * halfstep[i]];
            }
        };
        auto stage = [&](int b, int buf) {
#pragma unroll
            for (int i = 0; i < kSt; ++i) {
                const int e = i * 256 + threadIdx.x;
                const bool in = b * kCkpt + e / NS % kCkpt < tl.len && e % NS < P.ds;
                (&sBC[buf][0][0][0])[e] = in ? Raw<InBf16>::f(rBC[i]) : 0.f;
            }
        };
        fetch(blocks - 1);
        stage(blocks - 1, 0);
        __syncthreads();
        int buf = 0;
        const int mine = quads_sum4_value(lane);  // which of four states this lane's row sums
        float *pBC = W.pBC + (static_cast<int64_t>(group) * P.seq.rows() + tl.begin) * 2 * P.ds;
        for (int b = blocks - 1; b >= 0; --b, buf ^= 1) {
            float de[J], sl[J], us[J], xs[J], gp[J], gv[J], h[R], yv[J], gu[J], gd[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                de[j] = Raw<InBf16>::f(rdt[j]) + bias;
                sl[j] = 1.f;
            }
            if (P.softplus) {
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    sl[j] = sigmoid_f(de[j]);
                    de[j] = softplus_f(de[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const bool in = live && b * kCkpt + 4 * j + q < tl.len;
                de[j] = in ? de[j] : 0.f;
                us[j] = in ? Raw<InBf16>::f(ru[j]) : 0.f;
                gv[j] = in ? Raw<InBf16>::f(rg[j]) : 0.f;
                xs[j] = de[j] * us[j];
                gp[j] = gv[j];
                if (GATED) {
                    const float z = in ? Raw<InBf16>::f(rz[j]) : 0.f, sg = sigmoid_f(z);
                    gp[j] *= z * sg;
                    gv[j] *= sg * fmaf(z, 1.f - sg, 1.f);  // what dz takes of the output
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                h[r] = reinterpret_cast<const float *>(ck)[r];
                if (TILED) {  // a sequence's only tile has its true states stored
                    const float shifted = fmaf(__builtin_amdgcn_exp2f(cum * A2[r]), from[r], h[r]);
                    h[r] = chained ? shifted : h[r];
                }
            }
            if (b > 0) fetch(b - 1);
            // forwards: decay a and carried state c = a h of every token of the block, and its output sum
            float ha[kStash ? 1 : kCkpt][R], hc[kCkpt][R], dA8[R], part[4];
            auto ahead = [&](auto jc, auto ic) {
                constexpr int j = decltype(jc)::value, i = decltype(ic)::value, t = 4 * j + i;
                const float *bt = &sBC[buf][0][t][q * R], *ct = &sBC[buf][1][t][q * R];
                const float dl = lane_bcast<i>(de[j]), xl = lane_bcast<i>(xs[j]);
                float acc = 0.f;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float a = __builtin_amdgcn_exp2f(dl * A2[r]), c = a * h[r];
                    h[r] = fmaf(xl, bt[r], c);
                    ha[kStash ? 0 : t][r] = a;
                    hc[t][r] = c;
                    if (GATED) acc = fmaf(ct[r], h[r], acc);
                }
                if constexpr (kStash) sA[t][threadIdx.x] = make_float4(ha[0][0], ha[0][1], ha[0][2], ha[0][3]);
                part[i] = acc;
                if (GATED && i == 3) yv[j] = transpose_sum(part, q);
            };
            // backwards
            float Pn[4], Sn[4];
            auto back = [&](auto jc, auto ic) {
                constexpr int j = decltype(jc)::value, i = decltype(ic)::value, t = 4 * j + i;
                const float *bt = &sBC[buf][0][t][q * R], *ct = &sBC[buf][1][t][q * R];
                const float dl = lane_bcast<i>(de[j]), xl = lane_bcast<i>(xs[j]), g = lane_bcast<i>(gp[j]);
                float dB[R], dC[R], pn = 0.f, sn = 0.f;
                const float *a = kStash ? reinterpret_cast<const float *>(&sA[kStash ? t : 0][kStash ? threadIdx.x : 0])
                                        : ha[kStash ? 0 : t];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float gg = fmaf(ct[r], g, G[r]), c = hc[t][r], e = gg * c;
                    dC[r] = fmaf(xl, bt[r], c) * g;
                    dB[r] = gg * xl;
                    pn = fmaf(gg, bt[r], pn);
                    sn = fmaf(e, A2[r], sn);
                    dA8[r] = fmaf(e, dl, dA8[r]);
                    G[r] = a[r] * gg;
                }
                Pn[i] = pn;
                Sn[i] = sn;
#pragma unroll
                for (int r = 0; r < R; r += 4) {
                    const float sb = quads_sum4(dB[r], dB[r + 1], dB[r + 2], dB[r + 3]);
                    const float sc = quads_sum4(dC[r], dC[r + 1], dC[r + 2], dC[r + 3]);
                    // every quad of a row has the sums: one writes dB's, another dC's
                    if (!(lane & 8)) sR[buf][wave][t][(lane & 4 ? NS : 0) + q * R + r + mine] = lane & 4 ? sc : sb;
                }
                if (i > 0) return;
                const float p = transpose_sum(Pn, q), s = transpose_sum(Sn, q);
                gd[j] = sl[j] * fmaf(us[j], p, 0.6931471805599453f * s);  // s carries A log2(e)
                gu[j] = fmaf(skip, gp[j], de[j] * p);
                if (GATED) yv[j] = gv[j] * fmaf(skip, us[j], yv[j]);
                dD = fmaf(gp[j], us[j], dD);
                db += live && b * kCkpt + 4 * j + q < tl.len ? gd[j] : 0.f;
            };
#define KDA_I(v) std::integral_constant<int, v>{}
#pragma unroll
            for (int r = 0; r < R; ++r) dA8[r] = 0.f;
            ahead(KDA_I(0), KDA_I(0)); ahead(KDA_I(0), KDA_I(1)); ahead(KDA_I(0), KDA_I(2)); ahead(KDA_I(0), KDA_I(3));
            // The second group where the tile reaches it.  The branch also ends the basic block, which keeps the
            // scheduler from mixing the groups and paying in registers.
            if constexpr (J > 1) {
                if (b * kCkpt + 4 < tl.len) {
                    ahead(KDA_I(1), KDA_I(0)); ahead(KDA_I(1), KDA_I(1)); ahead(KDA_I(1), KDA_I(2)); ahead(KDA_I(1), KDA_I(3));
                    back(KDA_I(1), KDA_I(3)); back(KDA_I(1), KDA_I(2)); back(KDA_I(1), KDA_I(1)); back(KDA_I(1), KDA_I(0));
                }
            }
            back(KDA_I(0), KDA_I(3)); back(KDA_I(0), KDA_I(2)); back(KDA_I(0), KDA_I(1)); back(KDA_I(0), KDA_I(0));
#undef KDA_I
#pragma unroll
            for (int r = 0; r < R; ++r) dA[r] += dA8[r];
            ou.put(b * kCkpt, tl.len, q, live, P.du.bf16, gu);
            od.put(b * kCkpt, tl.len, q, live, P.ddt.bf16, gd);
            if (GATED) oz.put(b * kCkpt, tl.len, q, live, P.dz.bf16, yv);
            if (b > 0) stage(b - 1, buf ^ 1);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kSt; ++i) {
                const int e = i * 256 + threadIdx.x, t = e / (2 * NS), n = e % (2 * NS), half = n / NS, s = n % NS;
                if (b * kCkpt + t < tl.len && s < P.ds)
                    (pBC + static_cast<int64_t>(b) * kCkpt * 2 * P.ds)[static_cast<uint32_t>((t * 2 + half) * P.ds + s)] =
                        (sR[buf][0][t][n] + sR[buf][1][t][n]) + (sR[buf][2][t][n] + sR[buf][3][t][n]);
            }
        }
    }
    dD = quad_sum(dD);
    db = quad_sum(db);
    if (!live) return;
    float *par = W.par + slot * P.dim * (P.ds + 2);
    if (q == 0) {
        par[static_cast<int64_t>(P.dim) * P.ds + ch] = dD;
        par[static_cast<int64_t>(P.dim) * (P.ds + 1) + ch] = db;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (q * R + r >= P.ds) continue;
        par[static_cast<int64_t>(ch) * P.ds + q * R + r] = dA[r];
        if (P.dh0 && tl.valid && tl.k == 0)
            P.dh0[(static_cast<int64_t>(tl.n) * P.dim + ch) * P.ds + q * R + r] = G[r];
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

bool tiled(const SeqTiles &s) { return s.T > s.L; }

BwdSpace space(float *ws, const SeqTiles &seq, int dim, int ds) {
    const int64_t slots = seq.slots(), rows = seq.rows(), groups = (dim + 63) / 64;
    const int64_t padded = ds <= 16 ? 16 : ds <= 32 ? 32 : 64, blocks = rows / (ds <= 16 ? 8 : 4) + slots + 1;
    BwdSpace w{};
    int64_t at = 0;
    auto take = [&](int64_t n) {
        float *p = ws ? ws + at : nullptr;
        at += (n + 3) & ~int64_t{3};
        return p;
    };
    w.ck = take(blocks * dim * padded);
    if (tiled(seq)) {
        w.cum = take(blocks * dim);
        w.H = take(slots * dim * ds);
        w.G = take(slots * dim * ds);
        w.sum = take(slots * dim);
    }
    w.par = take(slots * dim * (ds + 2));
    w.pBC = take(groups * rows * 2 * ds);
    w.bytes = at * 4;
    return w;
}

template <int R, bool InBf16, bool GATED>
void launch_grad(const ScanBwdLaunch &P, const BwdSpace &w) {
    const int64_t slots = P.seq.slots();
    const int groups = (P.dim + 63) / 64;
    const unsigned grid = static_cast<unsigned>(slots * groups);
    if (tiled(P.seq)) {
        scan_states_kernel<R, InBf16, true, GATED><<<grid, 256, 0, P.stream>>>(P, w);
        const int64_t states = static_cast<int64_t>(P.dim) * P.ds;
        scan_bwd_combine_kernel<<<dim3(static_cast<unsigned>((states + 255) / 256), P.seq.N), 256, 0, P.stream>>>(P, w);
        scan_grad_kernel<R, InBf16, true, GATED><<<grid, 256, 0, P.stream>>>(P, w);
    } else {
        scan_states_kernel<R, InBf16, false, false><<<grid, 256, 0, P.stream>>>(P, w);
        scan_grad_kernel<R, InBf16, false, GATED><<<grid, 256, 0, P.stream>>>(P, w);
    }
    const int64_t n = P.seq.rows() * 2 * P.ds;
    if (n > 0) scan_bc_sum_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, P.stream>>>(P, w.pBC, groups);
}

template <int R, bool InBf16>
void launch_gated(const ScanBwdLaunch &P, const BwdSpace &w) {
    if (P.z.p) launch_grad<R, InBf16, true>(P, w);
    else launch_grad<R, InBf16, false>(P, w);
}

template <bool InBf16>
void launch_any(const ScanBwdLaunch &P, const BwdSpace &w) {
    if (P.ds <= 16) launch_gated<4, InBf16>(P, w);
    else if (P.ds <= 32) launch_gated<8, InBf16>(P, w);
    else launch_gated<16, InBf16>(P, w);
}

}  // namespace

// Whole sequences where they give two waves per SIMD by themselves, else tiles.  On MI355X, bf16: 16 x 1,024 x 4,096
// (1,024 workgroups) 1,207 us whole and 1,285 tiled, 8 x 1,024 x 4,096 (512) 696 and 693, 12 x 1,024 x 2,048 (384) 670
// and 520.  Packed ones go in tiles, as in the forward pass (8,000 tokens beside 80 of 100, 4,096 channels: 1,283 us
// against 3,781 whole; 16 x 1,024 x 4,096 1,285 against 1,213).
SeqTiles scan_bwd_tiles(const int32_t *cu, int N, int T, int dim, int ds) {
    SeqTiles s{cu, N, T, T > 0 ? T : 1};
    const int64_t groups = (dim + 63) / 64;
    if (cu || N * groups < 512) tile_for(s, groups);
    return s;
}

int64_t scan_bwd_threads(const SeqTiles &seq, int dim, int ds) {
    const int64_t walks = seq.slots() * ((dim + 63) / 64) * 256, sums = (seq.rows() * 2 * ds + 255) / 256 * 256;
    const int64_t params = column_sum_threads(static_cast<int64_t>(dim) * (ds + 2));
    return walks > sums ? walks > params ? walks : params : sums > params ? sums : params;
}

size_t scan_bwd_workspace_bytes(const SeqTiles &seq, int dim, int ds) { return space(nullptr, seq, dim, ds).bytes; }

hipError_t launch_scan_bwd(const ScanBwdLaunch &P) {
    const BwdSpace w = space(P.ws, P.seq, P.dim, P.ds);
    if (P.seq.N > 0) {
        if (P.u.bf16) launch_any<true>(P, w);
        else launch_any<false>(P, w);
    }
    const int64_t states = static_cast<int64_t>(P.dim) * P.ds;
    launch_column_sum(w.par, states + 2 * P.dim, P.seq.N > 0 ? static_cast<int>(P.seq.slots()) : 0,
                      {{P.dA, P.dD, P.ddt_bias}, {states, P.dim, P.dim}}, P.stream);
    return hipGetLastError();
}

}  // namespace kda
