// kda_selective_scan.hip - the selective state space scan, forward, for gfx950.
//
//     h_t = exp(delta_t A) h_{t-1} + delta_t u_t B_t,   y_t = (C_t . h_t + D u_t) silu(z_t)
//
// per channel d and state n, all in fp32.  The decay differs per (t, d, n), so nothing here is a matrix
// product: the bound is the vector unit, per (t, d, n) one exp2, two multiplications and two FMAs, about 6
// issue slots with exp2 at half rate, against 8 bytes per (t, d) of bf16 u, dt, z and y.
//
// Work split: four lanes hold one channel, R = ds / 4 states each; a wave holds 16 channels, a workgroup 64.
// Tokens go in groups of four: lane q of a quad loads token q's dt, u and z and computes its step size, gate
// and output, so that none of the per-channel work is done four times; DPP moves within the quad hand the
// values round and sum C . h.  B and C, the same for every channel, are widened to fp32 once per workgroup
// and block of 16 tokens in LDS (double buffered), and read as one 16-byte access per quad lane and token.
// Inputs of the next block are in flight while one is computed.  Tokens past a tile's end count as
// delta = 0, u = 0: decay 1, nothing added.
//
// Sequences too few to fill the chip are cut into tiles: a local pass walks every tile but a sequence's last
// from a zero state, a combine chains what they reach (a tile's decay needs only its sum of delta), and the
// output pass walks every tile from its true state.
#include "kda_layer.h"

namespace kda {

namespace {

constexpr int LPC = 4;             // lanes per channel
constexpr int kScanChannels = 64;  // channels per workgroup of 256

template <bool InBf16>
struct Raw {
    using T = typename Elem<InBf16>::T;
    static __device__ __forceinline__ float f(T x) { return Elem<InBf16>::load(&x, 0); }
};

// What a tiled scan keeps between its passes, in floats.
struct FwdSpace {
    float *H;    // [slot][dim][ds] the local pass: state a tile reaches from zero; after the combine: state it starts from
    float *sum;  // [slot][dim] sum of delta over the tile: its decay is exp(A sum)
    int64_t bytes;
};
__host__ __device__ inline FwdSpace fwd_space(float *ws, const SeqTiles &seq, int dim, int ds) {
    const int64_t slots = seq.slots();
    return {ws, ws ? ws + slots * dim * ds : nullptr, slots * dim * (ds + 1) * 4};
}

enum { kOutputs, kLocal };

// LPC lanes per channel with R states each; tokens in groups of LPC, one per lane.  Four give the most waves: two and
// one were slower at every size when they were compared (16,384 x 4,096: 536 and 695 us against 497, which are 465 by now).
template <int MODE, int R, bool InBf16, bool GATED>
__global__ void __launch_bounds__(256) scan_kernel(ScanFwdLaunch P) {
    using E = typename Raw<InBf16>::T;
    constexpr int NS = LPC * R, kTok = 16, J = kTok / LPC;  // tokens per block, per lane of it
    constexpr int kSt = kTok * NS / 256;                    // staged values per thread
    __shared__ __attribute__((aligned(16))) float sB[2][kTok][NS], sC[MODE == kLocal ? 1 : 2][kTok][NS];

    const int groups = (P.dim + kScanChannels - 1) / kScanChannels;
    const int64_t slot = blockIdx.x / groups;
    const Tile tl = find_tile(P.seq, slot);
    if (!tl.valid || (MODE == kLocal && tl.last())) return;  // nothing follows a last tile
    const int q = threadIdx.x % LPC;
    const int ch = static_cast<int>(blockIdx.x % groups) * kScanChannels + threadIdx.x / LPC;
    const bool live = ch < P.dim;
    const int chc = live ? ch : P.dim - 1;
    const FwdSpace W = fwd_space(P.ws, P.seq, P.dim, P.ds);

    float A2[R], h[R];
    const int64_t sbase = (static_cast<int64_t>(tl.n) * P.dim + chc) * P.ds + q * R;
    const int64_t wbase = (slot * P.dim + chc) * P.ds + q * R;
    // A sequence's only tile starts from its initial state; of several, all start from what the combine left
    // (the first too: the last may be writing the final state in the initial one's place).
    const float *from = MODE == kLocal ? nullptr : tl.count > 1 ? W.H + wbase : P.h0 ? P.h0 + sbase : nullptr;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool in = q * R + r < P.ds;
        A2[r] = in ? kLog2e * P.A[static_cast<int64_t>(chc) * P.ds + q * R + r] : 0.f;
        h[r] = in && from ? from[r] : 0.f;
    }
    const float skip = P.D ? P.D[chc] : 0.f, bias = P.dt_bias ? P.dt_bias[chc] : 0.f;

    const Column cu(P.u, tl.begin, chc), cd(P.dt, tl.begin, chc), cz(P.z, tl.begin, chc), cy(P.y, tl.begin, chc);
    const E *Bp = static_cast<const E *>(P.B.p) + tl.begin * P.B.stride;
    const E *Cp = static_cast<const E *>(P.C.p) + tl.begin * P.C.stride;
    E ru[J], rdt[J], rz[J], rB[kSt], rC[kSt];
    auto fetch = [&](int t0) {  // the block at t0 of the tile, into registers
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const Group g(t0 + LPC * j, tl.len, q);
            rdt[j] = cd.get<E>(g);
            ru[j] = cu.get<E>(g);
            if (GATED) rz[j] = cz.get<E>(g);
        }
#pragma unroll
        for (int i = 0; i < kSt; ++i) {
            const int e = i * 256 + threadIdx.x, n = e % NS < P.ds ? e % NS : P.ds - 1;
            const int left = tl.len - 1 - t0, t = e / NS < left ? e / NS : left;
            rB[i] = (Bp + t0 * P.B.stride)[static_cast<uint32_t>(t) * static_cast<uint32_t>(P.B.stride) + n];
            if (MODE == kOutputs)
                rC[i] = (Cp + t0 * P.C.stride)[static_cast<uint32_t>(t) * static_cast<uint32_t>(P.C.stride) + n];
        }
    };
    auto stage = [&](int t0, int buf) {
#pragma unroll
        for (int i = 0; i < kSt; ++i) {
            const int e = i * 256 + threadIdx.x;
            const bool in = t0 + e / NS < tl.len && e % NS < P.ds;
            (&sB[buf][0][0])[e] = in ? Raw<InBf16>::f(rB[i]) : 0.f;
            if (MODE == kOutputs) (&sC[buf][0][0])[e] = in ? Raw<InBf16>::f(rC[i]) : 0.f;
        }
    };

    float total = 0.f;  // of delta over this lane's tokens
    if (tl.len > 0) {
        fetch(0);
        stage(0, 0);
        __syncthreads();
    }
    for (int t0 = 0, buf = 0; t0 < tl.len; t0 += kTok, buf ^= 1) {
        float de[J], xs[J], us[J], y[J] = {};
#pragma unroll
        for (int j = 0; j < J; ++j) de[j] = Raw<InBf16>::f(rdt[j]) + bias;
        if (P.softplus) {
#pragma unroll
            for (int j = 0; j < J; ++j) de[j] = softplus_f(de[j]);
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const bool in = t0 + LPC * j + q < tl.len;
            de[j] = in ? de[j] : 0.f;
            us[j] = in ? Raw<InBf16>::f(ru[j]) : 0.f;
            xs[j] = de[j] * us[j];
            if (GATED) {
                const float z = Raw<InBf16>::f(rz[j]);
                y[j] = z * sigmoid_f(z);
            }
            if (MODE == kLocal) total += de[j];
        }
        const bool more = t0 + kTok < tl.len;
        if (more) fetch(t0 + kTok);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            // Also ends the basic block: across it the scheduler pulls every token's lane moves and loads to the
            // front of the unrolled block and pays in registers (134 against 56 in the local pass).
            if (t0 + LPC * j >= tl.len) break;
            float yp[LPC];
            auto token = [&](float dl, float xl, int i) {
                const float *bt = &sB[buf][LPC * j + i][q * R], *ct = &sC[MODE == kLocal ? 0 : buf][LPC * j + i][q * R];
                float acc = 0.f;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    h[r] = fmaf(__builtin_amdgcn_exp2f(dl * A2[r]), h[r], xl * bt[r]);
                    if (MODE == kOutputs) acc = fmaf(ct[r], h[r], acc);
                }
                yp[i] = acc;
            };
            token(lane_bcast<0>(de[j]), lane_bcast<0>(xs[j]), 0);
            token(lane_bcast<1>(de[j]), lane_bcast<1>(xs[j]), 1);
            token(lane_bcast<2>(de[j]), lane_bcast<2>(xs[j]), 2);
            token(lane_bcast<3>(de[j]), lane_bcast<3>(xs[j]), 3);
            if (MODE == kOutputs) {
                const float sum = fmaf(skip, us[j], transpose_sum(yp, q));
                y[j] = GATED ? sum * y[j] : sum;
            }
        }
        if (MODE == kOutputs) cy.put(t0, tl.len, q, live, P.y.bf16, y);
        if (more) stage(t0 + kTok, buf ^ 1);
        __syncthreads();
    }
    if (MODE == kLocal) {
        total = quad_sum(total);
        if (live) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (q * R + r < P.ds) W.H[wbase + r] = h[r];
            if (q == 0) W.sum[slot * P.dim + ch] = total;
        }
    } else if (P.hT && live && tl.last()) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (q * R + r < P.ds) P.hT[sbase + r] = h[r];
    }
}

// Chains the tiles of every sequence that has several: a tile starts from the state its predecessor leaves,
// exp(A sum) times what that started from plus what it reached from zero.
__global__ void __launch_bounds__(256) scan_combine_kernel(ScanFwdLaunch P) {
    const int n = blockIdx.y;
    const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, states = static_cast<int64_t>(P.dim) * P.ds;
    int64_t start;
    int len;
    P.seq.sequence(n, start, len);
    const int count = P.seq.tiles(len);
    if (e >= states || count <= 1) return;
    const FwdSpace W = fwd_space(P.ws, P.seq, P.dim, P.ds);
    const int64_t first = P.seq.first_slot(n, start);
    const int ch = static_cast<int>(e / P.ds);
    const float A2 = kLog2e * P.A[e];
    float carry = P.h0 ? P.h0[n * states + e] : 0.f;
    float *H = W.H + first * states + e;
    const float *sum = W.sum + first * P.dim + ch;
    constexpr int U = 8;  // tiles in flight: their loads do not wait for the chain
    for (int k = 0; k < count; k += U) {
        float h[U], d[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const bool in = k + i + 1 < count;  // the last tile has no successor
            h[i] = in ? H[(k + i) * states] : 0.f;
            d[i] = in ? sum[static_cast<int64_t>(k + i) * P.dim] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (k + i >= count) break;
            H[(k + i) * states] = carry;
            carry = fmaf(__builtin_amdgcn_exp2f(A2 * d[i]), carry, h[i]);
        }
    }
}

// R consecutive states of a channel; `wide`: the rows are exactly 4 R states, read 16 bytes at a time.
template <int R>
__device__ __forceinline__ void load_states(const float *p, bool wide, int left, float (&x)[R]) {
    if (wide) {
#pragma unroll
        for (int r = 0; r < R; r += 4) {
            const float4 v = load_stream(p + r);
            x[r] = v.x; x[r + 1] = v.y; x[r + 2] = v.z; x[r + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = r < left ? p[r] : 0.f;
    }
}

// One token per sequence: bound by the state, which streams through once, 16 bytes per lane where a row is 4 R
// states.  A workgroup takes its 64 channels through SEQS sequences, with A, D and the bias read once and the
// sequences' states in flight together: 256 sequences of 4,096 channels take 38 us with two (3.7 TB/s), 44 with
// one or four, 48 with two and without the non-temporal hint.
template <int R, bool InBf16, int SEQS>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanFwdLaunch P) {
    using E = typename Raw<InBf16>::T;
    const int groups = (P.dim + kScanChannels - 1) / kScanChannels;
    const int n0 = blockIdx.x / groups * SEQS, q = threadIdx.x & 3;
    const int ch = static_cast<int>(blockIdx.x % groups) * kScanChannels + (threadIdx.x >> 2);
    if (ch >= P.dim) return;
    const bool wide = P.ds == 4 * R;
    const int left = P.ds - q * R;
    float A2[R], h[SEQS][R], b[SEQS][R], c[SEQS][R], dl[SEQS], u[SEQS], z[SEQS];
    load_states<R>(P.A + static_cast<int64_t>(ch) * P.ds + q * R, wide, left, A2);
#pragma unroll
    for (int i = 0; i < SEQS; ++i) {
        const int n = n0 + i < P.seq.N ? n0 + i : P.seq.N - 1;
        const int64_t sbase = (static_cast<int64_t>(n) * P.dim + ch) * P.ds + q * R;
        if (P.h0) {
            load_states<R>(P.h0 + sbase, wide, left, h[i]);
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) h[i][r] = 0.f;
        }
        const E *Bp = static_cast<const E *>(P.B.p) + n * P.B.stride + q * R;
        const E *Cp = static_cast<const E *>(P.C.p) + n * P.C.stride + q * R;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            b[i][r] = r < left ? Raw<InBf16>::f(Bp[r]) : 0.f;
            c[i][r] = r < left ? Raw<InBf16>::f(Cp[r]) : 0.f;
        }
        u[i] = Raw<InBf16>::f(static_cast<const E *>(P.u.p)[n * P.u.stride + ch]);
        dl[i] = Raw<InBf16>::f(static_cast<const E *>(P.dt.p)[n * P.dt.stride + ch]);
        if (P.z.p) z[i] = Raw<InBf16>::f(static_cast<const E *>(P.z.p)[n * P.z.stride + ch]);
    }
    const float skip = P.D ? P.D[ch] : 0.f, bias = P.dt_bias ? P.dt_bias[ch] : 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) A2[r] *= kLog2e;
#pragma unroll
    for (int i = 0; i < SEQS; ++i) {
        if (n0 + i >= P.seq.N) break;
        const int64_t sbase = (static_cast<int64_t>(n0 + i) * P.dim + ch) * P.ds + q * R;
        const float d = dl[i] + bias, delta = P.softplus ? softplus_f(d) : d, xl = delta * u[i];
        float acc = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            h[i][r] = fmaf(__builtin_amdgcn_exp2f(delta * A2[r]), h[i][r], xl * b[i][r]);
            acc = fmaf(c[i][r], h[i][r], acc);
        }
        if (wide) {
#pragma unroll
            for (int r = 0; r < R; r += 4)
                store_stream(P.hT + sbase + r, make_float4(h[i][r], h[i][r + 1], h[i][r + 2], h[i][r + 3]));
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r < left) P.hT[sbase + r] = h[i][r];
        }
        acc = quad_sum(acc);
        if (q == 0) {
            float y = fmaf(skip, u[i], acc);
            if (P.z.p) y *= z[i] * sigmoid_f(z[i]);
            P.y.put(n0 + i, ch, y);
        }
    }
}

}  // namespace

// Whole sequences where they fill the chip by themselves, one pass; else tiles, and a second pass over the inputs.
// On MI355X, bf16: 8 x 1,024 x 4,096 (512 workgroups) 187 us whole and 241 tiled, 12 x 1,024 x 2,048 (384) 184
// and 186, 8 x 2,048 x 2,048 (256) 274 and 249, 2 x 4,096 x 4,096 (128) 539 and 248.  Packed sequences go in tiles:
// their lengths are on the device, and one long one would be what the call waits for (8,000 tokens beside 80 of 100, at
// 4,096 channels: 380 us in tiles of 256, 1,074 whole).  Equal ones pay for it (16 x 2,048 x 4,096: 863 against 600).
SeqTiles scan_fwd_tiles(const int32_t *cu, int N, int T, int dim, int ds) {
    SeqTiles s{cu, N, T, T > 0 ? T : 1};
    const int64_t groups = (dim + kScanChannels - 1) / kScanChannels;
    if (cu || N * groups < 384) tile_for(s, groups);
    return s;
}

static bool tiled(const SeqTiles &s) { return s.T > s.L; }

size_t scan_fwd_workspace_bytes(const SeqTiles &seq, int dim, int ds) {
    return tiled(seq) ? fwd_space(nullptr, seq, dim, ds).bytes : 0;
}

template <int R, bool InBf16>
static void launch_passes(const ScanFwdLaunch &P) {
    const unsigned grid = static_cast<unsigned>(P.seq.slots() * ((P.dim + kScanChannels - 1) / kScanChannels));
    if (tiled(P.seq)) {
        scan_kernel<kLocal, R, InBf16, false><<<grid, 256, 0, P.stream>>>(P);
        const int64_t states = static_cast<int64_t>(P.dim) * P.ds;
        scan_combine_kernel<<<dim3(static_cast<unsigned>((states + 255) / 256), P.seq.N), 256, 0, P.stream>>>(P);
    }
    if (P.z.p) scan_kernel<kOutputs, R, InBf16, true><<<grid, 256, 0, P.stream>>>(P);
    else scan_kernel<kOutputs, R, InBf16, false><<<grid, 256, 0, P.stream>>>(P);
}

template <bool InBf16>
static void launch_main(const ScanFwdLaunch &P) {
    if (P.ds <= 16) launch_passes<4, InBf16>(P);
    else if (P.ds <= 32) launch_passes<8, InBf16>(P);
    else launch_passes<16, InBf16>(P);
}

hipError_t launch_scan_fwd(const ScanFwdLaunch &P) {
    if (P.u.bf16) launch_main<true>(P);
    else launch_main<false>(P);
    return hipGetLastError();
}

template <bool InBf16, int SEQS>
static void launch_step(const ScanFwdLaunch &P) {
    const int64_t groups = (P.dim + kScanChannels - 1) / kScanChannels;
    const unsigned grid = static_cast<unsigned>((P.seq.N + SEQS - 1) / SEQS * groups);
    if (P.ds <= 16) scan_step_kernel<4, InBf16, SEQS><<<grid, 256, 0, P.stream>>>(P);
    else if (P.ds <= 32) scan_step_kernel<8, InBf16, SEQS><<<grid, 256, 0, P.stream>>>(P);
    else scan_step_kernel<16, InBf16, SEQS><<<grid, 256, 0, P.stream>>>(P);
}

hipError_t launch_scan_step(const ScanFwdLaunch &P) {
    // two sequences per workgroup once that leaves enough workgroups to fill the chip
    const int64_t groups = (P.dim + kScanChannels - 1) / kScanChannels;
    const bool many = P.seq.N * groups >= 4096;
    if (P.u.bf16) many ? launch_step<true, 2>(P) : launch_step<true, 1>(P);
    else many ? launch_step<false, 2>(P) : launch_step<false, 1>(P);
    return hipGetLastError();
}

}  // namespace kda
