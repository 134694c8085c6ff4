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
#include "kda_layer.h"

namespace kda {

namespace {

constexpr int kScanBlock = 16;     // tokens per LDS block
constexpr int kScanChannels = 64;  // channels per workgroup of 256

template <bool InBf16>
struct Raw {
    using T = typename Elem<InBf16>::T;
    static __device__ __forceinline__ float f(T x) { return Elem<InBf16>::load(&x, 0); }
};

template <int R, bool InBf16>
__global__ void __launch_bounds__(256) scan_kernel(ScanFwdLaunch P) {
    using E = typename Raw<InBf16>::T;
    constexpr int NS = 4 * R, kStage = kScanBlock * NS / 256;  // staged values per thread
    static_assert(kScanBlock * NS % 256 == 0 || NS < 16, "staging");
    constexpr int kSt = kStage > 0 ? kStage : 1;
    __shared__ __attribute__((aligned(16))) float sB[2][kScanBlock][NS], sC[2][kScanBlock][NS];

    const int groups = (P.dim + kScanChannels - 1) / kScanChannels;
    const int64_t slot = blockIdx.x / groups;
    const Tile tl = find_tile(P.seq, slot);
    if (!tl.valid) return;
    const int lane = threadIdx.x & 63, q = lane & 3;
    const int ch = static_cast<int>(blockIdx.x % groups) * kScanChannels + (threadIdx.x >> 2);
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
    const float skip = P.D ? P.D[chc] : 0.f, bias = P.dt_bias ? P.dt_bias[chc] : 0.f;

    const E *u = static_cast<const E *>(P.u.p), *dt = static_cast<const E *>(P.dt.p);
    const E *z = static_cast<const E *>(P.z.p);
    const E *Bp = static_cast<const E *>(P.B.p), *Cp = static_cast<const E *>(P.C.p);
    E ru[4], rdt[4], rz[4], rB[kSt], rC[kSt];
    auto fetch = [&](int t0) {  // the block at t0 of the tile, into registers
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = t0 + 4 * j + q;
            const int64_t row = tl.begin + (t < tl.len ? t : tl.len - 1);
            rdt[j] = dt[row * P.dt.stride + chc];
            ru[j] = u[row * P.u.stride + chc];
            if (z) rz[j] = z[row * P.z.stride + chc];
        }
#pragma unroll
        for (int i = 0; i < kSt; ++i) {
            const int e = i * 256 + threadIdx.x, t = t0 + e / NS, n = e % NS;
            rB[i] = rC[i] = 0;
            if (e < kScanBlock * NS && t < tl.len && n < P.ds) {
                rB[i] = Bp[(tl.begin + t) * P.B.stride + n];
                rC[i] = Cp[(tl.begin + t) * P.C.stride + n];
            }
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kSt; ++i) {
            const int e = i * 256 + threadIdx.x;
            if (e < kScanBlock * NS) {
                (&sB[buf][0][0])[e] = Raw<InBf16>::f(rB[i]);
                (&sC[buf][0][0])[e] = Raw<InBf16>::f(rC[i]);
            }
        }
    };

    if (tl.len > 0) {
        fetch(0);
        stage(0);
        __syncthreads();
    }
    for (int t0 = 0, buf = 0; t0 < tl.len; t0 += kScanBlock, buf ^= 1) {
        float de[4], xs[4], us[4], zs[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = t0 + 4 * j + q < tl.len;
            const float d = Raw<InBf16>::f(rdt[j]) + bias;
            us[j] = in ? Raw<InBf16>::f(ru[j]) : 0.f;
            de[j] = in ? (P.softplus ? softplus_f(d) : d) : 0.f;
            xs[j] = de[j] * us[j];
            zs[j] = z ? Raw<InBf16>::f(rz[j]) : 0.f;
        }
        const bool more = t0 + kScanBlock < tl.len;
        if (more) fetch(t0 + kScanBlock);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (t0 + 4 * j >= tl.len) break;
            float yp[4];
            auto token = [&](float dl, float xl, int i) {
                const float *bt = &sB[buf][4 * j + i][q * R], *ct = &sC[buf][4 * j + i][q * R];
                float acc = 0.f;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    h[r] = fmaf(__builtin_amdgcn_exp2f(dl * A2[r]), h[r], xl * bt[r]);
                    acc = fmaf(ct[r], h[r], acc);
                }
                yp[i] = acc;
            };
            token(quad_bcast<0>(de[j]), quad_bcast<0>(xs[j]), 0);
            token(quad_bcast<1>(de[j]), quad_bcast<1>(xs[j]), 1);
            token(quad_bcast<2>(de[j]), quad_bcast<2>(xs[j]), 2);
            token(quad_bcast<3>(de[j]), quad_bcast<3>(xs[j]), 3);
            float y = fmaf(skip, us[j], quad_transpose_sum(yp[0], yp[1], yp[2], yp[3], q));
            if (z) y *= zs[j] * sigmoid_f(zs[j]);
            const int t = t0 + 4 * j + q;
            if (live && t < tl.len) P.y.put(tl.begin + t, ch, y);
        }
        if (more) stage(buf ^ 1);
        __syncthreads();
    }
    if (P.hT && live && tl.last()) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (q * R + r < P.ds) P.hT[sbase + r] = h[r];
    }
}

// One token per sequence: the state streams through once, read and written by the lane that holds it (16
// bytes per lane where ds = 4 R), and there is nothing else to stage: each quad lane reads its own B and C.
template <int R, bool InBf16>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanFwdLaunch P) {
    using E = typename Raw<InBf16>::T;
    const int groups = (P.dim + kScanChannels - 1) / kScanChannels;
    const int n = blockIdx.x / groups, q = threadIdx.x & 3;
    const int ch = static_cast<int>(blockIdx.x % groups) * kScanChannels + (threadIdx.x >> 2);
    if (ch >= P.dim) return;
    const int64_t sbase = (static_cast<int64_t>(n) * P.dim + ch) * P.ds + q * R;
    const int64_t abase = static_cast<int64_t>(ch) * P.ds + q * R;
    const E *Bp = static_cast<const E *>(P.B.p) + n * P.B.stride + q * R;
    const E *Cp = static_cast<const E *>(P.C.p) + n * P.C.stride + q * R;
    const float u = P.u.get(n, ch);
    float dl = P.dt.get(n, ch) + (P.dt_bias ? P.dt_bias[ch] : 0.f);
    if (P.softplus) dl = softplus_f(dl);
    const float xl = dl * u;
    float acc = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (q * R + r >= P.ds) break;
        const float h = fmaf(__builtin_amdgcn_exp2f(dl * (kLog2e * P.A[abase + r])), P.h0 ? P.h0[sbase + r] : 0.f,
                             xl * Raw<InBf16>::f(Bp[r]));
        P.hT[sbase + r] = h;
        acc = fmaf(Raw<InBf16>::f(Cp[r]), h, acc);
    }
    acc = quad_sum(acc);
    if (q == 0) {
        float y = fmaf(P.D ? P.D[ch] : 0.f, u, acc);
        if (P.z.p) {
            const float zz = P.z.get(n, ch);
            y *= zz * sigmoid_f(zz);
        }
        P.y.put(n, ch, y);
    }
}

}  // namespace

SeqTiles scan_fwd_tiles(const int32_t *cu, int N, int T, int dim, int ds) {
    SeqTiles s{cu, N, T, T > 0 ? T : 1};
    return s;
}

size_t scan_fwd_workspace_bytes(const SeqTiles &seq, int dim, int ds) { return 0; }

template <bool InBf16>
static void launch_main(const ScanFwdLaunch &P, unsigned grid) {
    if (P.ds <= 16) scan_kernel<4, InBf16><<<grid, 256, 0, P.stream>>>(P);
    else if (P.ds <= 32) scan_kernel<8, InBf16><<<grid, 256, 0, P.stream>>>(P);
    else scan_kernel<16, InBf16><<<grid, 256, 0, P.stream>>>(P);
}

hipError_t launch_scan_fwd(const ScanFwdLaunch &P) {
    const int groups = (P.dim + kScanChannels - 1) / kScanChannels;
    const unsigned grid = static_cast<unsigned>(P.seq.slots() * groups);
    if (grid == 0) return hipSuccess;
    if (P.u.bf16) launch_main<true>(P, grid);
    else launch_main<false>(P, grid);
    return hipGetLastError();
}

template <bool InBf16>
static void launch_step(const ScanFwdLaunch &P, unsigned grid) {
    if (P.ds <= 16) scan_step_kernel<4, InBf16><<<grid, 256, 0, P.stream>>>(P);
    else if (P.ds <= 32) scan_step_kernel<8, InBf16><<<grid, 256, 0, P.stream>>>(P);
    else scan_step_kernel<16, InBf16><<<grid, 256, 0, P.stream>>>(P);
}

hipError_t launch_scan_step(const ScanFwdLaunch &P) {
    const int groups = (P.dim + kScanChannels - 1) / kScanChannels;
    const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(P.seq.N) * groups);
    if (P.u.bf16) launch_step<true>(P, grid);
    else launch_step<false>(P, grid);
    return hipGetLastError();
}

}  // namespace kda
