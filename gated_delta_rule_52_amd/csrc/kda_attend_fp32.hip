// kda_attend_fp32.hip - latent attention over expanded keys and values in fp32, forward and gradients (the formulas stand in
// kda_attend.hip and kda_attend_bwd.hip).
//
// The fp32 matrix unit bounds these kernels: a 32 x 32 tile of pairs takes a wave 10,000 cycles forward and 20,000 backward at
// the full head sizes, its operands 40 to 80 KiB.  So the operands come straight from the caches, without LDS, a few steps
// ahead of their products; what counts is that all waves have work.  A workgroup has 32 queries (or keys), and its waves,
// four of them or eight where there are few workgroups (`few`), share out the tiles of keys (or queries) that they meet and add up their
// results through LDS at the end, in the waves' order.  (With tiles in LDS, 64 rows to a workgroup of four waves, 256 rows of 8 heads
// took 61 us forward, 1,024 of 16 223, 4,096 of 16 1,326, and gradients of the last 3,506; as they are they take 21, 67, 730 and 3,330.)  At
// 4,096 rows of 16 heads that is 118 TFLOP/s forward and 67 for the gradients (93 with the products that are formed twice) of the
// unit's 157: the loads of operands that no product hides.
#include "kda_latent.h"

namespace kda {
namespace {

using namespace la;
typedef Mx<float> M;

constexpr int kAhead = 4;  // steps between an operand's load and its use

__device__ __forceinline__ void clear(f16 &x) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
}
// Row i of a lane's half of a 32 x 32 result, and the step of eight rows that it is in.
__device__ __forceinline__ int result_row(int i, int lane) { return 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3); }

// Rows of a tile in memory, as a buffer: rows behind the sequence read as zeros, and an operand costs at most one addition
// beside its load.  What lies behind a head's columns may be read but is not used.
struct TileRows {
    rsrc_t r;
    uint32_t stride;  // bytes
    __device__ __forceinline__ TileRows(const float *p, int64_t row0, int64_t step, int rows, int width)
        : r(rows_buffer(p + row0 * step, step, min(32, rows - static_cast<int>(row0)), width)), stride(static_cast<uint32_t>(step) * 4) {}
    // this lane's row, step i of eight elements
    __device__ __forceinline__ f4 row_step(int i, int lane) const {
        return __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(r, static_cast<int>((lane & 31) * stride + (lane >> 5) * 16) + 32 * i, 0, 0));
    }
    // column 32 c + lane % 32 of the rows that the lane's half has in a result's step of eight
    __device__ __forceinline__ f4 col_step(int step, int c, int lane) const {
        const int at = static_cast<int>((lane >> 5) * 4 * stride + (lane & 31) * 4);
        f4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, at + static_cast<int>((8 * step + j) * stride) + 128 * c, 0, 0));
        return v;
    }
};
// s += [A0 | A1] B, and d += A2 C where SV > 0: this lane's rows of A against operands in registers, as one run, so that the
// loads of one product hide behind the other.
template <int SN, int SR, int SV>
__device__ __forceinline__ void rows_products(f16 &s, f16 &d, const TileRows &a0, int w0, const TileRows &a1, int w1, const f4 *b,
                                              const TileRows &a2, int w2, const f4 *c, int lane) {
    pipelined<f4, SN + SR + SV, kAhead>(
        [&](int i) { return i < SN ? a0.row_step(i, lane) : i < SN + SR ? a1.row_step(i - SN, lane) : a2.row_step(i - SN - SR, lane); },
        [&](int i, f4 a) {
            if (i < SN) {
                if (8 * i < w0) s = M::mma32(a, b[i], s);
            } else if (i < SN + SR) {
                if (8 * (i - SN) < w1) s = M::mma32(a, b[i], s);
            } else if (8 * (i - SN - SR) < w2) {
                d = M::mma32(a, c[i - SN - SR], d);
            }
        });
}
__device__ __forceinline__ f4 rows_of(const f16 &b, int step) { return f4{b[4 * step], b[4 * step + 1], b[4 * step + 2], b[4 * step + 3]}; }
template <int STEPS>
__device__ __forceinline__ void load_rows(f4 *f, const float *row, int width, bool live, int lane) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) f[s] = row_operand<float>(row, s, width, live, lane);
}

// Adds up N tiles over the waves, PART at a time through LDS, and gives wave c % WAVES the sum of tile c.
template <int WAVES, int N, int PART, class Store>
__device__ __forceinline__ void join_waves(const f16 *acc, float *lds, int wave, int lane, Store store) {
#pragma unroll
    for (int first = 0; first < N; first += PART) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < PART; ++c)
            if (first + c < N) {
#pragma unroll
                for (int i = 0; i < 16; ++i) lds[((wave * PART + c) * 16 + i) * 64 + lane] = acc[first + c][i];
            }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < PART; ++c)
            if (first + c < N && (first + c) % WAVES == wave) {
                f16 x;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    x[i] = lds[(c * 16 + i) * 64 + lane];
#pragma unroll
                    for (int w = 1; w < WAVES; ++w) x[i] += lds[((w * PART + c) * 16 + i) * 64 + lane];
                }
                store(first + c, x);
            }
    }
}

template <int WAVES, int NP, int RP, int VP>
__global__ __launch_bounds__(64 * WAVES, 2) void attend_fwd_fp32_kernel(const AttendLaunch P) {
    constexpr int SN = NP / 8, SR = RP / 8, CV = VP / 32;
    __shared__ float sums[WAVES * CV * 1024];
    __shared__ float2 stats[WAVES][32];
    const Place w = place_of<true>(P, blockIdx.x);
    if (!w.valid || w.at >= w.nq) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int shift = w.nk - w.nq, q = w.at + (lane & 31);
    const bool live = q < w.nq;
    const int keys = P.causal ? max(0, min(w.nk, min(w.at + 32, w.nq) + shift)) : w.nk;
    const int limit = P.causal ? min(w.nk, q + shift + 1) : w.nk;

    f4 qf[SN + SR];
    const float *qp = head_row<float>(P.q, w.q_row + (live ? q : 0), w.h);
    load_rows<SN>(qf, qp, P.dn, live, lane);
    load_rows<SR>(qf + SN, qp + P.dn, P.dr, live, lane);
    const float *kp = head_row<float>(P.k, w.k_row, w.h), *rp = head_row<float>(P.kr, w.k_row, 0), *vp = head_row<float>(P.v, w.k_row, w.h);

    f16 acc[CV];
#pragma unroll
    for (int c = 0; c < CV; ++c) clear(acc[c]);
    float m = neg_inf(), l = 0.f;
    const float c2 = P.scale * kLog2e;
    for (int key0 = 32 * wave; key0 < keys; key0 += 32 * WAVES) {
        const int lane_ = afresh(lane);
        const TileRows K(kp, key0, P.k.stride, w.nk, P.dn), R(rp, key0, P.kr.stride, w.nk, P.dr), V(vp, key0, P.v.stride, w.nk, P.dv);
        f16 s;
        clear(s);
        rows_products<SN, SR, 0>(s, s, K, P.dn, R, P.dr, qf, V, 0, nullptr, lane_);
        float top = neg_inf();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (key0 + result_row(i, lane) >= limit) s[i] = neg_inf();
            top = fmaxf(top, s[i]);
        }
        top = halves_max(top) * c2;
        const bool move = top > m + 8.f;  // as in the bf16 kernel
        if (__any(move)) {
            const float to = move ? top : m, by = move ? exp2_f(m - to) : 1.f;
            m = to;
            l *= by;
#pragma unroll
            for (int c = 0; c < CV; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[c][i] *= by;
        }
        const float at = m == neg_inf() ? 0.f : m;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[i] = exp2_f(fmaf(s[i], c2, -at));
            l += s[i];
        }
        pipelined<f4, 4 * CV, kAhead>([&](int i) { return V.col_step(i / CV, i % CV, lane_); },
                                      [&](int i, f4 a) {
                                          if (32 * (i % CV) < P.dv) acc[i % CV] = M::mma32(a, rows_of(s, i / CV), acc[i % CV]);
                                      });
    }
    // each wave's sums relative to the largest reference point of all
    l = halves_sum(l);
    if (lane < 32) stats[wave][lane] = make_float2(m, l);
    __syncthreads();
    float top = neg_inf(), total = 0.f;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) top = fmaxf(top, stats[i][lane & 31].x);
    const float at = top == neg_inf() ? 0.f : top;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) total = fmaf(stats[i][lane & 31].y, exp2_f(stats[i][lane & 31].x - at), total);
    const float by = exp2_f(m - at), inv = total > 0.f ? 1.f / total : total == 0.f ? 0.f : total;  // NaN stays
#pragma unroll
    for (int c = 0; c < CV; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[c][i] *= by;
    const int64_t row = w.q_row + q, out = row * P.o.stride + w.h * P.o.head_stride;
    if (P.lse && live && threadIdx.x < 32) P.lse[row * P.H + w.h] = total == 0.f ? neg_inf() : (at + __log2f(total)) * kLn2;
    join_waves<WAVES, CV, CV>(acc, sums, wave, lane, [&](int c, const f16 &x) {
        if (!live) return;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int col = 32 * c + 8 * b + 4 * (lane >> 5);
            if (col < P.dv) store4(P.o.p, out + col, P.out_bf16, x[4 * b] * inv, x[4 * b + 1] * inv, x[4 * b + 2] * inv, x[4 * b + 3] * inv);
        }
    });
}

template <int WAVES, int NP, int RP, int VP>
__device__ __forceinline__ void dkv_fp32(const AttendLaunch &P, int64_t id, float *sums) {
    constexpr int SN = NP / 8, SR = RP / 8, SV = VP / 8, CN = NP / 32, CR = RP / 32, CV = VP / 32, PART = (CN + CR + CV + 1) / 2;
    const Place w = place_of<false>(P, id);
    if (!w.valid || w.at >= w.nk) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int shift = w.nk - w.nq, key = w.at + (lane & 31);
    const bool live = key < w.nk;

    f4 kf[SN + SR], vf[SV];
    const int64_t row = w.k_row + (live ? key : 0);
    load_rows<SN>(kf, head_row<float>(P.k, row, w.h), P.dn, live, lane);
    load_rows<SR>(kf + SN, head_row<float>(P.kr, row, 0), P.dr, live, lane);
    load_rows<SV>(vf, head_row<float>(P.v, row, w.h), P.dv, live, lane);
    const float *qp = head_row<float>(P.q, w.q_row, w.h), *gp = head_row<float>(P.go, w.q_row, w.h);
    const float *lp = P.lse + w.q_row * P.H + w.h, *ep = P.delta + w.q_row * P.H + w.h;

    f16 d[CN + CR + CV];  // dk, its shared part, dv
#pragma unroll
    for (int c = 0; c < CN + CR + CV; ++c) clear(d[c]);
    const float c2 = P.scale * kLog2e;
    const int first = P.causal ? max(0, w.at - shift) / 32 : 0;  // the tile of the first query that sees the first key
    for (int q0 = 32 * (first + wave); q0 < w.nq; q0 += 32 * WAVES) {
        const int lane_ = afresh(lane);
        const TileRows Q(qp, q0, P.q.stride, w.nq, P.dn), R(qp + P.dn, q0, P.q.stride, w.nq, P.dr), G(gp, q0, P.go.stride, w.nq, P.dv);
        f16 s, dp;
        clear(s);
        clear(dp);
        rows_products<SN, SR, SV>(s, dp, Q, P.dn, R, P.dr, kf, G, P.dv, vf, lane_);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int at = q0 + result_row(i, lane);
            const int64_t held = min(at, w.nq - 1) * static_cast<int64_t>(P.H);
            float p = exp2_f(fmaf(s[i], c2, -lp[held] * kLog2e));
            if (at >= w.nq || (P.causal && at + shift < key)) p = 0.f;
            s[i] = p;
            dp[i] = p * (dp[i] - ep[held]);
        }
        constexpr int C = CN + CR + CV;
        pipelined<f4, 4 * C, kAhead>(
            [&](int i) {
                const int k = i / C, c = i % C;
                return c < CN ? Q.col_step(k, c, lane_) : c < CN + CR ? R.col_step(k, c - CN, lane_) : G.col_step(k, c - CN - CR, lane_);
            },
            [&](int i, f4 a) {
                const int k = i / C, c = i % C;
                if (c < CN + CR ? c < CN ? 32 * c < P.dn : 32 * (c - CN) < P.dr : 32 * (c - CN - CR) < P.dv)
                    d[c] = M::mma32(a, rows_of(c < CN + CR ? dp : s, k), d[c]);
            });
    }
    const int64_t dk_at = row * P.dk.stride + w.h * P.dk.head_stride, dv_at = row * P.dvg.stride + w.h * P.dvg.head_stride;
    const int64_t part = (row * P.H + w.h) * P.dr;
    join_waves<WAVES, CN + CR + CV, PART>(d, sums, wave, lane, [&](int c, const f16 &x) {
        if (!live) return;
        const bool v = c >= CN + CR, r = !v && c >= CN;
        const float by = v ? 1.f : P.scale;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int col = 32 * (v ? c - CN - CR : r ? c - CN : c) + 8 * b + 4 * (lane >> 5);
            if (col >= (v ? P.dv : r ? P.dr : P.dn)) continue;
            store4(v ? P.dvg.p : r ? P.dkr_part : P.dk.p, (v ? dv_at : r ? part : dk_at) + col, !r && P.grad_bf16, x[4 * b] * by,
                   x[4 * b + 1] * by, x[4 * b + 2] * by, x[4 * b + 3] * by);
        }
    });
}

template <int WAVES, int NP, int RP, int VP>
__device__ __forceinline__ void dq_fp32(const AttendLaunch &P, int64_t id, float *sums) {
    constexpr int SN = NP / 8, SR = RP / 8, SV = VP / 8, CN = NP / 32, CR = RP / 32;
    const Place w = place_of<true>(P, id);
    if (!w.valid || w.at >= w.nq) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int shift = w.nk - w.nq, q = w.at + (lane & 31);
    const bool live = q < w.nq;
    const int keys = P.causal ? max(0, min(w.nk, min(w.at + 32, w.nq) + shift)) : w.nk;
    const int limit = P.causal ? min(w.nk, q + shift + 1) : w.nk;

    f4 qf[SN + SR], gf[SV];
    const int64_t row = w.q_row + (live ? q : 0);
    const float *qp = head_row<float>(P.q, row, w.h);
    load_rows<SN>(qf, qp, P.dn, live, lane);
    load_rows<SR>(qf + SN, qp + P.dn, P.dr, live, lane);
    load_rows<SV>(gf, head_row<float>(P.go, row, w.h), P.dv, live, lane);
    const float lse = P.lse[row * P.H + w.h] * kLog2e, delta = P.delta[row * P.H + w.h];
    const float *kp = head_row<float>(P.k, w.k_row, w.h), *rp = head_row<float>(P.kr, w.k_row, 0), *vp = head_row<float>(P.v, w.k_row, w.h);

    f16 dq[CN + CR];
#pragma unroll
    for (int c = 0; c < CN + CR; ++c) clear(dq[c]);
    const float c2 = P.scale * kLog2e;
    for (int key0 = 32 * wave; key0 < keys; key0 += 32 * WAVES) {
        const int lane_ = afresh(lane);
        const TileRows K(kp, key0, P.k.stride, w.nk, P.dn), R(rp, key0, P.kr.stride, w.nk, P.dr), V(vp, key0, P.v.stride, w.nk, P.dv);
        f16 s, dp;
        clear(s);
        clear(dp);
        rows_products<SN, SR, SV>(s, dp, K, P.dn, R, P.dr, qf, V, P.dv, gf, lane_);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float p = exp2_f(fmaf(s[i], c2, -lse));
            if (key0 + result_row(i, lane) >= limit) p = 0.f;
            dp[i] = p * (dp[i] - delta);
        }
        constexpr int C = CN + CR;
        pipelined<f4, 4 * C, kAhead>(
            [&](int i) {
                const int k = i / C, c = i % C;
                return c < CN ? K.col_step(k, c, lane_) : R.col_step(k, c - CN, lane_);
            },
            [&](int i, f4 a) {
                const int k = i / C, c = i % C;
                if (c < CN ? 32 * c < P.dn : 32 * (c - CN) < P.dr) dq[c] = M::mma32(a, rows_of(dp, k), dq[c]);
            });
    }
    const int64_t out = row * P.dq.stride + w.h * P.dq.head_stride;
    join_waves<WAVES, CN + CR, CN + CR>(dq, sums, wave, lane, [&](int c, const f16 &x) {
        if (!live) return;
        const bool r = c >= CN;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int col = 32 * (r ? c - CN : c) + 8 * b + 4 * (lane >> 5);
            if (col < (r ? P.dr : P.dn))
                store4(P.dq.p, out + col + (r ? P.dn : 0), P.grad_bf16, x[4 * b] * P.scale, x[4 * b + 1] * P.scale, x[4 * b + 2] * P.scale, x[4 * b + 3] * P.scale);
        }
    });
}

// Both in one launch: where there are few tiles they run side by side.  Keys' tiles first, each takes longer.
template <int WAVES, int NP, int RP, int VP>
__global__ __launch_bounds__(64 * WAVES, NP > 64 ? 1 : 2) void attend_grads_fp32_kernel(const AttendLaunch P, unsigned key_groups) {
    constexpr int N = (NP + RP) / 32, PART = (N + VP / 32 + 1) / 2;
    __shared__ float sums[WAVES * (N > PART ? N : PART) * 1024];
    if (blockIdx.x < key_groups) dkv_fp32<WAVES, NP, RP, VP>(P, blockIdx.x, sums);
    else dq_fp32<WAVES, NP, RP, VP>(P, blockIdx.x - key_groups, sums);
}

// Heads are padded with zeros to one of two sizes (2 sequences of 2,048 rows of 16 heads of 64 + 32 and 64: the gradients 800 us, padded
// to the larger one 1,300).
bool small(const AttendLaunch &P) { return P.dn <= 64 && P.dr <= 32 && P.dv <= 64; }

// Eight waves share a tile's work where there are few workgroups, and so the longest sequence's tiles decide; where there are
// many, more results to add up only cost (four waves and eight, forward at the full head sizes: 1,024 rows of 16 heads 91 and 67
// us, 1,536 rows 120 and 136; gradients at the small ones: 1,024 rows of 8 heads 105 and 80 us, 1,536 of 16 255 and 280).  Of packed
// sequences the launch's slots count, up to one more for each than it has tiles: what the lengths are the host does not know.
bool few(unsigned n) { return n <= 512; }

template <int WAVES, int NP, int RP, int VP>
void fwd(const AttendLaunch &L, unsigned n) {
    attend_fwd_fp32_kernel<WAVES, NP, RP, VP><<<n, 64 * WAVES, 0, L.stream>>>(L);
}
template <int WAVES, int NP, int RP, int VP>
void grads(const AttendLaunch &L, unsigned n, unsigned k) {
    attend_grads_fp32_kernel<WAVES, NP, RP, VP><<<n, 64 * WAVES, 0, L.stream>>>(L, k);
}

}  // namespace

void launch_attend_fwd_fp32(const AttendLaunch &P) {
    AttendLaunch L = P;
    L.q_seq.L = kAttendTileF32;
    const unsigned n = static_cast<unsigned>(tiles_of(L.q_seq) * L.H);
    if (small(L)) few(n) ? fwd<8, 64, 32, 64>(L, n) : fwd<4, 64, 32, 64>(L, n);
    else few(n) ? fwd<8, 128, 64, 128>(L, n) : fwd<4, 128, 64, 128>(L, n);
}
void launch_attend_grads_fp32(const AttendLaunch &P) {
    AttendLaunch L = P;
    L.q_seq.L = L.k_seq.L = kAttendTileF32;
    const unsigned k = L.k_seq.rows() ? static_cast<unsigned>(tiles_of(L.k_seq) * L.H) : 0;
    const unsigned n = k + (L.q_seq.rows() ? static_cast<unsigned>(tiles_of(L.q_seq) * L.H) : 0);
    if (small(L)) few(n) ? grads<8, 64, 32, 64>(L, n, k) : grads<4, 64, 32, 64>(L, n, k);
    else grads<4, 128, 64, 128>(L, n, k);  // one wave per SIMD has the registers
}

}  // namespace kda
