// kda_attend_bwd.hip - gradients of latent attention over expanded keys and values.
//
// With p_ij = exp(s_ij - lse_i) recomputed from the inputs, dp_ij = grad_o_i . v_j, delta_i = grad_o_i . o_i and
// ds_ij = p_ij (dp_ij - delta_i):
//     dv_j = sum_i p_ij grad_o_i,   dk_j = scale sum_i ds_ij q_i,   dq_i = scale sum_j ds_ij [k_j | k_rope_j],
// where dk's last dr elements are summed over the heads that share k_rope.  One kernel walks the queries for tiles of keys
// and one the keys for tiles of queries: seven products of a pair's tile instead of five, but no sum goes through atomics,
// and the same inputs give the same bits.
#include "kda_latent.h"

namespace kda {
namespace {

using namespace la;

// delta for fp32 (the bf16 kernel for dq forms its own): 16 lanes per (row, head), 8 elements each (dv <= 128).
__global__ __launch_bounds__(256) void attend_delta_kernel(const AttendLaunch P) {
    const int64_t rows = P.q_seq.rows() * P.H, at = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
    if (at >= rows) return;
    const int64_t row = at / P.H;
    const int h = static_cast<int>(at % P.H), c = 8 * (threadIdx.x & 15);
    float x = 0.f;
    if (c < P.dv) {
        const float *o = head_row<float>(P.o, row, h) + c, *g = head_row<float>(P.go, row, h) + c;
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
            const f4 a = *reinterpret_cast<const f4 *>(o + k), b = *reinterpret_cast<const f4 *>(g + k);
#pragma unroll
            for (int j = 0; j < 4; ++j) x = fmaf(a[j], b[j], x);
        }
    }
    x += dpp_mov<0xB1>(x);
    x += dpp_mov<0x4E>(x);
    x += dpp_mov<0x141>(x);
    x += dpp_mov<0x140>(x);
    if ((threadIdx.x & 15) == 0) P.delta[at] = x;
}

// A workgroup of four waves has 128 keys, 32 per wave, whose operands and gradients stay in registers (one wave per
// SIMD), and walks the queries that see them, 32 at a time.  Nothing but the wave itself can fill the time that its exponentials
// take: they are woven into the products of the block before, which wait in three buffers' worth of LDS until then (2
// sequences of 4,096 rows of 32 heads, 687 GFLOP: 790 us, 0.87 PFLOP/s, against 816 one after the other).  What is left beside the
// products is theirs to wait for: LDS delivers an operand per product, and the same kernel without those reads takes 623 us, without
// the next tile's loads 723, without the exponentials 715.
template <int NP, int RP, int VP>
__global__ __launch_bounds__(256, 1) void attend_dkv_kernel(const AttendLaunch P) {
    typedef uint16_t E;
    typedef Mx<E>::frag frag;
    constexpr int BQ = 64;  // queries per tile
    constexpr int SN = NP / 16, SR = RP / 16, SV = VP / 16, CN = NP / 32, CR = RP / 32, CV = VP / 32, C = CN + CR + CV;
    using NT = LdsTile<NP, E, 32>;
    using RT = LdsTile<RP, E, 32>;
    using VT = LdsTile<VP, E, 32>;
    constexpr int OR = BQ * NT::ROW, OV = OR + BQ * RT::ROW, OS = OV + BQ * VT::ROW, BUF = OS + 2 * BQ * 4;
    __shared__ __attribute__((aligned(1024))) char lds[3 * BUF];

    const Place w = place_of<false>(P, blockIdx.x);
    if (!w.valid || w.at >= w.nk) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int shift = w.nk - w.nq;
    const int k0 = w.at + 32 * wave, key = k0 + (lane & 31);
    const bool live = key < w.nk;

    frag kf[SN + SR], vf[SV];
    {
        const int64_t row = w.k_row + (live ? key : 0);
        const E *kp = head_row<E>(P.k, row, w.h), *rp = head_row<E>(P.kr, row, 0), *vp = head_row<E>(P.v, row, w.h);
#pragma unroll
        for (int s = 0; s < SN; ++s) kf[s] = row_operand<E>(kp, s, P.dn, live, lane);
#pragma unroll
        for (int s = 0; s < SR; ++s) kf[SN + s] = row_operand<E>(rp, s, P.dr, live, lane);
#pragma unroll
        for (int s = 0; s < SV; ++s) vf[s] = row_operand<E>(vp, s, P.dv, live, lane);
    }
    const E *qp = head_row<E>(P.q, w.q_row, w.h), *gp = head_row<E>(P.go, w.q_row, w.h);
    const float *lp = P.lse2 + w.q_row * P.H + w.h, *ep = P.delta + w.q_row * P.H + w.h;
    auto fetch = [&](int at, char *to, int lane) {
        const int rows = min(BQ, w.nq - at);
        const E *q = qp + at * P.q.stride;
        NT::template fill<BQ, 4>(to, rows_buffer(q, P.q.stride, rows, P.dn), P.q.stride * sizeof(E), P.dn * sizeof(E), wave, lane);
        RT::template fill<BQ, 4>(to + OR, rows_buffer(q + P.dn, P.q.stride, rows, P.dr), P.q.stride * sizeof(E), P.dr * sizeof(E), wave, lane);
        VT::template fill<BQ, 4>(to + OV, rows_buffer(gp + at * P.go.stride, P.go.stride, rows, P.dv), P.go.stride * sizeof(E), P.dv * sizeof(E), wave, lane);
        if (wave < 2) {  // the rows' statistics, behind one another; zeros behind the last row, where q and grad_o are too
            const rsrc_t r = rows_buffer((wave ? ep : lp) + at * static_cast<int64_t>(P.H), P.H, rows, 1);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)(to + OS + wave * BQ * 4), 4, lane * P.H * 4, 0, 0, 0);
        }
    };

    f16 d[C];  // dk, its shared part, dv
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) d[c][i] = 0.f;
    const float c2 = P.scale * kLog2e;

    // One block's scores become its weights p (in s) and gradients ds (in dp), element by element.
    auto stats = [&](const char *st, int r, f4 &lse, f4 &dl) {
        lse = *reinterpret_cast<const f4 *>(st + 32 * r);
        dl = *reinterpret_cast<const f4 *>(st + BQ * 4 + 32 * r);
    };
    auto element = [&](int i, int hidden, f16 &s, f16 &dp, const f4 &lse, const f4 &dl) {
        const int r = 8 * (i >> 2) + (i & 3);
        const float p = r < hidden ? 0.f : exp2_f(fmaf(s[i], c2, -lse[i & 3]));
        s[i] = p;
        dp[i] = p * (dp[i] - dl[i & 3]);
    };
    auto operand = [&](const char *t, int b, int i, int lane) {
        const int k = i / C, c = i % C;
        return c < CN ? NT::cols32(t, 32 * b, k, 32 * c, lane) : c < CN + CR ? RT::cols32(t + OR, 32 * b, k, 32 * (c - CN), lane)
                                                                            : VT::cols32(t + OV, 32 * b, k, 32 * (c - CN - CR), lane);
    };

    // the first query that sees the workgroup's first key
    const int first = P.causal ? max(0, w.at - shift) / BQ * BQ : 0;
    if (first < w.nq) fetch(first, lds, lane);
    // the block before: its weights and gradients as operands, its tile, its block in it; at first zeros, which meet the
    // first block itself
    frag pf[2], df[2];
    pf[0] = pf[1] = df[0] = df[1] = Mx<E>::zero();
    const char *before = nullptr;
    int before_b = 0, buf = 0;
    for (int at = first; at < w.nq; at += BQ, buf = buf == 2 ? 0 : buf + 1) {
        loads_landed();
        const char *t = lds + buf * BUF;
        if (at + BQ < w.nq) fetch(at + BQ, lds + (buf == 2 ? 0 : buf + 1) * BUF, lane);
#pragma unroll
        for (int b = 0; b < BQ / 32; ++b) {
            const int q0 = at + 32 * b;
            if (q0 >= w.nq || (P.causal && q0 + 31 + shift < k0)) continue;  // none of them sees the wave's keys
            f16 s, dp;
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.f;
            // the two products' steps alternate while both last: a step waits for the one before it in its own product
            auto step = [](int i) {
                constexpr int both = 2 * (SN + SR < SV ? SN + SR : SV);
                return i < both ? i / 2 + (i % 2 ? SN + SR : 0) : SN + SR < SV ? i : i - SV;
            };
            pipelined<frag, SN + SR + SV, 6>(
                [&](int j) {
                    const int i = step(j);
                    return i < SN ? NT::rows32(t, 32 * b, i, lane) : i < SN + SR ? RT::rows32(t + OR, 32 * b, i - SN, lane)
                                                                                 : VT::rows32(t + OV, 32 * b, i - SN - SR, lane);
                },
                [&](int j, frag f) {
                    const int i = step(j);
                    if (i < SN + SR) s = Mx<E>::mma32(f, kf[i], s);
                    else dp = Mx<E>::mma32(f, vf[i - SN - SR], dp);
                });
            before_b = before ? before_b : b;
            before = before ? before : t;
            const char *st = t + OS + 128 * b + 16 * (lane >> 5);
            // rows of the lane's half below this one do not see the lane's key
            const int hidden = P.causal ? key - shift - q0 - 4 * (lane >> 5) : 0;
            f4 lse[2], dl[2];
            stats(st, 0, lse[0], dl[0]);
            pipelined<frag, 2 * C, 4>([&](int i) { return operand(before, before_b, i, lane); },
                                      [&](int i, frag f) {
                                          const int k = i / C, c = i % C;
                                          d[c] = Mx<E>::mma32(f, c < CN + CR ? df[k] : pf[k], d[c]);
                                          // the elements spread over the products
                                          const int from = i * 16 / (2 * C), to = (i + 1) * 16 / (2 * C);
#pragma unroll
                                          for (int j = from; j < to; ++j) {
                                              const int r = j >> 2;
                                              if ((j & 3) == 0 && r < 3) stats(st, r + 1, lse[(r + 1) & 1], dl[(r + 1) & 1]);
                                              element(j, hidden, s, dp, lse[r & 1], dl[r & 1]);
                                          }
                                      });
#pragma unroll
            for (int k = 0; k < 2; ++k) pf[k] = result_operand(s, k), df[k] = result_operand(dp, k);
            before = t;
            before_b = b;
        }
    }
    if (before)
        pipelined<frag, 2 * C, 4>([&](int i) { return operand(before, before_b, i, lane); },
                                  [&](int i, frag f) {
                                      const int k = i / C, c = i % C;
                                      d[c] = Mx<E>::mma32(f, c < CN + CR ? df[k] : pf[k], d[c]);
                                  });
    __syncthreads();  // LDS holds outputs now
    char *mine = lds + wave * 32 * kStoreRow<(NP > VP ? NP : VP)>;
    const int64_t row = w.k_row + k0;
    const int rows = w.nk - k0;
    store_rows<NP>(mine, d, P.scale, out_row(P.dk, P.grad_bf16, row, w.h), P.grad_bf16, P.dk.stride, rows, P.dn, lane);
    store_rows<VP>(mine, d + CN + CR, 1.f, out_row(P.dvg, P.grad_bf16, row, w.h), P.grad_bf16, P.dvg.stride, rows, P.dv, lane);
    store_rows<RP>(mine, d + CN, P.scale, P.dkr_part + (row * P.H + w.h) * P.dr, false, static_cast<int64_t>(P.H) * P.dr, rows, P.dr, lane);
}

// As the forward pass: 128 queries per workgroup, 32 per wave, over the keys that they see.  Two workgroups share a CU: one's
// exponentials hide behind the other's products, and waves that are at a product go first (s_setprio: for 2 sequences of 4,096 rows of
// 32 heads all gradients take 1,416 us so and 1,445 without).  Blocks of 32 keys one after the other, not unrolled: two at a time do
// not fit the 256 registers beside q's, grad_o's and the sums'.  The same sequences: 590 us for 550 GFLOP, 0.93 PFLOP/s.
template <int NP, int RP, int VP>
__global__ __launch_bounds__(256, 2) void attend_dq_kernel(const AttendLaunch P) {
    typedef uint16_t E;
    typedef Mx<E>::frag frag;
    constexpr int BN = 64;  // keys per tile
    constexpr int SN = NP / 16, SR = RP / 16, SV = VP / 16, CN = NP / 32, CR = RP / 32, C = CN + CR;
    using KT = LdsTile<NP, E, 32>;
    using RT = LdsTile<RP, E, 32>;
    using VT = LdsTile<VP, E, 32>;
    constexpr int OR = BN * KT::ROW, OV = OR + BN * RT::ROW, BUF = OV + BN * VT::ROW;
    __shared__ __attribute__((aligned(1024))) char lds[2 * BUF];

    const Place w = place_of<true>(P, blockIdx.x);
    if (!w.valid || w.at >= w.nq) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int shift = w.nk - w.nq;
    const int q0 = w.at + 32 * wave, q = q0 + (lane & 31);
    const bool live = q < w.nq;
    const int tile_end = min(w.at + 128, w.nq);
    const int keys = P.causal ? max(0, min(w.nk, tile_end + shift)) : w.nk;
    const int wave_keys = P.causal ? min(w.nk, min(q0 + 32, w.nq) + shift) : w.nk;
    const int limit = P.causal ? min(w.nk, q + shift + 1) : w.nk;

    const E *kp = head_row<E>(P.k, w.k_row, w.h), *rp = head_row<E>(P.kr, w.k_row, 0), *vp = head_row<E>(P.v, w.k_row, w.h);
    auto fetch = [&](int key0, char *to, int lane) {
        const int rows = min(BN, w.nk - key0);
        KT::template fill<BN, 4>(to, rows_buffer(kp + key0 * P.k.stride, P.k.stride, rows, P.dn), P.k.stride * sizeof(E), P.dn * sizeof(E), wave, lane);
        RT::template fill<BN, 4>(to + OR, rows_buffer(rp + key0 * P.kr.stride, P.kr.stride, rows, P.dr), P.kr.stride * sizeof(E), P.dr * sizeof(E), wave, lane);
        VT::template fill<BN, 4>(to + OV, rows_buffer(vp + key0 * P.v.stride, P.v.stride, rows, P.dv), P.v.stride * sizeof(E), P.dv * sizeof(E), wave, lane);
    };
    if (keys > 0) fetch(0, lds, lane);

    frag qf[SN + SR], gf[SV];
    const int64_t row = w.q_row + (live ? q : 0);
    const E *qp = head_row<E>(P.q, row, w.h);
#pragma unroll
    for (int s = 0; s < SN; ++s) qf[s] = row_operand<E>(qp, s, P.dn, live, lane);
#pragma unroll
    for (int s = 0; s < SR; ++s) qf[SN + s] = row_operand<E>(qp + P.dn, s, P.dr, live, lane);
    const E *gp = head_row<E>(P.go, row, w.h);
#pragma unroll
    for (int s = 0; s < SV; ++s) gf[s] = row_operand<E>(gp, s, P.dv, live, lane);
    // The row's statistics, for the keys' kernel too: delta, and lse in powers of two, infinite for rows that see nothing, which
    // leaves them no weights.  In a kernel of their own they take 28 us more at 2 sequences of 4,096 rows of 32 heads.
    float delta = 0.f;
    const E *op = head_row<E>(P.o, row, w.h);
#pragma unroll
    for (int s = 0; s < SV; ++s) {
        const frag x = row_operand<E>(op, s, P.dv, live, lane);
#pragma unroll
        for (int j = 0; j < 8; ++j) delta = fmaf(static_cast<float>(x[j]), static_cast<float>(gf[s][j]), delta);
    }
    delta = halves_sum(delta);
    const int64_t stat = row * P.H + w.h;
    const float lse = P.lse[stat] == neg_inf() ? __builtin_inff() : P.lse[stat] * kLog2e;
    f16 dq[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) dq[c][i] = 0.f;
    const float c2 = P.scale * kLog2e;

    // o is rounded to bf16, and where few keys share the weights that rounding is of the size of dp - delta itself.  There a
    // walk over the keys in front of the other finds what delta is off by: sum_j p_j (dp_j - delta), which is 0 for the right one
    // (dq's errors relative to 64 bits, causal: sequences of 16 rows 0.0030 without and 0.0024 with it, 1,000 rows 0.0025 and 0.0024;
    // 256 rows of 8 heads take 46 us for 38, 1,024 of 16 98 for 97).
    bool exact = keys > 256;
    float off = 0.f;
    auto store_statistics = [&]() {
        if (live && lane < 32) {
            P.lse2[stat] = lse;
            P.delta[stat] = delta;
        }
    };
    if (exact || keys <= 0) store_statistics();

    int buf = 0;
    for (int key0 = 0; key0 < keys; buf ^= 1) {
        loads_landed();
        const char *t = lds + buf * BUF;
        const bool last = key0 + BN >= keys;
        if (!last || !exact) fetch(last ? 0 : key0 + BN, lds + (buf ^ 1) * BUF, afresh(lane));
#pragma unroll 1
        for (int b = 0; b < BN / 32; ++b) {
            const int kb = key0 + 32 * b;
            if (kb >= wave_keys) break;
            const int lane_ = afresh(lane);
            f16 s, dp;
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.f;
            __builtin_amdgcn_s_setprio(1);
            auto row_step = [](int i) {
                constexpr int both = 2 * (SN + SR < SV ? SN + SR : SV);
                return i < both ? i / 2 + (i % 2 ? SN + SR : 0) : SN + SR < SV ? i : i - SV;
            };
            pipelined<frag, SN + SR + SV, 4>(
                [&](int j) {
                    const int i = row_step(j);
                    return i < SN ? KT::rows32(t, 32 * b, i, lane_) : i < SN + SR ? RT::rows32(t + OR, 32 * b, i - SN, lane_) : VT::rows32(t + OV, 32 * b, i - SN - SR, lane_);
                },
                [&](int j, frag f) {
                    const int i = row_step(j);
                    if (i < SN + SR) s = Mx<E>::mma32(f, qf[i], s);
                    else dp = Mx<E>::mma32(f, gf[i - SN - SR], dp);
                });
            __builtin_amdgcn_s_setprio(0);
            const bool part = kb + 32 > w.nk || (P.causal && kb + 32 > q0 + shift + 1);  // some query does not see some key
            if (part) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (kb + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3) >= limit) s[i] = neg_inf();
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) dp[i] = exp2_f(fmaf(s[i], c2, -lse)) * (dp[i] - delta);
            if (!exact) {
#pragma unroll
                for (int i = 0; i < 16; ++i) off += dp[i];
                continue;
            }
            const frag df[2] = {result_operand(dp, 0), result_operand(dp, 1)};
            __builtin_amdgcn_s_setprio(1);
            pipelined<frag, 2 * C, 3>(
                [&](int i) {
                    const int k = i / C, c = i % C;
                    return c < CN ? KT::cols32(t, 32 * b, k, 32 * c, lane_) : RT::cols32(t + OR, 32 * b, k, 32 * (c - CN), lane_);
                },
                [&](int i, frag f) { dq[i % C] = Mx<E>::mma32(f, df[i / C], dq[i % C]); });
            __builtin_amdgcn_s_setprio(0);
        }
        key0 += BN;
        if (last && !exact) {
            delta += halves_sum(off);
            store_statistics();
            exact = true;
            key0 = 0;
        }
    }
    __syncthreads();  // LDS holds outputs now
    char *mine = lds + wave * 32 * kStoreRow<NP>;
    char *to = static_cast<char *>(out_row(P.dq, P.grad_bf16, w.q_row + q0, w.h));
    store_rows<NP>(mine, dq, P.scale, to, P.grad_bf16, P.dq.stride, w.nq - q0, P.dn, lane);
    store_rows<RP>(mine, dq + CN, P.scale, to + P.dn * (P.grad_bf16 ? 2 : 4), P.grad_bf16, P.dq.stride, w.nq - q0, P.dr, lane);
}

// k_rope's gradient: the heads' parts in their order, four columns per thread.
__global__ __launch_bounds__(256) void attend_rope_sum_kernel(const AttendLaunch P) {
    const int per = P.dr / 4;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, row = at / per;
    const int64_t first = P.k_seq.cu ? P.k_seq.offset(0) : 0, last = P.k_seq.cu ? P.k_seq.offset(P.k_seq.N) : P.k_seq.rows();
    if (row < first || row >= last) return;
    const int c = 4 * static_cast<int>(at % per);
    const float *p = P.dkr_part + row * P.H * P.dr + c;
    f4 x = {0, 0, 0, 0};
#pragma unroll 8
    for (int h = 0; h < P.H; ++h) x += *reinterpret_cast<const f4 *>(p + static_cast<int64_t>(h) * P.dr);
    store4(P.dkr.p, row * P.dkr.stride + c, P.grad_bf16, x[0], x[1], x[2], x[3]);
}

template <int NP, int RP, int VP>
void launch(const AttendLaunch &L, bool keys) {
    if (keys) attend_dkv_kernel<NP, RP, VP><<<static_cast<unsigned>(tiles_of(L.k_seq) * L.H), 256, 0, L.stream>>>(L);
    else attend_dq_kernel<NP, RP, VP><<<static_cast<unsigned>(tiles_of(L.q_seq) * L.H), 256, 0, L.stream>>>(L);
}

}  // namespace

hipError_t launch_attend_bwd(const AttendLaunch &P) {
    AttendLaunch L = P;
    L.q_seq.L = L.k_seq.L = kAttendTile;
    // as in the forward pass (2,048 rows of 32 heads of 64 + 32 and 64: 169 us, padded to the larger size 260; 90 of them
    // in each kernel, the matrix unit busy for 19% of dq's cycles and 24% of dk/dv's: twice the exponentials per product, and 512 workgroups
    // are one round of dq's and two of dk/dv's, whose longest decide)
    const bool small = P.dn <= 64 && P.dr <= 32 && P.dv <= 64;
    const int64_t rows_q = L.q_seq.rows() * L.H, rope = L.k_seq.rows() * (L.dr / 4);
    if (P.bf16) {
        if (rows_q) small ? launch<64, 32, 64>(L, false) : launch<128, 64, 128>(L, false);
        if (rope) small ? launch<64, 32, 64>(L, true) : launch<128, 64, 128>(L, true);
    } else {
        if (rows_q) attend_delta_kernel<<<static_cast<unsigned>((rows_q + 15) / 16), 256, 0, L.stream>>>(L);
        launch_attend_grads_fp32(P);
    }
    if (rope) attend_rope_sum_kernel<<<static_cast<unsigned>((rope + 255) / 256), 256, 0, L.stream>>>(L);
    return hipGetLastError();
}

// Of the largest launch.
int64_t attend_threads(const SeqTiles &q_, const SeqTiles &k_, int H, int dr, bool bf16, bool backward) {
    SeqTiles q = q_, k = k_;
    q.L = k.L = bf16 ? kAttendTile : kAttendTileF32;
    int64_t n = (tiles_of(q) + (backward && !bf16 ? tiles_of(k) : 0)) * H * (bf16 ? 256 : 512);
    if (backward) {
        const int64_t parts[] = {tiles_of(k) * H * 256, bf16 ? 0 : (q.rows() * H + 15) / 16 * 256, (k.rows() * (dr / 4) + 255) / 256 * 256};
        for (const int64_t p : parts) n = p > n ? p : n;
    }
    return n;
}

}  // namespace kda
