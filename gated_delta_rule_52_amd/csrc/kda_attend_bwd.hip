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

// delta: 16 lanes per (row, head), 8 elements each (dv <= 128).
template <class E>
__global__ __launch_bounds__(256) void attend_delta_kernel(const AttendLaunch P) {
    const int64_t rows = P.q_seq.rows() * P.H, at = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
    if (at >= rows) return;
    const int64_t row = at / P.H;
    const int h = static_cast<int>(at % P.H), c = 8 * (threadIdx.x & 15);
    float x = 0.f;
    if (c < P.dv) {
        const E *o = head_row<E>(P.o, row, h) + c, *g = head_row<E>(P.go, row, h) + c;
        constexpr int PER = Mx<E>::PER;
#pragma unroll
        for (int k = 0; k < 8; k += PER) {
            const typename Mx<E>::frag a = *reinterpret_cast<const typename Mx<E>::frag *>(o + k);
            const typename Mx<E>::frag b = *reinterpret_cast<const typename Mx<E>::frag *>(g + k);
#pragma unroll
            for (int j = 0; j < PER; ++j) x = fmaf(static_cast<float>(a[j]), static_cast<float>(b[j]), x);
        }
    }
    x += dpp_mov<0xB1>(x);
    x += dpp_mov<0x4E>(x);
    x += dpp_mov<0x141>(x);
    x += dpp_mov<0x140>(x);
    if ((threadIdx.x & 15) == 0) P.delta[at] = x;
}

// A workgroup of four waves has 128 keys, 32 per wave, whose operands and gradients stay in registers (one wave per
// SIMD), and walks the queries that see them.
template <class E, int NP, int RP, int VP>
__global__ __launch_bounds__(256, 1) void attend_dkv_kernel(const AttendLaunch P) {
    constexpr int BQ = sizeof(E) == 2 ? 64 : 32;  // queries per tile
    constexpr int SN = NP / (2 * Mx<E>::PER), SR = RP / (2 * Mx<E>::PER), SV = VP / (2 * Mx<E>::PER), ST = kSteps32<E>;
    using NT = LdsTile<NP, E>;
    using RT = LdsTile<RP, E>;
    using VT = LdsTile<VP, E>;
    constexpr int OR = BQ * NT::ROW, OV = OR + BQ * RT::ROW, OS = OV + BQ * VT::ROW, BUF = OS + 2 * BQ * 4;
    __shared__ __attribute__((aligned(1024))) char lds[2 * BUF];

    const Place w = place_of<false>(P, blockIdx.x);
    if (!w.valid || w.at >= w.nk) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int shift = w.nk - w.nq;
    const int k0 = w.at + 32 * wave, key = k0 + (lane & 31);
    const bool live = key < w.nk;

    typename Mx<E>::frag kf[SN + SR], vf[SV];
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
    const float *lp = P.lse + w.q_row * P.H + w.h, *dp_ = P.delta + w.q_row * P.H + w.h;
    auto fetch = [&](int at, char *to) {
        const int rows = min(BQ, w.nq - at);
        const E *q = qp + at * P.q.stride;
        NT::template fill<BQ, 4>(to, rows_buffer(q, P.q.stride, rows, P.dn), P.q.stride * sizeof(E), P.dn * sizeof(E), wave, lane);
        RT::template fill<BQ, 4>(to + OR, rows_buffer(q + P.dn, P.q.stride, rows, P.dr), P.q.stride * sizeof(E), P.dr * sizeof(E), wave, lane);
        VT::template fill<BQ, 4>(to + OV, rows_buffer(gp + at * P.go.stride, P.go.stride, rows, P.dv), P.go.stride * sizeof(E), P.dv * sizeof(E), wave, lane);
        if (wave < 2 && lane < BQ) {  // the rows' statistics, behind one another; zeros behind the last row
            const rsrc_t r = rows_buffer((wave ? dp_ : lp) + at * static_cast<int64_t>(P.H), P.H, rows, 1);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)(to + OS + wave * BQ * 4), 4, lane * P.H * 4, 0, 0, 0);
        }
    };

    f16 dk[(NP + RP) / 32], dv[VP / 32];
#pragma unroll
    for (int c = 0; c < (NP + RP) / 32; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) dk[c][i] = 0.f;
#pragma unroll
    for (int c = 0; c < VP / 32; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) dv[c][i] = 0.f;
    const float c2 = P.scale * kLog2e;

    // the first query that sees the workgroup's first key
    const int first = P.causal ? max(0, w.at - shift) / BQ * BQ : 0;
    if (first < w.nq) fetch(first, lds);
    int buf = 0;
    for (int at = first; at < w.nq; at += BQ, buf ^= 1) {
        loads_landed();
        const char *t = lds + buf * BUF;
        if (at + BQ < w.nq) fetch(at + BQ, lds + (buf ^ 1) * BUF);
#pragma unroll 1
        for (int b = 0; b < BQ / 32; ++b) {
            const int q0 = at + 32 * b;
            if (P.causal && q0 + 31 + shift < k0) continue;  // none of them sees the wave's keys
            f16 s, dp;
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.f;
#pragma unroll
            for (int k = 0; k < SN; ++k) s = Mx<E>::mma32(NT::rows32(t, 32 * b, k, lane), kf[k], s);
#pragma unroll
            for (int k = 0; k < SR; ++k) s = Mx<E>::mma32(RT::rows32(t + OR, 32 * b, k, lane), kf[SN + k], s);
#pragma unroll
            for (int k = 0; k < SV; ++k) dp = Mx<E>::mma32(VT::rows32(t + OV, 32 * b, k, lane), vf[k], dp);
            const float *st = reinterpret_cast<const float *>(t + OS) + 32 * b + 4 * (lane >> 5);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const f4 lse = *reinterpret_cast<const f4 *>(st + 8 * r), dl = *reinterpret_cast<const f4 *>(st + BQ + 8 * r);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float p = exp2_f(fmaf(s[4 * r + i], c2, -lse[i] * kLog2e));
                    if (P.causal && q0 + 8 * r + 4 * (lane >> 5) + i + shift < key) p = 0.f;
                    s[4 * r + i] = p;
                    dp[4 * r + i] = p * (dp[4 * r + i] - dl[i]);
                }
            }
#pragma unroll
            for (int k = 0; k < ST; ++k) {
                const typename Mx<E>::frag pf = result_operand<E>(s, k), df = result_operand<E>(dp, k);
#pragma unroll
                for (int c = 0; c < VP / 32; ++c) dv[c] = Mx<E>::mma32(VT::cols32(t + OV, 32 * b, k, 32 * c, lane), pf, dv[c]);
#pragma unroll
                for (int c = 0; c < NP / 32; ++c) dk[c] = Mx<E>::mma32(NT::cols32(t, 32 * b, k, 32 * c, lane), df, dk[c]);
#pragma unroll
                for (int c = 0; c < RP / 32; ++c)
                    dk[NP / 32 + c] = Mx<E>::mma32(RT::cols32(t + OR, 32 * b, k, 32 * c, lane), df, dk[NP / 32 + c]);
            }
        }
    }
    if (!live) return;
    const int64_t row = w.k_row + key;
    const int64_t dk_at = row * P.dk.stride + w.h * P.dk.head_stride, dv_at = row * P.dvg.stride + w.h * P.dvg.head_stride;
    const int64_t part = (row * P.H + w.h) * P.dr;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int col = 8 * b + 4 * (lane >> 5);
#pragma unroll
        for (int c = 0; c < NP / 32; ++c)
            if (32 * c + col < P.dn)
                store4(P.dk.p, dk_at + 32 * c + col, P.grad_bf16, dk[c][4 * b] * P.scale, dk[c][4 * b + 1] * P.scale,
                       dk[c][4 * b + 2] * P.scale, dk[c][4 * b + 3] * P.scale);
#pragma unroll
        for (int c = 0; c < RP / 32; ++c)
            if (32 * c + col < P.dr) {
                const f16 &d = dk[NP / 32 + c];
                store4(P.dkr_part, part + 32 * c + col, false, d[4 * b] * P.scale, d[4 * b + 1] * P.scale, d[4 * b + 2] * P.scale,
                       d[4 * b + 3] * P.scale);
            }
#pragma unroll
        for (int c = 0; c < VP / 32; ++c)
            if (32 * c + col < P.dv)
                store4(P.dvg.p, dv_at + 32 * c + col, P.grad_bf16, dv[c][4 * b], dv[c][4 * b + 1], dv[c][4 * b + 2], dv[c][4 * b + 3]);
    }
}

// As the forward pass: 128 queries per workgroup, 32 per wave, over the keys that they see.
template <class E, int NP, int RP, int VP>
__global__ __launch_bounds__(256, sizeof(E) == 2 ? 2 : 1) void attend_dq_kernel(const AttendLaunch P) {
    constexpr int BN = sizeof(E) == 2 ? 64 : 32;
    constexpr int SN = NP / (2 * Mx<E>::PER), SR = RP / (2 * Mx<E>::PER), SV = VP / (2 * Mx<E>::PER), ST = kSteps32<E>;
    using KT = LdsTile<NP, E>;
    using RT = LdsTile<RP, E>;
    using VT = LdsTile<VP, E>;
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

    typename Mx<E>::frag qf[SN + SR], gf[SV];
    const int64_t row = w.q_row + (live ? q : 0);
    {
        const E *qp = head_row<E>(P.q, row, w.h), *gp = head_row<E>(P.go, row, w.h);
#pragma unroll
        for (int s = 0; s < SN; ++s) qf[s] = row_operand<E>(qp, s, P.dn, live, lane);
#pragma unroll
        for (int s = 0; s < SR; ++s) qf[SN + s] = row_operand<E>(qp + P.dn, s, P.dr, live, lane);
#pragma unroll
        for (int s = 0; s < SV; ++s) gf[s] = row_operand<E>(gp, s, P.dv, live, lane);
    }
    const float lse = P.lse[row * P.H + w.h] * kLog2e, delta = P.delta[row * P.H + w.h];
    const E *kp = head_row<E>(P.k, w.k_row, w.h), *rp = head_row<E>(P.kr, w.k_row, 0), *vp = head_row<E>(P.v, w.k_row, w.h);
    auto fetch = [&](int key0, char *to) {
        const int rows = min(BN, w.nk - key0);
        KT::template fill<BN, 4>(to, rows_buffer(kp + key0 * P.k.stride, P.k.stride, rows, P.dn), P.k.stride * sizeof(E), P.dn * sizeof(E), wave, lane);
        RT::template fill<BN, 4>(to + OR, rows_buffer(rp + key0 * P.kr.stride, P.kr.stride, rows, P.dr), P.kr.stride * sizeof(E), P.dr * sizeof(E), wave, lane);
        VT::template fill<BN, 4>(to + OV, rows_buffer(vp + key0 * P.v.stride, P.v.stride, rows, P.dv), P.v.stride * sizeof(E), P.dv * sizeof(E), wave, lane);
    };

    f16 dq[(NP + RP) / 32];
#pragma unroll
    for (int c = 0; c < (NP + RP) / 32; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) dq[c][i] = 0.f;
    const float c2 = P.scale * kLog2e;

    if (keys > 0) fetch(0, lds);
    int buf = 0;
    for (int key0 = 0; key0 < keys; key0 += BN, buf ^= 1) {
        loads_landed();
        const char *t = lds + buf * BUF;
        if (key0 + BN < keys) fetch(key0 + BN, lds + (buf ^ 1) * BUF);
#pragma unroll 1
        for (int b = 0; b < BN / 32; ++b) {
            const int kb = key0 + 32 * b;
            if (kb >= wave_keys) break;
            f16 s, dp;
#pragma unroll
            for (int i = 0; i < 16; ++i) s[i] = dp[i] = 0.f;
#pragma unroll
            for (int k = 0; k < SN; ++k) s = Mx<E>::mma32(KT::rows32(t, 32 * b, k, lane), qf[k], s);
#pragma unroll
            for (int k = 0; k < SR; ++k) s = Mx<E>::mma32(RT::rows32(t + OR, 32 * b, k, lane), qf[SN + k], s);
#pragma unroll
            for (int k = 0; k < SV; ++k) dp = Mx<E>::mma32(VT::rows32(t + OV, 32 * b, k, lane), gf[k], dp);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float p = exp2_f(fmaf(s[i], c2, -lse));
                if (kb + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3) >= limit) p = 0.f;
                dp[i] = p * (dp[i] - delta);
            }
#pragma unroll
            for (int k = 0; k < ST; ++k) {
                const typename Mx<E>::frag df = result_operand<E>(dp, k);
#pragma unroll
                for (int c = 0; c < NP / 32; ++c) dq[c] = Mx<E>::mma32(KT::cols32(t, 32 * b, k, 32 * c, lane), df, dq[c]);
#pragma unroll
                for (int c = 0; c < RP / 32; ++c)
                    dq[NP / 32 + c] = Mx<E>::mma32(RT::cols32(t + OR, 32 * b, k, 32 * c, lane), df, dq[NP / 32 + c]);
            }
        }
    }
    if (!live) return;
    const int64_t out = row * P.dq.stride + w.h * P.dq.head_stride;
#pragma unroll
    for (int c = 0; c < (NP + RP) / 32; ++c)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int col = (c < NP / 32 ? 32 * c : 32 * c - NP) + 8 * b + 4 * (lane >> 5);
            if (col < (c < NP / 32 ? P.dn : P.dr))
                store4(P.dq.p, out + col + (c < NP / 32 ? 0 : P.dn), P.grad_bf16, dq[c][4 * b] * P.scale, dq[c][4 * b + 1] * P.scale,
                       dq[c][4 * b + 2] * P.scale, dq[c][4 * b + 3] * P.scale);
        }
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
    if (keys) attend_dkv_kernel<uint16_t, NP, RP, VP><<<static_cast<unsigned>(tiles_of(L.k_seq) * L.H), 256, 0, L.stream>>>(L);
    else attend_dq_kernel<uint16_t, NP, RP, VP><<<static_cast<unsigned>(tiles_of(L.q_seq) * L.H), 256, 0, L.stream>>>(L);
}

}  // namespace

hipError_t launch_attend_bwd(const AttendLaunch &P) {
    AttendLaunch L = P;
    L.q_seq.L = L.k_seq.L = kAttendTile;
    const bool small = P.dn <= 64 && P.dr <= 32 && P.dv <= 64;
    const int64_t rows_q = L.q_seq.rows() * L.H, rope = L.k_seq.rows() * (L.dr / 4);
    if (rows_q) {
        const unsigned n = static_cast<unsigned>((rows_q + 15) / 16);
        if (P.bf16) attend_delta_kernel<uint16_t><<<n, 256, 0, L.stream>>>(L);
        else attend_delta_kernel<float><<<n, 256, 0, L.stream>>>(L);
    }
    if (!P.bf16) launch_attend_grads_fp32(P);
    if (rope) {
        if (P.bf16) small ? launch<64, 32, 64>(L, true) : launch<128, 64, 128>(L, true);
        attend_rope_sum_kernel<<<static_cast<unsigned>((rope + 255) / 256), 256, 0, L.stream>>>(L);
    }
    if (rows_q && P.bf16) small ? launch<64, 32, 64>(L, false) : launch<128, 64, 128>(L, false);
    return hipGetLastError();
}

// Of the largest launch.
int64_t attend_threads(const SeqTiles &q_, const SeqTiles &k_, int H, int dr, bool bf16, bool backward) {
    SeqTiles q = q_, k = k_;
    q.L = k.L = bf16 ? kAttendTile : kAttendTileF32;
    int64_t n = (tiles_of(q) + (backward && !bf16 ? tiles_of(k) : 0)) * H * 256;
    if (backward) {
        const int64_t parts[] = {tiles_of(k) * H * 256, (q.rows() * H + 15) / 16 * 256, (k.rows() * (dr / 4) + 255) / 256 * 256};
        for (const int64_t p : parts) n = p > n ? p : n;
    }
    return n;
}

}  // namespace kda
