// kda_attend.hip - latent attention over expanded keys and values, forward.
//
// Per head, o_i = sum_j p_ij v_j with p_ij = exp(s_ij - lse_i), s_ij = scale (q_i[:dn] . k_j + q_i[dn:] . k_rope_j),
// lse_i = log sum_j exp(s_ij) over the keys that query i sees.
#include "kda_latent.h"

namespace kda {
namespace {

using namespace la;

// A workgroup has 128 queries, 32 per wave, and walks the keys that its last query sees, 64 at a time: q's operands, the scores of
// a tile and the output's sums stay in registers, keys and values come through two buffers in LDS (80 KiB at the full head sizes: two
// workgroups per CU, so that one's exponentials hide behind the other's products).  Scores are formed transposed, keys down and
// queries across: a lane then has 32 scores of one query, its maximum and sum need one exchange between the wave's halves, and
// the weights are the next product's operand as they lie.
//
// The matrix unit bounds it: 8,192 rows of 32 heads, causal, 128 + 64 and 128 wide (687 GFLOP), take 636 to 690 us on several
// cards, 1.0 to 1.08 PFLOP/s, and 16,384 rows of 16 heads 1,240 us, 1.11 PFLOP/s, where the same instructions with nothing beside
// them reach 1.7 to 1.9; what is between is exponentials that meet no other wave's products.  Waves that are at the scores' products
// go first (s_setprio): the first of these takes 641 us so and 670 without.
template <int NP, int RP, int VP>
__global__ __launch_bounds__(256, 2) void attend_fwd_kernel(const AttendLaunch P) {
    typedef uint16_t E;
    typedef Mx<E>::frag frag;
    constexpr int BN = 64;  // keys per tile
    constexpr int SN = NP / 16, SR = RP / 16;
    using KT = LdsTile<NP, E, 32>;
    using RT = LdsTile<RP, E, 32>;
    using VT = LdsTile<VP, E, 32>;
    constexpr int OR = BN * KT::ROW, OV = OR + BN * RT::ROW, BUF = OV + BN * VT::ROW;
    __shared__ __attribute__((aligned(1024))) char lds[2 * BUF];

    const Place w = place_of<true>(P, blockIdx.x);
    if (!w.valid || w.at >= w.nq) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int shift = w.nk - w.nq;              // query i sees keys up to i + shift
    const int q0 = w.at + 32 * wave, q = q0 + (lane & 31);
    const bool live = q < w.nq;
    const int tile_end = min(w.at + 128, w.nq);  // behind the workgroup's last query
    const int keys = P.causal ? max(0, min(w.nk, tile_end + shift)) : w.nk;
    const int wave_keys = P.causal ? min(w.nk, min(q0 + 32, w.nq) + shift) : w.nk;
    const int limit = P.causal ? min(w.nk, q + shift + 1) : w.nk;  // the lane's query sees keys below it

    frag qf[SN + SR];
    {
        const E *row = head_row<E>(P.q, w.q_row + (live ? q : 0), w.h);
#pragma unroll
        for (int s = 0; s < SN; ++s) qf[s] = row_operand<E>(row, s, P.dn, live, lane);
#pragma unroll
        for (int s = 0; s < SR; ++s) qf[SN + s] = row_operand<E>(row + P.dn, s, P.dr, live, lane);
    }
    const E *kp = head_row<E>(P.k, w.k_row, w.h), *rp = head_row<E>(P.kr, w.k_row, 0), *vp = head_row<E>(P.v, w.k_row, w.h);
    auto fetch = [&](int key0, char *to) {
        const int rows = min(BN, w.nk - key0);
        KT::template fill<BN, 4>(to, rows_buffer(kp + key0 * P.k.stride, P.k.stride, rows, P.dn), P.k.stride * sizeof(E), P.dn * sizeof(E), wave, lane);
        RT::template fill<BN, 4>(to + OR, rows_buffer(rp + key0 * P.kr.stride, P.kr.stride, rows, P.dr), P.kr.stride * sizeof(E), P.dr * sizeof(E), wave, lane);
        VT::template fill<BN, 4>(to + OV, rows_buffer(vp + key0 * P.v.stride, P.v.stride, rows, P.dv), P.v.stride * sizeof(E), P.dv * sizeof(E), wave, lane);
    };

    f16 acc[VP / 32];
#pragma unroll
    for (int c = 0; c < VP / 32; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[c][i] = 0.f;
    float m = neg_inf(), l = 0.f;  // in powers of two; l: this lane's half of the row
    const float c2 = P.scale * kLog2e;

    if (keys > 0) fetch(0, lds);
    int buf = 0;
    for (int key0 = 0; key0 < keys; key0 += BN, buf ^= 1) {
        loads_landed();
        const char *t = lds + buf * BUF;
        if (key0 + BN < keys) fetch(key0 + BN, lds + (buf ^ 1) * BUF);
        if (key0 >= wave_keys) continue;
        __builtin_amdgcn_s_setprio(1);
        f16 s[BN / 32];
#pragma unroll
        for (int b = 0; b < BN / 32; ++b) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[b][i] = 0.f;
#pragma unroll
            for (int k = 0; k < SN; ++k) s[b] = Mx<E>::mma32(KT::rows32(t, 32 * b, k, lane), qf[k], s[b]);
#pragma unroll
            for (int k = 0; k < SR; ++k) s[b] = Mx<E>::mma32(RT::rows32(t + OR, 32 * b, k, lane), qf[SN + k], s[b]);
        }
        __builtin_amdgcn_s_setprio(0);
        // a tile that some query of the wave sees only in part
        if (key0 + BN > w.nk || (P.causal && key0 + BN > q0 + shift + 1)) {
#pragma unroll
            for (int b = 0; b < BN / 32; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (key0 + 32 * b + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3) >= limit) s[b][i] = neg_inf();
        }
        float top = s[0][0];
#pragma unroll
        for (int b = 0; b < BN / 32; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
        top = halves_max(top) * c2;
        // The reference point follows the maximum only when it lags by 2^8: weights up to 2^8 lose nothing in fp32 or
        // bf16, and most tiles leave the sums as they are.
        const bool move = top > m + 8.f;
        if (__any(move)) {
            const float to = move ? top : m, by = move ? exp2_f(m - to) : 1.f;
            m = to;
            l *= by;
#pragma unroll
            for (int c = 0; c < VP / 32; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[c][i] *= by;
        }
        const float at = m == neg_inf() ? 0.f : m;
#pragma unroll
        for (int b = 0; b < BN / 32; ++b) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[b][i] = exp2_f(fmaf(s[b][i], c2, -at));
                l += s[b][i];
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const frag p = result_operand(s[b], k);
#pragma unroll
                for (int c = 0; c < VP / 32; ++c)
                    acc[c] = Mx<E>::mma32(VT::cols32(t + OV, 32 * b, k, 32 * c, lane), p, acc[c]);
            }
        }
    }
    l = halves_sum(l);
    const float by = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // NaN stays
    if (P.lse && live && lane < 32) P.lse[(w.q_row + q) * P.H + w.h] = l == 0.f ? neg_inf() : (m + __log2f(l)) * kLn2;
    __syncthreads();  // LDS holds outputs now
    store_rows<VP>(lds + wave * 32 * kStoreRow<VP>, acc, by, out_row(P.o, P.out_bf16, w.q_row + q0, w.h), P.out_bf16, P.o.stride, w.nq - q0, P.dv, lane);
}

}  // namespace

hipError_t launch_attend_fwd(const AttendLaunch &P) {
    if (!P.bf16) {
        launch_attend_fwd_fp32(P);
        return hipGetLastError();
    }
    AttendLaunch L = P;
    L.q_seq.L = kAttendTile;
    const unsigned n = static_cast<unsigned>(tiles_of(L.q_seq) * P.H);
    // Heads are padded with zeros to one of two sizes (2,048 rows of 32 heads of 64 + 32 and 64: 44 us, padded to the larger one 61).
    // At the smaller one a product has twice the exponentials beside it, and 512 workgroups are all there at once, of which the last has
    // twice the average's keys: the matrix unit is busy for 23% of the cycles, vector instructions for 34%.  At 8,192 rows, with
    // workgroups to follow, it is 390 us, 0.88 PFLOP/s.
    if (P.dn <= 64 && P.dr <= 32 && P.dv <= 64) attend_fwd_kernel<64, 32, 64><<<n, 256, 0, P.stream>>>(L);
    else attend_fwd_kernel<128, 64, 128><<<n, 256, 0, P.stream>>>(L);
    return hipGetLastError();
}

}  // namespace kda
