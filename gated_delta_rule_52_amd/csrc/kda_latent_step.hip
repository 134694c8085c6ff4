// kda_latent_step.hip - latent attention of one token per sequence over the paged cache, in the absorbed form: the
// cached row [c | r] is key and value of every head,
//     o_h = sum_j p_hj c_j,   p_hj = exp(s_hj - lse_h),   s_hj = scale (q_latent_h . c_j + q_rope_h . r_j).
#include "kda_latent.h"

namespace kda {
namespace {

using namespace la;

constexpr int kRopePad = 64;  // elements that r is padded to

// Keys per tile: 32 rows of 576 bf16, or 16 of fp32, are 36 KiB; two tiles let two workgroups share a CU.
template <class E>
constexpr int kTileKeys = sizeof(E) == 2 ? 32 : 16;

// A workgroup of four waves takes 16 HT heads of a sequence over one of `splits` runs of its keys.  The scores of a tile
// are shared out over the waves by heads (and by 16 keys where there are fewer than four tiles of heads), the products
// with the values by columns, so each wave's accumulators hold DLP / 4 columns of all the heads.
template <class E, int DLP, int HT>
__global__ __launch_bounds__(256, 2) void latent_step_kernel(const LatentStepLaunch P) {
    constexpr int BN = kTileKeys<E>, KT = BN / 16, KW = 4 / HT;  // tiles of 16 keys; waves that share a tile of heads
    constexpr int KPW = KT > KW ? KT / KW : 1;                   // tiles of keys per wave
    constexpr int KC = 4 * Mx<E>::PER, SL = DLP / KC, SR = kRopePad / KC, CT = DLP / 64;
    using LT = LdsTile<DLP, E>;
    using RT = LdsTile<kRopePad, E>;
    constexpr int OR = BN * LT::ROW, OM = OR + BN * RT::ROW, BUF = OM + BN * 4;
    constexpr int RPW = BN / 4;                // rows that a wave fetches
    constexpr int PROW = BN * sizeof(E) + 16;  // a head's weights, padded off the banks of the next
    __shared__ __attribute__((aligned(1024))) char lds[2 * BUF];
    __shared__ __attribute__((aligned(16))) char weights[HT * 16 * PROW];
    __shared__ float tops[HT * 16 * KW];

    const int n = blockIdx.z, h0 = blockIdx.y * HT * 16, split = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, col = lane & 15;
    const int length = P.pages.rows(P.lengths[n]);
    const int tiles = length > 0 ? (length - 1) / BN + 1 : 0;
    const int per = (tiles + P.splits - 1) / P.splits;
    const int t0 = min(tiles, split * per), t1 = min(tiles, t0 + per);

    const int ht = wave % HT, kt0 = wave / HT * KPW;  // the wave's share of the scores
    const bool scores = kt0 < KT;
    typename Mx<E>::frag qf[SL + SR];
    {
        const int h = h0 + 16 * ht + col;
        const bool live = h < P.H;
        const E *ql = static_cast<const E *>(P.ql.p) + n * P.ql.stride + (live ? h : 0) * P.ql.head_stride;
        const E *qr = static_cast<const E *>(P.qr.p) + n * P.qr.stride + (live ? h : 0) * P.qr.head_stride;
#pragma unroll
        for (int s = 0; s < SL; ++s) {
            const int c = (4 * s + g) * Mx<E>::PER;
            qf[s] = live && c < P.dl ? *reinterpret_cast<const typename Mx<E>::frag *>(ql + c) : Mx<E>::zero();
        }
#pragma unroll
        for (int s = 0; s < SR; ++s) {
            const int c = (4 * s + g) * Mx<E>::PER;
            qf[SL + s] = live && c < P.dr ? *reinterpret_cast<const typename Mx<E>::frag *>(qr + c) : Mx<E>::zero();
        }
    }

    // Lane i < RPW finds the wave's i-th row of a tile: its place in the cache, or none behind the sequence's end or on
    // a page that does not exist.
    const int64_t width = (P.dl + P.dr) * static_cast<int64_t>(sizeof(E));
    auto find = [&](int tile) -> int64_t {
        const int pos = tile * BN + wave * RPW + (lane < RPW ? lane : 0);
        return tile < t1 && pos < length ? P.pages.at(n, pos) : -1;
    };
    auto fetch = [&](int64_t row, char *to) {
        if (lane < RPW) reinterpret_cast<float *>(to + OM)[wave * RPW + lane] = row < 0 ? neg_inf() : 0.f;
#pragma unroll
        for (int i = 0; i < RPW; ++i) {
            const int lo = __builtin_amdgcn_readlane(static_cast<int>(row), i), hi = __builtin_amdgcn_readlane(static_cast<int>(row >> 32), i);
            const int64_t at = static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32 | static_cast<uint32_t>(lo));
            const bool there = at >= 0;
            const char *p = static_cast<const char *>(P.cache) + (there ? at * width : 0);
            const rsrc_t rl = buffer(p, there ? P.dl * sizeof(E) : 0), rr = buffer(p + P.dl * sizeof(E), there ? P.dr * sizeof(E) : 0);
            const int r = wave * RPW + i;
#pragma unroll
            for (int u = 0; u < LT::UNITS; u += 64) {
                if (LT::UNITS >= 64 || lane < LT::UNITS) {
                    const int unit = (u + lane) ^ LT::swz(r);
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(rl, (lds_ptr)(to + r * LT::ROW + u * 16), 16, unit * 16, 0, 0, 0);
                }
            }
            if (lane < RT::UNITS) {
                const int unit = lane ^ RT::swz(r);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rr, (lds_ptr)(to + OR + r * RT::ROW), 16, unit * 16, 0, 0, 0);
            }
        }
    };

    f4 acc[HT][CT];
#pragma unroll
    for (int a = 0; a < HT; ++a)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[a][c] = f4{0, 0, 0, 0};
    float m[HT], l = 0.f;  // the heads' reference points (head `col` of each tile of heads) in powers of two; the wave's own sum
#pragma unroll
    for (int a = 0; a < HT; ++a) m[a] = neg_inf();
    const float c2 = P.scale * kLog2e;

    if (t0 < t1) fetch(find(t0), lds);
    int64_t next = find(t0 + 1);
    int buf = 0;
    for (int tile = t0; tile < t1; ++tile, buf ^= 1) {
        loads_landed();
        const char *t = lds + buf * BUF;
        if (tile + 1 < t1) fetch(next, lds + (buf ^ 1) * BUF);
        next = find(tile + 2);
        f4 s[KPW];
        if (scores) {
            float top = neg_inf();
#pragma unroll
            for (int b = 0; b < KPW; ++b) {
                s[b] = f4{0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < SL; ++k) s[b] = Mx<E>::mma16(LT::rows16(t, 16 * (kt0 + b), k, lane), qf[k], s[b]);
#pragma unroll
                for (int k = 0; k < SR; ++k) s[b] = Mx<E>::mma16(RT::rows16(t + OR, 16 * (kt0 + b), k, lane), qf[SL + k], s[b]);
                const f4 mask = *reinterpret_cast<const f4 *>(t + OM + (16 * (kt0 + b) + 4 * g) * 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[b][i] = mask[i] < 0.f ? neg_inf() : s[b][i] * c2;
                    top = fmaxf(top, s[b][i]);
                }
            }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            if (g == 0) tops[(16 * ht + col) * KW + wave / HT] = top;
        }
        __syncthreads();
        bool moved = false;
        float by[HT];
#pragma unroll
        for (int a = 0; a < HT; ++a) {
            float top = neg_inf();
#pragma unroll
            for (int k = 0; k < (KT < KW ? KT : KW); ++k) top = fmaxf(top, tops[(16 * a + col) * KW + k]);
            // the reference point follows the maximum only when it lags by 2^8 (as in the prompts' kernel)
            const bool move = top > m[a] + 8.f;
            by[a] = move ? exp2_f(m[a] - top) : 1.f;
            if (a == ht) l *= by[a];
            m[a] = move ? top : m[a];
            moved |= move;
        }
        if (scores) {
            float at = m[0];
#pragma unroll
            for (int a = 1; a < HT; ++a) at = a == ht ? m[a] : at;
            at = at == neg_inf() ? 0.f : at;
            E *to = reinterpret_cast<E *>(weights + (16 * ht + col) * PROW);
#pragma unroll
            for (int b = 0; b < KPW; ++b) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[b][i] = exp2_f(s[b][i] - at);
                    l += s[b][i];
                }
                store4(to, 16 * (kt0 + b) + 4 * g, sizeof(E) == 2, s[b][0], s[b][1], s[b][2], s[b][3]);
            }
        }
        if (__any(moved)) {
#pragma unroll
            for (int a = 0; a < HT; ++a)
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[a][c][i] *= by[a];
        }
        __syncthreads();
        typename Mx<E>::frag p[HT];
#pragma unroll
        for (int a = 0; a < HT; ++a) p[a] = *reinterpret_cast<const typename Mx<E>::frag *>(weights + (16 * a + col) * PROW + 16 * g);
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            const typename Mx<E>::frag v = LT::cols16(t, 0, wave * (DLP / 4) + 16 * c, lane);
#pragma unroll
            for (int a = 0; a < HT; ++a) acc[a][c] = Mx<E>::mma16(v, p[a], acc[a][c]);
        }
    }

    // the heads' sums: over the quarters of a wave, then over the waves that share a tile of heads
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    __syncthreads();
    if (scores && g == 0) tops[(16 * ht + col) * KW + wave / HT] = l;
    __syncthreads();
    const bool whole = P.splits == 1;
    float *part = P.ws, *part_lse = P.ws + static_cast<int64_t>(P.N) * P.H * P.splits * P.dl;
#pragma unroll
    for (int a = 0; a < HT; ++a) {
        const int h = h0 + 16 * a + col;
        if (h >= P.H) continue;
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < (KT < KW ? KT : KW); ++k) sum += tops[(16 * a + col) * KW + k];
        const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;  // NaN stays
        const int64_t head = static_cast<int64_t>(n) * P.H + h;
        const float lse = sum == 0.f ? neg_inf() : (m[a] + __log2f(sum)) * kLn2;
        if (wave == 0 && g == 0) {
            if (!whole) part_lse[head * P.splits + split] = lse;
            else if (P.lse) P.lse[head] = lse;
        }
        void *to = whole ? P.o.p : part;
        const int64_t at = whole ? n * P.o.stride + h * P.o.head_stride : (head * P.splits + split) * P.dl;
        if (whole || sum != 0.f) {  // an empty run's part is not read
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const int d = wave * (DLP / 4) + 16 * c + 4 * g;
                if (d < P.dl) store4(to, at + d, whole && P.out_bf16, acc[a][c][0] * inv, acc[a][c][1] * inv, acc[a][c][2] * inv, acc[a][c][3] * inv);
            }
        }
    }
}

// Joins the runs of a (sequence, head): o = sum_s exp(lse_s - lse) o_s, lse = log sum_s exp(lse_s).
__global__ __launch_bounds__(128) void latent_join_kernel(const LatentStepLaunch P) {
    const int64_t head = blockIdx.x;
    const int n = static_cast<int>(head / P.H), h = static_cast<int>(head % P.H);
    const float *lses = P.ws + static_cast<int64_t>(P.N) * P.H * P.splits * P.dl + head * P.splits;
    const float *part = P.ws + head * P.splits * P.dl;
    float top = neg_inf(), sum = 0.f;
    bool bad = false;
    for (int s = 0; s < P.splits; ++s) {
        top = fmaxf(top, lses[s]);
        bad |= lses[s] != lses[s];
    }
    if (top != neg_inf())
        for (int s = 0; s < P.splits; ++s) sum += exp2_f((lses[s] - top) * kLog2e);
    if (bad) sum = __builtin_nanf("");
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    for (int d = 4 * threadIdx.x; d < P.dl; d += 512) {
        f4 x = {0, 0, 0, 0};
        for (int s = 0; s < P.splits; ++s) {
            if (lses[s] == neg_inf()) continue;
            x += *reinterpret_cast<const f4 *>(part + static_cast<int64_t>(s) * P.dl + d) * (exp2_f((lses[s] - top) * kLog2e) * inv);
        }
        store4(P.o.p, n * P.o.stride + h * P.o.head_stride + d, P.out_bf16, x[0], x[1], x[2], x[3]);
    }
    if (threadIdx.x == 0 && P.lse) P.lse[head] = sum == 0.f ? neg_inf() : top + __log2f(sum) * kLn2;
}

// Tiles of 16 heads per workgroup.
int head_tiles(int H, bool bf16) { return H <= 16 ? 1 : H <= 32 || !bf16 ? 2 : 4; }
int head_groups(int H, bool bf16) {
    const int per = 16 * head_tiles(H, bf16);
    return (H + per - 1) / per;
}

template <class E, int DLP, int HT>
void launch(const LatentStepLaunch &P) {
    const dim3 grid(P.splits, (P.H + 16 * HT - 1) / (16 * HT), P.N);
    latent_step_kernel<E, DLP, HT><<<grid, 256, 0, P.stream>>>(P);
}
template <class E, int HT>
void launch_dl(const LatentStepLaunch &P) {
    if (P.dl <= 128) launch<E, 128, HT>(P);
    else if (P.dl <= 256) launch<E, 256, HT>(P);
    else launch<E, 512, HT>(P);
}

}  // namespace

// Runs per sequence: as many as give every CU two workgroups, of at least 64 keys each.
int latent_step_splits(int N, int H, int dl, int64_t longest, bool bf16) {
    const int64_t groups = static_cast<int64_t>(N) * head_groups(H, bf16);
    int64_t s = groups > 0 ? (512 + groups - 1) / groups : 1;
    const int64_t most = (longest + 63) / 64;
    s = s < most ? s : most;
    return s < 1 ? 1 : static_cast<int>(s);
}
size_t latent_step_workspace_bytes(int N, int H, int dl, int splits) {
    return splits == 1 ? 0 : static_cast<size_t>(N) * H * splits * (static_cast<size_t>(dl) + 1) * 4;
}
int64_t latent_step_threads(int N, int H, bool bf16, int splits) {
    const int64_t step = static_cast<int64_t>(splits) * head_groups(H, bf16) * N * 256, join = static_cast<int64_t>(N) * H * 128;
    return step > join ? step : join;
}

hipError_t launch_latent_step(const LatentStepLaunch &P) {
    const int tiles = head_tiles(P.H, P.bf16);
    if (P.bf16) {
        if (tiles == 1) launch_dl<uint16_t, 1>(P);
        else if (tiles == 2) launch_dl<uint16_t, 2>(P);
        else launch_dl<uint16_t, 4>(P);
    } else {
        if (tiles == 1) launch_dl<float, 1>(P);
        else launch_dl<float, 2>(P);
    }
    if (P.splits > 1) latent_join_kernel<<<static_cast<unsigned>(P.N * static_cast<int64_t>(P.H)), 128, 0, P.stream>>>(P);
    return hipGetLastError();
}

}  // namespace kda
