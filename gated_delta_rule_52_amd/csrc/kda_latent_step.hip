// kda_latent_step.hip - latent attention of one token per sequence over the paged cache, in the absorbed form: the
// cached row [c | r] is key and value of every head,
//     o_h = sum_j p_hj c_j,   p_hj = exp(s_hj - lse_h),   s_hj = scale (q_latent_h . c_j + q_rope_h . r_j).
#include "kda_latent.h"

namespace kda {
namespace {

using namespace la;

constexpr int kRopePad = 64;  // elements that r is padded to

// How a workgroup is made up: HT tiles of 16 heads, W waves, tiles of BN keys.  Two tiles of 32 bf16 keys (16 of fp32) are
// 72 KiB, so two workgroups share a CU; with four tiles of heads one workgroup of eight waves fills it.
template <int HT>
constexpr int kWaves = HT == 4 ? 8 : 4;
template <class E, int HT>
struct Shape {
    static constexpr int W = kWaves<HT>, BN = HT == 4 ? 64 : sizeof(E) == 2 ? 32 : 16;
    static constexpr int KT = BN / 16, KG = KT < W / HT ? KT : W / HT, KPW = KT / KG;  // tiles of 16 keys, and who scores them
};

// How the tiles of all sequences are shared out: workgroup w takes tiles w * per .. + per - 1 of the sequences' tiles laid end
// to end.  A sequence that one workgroup has whole gets its result from it; of the others each workgroup leaves a part,
// in slot 2 w + 1 where the sequence begins in its run and in slot 2 w where it does not, and the sequence's first
// workgroup notes which workgroups they are.
struct Parts {
    float *o;    // [slots, heads of a group, dl]
    float *lse;  // [slots, heads of a group]
    int2 *span;  // [groups, N]: first and last workgroup
    __device__ __forceinline__ Parts(const LatentStepLaunch &P, int group, int groups, int heads) {
        const int64_t slots = 2 * static_cast<int64_t>(P.splits);
        o = P.ws + group * slots * heads * P.dl;
        lse = P.ws + groups * slots * heads * P.dl + group * slots * heads;
        span = reinterpret_cast<int2 *>(P.ws + groups * slots * heads * (P.dl + 1)) + static_cast<int64_t>(group) * P.N;
    }
};

// Sum over the threads in front of this one, and over all of them.
template <int W>
__device__ __forceinline__ int scan(int x, int *shared, int &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int y = x;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int z = __shfl_up(y, d);
        if (lane >= d) y += z;
    }
    if (lane == 63) shared[wave] = y;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        before += i < wave ? shared[i] : 0;
        total += shared[i];
    }
    return before + y - x;
}

// A workgroup's four or eight waves share the scores of a tile by heads (and by keys where there are fewer tiles of heads
// than waves) and the products with the values by columns: every accumulator then holds columns of all heads, and a
// value read from LDS serves all of them.  The weights, and the maxima of the waves that share heads, go through LDS.
template <class E, int DLP, int HT>
__global__ __launch_bounds__(64 * kWaves<HT>, sizeof(E) == 2 ? 2 : 1) void latent_step_kernel(const LatentStepLaunch P) {
    using S = Shape<E, HT>;
    constexpr int BN = S::BN, KG = S::KG, KPW = S::KPW, W = S::W;
    constexpr int KC = 4 * Mx<E>::PER, SL = DLP / KC, SR = kRopePad / KC, CT = DLP / (16 * W), ST = BN / KC;
    using LT = LdsTile<DLP, E, 16>;
    using RT = LdsTile<kRopePad, E, 16>;
    constexpr int OR = BN * LT::ROW, OM = OR + BN * RT::ROW, BUF = OM + BN * 4;
    constexpr int RPW = BN / W;                // rows that a wave fetches
    constexpr int AUX = sizeof(E) == 2 && HT <= 2 ? 2 : 0;  // rows that one workgroup reads once pass the caches by (non-temporal)
    constexpr int PROW = BN * sizeof(E) + 16;  // a head's weights, padded off the banks of the next
    __shared__ __attribute__((aligned(1024))) char lds[2 * BUF];
    __shared__ __attribute__((aligned(16))) char weights[HT * 16 * PROW];
    __shared__ float tops[HT * 16 * KG];
    __shared__ int shared[W + 2];

    const int w = blockIdx.x, group = blockIdx.y, h0 = group * HT * 16;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, col = lane & 15;
    auto tiles_of = [&](int n) {
        const int rows = P.pages.rows(P.lengths[n]);
        return rows > 0 ? (rows - 1) / BN + 1 : 0;
    };

    // the workgroup's run, and the sequence it begins in
    int n, before, left, run;  // sequence, tiles of it in front of the run, tiles left in the run; tiles of a whole run
    if (P.splits == 0) {       // a workgroup per sequence
        n = w, before = 0, left = run = tiles_of(w);
    } else {
        const int chunk = (P.N + (64 * W) - 1) / (64 * W), first = min(P.N, static_cast<int>(threadIdx.x) * chunk);
        int mine = 0, total;
        for (int i = first; i < min(P.N, first + chunk); ++i) mine += tiles_of(i);
        const int at = scan<W>(mine, shared, total);
        run = max(1, (total + P.splits - 1) / P.splits);
        const int64_t from = static_cast<int64_t>(w) * run;
        left = static_cast<int>(min(static_cast<int64_t>(run), total - from));
        if (left <= 0) return;
        const int lo = static_cast<int>(from);
        if (lo >= at && lo < at + mine) {
            int i = first, b = at;
            for (int t; i + 1 < P.N && lo >= b + (t = tiles_of(i)); ++i) b += t;
            shared[W] = i;
            shared[W + 1] = lo - b;
        }
        __syncthreads();
        n = __builtin_amdgcn_readfirstlane(shared[W]);
        before = __builtin_amdgcn_readfirstlane(shared[W + 1]);
    }

    const int ht = wave % HT, kt0 = wave / HT * KPW;  // the wave's share of the scores
    const bool scores = wave / HT < KG;
    const int64_t width = (P.dl + P.dr) * static_cast<int64_t>(sizeof(E));
    const uint32_t row_bytes = static_cast<uint32_t>(width), latent_bytes = P.dl * sizeof(E);
    const int own = wave + W * (lane < RPW ? lane : 0);
    const float c2 = P.scale * kLog2e;

    for (bool more = true; more; ) {
        const int length = P.pages.rows(P.lengths[n]), tiles = length > 0 ? (length - 1) / BN + 1 : 0;
        const int t0 = before, t1 = min(tiles, before + left);
        // Of a tile's rows a wave fetches wave + W i, and lane i < RPW looks after the i-th of them.  A block's number is read a tile ahead of the loads
        // that need it, and before those of the tile in between: a wait for it must not wait for them.
        auto block_of = [&](int tile) {
            const int pos = tile * BN + own;
            return tile < t1 && pos < length ? P.pages.block(n, pos) : -1;
        };
        // the row's place in the cache in bytes, -1 behind the sequence's end or on a page that does not exist
        auto place = [&](int tile, int block) -> int64_t {
            const int64_t row = P.pages.row(block, tile * BN + own);
            return row < 0 ? -1 : row * width;
        };
        auto fetch = [&](int64_t at, char *to, int lane) {
            if (lane < RPW) reinterpret_cast<float *>(to + OM)[own] = at < 0 ? neg_inf() : 0.f;
#pragma unroll
            for (int i = 0; i < RPW; ++i) {
                const int r = wave + W * i;
                const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(at), i);
                const int hi = __builtin_amdgcn_readlane(static_cast<int>(at >> 32), i);
                // no bytes, so zeros, where there is no row
                const rsrc_t row = buffer(static_cast<const char *>(P.cache) + (static_cast<int64_t>(hi) << 32 | lo), row_bytes & ~(hi >> 31));
#pragma unroll
                for (int u = 0; u < LT::UNITS; u += 64) {
                    if (LT::UNITS >= 64 || lane < LT::UNITS) {
                        const uint32_t off = static_cast<uint32_t>((u + lane) ^ LT::swz(r)) * 16;
                        __builtin_amdgcn_raw_ptr_buffer_load_lds(row, (lds_ptr)(to + r * LT::ROW + u * 16), 16, static_cast<int>(off < latent_bytes ? off : kOutside), 0, 0, AUX);
                    }
                }
                if (lane < RT::UNITS)
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(row, (lds_ptr)(to + OR + r * RT::ROW), 16, static_cast<int>(latent_bytes + (lane ^ RT::swz(r)) * 16), 0, 0, AUX);
            }
        };

        int block = block_of(t0);
        {
            const int64_t first = place(t0, block);
            block = block_of(t0 + 1);
            if (t0 < t1) fetch(first, lds, lane);
        }
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
        f4 acc[HT][CT];
#pragma unroll
        for (int a = 0; a < HT; ++a)
#pragma unroll
            for (int c = 0; c < CT; ++c) acc[a][c] = f4{0, 0, 0, 0};
        // the heads' reference points (head `col` of each tile of heads) in powers of two; the wave's own part of the sum
        float m[HT], l = 0.f;
#pragma unroll
        for (int a = 0; a < HT; ++a) m[a] = neg_inf();

        int buf = 0;
        for (int tile = t0; tile < t1; ++tile, buf ^= 1) {
            loads_landed();
            const char *t = lds + buf * BUF;
            const int64_t next = place(tile + 1, block);
            block = block_of(tile + 2);
            const int lane_ = afresh(lane), g_ = lane_ >> 4;
            if (tile + 1 < t1) fetch(next, lds + (buf ^ 1) * BUF, lane_);
            f4 s[KPW];
            if (scores) {
                float top = neg_inf();
#pragma unroll
                for (int b = 0; b < KPW; ++b) s[b] = f4{0, 0, 0, 0};
                pipelined<typename Mx<E>::frag, (SL + SR) * KPW, 6>(
                    [&](int i) {
                        const int k = i / KPW, b = i % KPW;
                        return k < SL ? LT::rows16(t, 16 * (kt0 + b), k, lane_) : RT::rows16(t + OR, 16 * (kt0 + b), k - SL, lane_);
                    },
                    [&](int i, typename Mx<E>::frag f) { s[i % KPW] = Mx<E>::mma16(f, qf[i / KPW], s[i % KPW]); });
#pragma unroll
                for (int b = 0; b < KPW; ++b) {
                    const f4 mask = *reinterpret_cast<const f4 *>(t + OM + (16 * (kt0 + b) + 4 * g_) * 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s[b][i] = mask[i] < 0.f ? neg_inf() : s[b][i] * c2;
                        top = fmaxf(top, s[b][i]);
                    }
                }
                top = quarters_max(top);
                if (g == 0) tops[(16 * ht + col) * KG + wave / HT] = top;
            }
            lds_barrier();
            bool moved = false;
            float by[HT];
#pragma unroll
            for (int a = 0; a < HT; ++a) {
                float top = neg_inf();
#pragma unroll
                for (int k = 0; k < KG; ++k) top = fmaxf(top, tops[(16 * a + col) * KG + k]);
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
                // in the order in which a step's operand takes them: of each 32 keys, 4 g .. + 3 of either half together
                char *to = weights + (16 * ht + col) * PROW + g_ * 16;
#pragma unroll
                for (int b = 0; b < KPW; ++b) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s[b][i] = exp2_f(s[b][i] - at);
                        l += s[b][i];
                    }
                    const int kt = kt0 + b;
                    store4(to + (sizeof(E) == 2 ? (kt >> 1) * 64 + (kt & 1) * 8 : kt * 64), 0, sizeof(E) == 2, s[b][0], s[b][1], s[b][2], s[b][3]);
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
            lds_barrier();
            typename Mx<E>::frag p[ST][HT];
#pragma unroll
            for (int k = 0; k < ST; ++k)
#pragma unroll
                for (int a = 0; a < HT; ++a) p[k][a] = *reinterpret_cast<const typename Mx<E>::frag *>(weights + (16 * a + col) * PROW + 64 * k + 16 * g_);
            pipelined<typename Mx<E>::frag, ST * CT, 4>(
                [&](int i) { return LT::cols16(t, i / CT * KC, wave * (DLP / W) + 16 * (i % CT), lane_); },
                [&](int i, typename Mx<E>::frag v) {
#pragma unroll
                    for (int a = 0; a < HT; ++a) acc[a][i % CT] = Mx<E>::mma16(v, p[i / CT][a], acc[a][i % CT]);
                });
        }

        // the heads' sums: over the quarters of a wave, then over the waves that share a tile of heads
        l = quarters_sum(l);
        __syncthreads();
        if (scores && g == 0) tops[(16 * ht + col) * KG + wave / HT] = l;
        __syncthreads();
        const bool whole = t0 == 0 && t1 == tiles;
        const Parts parts(P, group, gridDim.y, HT * 16);
        const int64_t slot = 2 * static_cast<int64_t>(w) + (t0 == 0);
        if (P.splits && t0 == 0 && threadIdx.x == 0) {  // the run that ends this sequence
            const int rest = tiles - (t1 - t0);
            parts.span[n] = int2{w, w + (rest + run - 1) / run};
        }
#pragma unroll
        for (int a = 0; a < HT; ++a) {
            const int h = h0 + 16 * a + col;
            if (h >= P.H) continue;
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < KG; ++k) sum += tops[(16 * a + col) * KG + k];
            const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;  // NaN stays
            const float lse = sum == 0.f ? neg_inf() : (m[a] + __log2f(sum)) * kLn2;
            if (wave == 0 && g == 0) {
                if (!whole) parts.lse[slot * (HT * 16) + 16 * a + col] = lse;
                else if (P.lse) P.lse[static_cast<int64_t>(n) * P.H + h] = lse;
            }
            void *to = whole ? P.o.p : parts.o;
            const int64_t at = whole ? n * P.o.stride + h * P.o.head_stride : (slot * (HT * 16) + 16 * a + col) * P.dl;
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                const int d = wave * (DLP / W) + 16 * c + 4 * g;
                if (d < P.dl) store4(to, at + d, whole && P.out_bf16, acc[a][c][0] * inv, acc[a][c][1] * inv, acc[a][c][2] * inv, acc[a][c][3] * inv);
            }
        }
        left -= t1 - t0;
        more = P.splits && left > 0;
        if (more) {
            ++n, before = 0;
            while (n < P.N && tiles_of(n) == 0) ++n;
            if (n >= P.N) return;
            __syncthreads();  // the sums are read before the next sequence's maxima are written
        }
    }
}

// Joins the parts of a (sequence, head): o = sum_s exp(lse_s - lse) o_s, lse = log sum_s exp(lse_s).  Sequences without rows
// get zeros here.  COLS columns per workgroup, COLS / 4 threads of four by those that share the parts out.
constexpr int kJoinParts = 512;
template <int COLS>
__global__ __launch_bounds__(256) void latent_join_kernel(const LatentStepLaunch P, int heads, int groups) {
    __shared__ float weight[kJoinParts];
    constexpr int T = COLS / 4, Q = 256 / T;
    __shared__ f4 sums[Q][T];
    __shared__ float2 stats[4];
    const int n = blockIdx.x / P.H, h = blockIdx.x % P.H, group = h / heads, hh = h % heads;
    const int64_t head = static_cast<int64_t>(n) * P.H + h, out = n * P.o.stride + h * P.o.head_stride;
    const int t = threadIdx.x % T, q = threadIdx.x / T, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = blockIdx.y * COLS + 4 * t;
    const Parts parts(P, group, groups, heads);
    int2 span = int2{0, -1};
    if (P.pages.rows(P.lengths[n]) > 0) {
        span = parts.span[n];
        if (span.x == span.y) return;
    }
    // part i of the sequence: slot 2 w + 1 of its first workgroup, slots 2 w of the others
    auto slot = [&](int i) { return (2 * static_cast<int64_t>(span.x + i) + (i == 0)) * heads + hh; };
    const int count = min(span.y - span.x + 1, kJoinParts);
    float lse[2], top = neg_inf(), sum = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int i = threadIdx.x + 256 * k;
        lse[k] = i < count ? parts.lse[slot(i)] : neg_inf();
        top = fmaxf(top, lse[k]);
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
    if (lane == 0) stats[wave].x = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) top = fmaxf(top, stats[i].x);
    const float at = top == neg_inf() ? 0.f : top;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float w = exp2_f((lse[k] - at) * kLog2e);
        weight[threadIdx.x + 256 * k] = w;
        sum += w;
    }
    sum = wave_sum(sum);
    if (lane == 0) stats[wave].y = sum;
    __syncthreads();
    sum = (stats[0].y + stats[1].y) + (stats[2].y + stats[3].y);
    f4 x = {0, 0, 0, 0};
    if (col < P.dl) {
#pragma unroll 4
        for (int i = q; i < count; i += Q) x += *reinterpret_cast<const f4 *>(parts.o + slot(i) * P.dl + col) * weight[i];
    }
    sums[q][t] = x;
    __syncthreads();
    if (q == 0 && col < P.dl) {
#pragma unroll
        for (int i = 1; i < Q; ++i) x += sums[i][t];
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        store4(P.o.p, out + col, P.out_bf16, x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    }
    if (threadIdx.x == 0 && blockIdx.y == 0 && P.lse) P.lse[head] = sum == 0.f ? neg_inf() : at + __log2f(sum) * kLn2;
}

// Tiles of 16 heads per workgroup, and groups of so many heads.
int head_tiles(int H, bool bf16) { return H <= 16 ? 1 : H <= 32 || !bf16 ? 2 : 4; }
int head_groups(int H, bool bf16) {
    const int per = 16 * head_tiles(H, bf16);
    return (H + per - 1) / per;
}

template <class E, int DLP, int HT>
void launch(const LatentStepLaunch &P) {
    const dim3 grid(P.splits ? P.splits : P.N, (P.H + 16 * HT - 1) / (16 * HT));
    latent_step_kernel<E, DLP, HT><<<grid, 64 * kWaves<HT>, 0, P.stream>>>(P);
}
template <class E, int HT>
void launch_dl(const LatentStepLaunch &P) {
    if (P.dl <= 128) launch<E, 128, HT>(P);
    else if (P.dl <= 256) launch<E, 256, HT>(P);
    else launch<E, 512, HT>(P);
}
template <class E>
void launch_heads(const LatentStepLaunch &P) {
    const int tiles = head_tiles(P.H, P.bf16);
    if (tiles == 1) launch_dl<E, 1>(P);
    else if (tiles == 2) launch_dl<E, 2>(P);
    else if constexpr (sizeof(E) == 2) launch_dl<E, 4>(P);
}

}  // namespace

// Workgroups over which the sequences' tiles are shared out: what the CUs hold at once (two workgroups each, one where it has eight
// waves), no more than there can be pairs of tiles.  0: a workgroup per sequence, where there are many.
int latent_step_splits(int N, int H, int dl, int64_t longest, bool bf16) {
    const int groups = head_groups(H, bf16), tiles = head_tiles(H, bf16);
    if (N >= 1024) return 0;
    int64_t s = (tiles == 4 ? 256 : kJoinParts) / groups;
    const int64_t most = static_cast<int64_t>(N) * ((longest + 31) / 32);
    s = s < most ? s : most;
    return s < 1 ? 1 : static_cast<int>(s);
}
size_t latent_step_workspace_bytes(int N, int H, int dl, int splits, bool bf16) {
    const size_t groups = head_groups(H, bf16), heads = 16 * head_tiles(H, bf16);
    return splits == 0 ? 0 : groups * 2 * splits * heads * (static_cast<size_t>(dl) + 1) * 4 + groups * N * sizeof(int2);
}
int64_t latent_step_threads(int N, int H, bool bf16, int splits) {
    const int64_t step = static_cast<int64_t>(splits ? splits : N) * head_groups(H, bf16) * 512, join = static_cast<int64_t>(N) * H * 256;
    return step > join ? step : join;
}

hipError_t launch_latent_step(const LatentStepLaunch &P) {
    if (P.bf16) launch_heads<uint16_t>(P);
    else launch_heads<float>(P);
    if (P.splits) {
        const int64_t rows = P.N * static_cast<int64_t>(P.H);
        const int heads = 16 * head_tiles(P.H, P.bf16), groups = head_groups(P.H, P.bf16);
        // All columns at once where there are rows enough for every CU (64 sequences of 32 heads JOIN_A), a quarter where a few rows
        // have many parts (one sequence of 65,536 rows JOIN_B).
        if (rows >= 512) latent_join_kernel<512><<<static_cast<unsigned>(rows), 256, 0, P.stream>>>(P, heads, groups);
        else latent_join_kernel<128><<<dim3(static_cast<unsigned>(rows), (P.dl + 127) / 128), 256, 0, P.stream>>>(P, heads, groups);
    }
    return hipGetLastError();
}

}  // namespace kda
