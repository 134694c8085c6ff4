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
    static constexpr int KT = BN / 16, KG = KT < W / HT ? KT : W / HT, KPW = KT / KG;  // tiles of 16 keys; KG waves score a tile of heads
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

// A tile of a sequence: its number in it, and the sequence's rows.
struct Where {
    int n, tile, length;
};
template <int BN>
struct Tiles {
    const LatentStepLaunch &P;
    __device__ __forceinline__ static int of(int length) { return pieces(length, BN); }
    __device__ __forceinline__ int length(int n) const { return P.pages.rows(P.lengths[n]); }
    __device__ __forceinline__ void next(Where &x) const {
        if (++x.tile < of(x.length)) return;
        x.tile = 0;
        do {
            x.length = ++x.n < P.N ? length(x.n) : 0;
        } while (x.n < P.N && x.length == 0);
    }
    // The tile where workgroup w's run begins; `left` tiles in it, `run` in a whole one.
    template <int W>
    __device__ __forceinline__ Where first(int w, int *shared, int &left, int &run) const {
        Where x{w, 0, 0};
        if (P.splits == 0) {  // a workgroup per sequence
            x.length = length(w);
            left = run = of(x.length);
            return x;
        }
        const int chunk = (P.N + 64 * W - 1) / (64 * W), from = min(P.N, static_cast<int>(threadIdx.x) * chunk);
        int mine = 0, total;
        for (int i = from; i < min(P.N, from + chunk); ++i) mine += of(length(i));
        const int at = scan<W>(mine, shared, total);
        const TileRun part(total, P.splits, w);
        run = part.run;
        left = part.left;
        const int lo = part.begin;
        if (left > 0 && lo >= at && lo < at + mine) {
            int i = from, b = at, rows = length(i);
            while (i + 1 < P.N && lo >= b + of(rows)) {
                b += of(rows);
                rows = length(++i);
            }
            shared[W] = i;
            shared[W + 1] = lo - b;
            shared[W + 2] = rows;
        }
        __syncthreads();
        if (left > 0) {
            x.n = __builtin_amdgcn_readfirstlane(shared[W]);
            x.tile = __builtin_amdgcn_readfirstlane(shared[W + 1]);
            x.length = __builtin_amdgcn_readfirstlane(shared[W + 2]);
        }
        return x;
    }
};

// How W waves bring tiles of BN rows into LDS: latent parts, rotated parts, and 0 or -infinity for a row that is there or not.
template <class E, int DLP, int W, int BN, int AUX>
struct Fetch {
    using LT = LdsTile<DLP, E, 16>;
    using RT = LdsTile<kRopePad, E, 16>;
    static constexpr int OR = BN * LT::ROW, OM = OR + BN * RT::ROW, BUF = OM + BN * 4, RPW = BN / W;
    const LatentStepLaunch &P;
    int wave;
    uint32_t latent, row;  // bytes
    __device__ __forceinline__ Fetch(const LatentStepLaunch &P_, int wave_)
        : P(P_), wave(wave_), latent(P_.dl * sizeof(E)), row((P_.dl + P_.dr) * sizeof(E)) {}
    // of a tile's rows a wave fetches RPW that follow each other, and RT::UNITS lanes look after each
    __device__ __forceinline__ int own(int lane) const { return wave * RPW + min(lane / RT::UNITS, RPW - 1); }
    // the block of the lane's row; read a tile ahead of the loads that need it, and before those of the tile in between: a
    // wait for it must not wait for them
    __device__ __forceinline__ int block(const Where &x, int lane) const {
        const int pos = x.tile * BN + own(lane);
        return pos < x.length ? P.pages.block(x.n, pos) : -1;
    }
    // its place in the cache in bytes, -1 behind the sequence's end or on a page that does not exist
    __device__ __forceinline__ int64_t place(const Where &x, int block, int lane) const {
        const int64_t r = P.pages.row(block, x.tile * BN + own(lane));
        return r < 0 ? -1 : r * row;
    }
    // What a load leaves out of the rotated part's columns stays zero.
    __device__ __forceinline__ void clear(char *buffers) const {
        if (P.dr == kRopePad) return;
        for (int b = 0; b < 2; ++b)
            for (int i = threadIdx.x * 16; i < BN * RT::ROW; i += 64 * W * 16) *reinterpret_cast<f4 *>(buffers + b * BUF + OR + i) = f4{0, 0, 0, 0};
        __syncthreads();
    }
    // Latent parts of the wave's rows from the first one to the last.
    template <int FIRST, int LAST>
    __device__ __forceinline__ void load_latent(int64_t at, char *to, int lane) const {
#pragma unroll
        for (int i = FIRST; i < LAST; ++i) {
            const int r = wave * RPW + i;
            const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(at), RT::UNITS * i);
            const int hi = __builtin_amdgcn_readlane(static_cast<int>(at >> 32), RT::UNITS * i);
            // no bytes, so zeros, where there is no row
            const rsrc_t src = buffer(static_cast<const char *>(P.cache) + (static_cast<int64_t>(hi) << 32 | lo), row & ~(hi >> 31));
#pragma unroll
            for (int u = 0; u < LT::UNITS; u += 64) {
                if (LT::UNITS >= 64 || lane < LT::UNITS) {
                    const uint32_t off = static_cast<uint32_t>((u + lane) ^ LT::swz(r)) * 16;
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (lds_ptr)(to + r * LT::ROW + u * 16), 16, static_cast<int>(off < latent ? off : kOutside), 0, 0, AUX);
                }
            }
        }
    }
    // A tile in two parts, the second behind the scores of the tile before: all at once take their time to issue, and the products
    // wait (128 heads, 4 sequences of 65,536 rows: 138 us against 145; 64 of 8,192 rows of 64 heads 108 against 114).
    __device__ __forceinline__ void load(int64_t at, char *to, int lane) const {
        load_front(at, to, lane);
        load_back(at, to, lane);
    }
    __device__ __forceinline__ void load_back(int64_t at, char *to, int lane) const { load_latent<RPW / 2, RPW>(at, to, lane); }
    __device__ __forceinline__ void load_front(int64_t at, char *to, int lane) const {
        const int unit = lane % RT::UNITS, mine = own(lane);
        // in front of the loads: a write to LDS would wait for those on their way there
        if (unit == 0) reinterpret_cast<float *>(to + OM)[mine] = at < 0 ? neg_inf() : 0.f;
        load_latent<0, RPW / 2>(at, to, lane);
        // The rotated parts of all these rows at once.  Where there is no row the scores are not used: what is in LDS may stay.
        if (lane < RPW * RT::UNITS) {
            const uint32_t off = latent + (unit ^ RT::swz(mine)) * 16;
            if (at >= 0 && off < row)
                __builtin_amdgcn_global_load_lds((glb_ptr)(const_cast<char *>(static_cast<const char *>(P.cache)) + at + off), (lds_ptr)(to + OR + wave * RPW * RT::ROW), 16, 0, AUX);
        }
    }
};

// The operands of head h's query of sequence n.
template <class E, int SL, int SR>
__device__ __forceinline__ void load_query(typename Mx<E>::frag *qf, const LatentStepLaunch &P, int n, int h, int lane) {
    const bool live = h < P.H;
    const int g = lane >> 4;
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

// Where a head's result goes: the whole one to o and lse, a part to its slot.
struct Target {
    void *o;
    int64_t at;
    float *lse;
    bool bf16;
    float inv, l;
    __device__ __forceinline__ Target(const LatentStepLaunch &P, const Parts &parts, bool whole, int64_t slot, int heads, int n, int h, int hh,
                                      float sum, float m)
        : inv(sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum),  // NaN stays
          l(sum == 0.f ? neg_inf() : (m + __log2f(sum)) * kLn2) {
        o = whole ? P.o.p : parts.o;
        at = whole ? n * P.o.stride + h * P.o.head_stride : (slot * heads + hh) * P.dl;
        lse = whole ? (P.lse ? P.lse + static_cast<int64_t>(n) * P.H + h : nullptr) : parts.lse + slot * heads + hh;
        bf16 = whole && P.out_bf16;
    }
    __device__ __forceinline__ void store(int d, const f4 &x) const { store4(o, at + d, bf16, x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv); }
};

// A sequence without rows in a workgroup of its own: zeros.
__device__ __forceinline__ void store_empty(const LatentStepLaunch &P, int n, int h0, int heads) {
    for (int h = h0; h < min(P.H, h0 + heads); ++h) {
        for (int d = 4 * threadIdx.x; d < P.dl; d += 4 * blockDim.x) store4(P.o.p, n * P.o.stride + h * P.o.head_stride + d, P.out_bf16, 0.f, 0.f, 0.f, 0.f);
        if (threadIdx.x == 0 && P.lse) P.lse[static_cast<int64_t>(n) * P.H + h] = neg_inf();
    }
}

// A workgroup's four or eight waves share the scores of a tile by heads (and by keys where there are fewer tiles of heads
// than waves) and the products with the values by columns: every accumulator then holds columns of all heads, and a
// value read from LDS serves all of them.  The weights, and the maxima of the waves that share heads, go through LDS.
//
// A workgroup goes through its run of tiles as one stream: the next tile's rows are on their way, and the block numbers of the one
// after it, whether or not it is of the same sequence.  With 32 heads of 512 + 64 in bf16, 64 ragged sequences of up to 8,192 rows
// (302 MB) take 79 us with the join (3.9 TB/s; 73 with the loads alone, 55 without them), of up to 32,768 219 us (5.6 TB/s; 6.6 from
// one to the other): the cache's bandwidth bounds it, and what a call costs that reads little, 16 us for 2,000 rows, where the
// lengths, the block numbers, the rows and the join follow each other.  With 128 heads, 4 of 65,536 rows take 139 us (530 TFLOP/s; 99
// with the loads alone, 110 without them): there each tile's scores, softmax and products follow each other in waves that meet
// twice.  In fp32 a tile has 16 rows and its scores come from one wave for 16 heads and two for 32 while the others wait: 64 ragged
// sequences of 16 heads 220 us (2.8 TB/s), of 32 heads 379.
template <class E, int DLP, int HT>
__global__ __launch_bounds__(64 * kWaves<HT>, sizeof(E) == 2 ? 2 : 1) void latent_step_kernel(const LatentStepLaunch P) {
    using S = Shape<E, HT>;
    constexpr int W = S::W, BN = S::BN, KG = S::KG, KPW = S::KPW;
    constexpr int KC = 4 * Mx<E>::PER, SL = DLP / KC, SR = kRopePad / KC, CT = DLP / (16 * W), ST = BN / KC, HEADS = 16 * HT;
    constexpr int AUX = sizeof(E) == 2 && HT <= 2 ? 2 : 0;  // rows that one workgroup reads once pass the caches by (non-temporal)
    using F = Fetch<E, DLP, W, BN, AUX>;
    typedef typename Mx<E>::frag frag;
    constexpr int PROW = BN * sizeof(E) + 16;  // a head's weights, padded off the banks of the next
    __shared__ __attribute__((aligned(1024))) char lds[2 * F::BUF];
    __shared__ __attribute__((aligned(16))) char weights[HEADS * PROW];
    __shared__ float tops[HEADS * KG];
    __shared__ int shared[W + 3];

    const int w = blockIdx.x, group = blockIdx.y, h0 = group * HEADS;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Tiles<BN> tiles{P};
    int left, run;
    Where x = tiles.template first<W>(w, shared, left, run);
    if (left == 0) {
        if (P.splits == 0) store_empty(P, w, h0, HEADS);
        return;
    }
    const F fetch(P, wave);
    const int ht = wave % HT, kt0 = wave / HT * KPW;  // the wave's share of the scores
    const bool scores = wave / HT < KG;
    const float c2 = P.scale * kLog2e;

    fetch.clear(lds);
    frag qf[SL + SR];
    int block = fetch.block(x, lane);
    load_query<E, SL, SR>(qf, P, x.n, h0 + 16 * ht + (lane & 15), lane);
    const int64_t begin = fetch.place(x, block, lane);
    Where y = x;
    tiles.next(y);
    block = left > 1 ? fetch.block(y, lane) : -1;
    fetch.load(begin, lds, lane);

    f4 acc[HT][CT];
    // the heads' reference points (head `col` of each tile of heads) in powers of two; the wave's own part of the sum
    float m[HT], l;
    int t0;  // the first of the sequence's tiles that are summed up
    auto begin_sequence = [&]() {
        t0 = x.tile;
        l = 0.f;
#pragma unroll
        for (int a = 0; a < HT; ++a) {
            m[a] = neg_inf();
#pragma unroll
            for (int c = 0; c < CT; ++c) acc[a][c] = f4{0, 0, 0, 0};
        }
    };
    begin_sequence();
    for (int i = 0, buf = 0; i < left; ++i, buf ^= 1) {
        loads_landed();
        const char *t = lds + buf * F::BUF;
        const int lane_ = afresh(lane), g = lane_ >> 4, col = lane_ & 15;
        const int64_t next = fetch.place(y, block, lane_);
        Where z = y;
        tiles.next(z);
        block = i < left - 2 ? fetch.block(z, lane_) : -1;
        if (i > 0 && x.tile == 0) {
            const int lane_ = afresh(lane);  // or its addresses would be kept from tile to tile
            load_query<E, SL, SR>(qf, P, x.n, h0 + 16 * ht + (lane_ & 15), lane_);
            loads_done();  // here, or every tile's first product would wait for all loads
            begin_sequence();
        }
        char *to = lds + (buf ^ 1) * F::BUF;
        if (i + 1 < left) fetch.load_front(next, to, lane_);
        f4 s[KPW];
        if (scores) {
            float top = neg_inf();
#pragma unroll
            for (int b = 0; b < KPW; ++b) s[b] = f4{0, 0, 0, 0};
            pipelined<frag, (SL + SR) * KPW, 6>(
                [&](int i) {
                    const int k = i / KPW, b = i % KPW;
                    return k < SL ? F::LT::rows16(t, 16 * (kt0 + b), k, lane_) : F::RT::rows16(t + F::OR, 16 * (kt0 + b), k - SL, lane_);
                },
                [&](int i, frag f) { s[i % KPW] = Mx<E>::mma16(f, qf[i / KPW], s[i % KPW]); });
#pragma unroll
            for (int b = 0; b < KPW; ++b) {
                const f4 mask = *reinterpret_cast<const f4 *>(t + F::OM + (16 * (kt0 + b) + 4 * g) * 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[b][i] = mask[i] < 0.f ? neg_inf() : s[b][i] * c2;
                    top = fmaxf(top, s[b][i]);
                }
            }
            top = quarters_max(top);
            if (g == 0) tops[(16 * ht + col) * KG + wave / HT] = top;
        }
        if (i + 1 < left) fetch.load_back(next, to, lane_);
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
            // in the order in which a step's operand takes them: of each 32 keys, 4 g .. + 3 of either half together; in bf16 rounded as
            // the matrix unit takes them (result_operand), while l sums them as they are
            char *to = weights + (16 * ht + col) * PROW + g * 16;
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
        frag p[ST][HT];
#pragma unroll
        for (int k = 0; k < ST; ++k)
#pragma unroll
            for (int a = 0; a < HT; ++a) p[k][a] = *reinterpret_cast<const frag *>(weights + (16 * a + col) * PROW + 64 * k + 16 * g);
        pipelined<frag, ST * CT, 4>([&](int i) { return F::LT::cols16(t, i / CT * KC, wave * (DLP / W) + 16 * (i % CT), lane_); },
                                    [&](int i, frag v) {
#pragma unroll
                                        for (int a = 0; a < HT; ++a) acc[a][i % CT] = Mx<E>::mma16(v, p[i / CT][a], acc[a][i % CT]);
                                    });
        if (i + 1 == left || y.tile == 0) {  // the last tile of the sequence, or of the run
            const int lane_ = afresh(lane), g = lane_ >> 4, col = lane_ & 15;  // not kept from tile to tile
            // the heads' sums: over the quarters of a wave, then over the waves that share a tile of heads
            l = quarters_sum(l);
            lds_barrier();
            if (scores && g == 0) tops[(16 * ht + col) * KG + wave / HT] = l;
            lds_barrier();
            const int count = x.tile + 1 - t0, all = Tiles<BN>::of(x.length);
            const Parts parts(P, group, gridDim.y, HEADS);
            if (P.splits && t0 == 0 && threadIdx.x == 0) parts.span[x.n] = int2{w, w + pieces(all - count, run)};
#pragma unroll
            for (int a = 0; a < HT; ++a) {
                const int h = h0 + 16 * a + col;
                if (h >= P.H) continue;
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < KG; ++k) sum += tops[(16 * a + col) * KG + k];
                const Target to(P, parts, count == all, 2 * static_cast<int64_t>(w) + (t0 == 0), HEADS, x.n, h, 16 * a + col, sum, m[a]);
                if (wave == 0 && g == 0 && to.lse) *to.lse = to.l;
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    const int d = wave * (DLP / W) + 16 * c + 4 * g;
                    if (d < P.dl) to.store(d, acc[a][c]);
                }
            }
        }
        x = y;
        y = z;
    }
}

// Joins the parts of a (sequence, head): o = sum_s exp(lse_s - lse) o_s, lse = log sum_s exp(lse_s).  Sequences without rows
// get zeros here.  COLS columns per workgroup, COLS / 4 threads of four by those that share the parts out.
constexpr int kJoinParts = 512, kJoinWhole = 512;  // the most parts; rows from which a workgroup has all columns
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

// Tiles of 16 heads per workgroup, and groups of so many heads.  No more tiles than the heads fill: 64 sequences of 16 heads
// take 72 us, of 32 heads 79, of 64 heads 108.  More than four were slower at short contexts, with twice the parts to join (measured
// before a tile's rows were loaded in two parts, 128 heads as one group and as two: 4 sequences of 16,384 rows 70 us and 57, of
// 65,536 rows 145 and 152; as two groups they take 52 and 138 now).
int head_tiles(int H, bool bf16) { return H <= 16 ? 1 : H <= 32 || !bf16 ? 2 : 4; }
int head_groups(int H, bool bf16) {
    const int per = 16 * head_tiles(H, bf16);
    return (H + per - 1) / per;
}

template <class E, int DLP>
void launch(const LatentStepLaunch &P) {
    const int tiles = head_tiles(P.H, P.bf16);
    const dim3 grid(P.splits ? P.splits : P.N, head_groups(P.H, P.bf16));
    if (tiles == 1) latent_step_kernel<E, DLP, 1><<<grid, 64 * kWaves<1>, 0, P.stream>>>(P);
    else if (tiles == 2) latent_step_kernel<E, DLP, 2><<<grid, 64 * kWaves<2>, 0, P.stream>>>(P);
    else if constexpr (sizeof(E) == 2) latent_step_kernel<E, DLP, 4><<<grid, 64 * kWaves<4>, 0, P.stream>>>(P);
}
template <class E>
void launch_dl(const LatentStepLaunch &P) {
    if (P.dl <= 128) launch<E, 128>(P);
    else if (P.dl <= 256) launch<E, 256>(P);
    else launch<E, 512>(P);
}

}  // namespace

// Workgroups over which the sequences' tiles are shared out: what the CUs hold at once (two workgroups each, one where it has eight
// waves), no more than there can be tiles.  0: a workgroup per sequence and no parts, where there are enough of them and none can be
// so long that the others wait for it (32 heads, ragged, that way and shared out: 1,024 sequences of up to 256 rows 58 and 97 us,
// of up to 1,024 170 and 186, of up to 4,096 591 and 500; 4,096 of up to 512 324 and 432).  `longest` is what the block table has
// room for: the lengths are on the device.  A caller whose sequences are all much shorter gives the table's first columns.
int latent_step_splits(int N, int H, int64_t longest, bool bf16) {
    if (N >= 1024 && longest <= 2048) return 0;
    int64_t s = (head_tiles(H, bf16) == 4 ? 256 : kJoinParts) / head_groups(H, bf16);
    const int64_t most = N * ((longest + 15) / 16);
    s = s < most ? s : most;
    return s < 1 ? 1 : static_cast<int>(s);
}
size_t latent_step_workspace_bytes(int N, int H, int dl, int splits, bool bf16) {
    const size_t groups = head_groups(H, bf16), heads = 16 * head_tiles(H, bf16);
    return splits == 0 ? 0 : groups * 2 * splits * heads * (static_cast<size_t>(dl) + 1) * 4 + groups * N * sizeof(int2);
}
int64_t latent_step_threads(int N, int H, bool bf16, int splits) {
    const int64_t step = static_cast<int64_t>(splits ? splits : N) * head_groups(H, bf16) * 512, rows = static_cast<int64_t>(N) * H;
    const int64_t join = splits == 0 ? 0 : rows * (rows >= kJoinWhole ? 256 : 256 * 4);
    return step > join ? step : join;
}

hipError_t launch_latent_step(const LatentStepLaunch &P) {
    if (P.bf16) launch_dl<uint16_t>(P);
    else launch_dl<float>(P);
    if (P.splits) {
        const int64_t rows = P.N * static_cast<int64_t>(P.H);
        const int heads = 16 * head_tiles(P.H, P.bf16), groups = head_groups(P.H, P.bf16);
        // All columns at once where there are rows enough for every CU (64 sequences of 32 heads 79 us for both kernels against 84), a
        // quarter where a few rows have many parts (one sequence of 65,536 rows 41 us against 59).
        if (rows >= kJoinWhole) latent_join_kernel<512><<<static_cast<unsigned>(rows), 256, 0, P.stream>>>(P, heads, groups);
        else latent_join_kernel<128><<<dim3(static_cast<unsigned>(rows), (P.dl + 127) / 128), 256, 0, P.stream>>>(P, heads, groups);
    }
    return hipGetLastError();
}

}  // namespace kda
