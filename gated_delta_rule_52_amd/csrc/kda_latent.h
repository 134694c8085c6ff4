// kda_latent.h - what the latent attention kernels share: launch structs, matrix products of 32 x 32 and 16 x 16 tiles
// in bf16 or fp32, and tiles of rows in LDS that are filled by loads past the registers.
#pragma once

#include <type_traits>

#include "kda_device.h"
#include "kda_latent_pages.h"
#include "kda_seq_tiles.h"

namespace kda {

// [rows, heads, width] elements, rows and heads any distance apart.
struct Heads {
    void *p;
    int64_t stride, head_stride;  // elements
};

struct RotaryLaunch {
    Heads x, y;
    const int32_t *positions;
    const float *inv_freq;
    int64_t rows;
    int heads, dim, rot, offset;
    float scale;
    int interleaved, inverse, bf16;
    hipStream_t stream;
};
hipError_t launch_rotary(const RotaryLaunch &P);
int64_t rotary_threads(const RotaryLaunch &P);

struct AppendLaunch {
    Heads latent, rope;  // head_stride unused
    void *cache;
    const int32_t *slots, *positions;
    const float *inv_freq;  // null: no rotation
    int64_t rows, cache_rows;
    int dl, dr;
    float scale;
    int interleaved, bf16;
    hipStream_t stream;
};
hipError_t launch_append(const AppendLaunch &P);

struct LatentStepLaunch {
    Heads ql, qr, o;
    const void *cache;
    CachePages pages;
    const int32_t *lengths;
    float *lse;  // may be null
    int N, H, dl, dr;
    float scale;
    int bf16, out_bf16;
    int splits;
    float *ws;
    hipStream_t stream;
};
int latent_step_splits(int N, int H, int64_t longest, bool bf16);
size_t latent_step_workspace_bytes(int N, int H, int dl, int splits, bool bf16);
hipError_t launch_latent_step(const LatentStepLaunch &P);
int64_t latent_step_threads(int N, int H, bool bf16, int splits);

struct AttendLaunch {
    Heads q, k, v, o;
    Heads kr;    // head_stride unused
    float *lse;  // [rows_q, H]
    SeqTiles q_seq, k_seq;  // L set by the kernel that walks them
    int H, dn, dr, dv;
    float scale;
    int causal, bf16, out_bf16;
    hipStream_t stream;
    // gradients
    Heads go, dq, dk, dkr, dvg;
    int grad_bf16;
    float *delta;     // [rows_q, H]
    float *lse2;      // [rows_q, H], lse in powers of two (bf16)
    float *dkr_part;  // [rows_k, H, dr]
};
// Rows per workgroup: bf16 and fp32.
constexpr int kAttendTile = 128, kAttendTileF32 = 32;
inline int64_t tiles_of(const SeqTiles &s) { return s.cu ? s.slots() : s.N * static_cast<int64_t>(s.per_seq()); }
hipError_t launch_attend_fwd(const AttendLaunch &P);
hipError_t launch_attend_bwd(const AttendLaunch &P);
int64_t attend_threads(const SeqTiles &q, const SeqTiles &k, int H, int dr, bool bf16, bool backward);
void launch_attend_fwd_fp32(const AttendLaunch &P);
void launch_attend_grads_fp32(const AttendLaunch &P);

// ---- device side ---------------------------------------------------------------------------------------

namespace la {

typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef __bf16 b4 __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16 __attribute__((ext_vector_type(16)));
typedef unsigned u4 __attribute__((ext_vector_type(4)));
typedef unsigned u2 __attribute__((ext_vector_type(2)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef __attribute__((address_space(3))) void *lds_ptr;
typedef __attribute__((address_space(1))) void *glb_ptr;
typedef __attribute__((address_space(3))) s4 *lds_s4;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }
__device__ __forceinline__ float exp2_f(float x) { return __builtin_amdgcn_exp2f(x); }

// Bytes [base, base + bytes) as a buffer: loads at or past its end give zeros, so rows behind a sequence and columns
// behind a head need no branch.
__device__ __forceinline__ rsrc_t buffer(const void *base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, static_cast<int>(bytes), 0x00020000);
}
constexpr uint32_t kOutside = 0x7ffffff0u;  // an offset past the end of every buffer here (all are below 2^30 bytes)

// Four consecutive elements stored from fp32.
__device__ __forceinline__ void store4(void *p, int64_t i, bool bf16, float a, float b, float c, float d) {
    if (bf16) {
        b4 v = {static_cast<__bf16>(a), static_cast<__bf16>(b), static_cast<__bf16>(c), static_cast<__bf16>(d)};
        *reinterpret_cast<u2 *>(static_cast<uint16_t *>(p) + i) = __builtin_bit_cast(u2, v);
    } else {
        *reinterpret_cast<f4 *>(static_cast<float *>(p) + i) = f4{a, b, c, d};
    }
}

// Matrix products.  A `step` multiplies what one 16-byte operand per lane holds: for a 32 x 32 tile lane l has row
// (or column) l % 32 and half h = l / 32 of the step's elements along the contraction, for 16 x 16 row l % 16 and
// quarter l / 16.  fp32 spends four instructions on it, each with the operand's next element; which element of the
// contraction a lane's element is does not matter as long as both operands agree.
template <class E>
struct Mx;
template <>
struct Mx<uint16_t> {
    typedef b8 frag;
    static constexpr int PER = 8;  // elements of an operand
    __device__ __forceinline__ static f16 mma32(frag a, frag b, f16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    __device__ __forceinline__ static f4 mma16(frag a, frag b, f4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    __device__ __forceinline__ static frag zero() { return __builtin_bit_cast(frag, (u4{0, 0, 0, 0})); }
};
template <>
struct Mx<float> {
    typedef f4 frag;
    static constexpr int PER = 4;
    __device__ __forceinline__ static f16 mma32(frag a, frag b, f16 c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
        return c;
    }
    __device__ __forceinline__ static f4 mma16(frag a, frag b, f4 c) {
#pragma unroll
        for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
        return c;
    }
    __device__ __forceinline__ static frag zero() { return f4{0, 0, 0, 0}; }
};

// A transposing read: of four rows of 16 bf16 per 16 lanes, the lanes giving the addresses of four consecutive elements
// each, lane i gets column i.  The restrict qualifier tells the compiler what the kernels see to themselves (by
// loads_landed): that no load into LDS in flight writes what is read; without it every such read waits for all of them.
__device__ __forceinline__ s4 read_columns(const char *__restrict__ p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)p);
}

// Rows of W elements in LDS, in 16-byte units.  Unit u of row r lies at place u ^ swz(r), so that what LDS serves at once, 256
// bytes, comes from all of its 64 banks: a transposing read takes 32 COLS bytes of consecutive rows, four of them for COLS = 32 and
// eight for COLS = 16, and an operand read 16 bytes for each of lanes 0-3, 12-15 and 20-27 together (and of the rest of 32): for
// COLS = 32 those are 16 rows, for COLS = 16 eight rows' one unit and the other eight's next one, so that rows 0-3 and 12-15 have
// whole pairs of places (of the cycles that LDS is busy in the step's kernel with 128 heads, conflicts take 2.1 of 17.7 million so,
// 11.5 of 27.1 with rows in plain order).  swz repeats after 16 rows.  In long rows the swap stays within 16 units: what lies beyond is a constant distance.
template <int W, class E, int COLS>
struct LdsTile {
    static constexpr int ROW = W * static_cast<int>(sizeof(E)), UNITS = ROW / 16;
    static_assert(UNITS >= 4 && (UNITS & (UNITS - 1)) == 0, "rows of 64 bytes or a power of two more");
    __device__ __forceinline__ static int swz(int row) {
        if (COLS == 16) {
            constexpr int ROWS = UNITS == 8 ? 2 : 1, H = 8 / ROWS;  // rows in 256 bytes
            const int r = row / ROWS;
            return ((r & (H - 1)) ^ (r & H) / 2) << 1 | ((r & H) != 0);
        }
        if (UNITS == 4) return (row >> 2) & 3;                            // four rows in 256 bytes
        if (UNITS == 8) return ((row >> 1) & 1) << 2 | ((row >> 2) & 3);  // two
        return (row & 3) << 2 | ((row >> 2) & 3);
    }
    __device__ __forceinline__ static int at(int row, int unit) {
        return row * ROW + (unit & ~15) * 16 + (((unit & 15) ^ swz(row)) << 4);
    }

    // Fills ROWS rows from rows `stride` bytes apart of a buffer, `width` bytes of each (a multiple of 16), zeros
    // behind them and behind the buffer, past the registers: the data has arrived after a wait for the wave's loads.
    template <int ROWS, int WAVES>
    __device__ __forceinline__ static void fill(char *lds, rsrc_t from, uint32_t stride, uint32_t width, int wave, int lane) {
        constexpr int LOADS = ROWS * UNITS / 64;
        static_assert(LOADS > 0, "");
#pragma unroll
        for (int i = 0; i < (LOADS + WAVES - 1) / WAVES; ++i) {
            const int u = wave + WAVES * i;
            if (LOADS % WAVES != 0 && u >= LOADS) break;
            const int c = u * 64 + lane, row = c / UNITS, unit = (c % UNITS) ^ swz(row);
            const uint32_t off = static_cast<uint32_t>(unit) * 16 < width ? row * stride + unit * 16 : kOutside;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_ptr)(lds + u * 1024), 16, static_cast<int>(off), 0, 0, 0);
        }
    }
    // A step's operand whose rows are the tile's.
    __device__ __forceinline__ static typename Mx<E>::frag rows32(const char *lds, int row0, int step, int lane) {
        return *reinterpret_cast<const typename Mx<E>::frag *>(lds + at(row0 + (lane & 31), 2 * step | (lane >> 5)));
    }
    __device__ __forceinline__ static typename Mx<E>::frag rows16(const char *lds, int row0, int step, int lane) {
        return *reinterpret_cast<const typename Mx<E>::frag *>(lds + at(row0 + (lane & 15), 4 * step | (lane >> 4)));
    }
    // A step's operand whose rows are the tile's columns col0 .. + 31, contracted over the tile's rows, in the order
    // in which a lane holds the rows of a 32 x 32 result (lane half h: rows 8 b + 4 h + i), 16 rows a step.
    __device__ __forceinline__ static b8 cols32(const char *lds, int row0, int step, int col0, int lane) {
        static_assert(sizeof(E) == 2, "");
        const int h = lane >> 5, i = lane & 15, row = row0 + 16 * step + 4 * h + (i >> 2);
        const int unit = (col0 >> 3) | ((lane >> 3) & 2) | ((i >> 1) & 1);
        const char *p = lds + (i & 1) * 8;
        const s4 lo = read_columns(p + at(row, unit));
        const s4 hi = read_columns(p + at(row + 8, unit));
        return __builtin_bit_cast(b8, (__attribute__((ext_vector_type(8))) short){lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
    }
    // The same for 16 columns and the rows that a lane holds of 16 x 16 results (quarter g: rows 4 g + i), one result for
    // fp32 and two, 16 rows apart, for bf16.
    __device__ __forceinline__ static typename Mx<E>::frag cols16(const char *lds, int row0, int col0, int lane) {
        const int g = lane >> 4, i = lane & 15;
        if constexpr (sizeof(E) == 2) {
            const char *p = lds + (i & 1) * 8 + at(row0 + 4 * g + (i >> 2), (col0 >> 3) | ((i >> 1) & 1));
            const s4 lo = read_columns(p);
            const s4 hi = read_columns(p + 16 * ROW);
            return __builtin_bit_cast(b8, (__attribute__((ext_vector_type(8))) short){lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
        } else {
            const int col = col0 + i;
            f4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const float *>(lds + at(row0 + 4 * g + j, col >> 2) + (col & 3) * 4);
            return v;
        }
    }
};

// Rows of a 32 x 32 result as a step's operand (the order that cols32 reads in): weights and their gradients, rounded to bf16 as the
// matrix unit takes them.  Each is off by 2^-8 of itself at most, about what the result's own rounding to bf16 costs; operands in
// two parts would take that away for as many products again.
__device__ __forceinline__ b8 result_operand(const f16 &s, int step) {
    b8 v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = static_cast<__bf16>(s[8 * step + j]);
    return v;
}

// A row's operands straight from memory: element 2 PER step + PER h on; zeros from `width` on or where !live.
template <class E>
__device__ __forceinline__ typename Mx<E>::frag row_operand(const E *row, int step, int width, bool live, int lane) {
    const int c = (2 * step + (lane >> 5)) * Mx<E>::PER;
    return live && c < width ? *reinterpret_cast<const typename Mx<E>::frag *>(row + c) : Mx<E>::zero();
}

// Maximum and sum over the two halves of a wave, and over its four quarters, in every lane: a swap of rows or halves
// between two copies of a value leaves the partners' values side by side.
__device__ __forceinline__ u2 swap_halves(float x) {
    return __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
}
__device__ __forceinline__ u2 swap_rows(float x) {
    return __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
}
__device__ __forceinline__ float halves_max(float x) {
    const u2 r = swap_halves(x);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float halves_sum(float x) {
    const u2 r = swap_halves(x);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float quarters_max(float x) {
    const u2 r = swap_rows(x);
    return halves_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float quarters_sum(float x) {
    const u2 r = swap_rows(x);
    return halves_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// All of the wave's loads have arrived.
__device__ __forceinline__ void loads_done() { __builtin_amdgcn_s_waitcnt(0x0f70); }  // vmcnt(0)
// Those into LDS too, and every wave is here.
__device__ __forceinline__ void loads_landed() {
    loads_done();
    __syncthreads();
}

// The rows of a wave's results: row lane % 32 has, in tile c, columns 32 c + 8 b + 4 (lane / 32) .. + 3 as elements 4 b .. + 3.
// Rows of bf16 are put together in LDS (32 * kStoreRow<W> bytes of the wave's own) and leave 16 bytes per lane and whole rows at
// a time (measured together: the forward kernel at 8,192 rows of 32 heads 646 us so and 658 with eight bytes to each of 64 places,
// the gradients' query kernel at 2 sequences of 4,096 rows 590 and 600).  `to`: the wave's first row.
template <int W>
constexpr int kStoreRow = 2 * W + 16;
template <int W>
__device__ __forceinline__ void store_rows(char *lds, const f16 *x, float by, void *to, bool bf16, int64_t stride, int rows, int width, int lane) {
    const int r = lane & 31, h = lane >> 5;
    if (!bf16) {
        if (r < rows)
#pragma unroll
            for (int c = 0; c < W / 32; ++c)
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (32 * c + 8 * b + 4 * h < width)
                        store4(to, r * stride + 32 * c + 8 * b + 4 * h, false, x[c][4 * b] * by, x[c][4 * b + 1] * by, x[c][4 * b + 2] * by, x[c][4 * b + 3] * by);
        return;
    }
#pragma unroll
    for (int c = 0; c < W / 32; ++c)
#pragma unroll
        for (int b = 0; b < 4; ++b)
            store4(lds + r * kStoreRow<W> + (32 * c + 8 * b + 4 * h) * 2, 0, true, x[c][4 * b] * by, x[c][4 * b + 1] * by, x[c][4 * b + 2] * by, x[c][4 * b + 3] * by);
    constexpr int PER = 512 / W;  // rows at a time
#pragma unroll
    for (int i = 0; i < 32 / PER; ++i) {
        const int row = PER * i + lane / (W / 8), col = lane % (W / 8) * 8;
        const u4 v = *reinterpret_cast<const u4 *>(lds + row * kStoreRow<W> + col * 2);
        if (row < rows && col < width) *reinterpret_cast<u4 *>(static_cast<uint16_t *>(to) + row * stride + col) = v;
    }
}
__device__ __forceinline__ void *out_row(const Heads &t, bool bf16, int64_t row, int h) {
    return static_cast<char *>(t.p) + (row * t.stride + h * t.head_stride) * (bf16 ? 2 : 4);
}

// ---- attention over expanded keys and values -------------------------------------------------------------

// Where a workgroup's tile lies: the sequence's rows of queries and keys.
struct Place {
    int h;
    int64_t q_row, k_row;  // the sequences' first rows
    int nq, nk;            // their lengths
    int at;                // first row of the tile in its sequence
    bool valid;
};
// Workgroups go round-robin over the 8 XCDs: heads (of sequences, where they have equal lengths) are dealt to the XCDs
// whole where their number allows, so that an L2 fetches a head's keys once.  The tiles that meet the most start first: a
// head's last queries, its first keys.
template <bool QUERIES>
__device__ __forceinline__ Place place_of(const AttendLaunch &P, int64_t id) {
    const SeqTiles &tiled = QUERIES ? P.q_seq : P.k_seq;
    const int64_t per = tiled.cu ? tiled.slots() : tiled.per_seq();
    const int64_t groups = static_cast<int64_t>(P.H) * (tiled.cu ? 1 : tiled.N);
    int64_t group, k;
    if (groups % 8 == 0) {
        const int64_t r = id >> 3;
        group = (id & 7) + 8 * (r / per);
        k = r % per;
    } else {
        group = id / per;
        k = id % per;
    }
    if (QUERIES) k = per - 1 - k;
    Place w;
    w.h = static_cast<int>(group % P.H);
    const Tile t = tile_at(tiled, (tiled.cu ? 0 : group / P.H * per) + k);
    const int n = __builtin_amdgcn_readfirstlane(t.n);
    w.valid = t.valid;
    P.q_seq.sequence(n, w.q_row, w.nq);
    P.k_seq.sequence(n, w.k_row, w.nk);
    w.at = __builtin_amdgcn_readfirstlane(t.k) * tiled.L;
    return w;
}

template <class E>
__device__ __forceinline__ const E *head_row(const Heads &t, int64_t row, int h) {
    return static_cast<const E *>(t.p) + row * t.stride + h * t.head_stride;
}
// A buffer over `rows` rows of `width` elements from there.
template <class E>
__device__ __forceinline__ rsrc_t rows_buffer(const E *p, int64_t stride, int rows, int width) {
    return buffer(p, rows > 0 ? static_cast<uint32_t>(((rows - 1) * stride + width) * static_cast<int64_t>(sizeof(E))) : 0);
}

// What a wave has written to LDS is there, and every wave is here.  Unlike __syncthreads() it does not wait for loads: those
// into LDS for a later tile stay in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The same value, of which the compiler does not know that: what is formed from it inside a loop is formed there, and takes
// no register from one round to the next.
__device__ __forceinline__ int afresh(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// N operands, each read from LDS and then used, with DEPTH reads in flight: left alone the compiler, which prefers few
// registers, reads one at a time and waits for it.
template <class F, int N, int DEPTH, class Read, class Use>
__device__ __forceinline__ void pipelined(Read read, Use use) {
    F f[DEPTH];
#pragma unroll
    for (int i = 0; i < DEPTH && i < N; ++i) f[i] = read(i);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        use(i, f[i % DEPTH]);
        if (i + DEPTH < N) f[i % DEPTH] = read(i + DEPTH);
        __builtin_amdgcn_sched_barrier(0);
    }
}

}  // namespace la
}  // namespace kda
