// kda_layer.h - what the layer operators (selective scan, short convolution, layer norm) share: launch
// structs, the map from launch slots to sequence tiles, strided typed access, and the column sum that
// finishes every parameter gradient.
#pragma once

#include "kda_device.h"

namespace kda {

// A [rows, width] tensor whose rows are `stride` elements apart, in bf16 or fp32.
struct Rows {
    void *p;
    int64_t stride;
    int bf16;
    __device__ __forceinline__ float get(int64_t row, int col) const {
        const int64_t i = row * stride + col;
        return bf16 ? bf16_to_f32(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
    }
    __device__ __forceinline__ void put(int64_t row, int col, float x) const {
        const int64_t i = row * stride + col;
        if (bf16) static_cast<uint16_t *>(p)[i] = f32_to_bf16(x);
        else static_cast<float *>(p)[i] = x;
    }
};
// A parameter vector in bf16 or fp32.
__device__ __forceinline__ float param(const void *p, int bf16, int64_t i) {
    return bf16 ? bf16_to_f32(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}

// Sequences cut into tiles of L tokens.  A launch has one slot per possible tile: sequence n's tiles take
// the slots from (start_n / L + n) on.  As ceil(len / L) <= (start + len) / L - start / L + 1 these ranges
// are disjoint, so a slot finds its tile by a binary search over the offsets alone, without a table made
// beforehand; slots that no tile takes end at once.  Offsets are clamped to the rows that exist, so wrong
// ones cannot lead out of the tensors.
struct SeqTiles {
    const int32_t *cu;  // N + 1 offsets, or nullptr: N sequences of T tokens
    int N, T;           // T: per sequence, or all rows with cu
    int L;              // tokens per tile
    __host__ __device__ int64_t rows() const { return cu ? T : static_cast<int64_t>(N) * T; }
    __host__ __device__ int per_seq() const { return T > L ? (T + L - 1) / L : 1; }  // without cu
    __host__ __device__ int64_t slots() const {
        return cu ? static_cast<int64_t>(T) / L + N : static_cast<int64_t>(N) * per_seq();
    }
    __device__ __forceinline__ int offset(int n) const {
        const int c = cu[n];
        return c < 0 ? 0 : c > T ? T : c;
    }
    __device__ __forceinline__ void sequence(int n, int64_t &start, int &len) const {
        if (cu) {
            const int s = offset(n), e = offset(n + 1);
            start = s;
            len = e > s ? e - s : 0;
        } else {
            start = static_cast<int64_t>(n) * T;
            len = T;
        }
    }
    __device__ __forceinline__ int64_t first_slot(int n, int64_t start) const {
        return cu ? start / L + n : static_cast<int64_t>(n) * per_seq();
    }
};

struct Tile {
    int n, k, count;      // sequence, tile within it, tiles of it (0: an empty sequence's only slot)
    int64_t begin;        // first row
    int len;              // rows in the tile
    bool valid;           // false: no tile takes this slot
    __device__ __forceinline__ bool last() const { return k + 1 >= count; }
};

__device__ __forceinline__ Tile find_tile(const SeqTiles &s, int64_t slot) {
    Tile t;
    if (s.cu) {
        int lo = 0, hi = s.N - 1;
        while (lo < hi) {  // the last sequence whose first slot is not behind this one
            const int mid = (lo + hi + 1) >> 1;
            if (s.offset(mid) / s.L + static_cast<int64_t>(mid) <= slot) lo = mid;
            else hi = mid - 1;
        }
        t.n = lo;
    } else {
        t.n = static_cast<int>(slot / s.per_seq());
    }
    int64_t start;
    int len;
    s.sequence(t.n, start, len);
    t.count = (len + s.L - 1) / s.L;
    const int64_t k = slot - s.first_slot(t.n, start);
    t.valid = k >= 0 && k < (t.count > 0 ? t.count : 1);
    t.k = t.valid ? static_cast<int>(k) : 0;
    t.begin = start + static_cast<int64_t>(t.k) * s.L;
    const int left = len - t.k * s.L;
    t.len = left < s.L ? left : s.L;
    // uniform over the workgroup: kept in scalar registers
    t.n = __builtin_amdgcn_readfirstlane(t.n);
    t.k = __builtin_amdgcn_readfirstlane(t.k);
    t.count = __builtin_amdgcn_readfirstlane(t.count);
    t.len = __builtin_amdgcn_readfirstlane(t.len);
    t.begin = static_cast<int64_t>(static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(t.begin))));
    return t;
}

// One channel's column of a tile's rows, read or written four rows at a time by the lanes q = 0..3 of a quad:
// a uniform address per group of four rows plus a 32-bit lane offset that stays the same, so that a step
// costs scalar additions only.  Strides are at most 2^27 elements, which keeps 3 rows inside 32 bits.
struct QuadColumn {
    char *at;           // the tile's first row
    int64_t step;       // bytes per row
    uint32_t off, tail; // lane offset; the same in a last group of fewer than four rows, held to its last row
    __device__ __forceinline__ QuadColumn(const Rows &r, int64_t begin, int len, int ch, int q) {
        const int e = r.bf16 ? 2 : 4, left = (len & 3) - 1;
        at = static_cast<char *>(r.p) + begin * r.stride * e;
        step = r.stride * e;
        off = (static_cast<uint32_t>(q) * static_cast<uint32_t>(r.stride) + static_cast<uint32_t>(ch)) * e;
        const int qt = left >= 0 && q > left ? left : q;
        tail = (static_cast<uint32_t>(qt) * static_cast<uint32_t>(r.stride) + static_cast<uint32_t>(ch)) * e;
    }
    // the group of rows t .. t + 3 of the tile; whole: all four exist
    template <typename E>
    __device__ __forceinline__ E get(int t, bool whole) const {
        return *reinterpret_cast<const E *>(at + t * step + (whole ? off : tail));
    }
    __device__ __forceinline__ void put(int t, int bf16, float x) const {
        char *p = at + t * step + off;
        if (bf16) *reinterpret_cast<uint16_t *>(p) = f32_to_bf16(x);
        else *reinterpret_cast<float *>(p) = x;
    }
};

// x * sigmoid(x) and the sigmoid.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float sigmoid_f(float x) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

// softplus(x) = max(x, 0) + log1p(e), e = exp(-|x|) in (0, 1].  log1p(e) = 2 atanh(r), r = e / (2 + e) <= 1/3,
// by atanh's series to r^13 (the next term is below 1e-8 of the value): small e keep their relative precision,
// which 1 + e would round away.
__device__ __forceinline__ float softplus_f(float x) {
    const float e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(x));
    const float r = e * __builtin_amdgcn_rcpf(2.f + e), q = r * r;
    float s = 1.f / 13.f;
    s = fmaf(s, q, 1.f / 11.f);
    s = fmaf(s, q, 1.f / 9.f);
    s = fmaf(s, q, 1.f / 7.f);
    s = fmaf(s, q, 1.f / 5.f);
    s = fmaf(s, q, 1.f / 3.f);
    s = fmaf(s, q, 1.f);
    return fmaxf(x, 0.f) + 2.f * r * s;
}

// A value of lane I of each quad, in all four lanes.
template <int I>
__device__ __forceinline__ float quad_bcast(float x) {
    return dpp_mov<I * 0x55>(x);
}
// Lane q of each quad gets the quad's sum of v[q].
__device__ __forceinline__ float quad_transpose_sum(float v0, float v1, float v2, float v3, int q) {
    const bool b0 = q & 1, b1 = q & 2;
    const float r01 = (b0 ? v1 : v0) + dpp_mov<0xB1>(b0 ? v0 : v1);
    const float r23 = (b0 ? v3 : v2) + dpp_mov<0xB1>(b0 ? v2 : v3);
    return (b1 ? r23 : r01) + dpp_mov<0x4E>(b1 ? r01 : r23);
}

// ---- launch structs ------------------------------------------------------------------------------------

struct ScanFwdLaunch {
    Rows u, dt, B, C, z, y;  // z.p may be null
    const float *A, *D, *dt_bias, *h0;
    float *hT;
    SeqTiles seq;
    int dim, ds;
    int softplus;
    float *ws;
    hipStream_t stream;
};
size_t scan_fwd_workspace_bytes(const SeqTiles &seq, int dim, int ds);
hipError_t launch_scan_fwd(const ScanFwdLaunch &P);
hipError_t launch_scan_step(const ScanFwdLaunch &P);
// tiles for these sizes (cu only tells packed from fixed)
SeqTiles scan_fwd_tiles(const int32_t *cu, int N, int T, int dim, int ds);

struct ScanBwdLaunch {
    Rows u, dt, B, C, z, gy, du, ddt, dB, dC, dz;
    const float *A, *D, *dt_bias, *h0, *dhT;
    float *dA, *dD, *ddt_bias, *dh0;
    SeqTiles seq;
    int dim, ds;
    int softplus;
    float *ws;
    hipStream_t stream;
};
SeqTiles scan_bwd_tiles(const int32_t *cu, int N, int T, int dim, int ds);
size_t scan_bwd_workspace_bytes(const SeqTiles &seq, int dim, int ds);
hipError_t launch_scan_bwd(const ScanBwdLaunch &P);

struct ConvLaunch {
    Rows x, y;
    const void *w, *bias;
    int w_bf16;
    const void *h0;
    void *hT;
    const int32_t *cu;
    int N, T, dim, width;
    int silu;
    hipStream_t stream;
};
hipError_t launch_conv_fwd(const ConvLaunch &P);
hipError_t launch_conv_step(const ConvLaunch &P);

struct ConvBwdLaunch {
    Rows x, gy, dx;
    const void *w, *bias;
    int w_bf16;
    const void *h0;
    const float *dhT;
    float *dw, *db, *dh0;
    const int32_t *cu;
    int N, T, dim, width;
    int silu;
    float *ws;
    hipStream_t stream;
};
size_t conv_bwd_workspace_bytes(int64_t rows, int dim, int width);
hipError_t launch_conv_bwd(const ConvBwdLaunch &P);

struct NormFwdLaunch {
    Rows x, res, y, res_out;
    const void *w, *b;
    int w_bf16;
    int64_t rows;
    int dim;
    float eps;
    hipStream_t stream;
};
hipError_t launch_norm_fwd(const NormFwdLaunch &P);

struct NormBwdLaunch {
    Rows x, gy, gres, dx;
    const void *w;
    int w_bf16;
    float *dw, *db;
    int64_t rows;
    int dim;
    float eps;
    float *ws;
    hipStream_t stream;
};
size_t norm_bwd_workspace_bytes(int64_t rows, int dim);
hipError_t launch_norm_bwd(const NormBwdLaunch &P);

// out[c] = sum over p < parts of in[p * ld + c] for c < cols, in a fixed order (kda_layer_norm.hip).
void launch_column_sum(const float *in, int64_t ld, int parts, int64_t cols, float *out, hipStream_t stream);

}  // namespace kda
