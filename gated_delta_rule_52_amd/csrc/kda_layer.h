// kda_layer.h - what the layer operators (selective scan, short convolution, layer norm) share: launch
// structs, strided typed access, and the column sum that finishes every parameter gradient.
#pragma once

#include <type_traits>

#include "kda_device.h"
#include "kda_seq_tiles.h"

namespace kda {

// fp32 to bf16, nearest even, by the conversion instruction.
__device__ __forceinline__ uint16_t to_bf16(float x) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}

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
        if (bf16) static_cast<uint16_t *>(p)[i] = to_bf16(x);
        else static_cast<float *>(p)[i] = x;
    }
};

// A workgroup's tile, uniform over it: kept in scalar registers.
__device__ __forceinline__ Tile find_tile(const SeqTiles &s, int64_t slot) {
    Tile t = tile_at(s, slot);
    t.n = __builtin_amdgcn_readfirstlane(t.n);
    t.k = __builtin_amdgcn_readfirstlane(t.k);
    t.count = __builtin_amdgcn_readfirstlane(t.count);
    t.len = __builtin_amdgcn_readfirstlane(t.len);
    t.begin = static_cast<int64_t>(static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(t.begin))));
    return t;
}

// Where the four lanes q of a quad stand in a group of four rows, held to the tile's last row: a scalar row for the
// group and a lane's distance from it.  Loads through it need no branch at a tile's end; what lies past the end
// is masked where it is used.
struct Group {
    int row;
    uint32_t lane;
    __device__ __forceinline__ Group(int t, int len, int q) {
        row = t < len ? t : len - 1;
        const int left = len - 1 - row;
        lane = q < left ? q : left;
    }
};
// One channel's column of a tile: a uniform address per group of rows and a 32-bit lane offset, one 24-bit
// multiply-add.  Strides are below 2^22 elements, which keeps a row's bytes within 24 bits.
struct Column {
    char *at;      // the tile's first row
    int64_t step;  // bytes per row
    uint32_t ch;   // the channel's byte in a row
    __device__ __forceinline__ Column(const Rows &r, int64_t row, int c) {
        const int e = r.bf16 ? 2 : 4;
        at = static_cast<char *>(r.p) + row * r.stride * e;
        step = r.stride * e;
        ch = static_cast<uint32_t>(c) * e;
    }
    __device__ __forceinline__ char *of(const Group &g) const {
        return at + g.row * step + (__umul24(g.lane, static_cast<uint32_t>(step)) + ch);
    }
    template <typename E>
    __device__ __forceinline__ E get(const Group &g) const {
        return *reinterpret_cast<const E *>(of(g));
    }
    // one value of each of a block's J groups, masked by the tile's end
    template <int J>
    __device__ __forceinline__ void put(int t0, int len, int q, bool live, int bf16, const float (&x)[J]) const {
        if (!live) return;
        auto all = [&](auto bf) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const Group g(t0 + 4 * j, len, q);
                if (t0 + 4 * J > len && t0 + 4 * j + q >= len) continue;
                if constexpr (decltype(bf)::value) *reinterpret_cast<uint16_t *>(of(g)) = to_bf16(x[j]);
                else *reinterpret_cast<float *>(of(g)) = x[j];
            }
        };
        if (bf16) all(std::true_type{});
        else all(std::false_type{});
    }
};

// x * sigmoid(x) and the sigmoid.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float sigmoid_f(float x) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

// softplus(x) = max(x, 0) + log1p(e), e = exp(-|x|) in (0, 1].  log1p(e) is log(s), s = fl(1 + e), plus what the
// rounding of s left out, e - (s - 1) (exact; its 1 / s is below half a rounding): small e keep their relative
// precision, 2e-7 measured over 2^-30 .. 1, at half the cost of atanh's series.
__device__ __forceinline__ float softplus_f(float x) {
    const float e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(x)), s = 1.f + e;
    return fmaxf(x, 0.f) + fmaf(__builtin_amdgcn_logf(s), 0.6931471805599453f, e - (s - 1.f));
}

// A value of lane I of each quad, in all four lanes.
template <int I>
__device__ __forceinline__ float lane_bcast(float x) {
    return dpp_mov<I * 0x55>(x);
}
// Lane q of each quad gets the quad's sum of v[q].
__device__ __forceinline__ float transpose_sum(const float (&v)[4], int q) {
    const bool b0 = q & 1, b1 = q & 2;
    const float r01 = (b0 ? v[1] : v[0]) + dpp_mov<0xB1>(b0 ? v[0] : v[1]);
    const float r23 = (b0 ? v[3] : v[2]) + dpp_mov<0xB1>(b0 ? v[2] : v[3]);
    return (b1 ? r23 : r01) + dpp_mov<0x4E>(b1 ? r01 : r23);
}
// Sums over the 16 quads of a wave (the lanes that hold the same states of different channels) of four values.
// permlane swaps sum pairs of values over halves and rows at once: row k of 16 lanes ends with value
// quads_sum4_value, which two rotations sum within the row; every lane of the row has the result.
__device__ __forceinline__ float swap_add(float a, float b, bool rows) {
    typedef unsigned u2 __attribute__((ext_vector_type(2)));
    const u2 r = rows ? __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false)
                      : __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float quads_sum4(float v0, float v1, float v2, float v3) {
    float x = swap_add(swap_add(v0, v1, false), swap_add(v2, v3, false), true);
    x += dpp_mov<0x124>(x);         // row rotate by 4
    return x + dpp_mov<0x128>(x);   // by 8
}
// which of the four values a lane ends with: rows 0, 1, 2, 3 hold values 0, 2, 1, 3
__device__ __forceinline__ int quads_sum4_value(int lane) { return ((lane >> 5) & 1) | ((lane >> 3) & 2); }

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
int64_t scan_bwd_threads(const SeqTiles &seq, int dim, int ds);

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
int64_t conv_fwd_threads(int64_t rows, int dim);  // of its largest launch over the rows
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
size_t conv_bwd_workspace_bytes(int64_t rows, int dim, int width, bool bf16);
hipError_t launch_conv_bwd(const ConvBwdLaunch &P);
int64_t conv_bwd_threads(int64_t rows, int dim, bool bf16);

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
int64_t norm_fwd_threads(int64_t rows, int dim);

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

// Sums parts rows of `in`, ld apart, in a fixed order, into up to three outputs that take consecutive runs of the
// columns (a null output's run is skipped) (kda_layer_norm.hip).
struct ColumnSums {
    float *out[3];
    int64_t cols[3];
};
int64_t column_sum_threads(int64_t cols);
void launch_column_sum(const float *in, int64_t ld, int parts, const ColumnSums &to, hipStream_t stream);

}  // namespace kda
