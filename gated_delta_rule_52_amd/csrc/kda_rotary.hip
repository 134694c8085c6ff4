// kda_rotary.hip - rotary positions, and rows of latent vectors and rotated keys into a paged cache.
//
// A pair (a, b) of a head at position p turns by the angle p f of its frequency f:
//     (a, b) -> scale (a cos - b sin, b cos + a sin).
// The angle is formed in 64 bits and reduced to a turn's fraction there: at position 10^6 an angle rounded to fp32 is
// off by up to 0.03.
#include "kda_latent.h"

namespace kda {
namespace {

using namespace la;

// cos and sin of p f, times scale; inverse: of -p f.
__device__ __forceinline__ float2 turn(int p, float f, float scale, int inverse) {
    const double t = static_cast<double>(p) * static_cast<double>(f) * 0.15915494309189535;  // turns
    const float half = 2.f * static_cast<float>(t - __builtin_rint(t));
    float s, c;
    sincospif(half, &s, &c);
    return make_float2(c * scale, (inverse ? -s : s) * scale);
}

// V consecutive elements.
template <class E, int V>
struct Vec {
    E x[V];
};
template <class E, int V>
__device__ __forceinline__ Vec<E, V> load(const E *p) {
    Vec<E, V> v;
    if constexpr (V * sizeof(E) == 16) {
        const u4 w = *reinterpret_cast<const u4 *>(p);
        __builtin_memcpy(v.x, &w, 16);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v.x[i] = p[i];
    }
    return v;
}
template <class E, int V>
__device__ __forceinline__ void store(E *p, const Vec<E, V> &v) {
    if constexpr (V * sizeof(E) == 16) {
        u4 w;
        __builtin_memcpy(&w, v.x, 16);
        *reinterpret_cast<u4 *>(p) = w;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = v.x[i];
    }
}
__device__ __forceinline__ float wide(uint16_t x) { return bf16_to_f32(x); }
__device__ __forceinline__ float wide(float x) { return x; }
__device__ __forceinline__ void narrow(float x, uint16_t &to) { to = __builtin_bit_cast(uint16_t, static_cast<__bf16>(x)); }
__device__ __forceinline__ void narrow(float x, float &to) { to = x; }

// n / d for n d < 2^32, by = ceil(2^32 / d).  The largest here is a head's units, of which there are at most 2^15, by their number.
__device__ __forceinline__ unsigned quotient(unsigned n, unsigned d, unsigned by) { return d == 1 ? n : __umulhi(n, by); }
unsigned reciprocal(unsigned d) { return d == 1 ? 0 : static_cast<unsigned>(((uint64_t{1} << 32) + d - 1) / d); }

// How a workgroup's work is cut: `rows` rows of `heads` heads, each in units: first the rotated part's, V pairs that
// start V apart (halves) or V / 2 adjacent pairs (interleaved), then the copied part's.
struct RotaryCut {
    int rows, heads, groups;  // groups: workgroups per run of rows
    int turned, units;        // per head: rotated units, all units
    unsigned by_units, by_heads, by_pairs;
};

constexpr int kTable = 2048;  // angles of a workgroup

// A workgroup first forms the angles of its rows, once for all their heads, and then turns and copies 16 bytes per lane.  Memory
// bounds it: 16,384 tokens of 32 heads of 192 in bf16 (403 MB both ways) take 77 us, 5.2 TB/s.
template <class E, int V>
__global__ __launch_bounds__(256) void rotary_kernel(const RotaryLaunch P, const RotaryCut C) {
    __shared__ float2 angles[kTable];
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) / C.groups * C.rows;
    const int head0 = static_cast<int>(blockIdx.x % C.groups) * C.heads;
    const int rows = static_cast<int>(min(static_cast<int64_t>(C.rows), P.rows - row0)), heads = min(C.heads, P.heads - head0);
    const unsigned half = P.rot / 2;
    for (unsigned i = threadIdx.x; i < rows * half; i += 256) {
        const unsigned r = quotient(i, half, C.by_pairs), j = i - r * half;
        angles[i] = turn(P.positions[row0 + r], P.inv_freq[j], P.scale, P.inverse);
    }
    __syncthreads();
    for (unsigned i = threadIdx.x; i < static_cast<unsigned>(rows) * heads * C.units; i += 256) {
        const unsigned rh = quotient(i, C.units, C.by_units), u = i - rh * C.units;
        const unsigned r = quotient(rh, C.heads, C.by_heads), h = rh - r * C.heads;
        if (h >= static_cast<unsigned>(heads)) continue;
        const E *x = static_cast<const E *>(P.x.p) + (row0 + r) * P.x.stride + (head0 + h) * P.x.head_stride;
        E *y = static_cast<E *>(P.y.p) + (row0 + r) * P.y.stride + (head0 + h) * P.y.head_stride;
        const float2 *t = angles + r * half;
        if (u >= static_cast<unsigned>(C.turned)) {
            int c = static_cast<int>(u - C.turned) * V;
            if (c >= P.offset) c += P.rot;
            store<E, V>(y + c, load<E, V>(x + c));
        } else if (P.interleaved) {
            constexpr int W = V == 1 ? 2 : V;
            const int c = P.offset + static_cast<int>(u) * W;
            Vec<E, W> v = load<E, W>(x + c);
#pragma unroll
            for (int k = 0; k < W; k += 2) {
                const float2 w = t[u * (W / 2) + k / 2];
                const float a = wide(v.x[k]), b = wide(v.x[k + 1]);
                narrow(a * w.x - b * w.y, v.x[k]);
                narrow(b * w.x + a * w.y, v.x[k + 1]);
            }
            store<E, W>(y + c, v);
        } else {
            const int j = static_cast<int>(u) * V, c = P.offset + j;
            Vec<E, V> a = load<E, V>(x + c), b = load<E, V>(x + c + half);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float2 w = t[j + k];
                const float p = wide(a.x[k]), q = wide(b.x[k]);
                narrow(p * w.x - q * w.y, a.x[k]);
                narrow(q * w.x + p * w.y, b.x[k]);
            }
            store<E, V>(y + c, a);
            store<E, V>(y + c + half, b);
        }
    }
}

bool aligned(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// 16 bytes per access where every head's parts allow it, single elements elsewhere: the rotation above with its part from element 126
// on takes 244 us against 77, two thirds of its cycles for 87 million vector instructions against 20.
bool rotary_wide(const RotaryLaunch &P) {
    const int v = P.bf16 ? 8 : 4;
    auto whole = [&](int64_t n) { return n % v == 0; };
    return aligned(P.x.p, 16) && aligned(P.y.p, 16) && whole(P.x.stride) && whole(P.y.stride) &&
           whole(P.x.head_stride) && whole(P.y.head_stride) && whole(P.offset) && whole(P.dim) &&
           whole(P.interleaved ? P.rot : P.rot / 2);
}

RotaryCut rotary_cut(int64_t rows, int heads, int dim, int rot, int v, bool interleaved) {
    RotaryCut c{};
    c.turned = interleaved ? rot / (v == 1 ? 2 : v) : rot / 2 / v;
    c.units = c.turned + (dim - rot) / v;
    // about 1,024 units per workgroup: heads of a row first, then rows, as many as the table of angles holds
    c.heads = heads < 1024 / c.units ? heads : 1024 / c.units;
    c.heads = c.heads < 1 ? 1 : c.heads;
    c.groups = (heads + c.heads - 1) / c.heads;
    int64_t r = c.groups > 1 ? 1 : 1024 / (static_cast<int64_t>(c.heads) * c.units);
    r = r < 1 ? 1 : r;
    if (rot && r > kTable / (rot / 2)) r = kTable / (rot / 2);
    // fewer rows each where that would leave CUs without work
    const int64_t spread = (rows * c.groups + 511) / 512;
    if (r > spread) r = spread < 1 ? 1 : spread;
    c.rows = static_cast<int>(r);
    c.by_units = reciprocal(c.units);
    c.by_heads = reciprocal(c.heads);
    c.by_pairs = reciprocal(rot / 2);
    return c;
}

RotaryCut rotary_cut(const RotaryLaunch &P) {
    const bool in_place = P.x.p == P.y.p;  // then nothing is copied
    return rotary_cut(P.rows, P.heads, in_place ? P.rot : P.dim, P.rot, !rotary_wide(P) ? 1 : P.bf16 ? 8 : 4, P.interleaved);
}

template <class E, int V>
hipError_t launch(const RotaryLaunch &P) {
    const RotaryCut c = rotary_cut(P);
    const int64_t grid = (P.rows + c.rows - 1) / c.rows * c.groups;
    rotary_kernel<E, V><<<static_cast<unsigned>(grid), 256, 0, P.stream>>>(P, c);
    return hipGetLastError();
}

// ---- the cache ------------------------------------------------------------------------------------------

// A wave per row: its latent part is copied while the angles of the rest are formed.  One decode step's 64 rows take 2.8 us, less
// than a launch; 16,384 rows (38 MB both ways) 9.1 us, what lies above those 2.8 at 6.0 TB/s.
template <class E, int V>
__global__ __launch_bounds__(256) void append_kernel(const AppendLaunch P) {
    const int lane = threadIdx.x & 63;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (row >= P.rows) return;
    const int64_t slot = slot_row(P.slots[row], P.cache_rows);
    if (slot < 0) return;
    const E *c = static_cast<const E *>(P.latent.p) + row * P.latent.stride;
    const E *r = static_cast<const E *>(P.rope.p) + row * P.rope.stride;
    E *to = static_cast<E *>(P.cache) + slot * (P.dl + P.dr);
    for (int i = lane * V; i < P.dl; i += 64 * V) store<E, V>(to + i, load<E, V>(c + i));
    to += P.dl;
    if (!P.inv_freq) {
        for (int i = lane * V; i < P.dr; i += 64 * V) store<E, V>(to + i, load<E, V>(r + i));
        return;
    }
    const int p = P.positions[row], half = P.dr / 2;
    for (int j = lane; j < half; j += 64) {
        const int ia = P.interleaved ? 2 * j : j, ib = P.interleaved ? 2 * j + 1 : j + half;
        const float a = wide(r[ia]), b = wide(r[ib]);
        const float2 w = turn(p, P.inv_freq[j], P.scale, 0);
        narrow(a * w.x - b * w.y, to[ia]);
        narrow(b * w.x + a * w.y, to[ib]);
    }
}

template <class E, int V>
void append(const AppendLaunch &P) {
    append_kernel<E, V><<<static_cast<unsigned>((P.rows + 3) / 4), 256, 0, P.stream>>>(P);
}

}  // namespace

hipError_t launch_rotary(const RotaryLaunch &P) {
    const bool wide_ = rotary_wide(P);
    if (P.bf16) return wide_ ? launch<uint16_t, 8>(P) : launch<uint16_t, 1>(P);
    return wide_ ? launch<float, 4>(P) : launch<float, 1>(P);
}
int64_t rotary_threads(const RotaryLaunch &P) { return P.rows * rotary_cut(P).groups * 256; }  // as if each row had its own workgroups

hipError_t launch_append(const AppendLaunch &P) {
    const int v = P.bf16 ? 8 : 4;
    auto whole = [&](int64_t n) { return n % v == 0; };
    const bool wide_ = aligned(P.latent.p, 16) && aligned(P.rope.p, 16) && aligned(P.cache, 16) && whole(P.latent.stride) &&
                       whole(P.rope.stride) && whole(P.dl) && whole(P.dr);
    if (P.bf16) wide_ ? append<uint16_t, 8>(P) : append<uint16_t, 1>(P);
    else wide_ ? append<float, 4>(P) : append<float, 1>(P);
    return hipGetLastError();
}

}  // namespace kda
