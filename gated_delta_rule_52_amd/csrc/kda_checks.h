// kda_checks.h - what the host entry points of the layer operators share: status texts, the memory of strided tensors and
// its overlaps, strides, launch sizes.
#pragma once

#include <cstdarg>
#include <cstddef>
#include <cstdint>
#include <cstdio>

#include "kda.h"
#include "kda_internal.h"
#include "kda_spans.h"

namespace {

kda_status fail(kda_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
kda_status fail(kda_status s, const char *fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    kda::set_last_error(buf);
    return s;
}

kda_status hip_status(hipError_t e, const char *what) {
    if (e == hipSuccess) return KDA_OK;
    return fail(KDA_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool valid_dtype(kda_dtype d) { return d == KDA_DTYPE_BF16 || d == KDA_DTYPE_FP32; }
int64_t dsize(kda_dtype d) { return d == KDA_DTYPE_BF16 ? 2 : 4; }

using kda::Span;
using kda::overlap;
Span flat(const char *name, const void *p, int64_t bytes) {
    return {name, reinterpret_cast<uintptr_t>(p), 1, bytes, bytes};
}
Span strided(const char *name, const void *p, int64_t rows, int64_t width, int64_t stride, kda_dtype d) {
    return {name, reinterpret_cast<uintptr_t>(p), rows, width * dsize(d), stride * dsize(d)};
}
// Every output against every input and the other outputs.
template <size_t NI, size_t NO>
kda_status check_overlaps(const Span (&ins)[NI], const Span (&outs)[NO]) {
    for (size_t i = 0; i < NO; ++i) {
        for (const Span &s : ins)
            if (overlap(outs[i], s)) return fail(KDA_ERR_ALIAS, "%s overlaps %s", outs[i].name, s.name);
        for (size_t j = i + 1; j < NO; ++j)
            if (overlap(outs[i], outs[j])) return fail(KDA_ERR_ALIAS, "%s overlaps %s", outs[i].name, outs[j].name);
    }
    return KDA_OK;
}

constexpr int64_t kAnyStride = int64_t{1} << 40;

kda_status check_stride(const char *name, const void *p, int64_t stride, int64_t width, int64_t rows, int64_t below) {
    if (p && (stride < width || stride >= below || stride > (int64_t{1} << 40) / (rows > 0 ? rows : 1)))
        return fail(KDA_ERR_BAD_SHAPE, "%s: stride %lld for rows of %lld", name, static_cast<long long>(stride),
                    static_cast<long long>(width));
    return KDA_OK;
}
#define KDA_TRY(x)                          \
    do {                                    \
        const kda_status st_ = (x);         \
        if (st_ != KDA_OK) return st_;      \
    } while (0)

// Threads of one launch stay below 2^32.
kda_status check_grid(int64_t threads) {
    if (threads < 0 || threads >= (int64_t{1} << 32)) return fail(KDA_ERR_UNSUPPORTED, "problem too large for one launch");
    return KDA_OK;
}

template <class A>
kda_status check_struct(const A *a) {
    if (!a) return fail(KDA_ERR_NULL_POINTER, "args is NULL");
    if (a->struct_size != sizeof(A))
        return fail(KDA_ERR_BAD_STRUCT, "struct_size %u (expected %zu)", a->struct_size, sizeof(A));
    return KDA_OK;
}

}  // namespace
