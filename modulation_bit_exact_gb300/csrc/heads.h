// heads.h -- argument checks shared by the translation units of the training
// path's C ABI: types, workspaces, and views of heads with the rotation's
// positions, frequencies and axes.  Internal; not part of the ABI.
#pragma once

#include "views.h"

namespace {

// Activations are bfloat16 or binary32, one type a call; parameters have the
// activations' type, or binary32 with bfloat16 activations.
inline bool act_dtype(int32_t d) { return d == MBX_BF16 || d == MBX_F32; }
inline bool param_dtype(int32_t p, int32_t act) { return p == act || p == MBX_F32; }

inline int check_eps(float eps) { return eps >= 0.0f && std::isfinite(eps) ? MBX_OK : MBX_E_ARG; }

// The workspace of a call that needs `need` bytes of it, overlapping none of
// the n views.
inline int check_workspace(const float* ws, int64_t bytes, int64_t need, const V* views, int n) {
    if (!ws) return MBX_E_NULL;
    if (bytes < need) return MBX_E_BOUNDS;
    if (reinterpret_cast<uintptr_t>(ws) % 16) return MBX_E_ALIGN;
    const V w{ws, 1, need / 4, need / 4, MBX_F32};
    MBX_TRY(extent_ok(w));
    for (int i = 0; i < n; ++i)
        if (overlaps(w, views[i])) return MBX_E_ALIAS;
    return MBX_OK;
}

// A heads view in one form.  Strides of dimensions of size 1 address nothing
// and are taken as 0.
struct H4 {
    const void* data;
    int64_t b, t, h, hd, sb, st, sh;
    int32_t dtype;
    int64_t es() const { return esize(dtype); }
    int64_t head_span() const { return (h - 1) * sh + hd; }
    int64_t token_span() const { return (t - 1) * st + head_span(); }
    int64_t span() const { return (b - 1) * sb + token_span(); }
};

template <class W>
H4 of4(const W* w) {
    return H4{w->data,
              w->batch,
              w->tokens,
              w->heads,
              w->head_dim,
              w->batch > 1 ? w->batch_stride : 0,
              w->tokens > 1 ? w->token_stride : 0,
              w->heads > 1 ? w->head_stride : 0,
              w->dtype};
}

inline int basic4(const H4& v) {
    if (!v.data) return MBX_E_NULL;
    if (!act_dtype(v.dtype)) return MBX_E_DTYPE;
    if (v.b <= 0 || v.t <= 0 || v.h <= 0 || v.hd <= 0) return MBX_E_EMPTY;
    if (v.hd > 256) return MBX_E_DIM_TOO_LARGE;
    if (v.h > (int64_t)1 << 20 || v.b > (int64_t)1 << 40 || v.t > (int64_t)1 << 40) return MBX_E_ARG;
    if (v.sb < 0 || v.st < 0 || v.sh < 0) return MBX_E_STRIDE;
    if (reinterpret_cast<uintptr_t>(v.data) % v.es()) return MBX_E_ALIGN;
    int64_t a = 0, bb = 0, c = 0, n = 0, bytes = 0;
    uintptr_t end = 0;
    if (__builtin_mul_overflow(v.b - 1, v.sb, &a) || __builtin_mul_overflow(v.t - 1, v.st, &bb) ||
        __builtin_mul_overflow(v.h - 1, v.sh, &c) || __builtin_add_overflow(a, bb, &n) ||
        __builtin_add_overflow(n, c, &n) || __builtin_add_overflow(n, v.hd, &n) ||
        __builtin_mul_overflow(n, v.es(), &bytes) ||
        __builtin_add_overflow(reinterpret_cast<uintptr_t>(v.data), (uintptr_t)bytes, &end))
        return MBX_E_BOUNDS;
    return MBX_OK;
}

// No two elements of an output share an address: sorted by stride, each
// dimension's stride covers the span of those below it.
inline int injective4(const H4& v) {
    int64_t n[3] = {v.h, v.t, v.b}, s[3] = {v.sh, v.st, v.sb};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (s[j] < s[i]) {
                const int64_t a = n[i], c = s[i];
                n[i] = n[j];
                s[i] = s[j];
                n[j] = a;
                s[j] = c;
            }
    int64_t span = v.hd;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        if (s[i] < span) return MBX_E_STRIDE;
        span += (n[i] - 1) * s[i];
    }
    return MBX_OK;
}

inline bool same4(const H4& a, const H4& b) {
    return a.data == b.data && a.b == b.b && a.t == b.t && a.h == b.h && a.hd == b.hd && a.sb == b.sb &&
           a.st == b.st && a.sh == b.sh;
}

// Whether two views share no element: their address ranges are apart, or they
// repeat with one period (the batch's, the token's or the head's stride) and lie
// in disjoint parts of it, as Q and K inside a merged QKV buffer do.
inline bool disjoint4(const H4& a, const H4& b) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.data), b0 = reinterpret_cast<uintptr_t>(b.data);
    if (a0 + a.span() * a.es() <= b0 || b0 + b.span() * b.es() <= a0) return true;
    if (a.dtype != b.dtype || (b0 > a0 ? b0 - a0 : a0 - b0) % a.es()) return false;
    const bool a_first = a0 <= b0;
    const H4 &lo = a_first ? a : b, &hi = a_first ? b : a;
    const int64_t delta = (int64_t)((a_first ? b0 - a0 : a0 - b0) / a.es());
    auto apart = [&](int64_t period, int64_t span_lo, int64_t span_hi) {
        return period > 0 && delta >= span_lo && delta + span_hi <= period;
    };
    if (a.b > 1 && b.b > 1 && a.sb == b.sb && apart(a.sb, lo.token_span(), hi.token_span())) return true;
    // a dimension of n entries, stride s, whose entries lie whole periods apart
    auto whole = [](int64_t na, int64_t nb, int64_t sa, int64_t sb, int64_t period) {
        return (na == 1 && nb == 1) || (sa == sb && period > 0 && sa % period == 0);
    };
    if (a.t > 1 && b.t > 1 && a.st == b.st && whole(a.b, b.b, a.sb, b.sb, a.st) &&
        apart(a.st, lo.head_span(), hi.head_span()))
        return true;
    return a.h > 1 && b.h > 1 && a.sh == b.sh && whole(a.b, b.b, a.sb, b.sb, a.sh) &&
           whole(a.t, b.t, a.st, b.st, a.sh) && apart(a.sh, a.hd, b.hd);
}

// The power of two up to 16 bytes that every head's start is a multiple of.
inline int align4(const H4& v) {
    const uint64_t bits = reinterpret_cast<uintptr_t>(v.data) | (uint64_t)((v.sb | v.st | v.sh) * v.es()) | 16;
    return (int)(bits & (~bits + 1));
}

inline V flat4(const H4& v) { return V{v.data, 1, v.span(), v.span(), v.dtype}; }

// The rotation's operands as views: positions MBX_I32 or MBX_F32, frequencies MBX_F64.
inline int check_turn_views(const V& pv, const V& fv) {
    if (pv.dtype != MBX_I32 && pv.dtype != MBX_F32) return MBX_E_DTYPE;
    if (fv.dtype != MBX_F64) return MBX_E_DTYPE;
    for (const V* v : {&pv, &fv}) {
        if (v->rows <= 0 || v->cols <= 0) return MBX_E_EMPTY;
        if (!stride_ok(*v)) return MBX_E_STRIDE;
        if (reinterpret_cast<uintptr_t>(v->data) % esize(v->dtype)) return MBX_E_ALIGN;
        MBX_TRY(extent_ok(*v));
    }
    return MBX_OK;
}

// The axes against the heads x, the positions and the frequencies.
inline int check_turn(const H4& x, const V& pv, const V& fv, const int32_t* axes, int n_axes) {
    int64_t tokens = 0;
    if (__builtin_mul_overflow(x.b, x.t, &tokens) || tokens > 0x7fffffff) return MBX_E_ARG;
    if (n_axes < 1 || n_axes > 4) return MBX_E_ARG;
    int64_t rot = 0;
    for (int i = 0; i < n_axes; ++i) {
        if (axes[i] < 2 || axes[i] % 2) return MBX_E_ARG;
        rot += axes[i];
    }
    if (rot > x.hd) return MBX_E_ARG;
    if (pv.cols != n_axes || (pv.rows != x.t && pv.rows != tokens)) return MBX_E_SHAPE;
    if (fv.rows != 1 || fv.cols != rot / 2) return MBX_E_SHAPE;
    return MBX_OK;
}

}  // namespace
