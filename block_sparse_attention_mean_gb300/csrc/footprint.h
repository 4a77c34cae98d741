// footprint.h -- host checks of strided tensors shared by the C entry points (block_api.cu, cache_api.cu): alignment,
// strides, and which outputs may overlap what. Not part of the public C ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cstring>

namespace {

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The bytes that a strided tensor covers: three dimensions (sizes, byte strides) of `inner` bytes each.
struct Footprint {
    uintptr_t at, end;  // end: one past the last
    int64_t size[3], stride[3], inner;

    // bytes from the first to one past the last, over dimensions whose stride is below `under`
    int64_t span(int64_t under) const
    {
        int64_t s = inner;
        for (int i = 0; i < 3; ++i)
            if (stride[i] < under) s += (size[i] - 1) * stride[i];
        return s;
    }
};

// Strides for the kernels: non-negative multiples of 16 bytes, the whole tensor within the address space.
// A dimension of length one gets stride 0: it is never stepped.
inline bool make_footprint(const void *p, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t inner,
                    int elem, Footprint *f)
{
    if (!p || !aligned(p, 16)) return false;
    f->at = reinterpret_cast<uintptr_t>(p);
    const int64_t n[3] = {n0, n1, n2}, s[3] = {s0, s1, s2};
    double end = static_cast<double>(inner) * elem;
    for (int i = 0; i < 3; ++i) {
        f->size[i] = n[i];
        f->stride[i] = 0;
        if (n[i] <= 1) continue;
        if (s[i] < 0 || s[i] > (INT64_MAX >> 8) || s[i] * elem % 16 != 0) return false;
        f->stride[i] = s[i] * elem;
        end += static_cast<double>(n[i] - 1) * static_cast<double>(f->stride[i]);
    }
    f->inner = inner * elem;
    if (end >= 4.0e18) return false;
    f->end = f->at + f->span(INT64_MAX);
    return true;
}

// `count` of `bytes` each, `step` bytes apart, at any address
inline Footprint block_of(const void *p, int64_t bytes, int64_t count = 1, int64_t step = 0)
{
    Footprint f{};
    f.at = reinterpret_cast<uintptr_t>(p);
    f.size[0] = count, f.size[1] = f.size[2] = 1;
    f.stride[0] = count > 1 ? step : 0;
    f.inner = bytes;
    f.end = f.at + f.span(INT64_MAX);
    return f;
}

// Whether no two elements of an output share an address: each stride steps over what lies below it.
inline bool steps_clear(const Footprint &f)
{
    for (int i = 0; i < 3; ++i) {
        if (f.size[i] <= 1) continue;
        if (f.stride[i] < f.span(f.stride[i])) return false;
        for (int j = 0; j < i; ++j)
            if (f.size[j] > 1 && f.stride[j] == f.stride[i]) return false;
    }
    return true;
}

// Whether a (an output: steps_clear) and b are shown to be disjoint: by their address ranges, or, with the same
// strides, because they lie beside each other within one step of some dimension.
inline bool disjoint(const Footprint &a, const Footprint &b)
{
    if (a.end <= b.at || b.end <= a.at) return true;
    const Footprint &lo = a.at <= b.at ? a : b, &hi = a.at <= b.at ? b : a;
    int64_t step[3];
    for (int i = 0; i < 3; ++i) {
        if (a.stride[i] != b.stride[i] && a.stride[i] && b.stride[i]) return false;
        step[i] = a.stride[i] > b.stride[i] ? a.stride[i] : b.stride[i];
    }
    const int64_t delta = static_cast<int64_t>(hi.at - lo.at);
    for (int i = 0; i < 3; ++i) {
        const int64_t s = step[i];
        if (s == 0) continue;
        bool beside = delta >= lo.span(s) && delta + hi.span(s) <= s;
        for (int j = 0; j < 3 && beside; ++j)  // and no step of an outer dimension brings them together
            if (step[j] > s) beside = lo.span(step[j]) <= step[j] && delta + hi.span(step[j]) <= step[j];
        for (int j = 0; j < 3 && beside; ++j)
            if (j != i && step[j] == s) beside = false;
        if (beside) return true;
    }
    return false;
}

inline bool same(const Footprint &a, const Footprint &b)
{
    return a.at == b.at && a.inner == b.inner && std::memcmp(a.size, b.size, sizeof(a.size)) == 0 &&
           std::memcmp(a.stride, b.stride, sizeof(a.stride)) == 0;
}

// What a call reads and writes, weights, modulations, positions and the workspace among it: outputs must be clear of
// themselves, of each other and of every input but those they may replace.
struct Tensors {
    static constexpr int kMax = 12;
    Footprint in[kMax], out[kMax];
    int n_in = 0, n_out = 0;
    unsigned may_be[kMax];  // out[i] may be in[k] for the bits k

    // a contiguous operand, where there is one
    void reads(const void *p, int64_t bytes)
    {
        if (p) in[n_in++] = block_of(p, bytes);
    }
    void writes(const void *p, int64_t bytes)
    {
        if (!p) return;
        may_be[n_out] = 0;
        out[n_out++] = block_of(p, bytes);
    }

    bool check() const
    {
        for (int i = 0; i < n_out; ++i) {
            if (!steps_clear(out[i])) return false;
            for (int j = 0; j < i; ++j)
                if (!disjoint(out[i], out[j])) return false;
            for (int k = 0; k < n_in; ++k) {
                if ((may_be[i] >> k & 1u) && same(out[i], in[k])) continue;
                if (!disjoint(out[i], in[k])) return false;
            }
        }
        return true;
    }
};

}  // namespace
