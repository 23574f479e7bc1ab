// views.hpp -- strided views of memory and whether two of them share a byte.
// Plain C++ (marshal.cpp, tests/test_host_headers.py).
#pragma once
#include <cstdint>
#include <initializer_list>

namespace ck {

// The bytes at + sum_i n_i stride[i] + [0, width), 0 <= n_i < size[i].
struct View {
    static constexpr int kDims = 4;
    uintptr_t at = 0;
    int64_t width = 0;   // 0: no bytes
    int dims = 0;
    int64_t size[kDims] = {}, stride[kDims] = {};   // sizes over 1, strides in bytes, over 0

    // A view of n <= 4 dimensions, strides in elements of `bytes` bytes.  Where
    // a stride is 0 the same bytes again are no others.
    static View of(const void* data, int64_t bytes, const int64_t* sizes, const int64_t* strides, int n)
    {
        View v;
        v.at = (uintptr_t)data;
        v.width = bytes;
        for (int i = n - 1; i >= 0; --i) {
            if (sizes[i] == 0) v.width = 0;
            if (sizes[i] < 2 || strides[i] == 0 || v.width == 0) continue;
            const int64_t st = strides[i] * bytes;
            if (st == v.width) {   // follows on without a gap
                v.width *= sizes[i];
            } else {
                v.size[v.dims] = sizes[i];
                v.stride[v.dims++] = st;
            }
        }
        return v;
    }
    // Bytes from the first to the last, over the dimensions of strides below `pitch`.
    int64_t extent(int64_t pitch) const
    {
        int64_t n = width;
        for (int i = 0; i < dims; ++i)
            if (stride[i] < pitch) n += (size[i] - 1) * stride[i];
        return n;
    }
    // Whether no byte is part of two elements: each stride is at least the extent
    // of all smaller ones.
    bool distinct() const
    {
        for (int i = 0; i < dims; ++i)
            if (stride[i] < extent(stride[i])) return false;
        for (int i = 0; i < dims; ++i)
            for (int j = 0; j < i; ++j)
                if (stride[i] == stride[j]) return false;
        return true;
    }
    bool rows_of(int64_t pitch) const   // whether all its larger strides are multiples of pitch
    {
        for (int i = 0; i < dims; ++i)
            if (stride[i] >= pitch && stride[i] % pitch != 0) return false;
        return true;
    }
};

// Whether a and b share no byte: one ends before the other begins, or both are
// column ranges of rows of one pitch (any stride of theirs) and the ranges are
// apart.  Views that are apart for neither reason count as sharing.
inline bool disjoint(const View& a, const View& b)
{
    if (a.width == 0 || b.width == 0) return true;
    if (a.at + a.extent(INT64_MAX) <= b.at || b.at + b.extent(INT64_MAX) <= a.at) return true;
    for (const View* v : {&a, &b}) {
        for (int i = 0; i < v->dims; ++i) {
            const int64_t pitch = v->stride[i];
            if (!a.rows_of(pitch) || !b.rows_of(pitch)) continue;
            int64_t gap = (int64_t)(b.at - a.at) % pitch;   // b's columns start `gap` after a's
            if (gap < 0) gap += pitch;
            if (a.extent(pitch) <= gap && gap + b.extent(pitch) <= pitch) return true;
        }
    }
    return false;
}

}  // namespace ck
