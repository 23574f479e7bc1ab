// heads.hpp -- what the per-head kernels (qknorm.hip, attn.hip) share: the two
// 16-bit types, their packing, and a division by a number known on the host.
#pragma once
#include "ck_device.hpp"

namespace ck {

typedef __bf16 bf16;
typedef _Float16 f16;
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

// What the Infinity Cache behind the XCDs' L2s holds.  A stream of more than
// that finds nothing of itself there on the next call, and loads and stores
// marked nontemporal (not kept) run faster; a smaller one does find it, and they
// run slower.
constexpr int64_t kInfinityCacheBytes = 256 << 20;

// 16 bytes, nontemporal or not.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <bool NT>
__device__ __forceinline__ uint4 load16(const uint16_t* p)
{
    if constexpr (NT) return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)));
    return *reinterpret_cast<const uint4*>(p);
}
template <bool NT>
__device__ __forceinline__ void store16(uint16_t* p, uint4 v)
{
    if constexpr (NT)
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4*>(p));
    else
        *reinterpret_cast<uint4*>(p) = v;
}

// n / d for n < 2^31 and 1 <= d < 2^31 as one high product and a shift, after
// Granlund and Montgomery, "Division by invariant integers using
// multiplication" (1994): with s = ceil(log2 d) - 1 and m = floor(2^(32+s) / d)
// + 1, m d exceeds 2^(32+s) by at most d <= 2^(s+1), so n m / 2^(32+s) exceeds
// n / d by less than n 2^(s+1) / (d 2^(32+s)) < 1 / d and the floor is the same.
struct FastDiv {
    uint32_t d = 1, m = 0, s = 0;
    FastDiv() = default;
    explicit FastDiv(uint32_t div) : d(div)
    {
        if (div <= 1) return;
        while ((2ull << s) < div) ++s;
        m = (uint32_t)((1ull << (32 + s)) / div) + 1u;
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return d == 1 ? n : __umulhi(n, m) >> s; }
};

// Two 16-bit values of a word as FP32.
template <typename T>
__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b)
{
    if constexpr (__is_same(T, f16)) {
        const f16x2_t h = __builtin_bit_cast(f16x2_t, w);
        a = (float)h.x;
        b = (float)h.y;
    } else {
        a = bf16_lo(w);
        b = bf16_hi(w);
    }
}

// Two FP32 values as 16-bit ones, round-to-nearest-even.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if constexpr (__is_same(T, f16)) {
        const f16x2_t h = {(_Float16)a, (_Float16)b};
        return __builtin_bit_cast(uint32_t, h);
    } else {
        return pack_bf16x2(a, b);
    }
}

template <typename T>
__device__ __forceinline__ void unpack8(uint4 r, float (&v)[8])
{
    unpack2<T>(r.x, v[0], v[1]);
    unpack2<T>(r.y, v[2], v[3]);
    unpack2<T>(r.z, v[4], v[5]);
    unpack2<T>(r.w, v[6], v[7]);
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&v)[8])
{
    return make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
}

}  // namespace ck
