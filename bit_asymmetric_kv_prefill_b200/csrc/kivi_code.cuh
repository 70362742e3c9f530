// kivi_code.cuh -- device helpers of the quantizers: 16-bit inputs, the code
// thresholds of a group as input values, and asynchronous copies into shared
// memory.  Internal to the library.
#pragma once

#include <cstring>

#include "kivi_common.cuh"

namespace kivi {

// ---- input dtype helpers (bits are carried as uint16 / packed uint32) ----------
template <int DT>
struct In;

template <>
struct In<1> {  // bfloat16
    static constexpr uint16_t kInf = 0x7F80u, kNegInf = 0xFF80u;
    __device__ static float f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
    __device__ static uint16_t from_float_rd(float y) { return __bfloat16_as_ushort(__float2bfloat16_rd(y)); }
    __device__ static __nv_bfloat162 v(uint32_t u)
    {
        __nv_bfloat162 r;
        memcpy(&r, &u, 4);
        return r;
    }
    __device__ static uint32_t u(__nv_bfloat162 x)
    {
        uint32_t r;
        memcpy(&r, &x, 4);
        return r;
    }
    __device__ static uint32_t vmin(uint32_t a, uint32_t b) { return u(__hmin2(v(a), v(b))); }
    __device__ static uint32_t vmax(uint32_t a, uint32_t b) { return u(__hmax2(v(a), v(b))); }
    __device__ static uint32_t ge_mask(uint32_t a, uint32_t b) { return __hge2_mask(v(a), v(b)); }
};

template <>
struct In<0> {  // IEEE fp16
    static constexpr uint16_t kInf = 0x7C00u, kNegInf = 0xFC00u;
    __device__ static float f(uint16_t b) { return __half2float(__ushort_as_half(b)); }
    __device__ static uint16_t from_float_rd(float y) { return __half_as_ushort(__float2half_rd(y)); }
    __device__ static __half2 v(uint32_t u)
    {
        __half2 r;
        memcpy(&r, &u, 4);
        return r;
    }
    __device__ static uint32_t u(__half2 x)
    {
        uint32_t r;
        memcpy(&r, &x, 4);
        return r;
    }
    __device__ static uint32_t vmin(uint32_t a, uint32_t b) { return u(__hmin2(v(a), v(b))); }
    __device__ static uint32_t vmax(uint32_t a, uint32_t b) { return u(__hmax2(v(a), v(b))); }
    __device__ static uint32_t ge_mask(uint32_t a, uint32_t b) { return __hge2_mask(v(a), v(b)); }
};

// Neighbours in value order of a 16-bit sign-magnitude float (both zeros are
// the value 0; the infinities are fixed points).
template <int DT>
__device__ __forceinline__ uint16_t next_up(uint16_t b)
{
    // Value order: +-0 -> smallest positive subnormal, negatives step towards
    // zero, positives away from it, +inf stays (selects, no branches).
    const uint16_t up = (b & 0x8000u) ? (uint16_t)(b - 1) : (uint16_t)(b + 1);
    const uint16_t r = (b & 0x7fffu) == 0 ? (uint16_t)0x0001u : up;
    return b == In<DT>::kInf ? b : r;
}
template <int DT>
__device__ __forceinline__ uint16_t next_down(uint16_t b)
{
    if ((b & 0x7fffu) == 0) return 0x8001u;
    if (b & 0x8000u) return b == In<DT>::kNegInf ? b : (uint16_t)(b + 1);
    return (uint16_t)(b - 1);
}

// Does input value x reach threshold e: fl32(x - z) > e (the definition's
// fp32 subtraction, compared against the exact fp32 bound)?
template <int DT>
__device__ __forceinline__ bool passes(uint16_t x, float e, float z)
{
    return __fsub_rn(In<DT>::f(x), z) > e;
}

// Smallest input value x (as bits) with fl32(x - z) > e; +inf when none.
// fl32(x - z) is non-decreasing in x, so {x : passes} is an upper set.  The
// start c = RD_dtype(RD_fp32(z + e)) satisfies c - z <= e (rounding to
// nearest is monotone and e is an fp32 value), so it never passes.  Its
// successor x1 lies above z + e, so it passes whenever x1 - z is exact in
// fp32, i.e. unless x1 and z are many binades apart; otherwise stepping on,
// and after three more steps a binary search over the value-ordered 16-bit
// patterns, settles it.
template <int DT>
__device__ __noinline__ uint16_t min_passing_slow(uint16_t x, float e, float z);

template <int DT>
__device__ __forceinline__ uint16_t min_passing(float e, float z)
{
    if (!(e < __int_as_float(0x7f800000))) return In<DT>::kInf;
    const uint16_t c = In<DT>::from_float_rd(__fadd_rd(z, e));
    // The successor of c in value order (c is finite: a rounding down of a
    // finite sum never gives +inf).
    const uint16_t x1 = (c & 0x7fffu) == 0 ? (uint16_t)0x0001u
                        : (c & 0x8000u)    ? (uint16_t)(c - 1)
                                           : (uint16_t)(c + 1);
    if (passes<DT>(x1, e, z)) return x1;
    return min_passing_slow<DT>(x1, e, z);
}

// Continuation from x (not passing): three more steps, then a bisection.
template <int DT>
__device__ __noinline__ uint16_t min_passing_slow(uint16_t x, float e, float z)
{
#pragma unroll 1
    for (int i = 0; i < 3; ++i) {
        x = next_up<DT>(x);
        if (passes<DT>(x, e, z)) return x;
    }
    // Value-order key of a pattern: negatives reversed below the positives.
    auto key_bits = [](int k) -> uint16_t {
        return k < 0x8000 ? (uint16_t)(0xffff - k) : (uint16_t)(k - 0x8000);
    };
    int lo = 0x8000 - (In<DT>::kInf & 0x7fff), hi = 0x8000 + In<DT>::kInf;  // -inf .. +inf
#pragma unroll 1
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (passes<DT>(key_bits(mid), e, z)) hi = mid;
        else lo = mid + 1;
    }
    return key_bits(lo);
}

// Two codes of a channel pair x against packed thresholds t1..t3, placed at
// the word bits K1 (0x00010001 << 2i) and K3 (0x00030003 << 2i) of pair i.
// Masks m_k are 0xffff per half where x >= t_k; as m1 >= m2 >= m3, bit 1 of
// a code is m2 and bit 0 is m1 ^ m2 ^ m3.
template <int DT>
__device__ __forceinline__ uint32_t code_pair_at(uint32_t x, uint32_t t1, uint32_t t2, uint32_t t3, uint32_t K1,
                                                 uint32_t K3)
{
    const uint32_t m1 = In<DT>::ge_mask(x, t1), m2 = In<DT>::ge_mask(x, t2), m3 = In<DT>::ge_mask(x, t3);
    uint32_t a, r;
    asm("lop3.b32 %0, %1, %2, %3, 0x28;" : "=r"(a) : "r"(m1), "r"(m3), "r"(K1));  // (m1^m3)&K1
    asm("lop3.b32 %0, %1, %2, %3, 0x78;" : "=r"(r) : "r"(a), "r"(m2), "r"(K3));   // a^(m2&K3)
    return r;
}

// Packed (a.lo, b.lo) and (a.hi, b.hi) of two 16-bit pairs.
__device__ __forceinline__ uint32_t lo_halves(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
__device__ __forceinline__ uint32_t hi_halves(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

__device__ __forceinline__ void cp_async16(void *smem, const void *gmem)
{
    const uint32_t s = (uint32_t)__cvta_generic_to_shared(smem);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(gmem) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

}  // namespace kivi
