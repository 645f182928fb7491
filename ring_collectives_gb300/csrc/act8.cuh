// act8.cuh -- rows of bf16 activations and their 8-bit form, in registers: eight
// channels a thread, four neighbouring lanes a group of 32.
//
// A group's power of two is the least 2^k with max |x| <= 127 * 2^k.  For a bf16
// maximum (1 + m / 128) 2^E that is E - 6, or E - 5 when m = 127: adding one to
// the maximum's bits carries into the exponent exactly then.
#pragma once
#include <stdint.h>

#include "dev.cuh"
#include "f32x2.cuh"
#include "ringcoll.h"

namespace rc {

typedef uint64_t f32x2;

// ------------------------------------------------------------ places
struct Rows {
    char *base;
    size_t slot, row;
    __device__ __forceinline__ char *at(uint32_t r, uint32_t t) const { return base + r * slot + t * row; }
};
struct Act8 {
    Rows q, e;                       // q.base null: not given
};

// n / d for 0 <= n < 2^31 and 1 <= d < 2^31, by one high product: with 2^(l-1) < d <= 2^l
// and m = ceil(2^(31+l) / d) the error n (m d - 2^(31+l)) / d is below 2^(31+l) / d.
struct FastDiv {
    uint32_t d, m, s;
    static FastDiv of(uint32_t d)
    {
        uint32_t l = 0;
        while ((1ull << l) < d) ++l;
        if (l == 0) return FastDiv{1, 0, 0};
        return FastDiv{d, (uint32_t)(((1ull << (31 + l)) + d - 1) / d), l - 1};
    }
    __host__ __device__ __forceinline__ uint32_t operator()(uint32_t n) const
    {
        const uint32_t q = (uint32_t)(((uint64_t)n * m) >> 32) >> s;
        return d == 1 ? n : q;
    }
};

// Elementwise work on [P][T][N]: all rows behind one another, 16 channels a lane and two
// neighbouring lanes a group of 32, so that groups never leave a warp and narrow rows fill
// it too.
struct Flat {
    FastDiv lanes, tokens;           // lanes of a row: 2 ceil(N / 32); rows of a slot
    uint32_t rows, N;
    static Flat of(int P, int T, int N)
    {
        return Flat{FastDiv::of(2u * (uint32_t)((N + 31) / 32)), FastDiv::of((uint32_t)T), (uint32_t)P * (uint32_t)T, (uint32_t)N};
    }
    // blocks of `lanes_a_block` lanes, an even number
    uint64_t blocks(uint32_t lanes_a_block) const { return ((uint64_t)rows * lanes.d + lanes_a_block - 1) / lanes_a_block; }
};
// Place of lane `off` behind the first lane (row0, rem0) of a block: channels c.. of row t
// of slot r, if `on`; the last 8 of the 16 exist if `all`.
struct Spot {
    uint32_t r, t, c;
    bool on, all;
    __device__ __forceinline__ Spot(const Flat &f, uint32_t row0, uint32_t rem0, uint32_t off)
    {
        const uint32_t d = f.lanes(rem0 + off), row = row0 + d;
        c = (rem0 + off - d * f.lanes.d) * 16;
        on = row < f.rows && c < f.N;
        all = on && c + 8 < f.N;
        r = f.tokens(row);
        t = row - r * f.tokens.d;
    }
};

// ------------------------------------------------------------ eight channels
__device__ __forceinline__ float lo(f32x2 v)
{
    float a, b;
    unf2(v, a, b);
    return a;
}
__device__ __forceinline__ float hi(f32x2 v)
{
    float a, b;
    unf2(v, a, b);
    return b;
}
__device__ __forceinline__ float hsum(f32x2 v) { return lo(v) + hi(v); }
__device__ __forceinline__ f32x2 both(float a) { return f2(a, a); }

__device__ __forceinline__ f32x2 wide2(uint32_t w) { return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
__device__ __forceinline__ void wide8(const uint4 &w, f32x2 (&f)[4])
{
    f[0] = wide2(w.x);
    f[1] = wide2(w.y);
    f[2] = wide2(w.z);
    f[3] = wide2(w.w);
}
__device__ __forceinline__ uint32_t narrow2(f32x2 v)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi(v)), "f"(lo(v)));
    return r;
}
__device__ __forceinline__ uint4 narrow8(const f32x2 (&f)[4])
{
    return make_uint4(narrow2(f[0]), narrow2(f[1]), narrow2(f[2]), narrow2(f[3]));
}

// ------------------------------------------------------------ 8 bits
// The values of 8 bytes with their group's byte e.  A byte b + 128 as the low bits of 2^23
// gives an exact difference, and a power of two an exact product; e = 255 is an infinity,
// which makes a NaN of a zero.
__device__ __forceinline__ void bytes8(const uint2 &q, f32x2 (&f)[4])
{
    const f32x2 zero = both(-8388736.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = (i < 2 ? q.x : q.y) ^ 0x80808080u;
        const uint32_t a = __byte_perm(w, 0x4B000000u, i & 1 ? 0x7652 : 0x7650);
        const uint32_t b = __byte_perm(w, 0x4B000000u, i & 1 ? 0x7653 : 0x7651);
        f[i] = add2(f2(__uint_as_float(a), __uint_as_float(b)), zero);
    }
}
__device__ __forceinline__ void held8(const uint2 &q, uint32_t e, f32x2 (&f)[4])
{
    const f32x2 scale = both(__uint_as_float(e << 23));
    bytes8(q, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], scale);
}

// The same in one multiply-add, for e <= kLowMost (gemm_wgrad of 8 x 768x4096 over 8192 tokens: 260 -> 255
// us): above, 2^23 + 128 times the power of two, 2^104 there, is no number.
constexpr uint32_t kLowMost = 231;
__device__ __forceinline__ void held8_low(const uint2 &q, uint32_t e, f32x2 (&f)[4])
{
    const float s = __uint_as_float(e << 23);
    const f32x2 scale = both(s), bias = both(s * -8388736.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = (i < 2 ? q.x : q.y) ^ 0x80808080u;
        const uint32_t a = __byte_perm(w, 0x4B000000u, i & 1 ? 0x7652 : 0x7650);
        const uint32_t b = __byte_perm(w, 0x4B000000u, i & 1 ? 0x7653 : 0x7651);
        f[i] = fma2(f2(__uint_as_float(a), __uint_as_float(b)), scale, bias);
    }
}

// The larger of each pair of halves, as unsigned numbers: for magnitudes of bf16 numbers
// their order, infinities and NaNs above all.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The 8-bit form of V vectors of 8 bf16 channels; all 32 lanes call it, and 4 / V neighbouring
// lanes hold a group (zeros behind a row's end).  The sum x 2^-k + 1.5 * 2^23 rounds to the
// nearest integer, ties to even, and leaves it in the low byte.
template <int V>
__device__ __forceinline__ void pack8(const uint4 (&w)[V], uint2 (&q)[V], uint32_t &e)
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
        top = max2(max2(top, max2(w[i].x & 0x7FFF7FFFu, w[i].y & 0x7FFF7FFFu)), max2(w[i].z & 0x7FFF7FFFu, w[i].w & 0x7FFF7FFFu));
#pragma unroll
    for (int o = 1; o < 4 / V; o *= 2) top = max2(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    top = max(top & 0xFFFFu, top >> 16);
    const int k = min(max((int)((top + 1u) >> 7) - 6, 1), 248);
    const f32x2 scale = both(__uint_as_float((uint32_t)(254 - k) << 23)), magic = both(12582912.f);
    e = top >= 0x7F80u ? 255u : (uint32_t)k;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        f32x2 f[4];
        wide8(w[i], f);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = fma2(f[j], scale, magic);
        if (top >= 0x7F7Fu) {                  // the largest bf16 number is 127.5 * 2^121; what is not finite is 0
#pragma unroll
            for (int j = 0; j < 4; ++j)
                f[j] = top > 0x7F7Fu ? magic
                                     : f2(fminf(fmaxf(lo(f[j]), 12582912.f - 127.f), 12582912.f + 127.f),
                                          fminf(fmaxf(hi(f[j]), 12582912.f - 127.f), 12582912.f + 127.f));
        }
        uint32_t r[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) r[2 * j] = __float_as_uint(lo(f[j])), r[2 * j + 1] = __float_as_uint(hi(f[j]));
        q[i].x = __byte_perm(__byte_perm(r[0], r[1], 0x0040), __byte_perm(r[2], r[3], 0x0040), 0x5410);
        q[i].y = __byte_perm(__byte_perm(r[4], r[5], 0x0040), __byte_perm(r[6], r[7], 0x0040), 0x5410);
    }
}

// Vector v (channels 8 v..) of a row to its place, four lanes a group; lane 4 i writes the
// group's byte.
__device__ __forceinline__ void put8(const Act8 &o, uint32_t r, uint32_t t, uint32_t v, bool on, const uint4 &w)
{
    const uint4 one[1] = {w};
    uint2 q[1];
    uint32_t e;
    pack8(one, q, e);
    if (!on) return;
    __stcs((uint2 *)(o.q.at(r, t) + v * 8), q[0]);
    if (v % 4 == 0) *(uint8_t *)(o.e.at(r, t) + v / 4) = (uint8_t)e;
}

// ------------------------------------------------------------ 16 channels of a Spot
// WIDE: bf16 rows on 32-byte and bytes on 16-byte boundaries, N a multiple of 16.
template <bool WIDE>
__device__ __forceinline__ void get16(const Rows &o, const Spot &s, uint4 (&w)[2])
{
    w[0] = w[1] = make_uint4(0, 0, 0, 0);
    if (!s.on) return;
    const char *const p = o.at(s.r, s.t) + s.c * 2;
    if (WIDE) {
        ld8_ef(p, w[0], w[1]);
    } else {
        w[0] = __ldcs((const uint4 *)p);
        if (s.all) w[1] = __ldcs((const uint4 *)p + 1);
    }
}
template <bool WIDE>
__device__ __forceinline__ void set16(const Rows &o, const Spot &s, const uint4 &a, const uint4 &b)
{
    if (!s.on) return;
    char *const p = o.at(s.r, s.t) + s.c * 2;
    if (WIDE) {
        st8<kStEvictFirst>(p, a, b);
    } else {
        __stcs((uint4 *)p, a);
        if (s.all) __stcs((uint4 *)p + 1, b);
    }
}
template <bool WIDE>
__device__ __forceinline__ void get16(const Act8 &o, const Spot &s, uint4 &q, uint32_t &e)
{
    q = make_uint4(0, 0, 0, 0);
    e = 1;
    if (!s.on) return;
    const char *const p = o.q.at(s.r, s.t) + s.c;
    e = __ldcs((const uint8_t *)o.e.at(s.r, s.t) + s.c / 32);
    if (WIDE) {
        q = __ldcs((const uint4 *)p);
    } else {
        const uint2 a = __ldcs((const uint2 *)p);
        q.x = a.x;
        q.y = a.y;
        if (!s.all) return;
        const uint2 b = __ldcs((const uint2 *)p + 1);
        q.z = b.x;
        q.w = b.y;
    }
}
template <bool WIDE>
__device__ __forceinline__ void set16(const Act8 &o, const Spot &s, const uint4 (&w)[2])
{
    uint2 q[2];
    uint32_t e;
    pack8(w, q, e);
    if (!s.on) return;
    char *const p = o.q.at(s.r, s.t) + s.c;
    if (WIDE) {
        __stcs((uint4 *)p, make_uint4(q[0].x, q[0].y, q[1].x, q[1].y));
    } else {
        __stcs((uint2 *)p, q[0]);
        if (s.all) __stcs((uint2 *)p + 1, q[1]);
    }
    if (s.c % 32 == 0) *(uint8_t *)(o.e.at(s.r, s.t) + s.c / 32) = (uint8_t)e;
}

// ------------------------------------------------------------ host
inline Rows rows_of(const rc_rows &r) { return Rows{(char *)r.base, r.slot, r.row}; }
inline bool wide_of(const rc_rows &r, size_t bytes) { return !(((uintptr_t)r.base | r.slot | r.row) & (bytes - 1)); }
inline Act8 act8_of(const rc_act8 &a) { return Act8{rows_of(a.q), rows_of(a.e)}; }

} // namespace rc
