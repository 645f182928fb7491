// qk_norm.cu -- RMS norm of every query and key head and the rotary position
// rotation in one pass, and its gradient.
//
//   r = (mean_i x_i^2 + eps)^(-1/2),  y = x r g,
//   (z_a, z_b) = (y_a cos - y_b sin, y_a sin + y_b cos)
// for every rotated pair (a, b) of the head: (i, i + D/2) or (2i, 2i + 1).
// Gradient: dy is dz rotated back; with xh = x r and t = dy g,
//   dx = r (t - xh mean_i(t_i xh_i)),   dg = sum over rows of dy xh.
//
// Bound by memory: each head is read and written once (three passes in the
// gradient), the rows of cos and sin once per token, rank and run of heads.
// Lanes hold two chunks of V elements, c and c + D/2 further on, so both
// members of either kind of pair are in one thread and only the mean crosses
// lanes: a group of D / 2V lanes (rounded up to a power of two) covers a head.
// All arithmetic is on pairs of binary32 (one issue slot for two), and norm
// weight and rotation become two factors an element, z = r (x a + x' b) with x'
// the element's partner, formed once per token for a run of heads: with the
// plain formula the kernel was bound by issue, not by memory.
//
// Measured: 16383 tokens x 8 ranks x 5 heads of 128, 65.5 us, 5.25 TB/s with the
// tables (79 % of the copy rate; ncu: issue slots 42 % busy); the gradient on 8192
// tokens, 46.7 us + 2.5 us for the sums of the weight gradient, 5.2 TB/s.
#include <climits>
#include <cmath>
#include <cuda_bf16.h>

#include "internal.h"
#include "ringcoll.h"
#include "dev.cuh"
#include "f32x2.cuh"
#include "heads.h"
#include "per_device.h"

namespace rc {
namespace qkn {

constexpr int THREADS = 128;     // three blocks per SM: up to 168 registers, 576 bytes of staging a thread
constexpr int STAGES = 3;        // steps of a thread's staging ring
constexpr int HB = 4;            // heads of a step of qk_norm_rope
constexpr int GB = 2;            // heads of a step of its gradient (two tensors)

struct Heads {
    char *base;
    size_t slot, token, head;
};

struct Params {
    Heads x[2], z[2], dx[2];     // query and key heads: inputs, (gradients of the) outputs, input gradients
    const float *g[2], *cos, *sin;
    const int32_t *pos;
    float *part;                 // gradient: [blocks of a slot][slot][2][D] partial weight gradients
    float *dg[2];                // [P][D]
    int P, T, H[2], D, npos, pairs;
    int blocks;                  // gradient: rows of `part`
    int clear;                   // gradient: 1: `part` is zeroed once read (a caller's workspace)
    float eps;
};

// ------------------------------------------------------------ pairs of binary32
typedef uint64_t f32x2;
__device__ __forceinline__ f32x2 swap(f32x2 v)
{
    float a, b;
    unf2(v, a, b);
    return f2(b, a);
}
__device__ __forceinline__ float hsum(f32x2 v)
{
    float a, b;
    unf2(v, a, b);
    return a + b;
}

// ------------------------------------------------------------ staging
// Every thread copies what it will use itself into its own shared-memory slots
// (cp.async, STAGES - 1 steps ahead) and reads it back: no barrier, and the
// loads in flight do not depend on registers or on which phase a block is in.
// Loading into registers instead, with whole blocks taking turns, reached
// 4.6 TB/s on 16383 tokens x 8 ranks x 5 heads of 128.
// A slot: W chunks of V elements, then V cosines and V sines.
template <int V, int W>
struct Stage {
    static constexpr int CHUNK = 2 * V, BYTES = W * CHUNK + 8 * V;
    static constexpr int TOTAL = STAGES * BYTES * THREADS;
    // 16-byte pieces (8 for V = 4) of the threads side by side: no bank conflicts
    static __device__ __forceinline__ uint32_t chunk(uint32_t base, int stage, int i)
    {
        return base + stage * (BYTES * THREADS) + (i * THREADS + threadIdx.x) * CHUNK;
    }
    // piece i of 16 bytes of the angles: V / 4 of cosines, V / 4 of sines
    static __device__ __forceinline__ uint32_t angle(uint32_t base, int stage, int i)
    {
        return base + stage * (BYTES * THREADS) + W * CHUNK * THREADS + (i * THREADS + threadIdx.x) * 16;
    }
};

template <int B>
__device__ __forceinline__ void copy(uint32_t dst, const void *src)
{
    if (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void wait_oldest() { asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory"); }
__device__ __forceinline__ void lds4(uint32_t a, uint32_t &x, uint32_t &y, uint32_t &z, uint32_t &w)
{
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x), "=r"(y), "=r"(z), "=r"(w) : "r"(a) : "memory");
}

// A thread's share of a head: V elements from c and V from c + D/2, as the
// pairs 2i, 2i + 1 of the first chunk, then of the second.
template <int V>
__device__ __forceinline__ void take(uint32_t lo, uint32_t hi, f32x2 (&f)[V])
{
    uint32_t w[V];
    if (V == 8) {
        lds4(lo, w[0], w[1], w[2], w[3]);
        lds4(hi, w[V - 4], w[V - 3], w[V - 2], w[V - 1]);
    } else {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(lo) : "memory");
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[2]), "=r"(w[3]) : "r"(hi) : "memory");
    }
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t pack(f32x2 v)
{
    float a, b;
    uint32_t r;
    unf2(v, a, b);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

template <int V>
__device__ __forceinline__ void st(char *p, int half_bytes, const f32x2 (&f)[V])
{
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (V == 8)
            __stcs((uint4 *)(p + k * half_bytes), make_uint4(pack(f[4 * k]), pack(f[4 * k + 1]), pack(f[V / 2 * k + 2]), pack(f[V / 2 * k + V / 2 - 1])));
        else
            __stcs((uint2 *)(p + k * half_bytes), make_uint2(pack(f[2 * k]), pack(f[2 * k + 1])));
}

// The elements' partners: the other chunk, or the other element of the pair.
template <int V, bool PAIRS>
__device__ __forceinline__ void partners(const f32x2 (&f)[V], f32x2 (&q)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) q[i] = PAIRS ? swap(f[i]) : f[(i + V / 2) % V];
}

// 2V floats in the same order.
template <int V>
__device__ __forceinline__ void ldf(const float *p, int half, f32x2 (&f)[V])
{
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 v = __ldg((const float4 *)(p + k * half + i));
            f[k * V / 2 + i / 2] = f2(v.x, v.y);
            f[k * V / 2 + i / 2 + 1] = f2(v.z, v.w);
        }
}

// Sum over the L lanes of a group.
template <int L>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Starts the copies of position pos's angles: with halves the V angles from c
// (both chunks turn by them), with adjacent pairs the V / 2 from c / 2 and the
// V / 2 from D / 4 + c / 2.  A position outside the table gives NaN.
template <int V, int W, bool PAIRS>
__device__ __forceinline__ void fetch_angles(const Params &p, uint32_t base, int stage, int pos, int c)
{
    using S = Stage<V, W>;
    if (pos < 0 || pos >= p.npos) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(S::angle(base, stage, i)), "r"(0x7FC00000) : "memory");
        return;
    }
    const size_t row = (size_t)pos * (p.D / 2);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float *const t = (k ? p.sin : p.cos) + row;
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const uint32_t dst = S::angle(base, stage, k * (V / 4) + i);
            if (!PAIRS) {
                copy<16>(dst, t + c + 4 * i);
            } else if (V == 8) {
                copy<16>(dst, t + i * (p.D / 4) + c / 2);
            } else {
                copy<8>(dst, t + c / 2);
                copy<8>(dst + 8, t + p.D / 4 + c / 2);
            }
        }
    }
}

// cos of every element's angle, and sin with the sign it has on the element's
// partner in the forward rotation: z = x cs + x' sn.
template <int V, int W, bool PAIRS>
__device__ __forceinline__ void angles(uint32_t base, int stage, f32x2 (&cs)[V], f32x2 (&sn)[V])
{
    using S = Stage<V, W>;
    float c[V], s[V];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
        uint32_t w[4];
        lds4(S::angle(base, stage, i), w[0], w[1], w[2], w[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k) c[4 * i + k] = __uint_as_float(w[k]);
        lds4(S::angle(base, stage, V / 4 + i), w[0], w[1], w[2], w[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k) s[4 * i + k] = __uint_as_float(w[k]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (PAIRS) {
            cs[i] = f2(c[i], c[i]);
            sn[i] = f2(-s[i], s[i]);
        } else {
            const int k = 2 * (i % (V / 2));
            const float g = i < V / 2 ? -1.f : 1.f;
            cs[i] = f2(c[k], c[k + 1]);
            sn[i] = f2(g * s[k], g * s[k + 1]);
        }
    }
}

// The steps of a block: its token groups, y, y + gridDim.y, ..., and for each the
// batches [b0, b1) of heads.  Every lane of a warp takes every step.
struct Walk {
    int t, b;
    __device__ __forceinline__ void next(int b0, int b1, int stride)
    {
        if (++b == b1) b = b0, t += stride;
    }
};

// Block (x, y, z): slot x, token groups y.., share z of the batches of HB heads
// (those of the queries, then those of the keys).
template <int V, int L, bool PAIRS>
__global__ void __launch_bounds__(THREADS, 3) k_qk_norm(const Params p)
{
    using S = Stage<V, 2 * HB>;
    extern __shared__ __align__(16) uint8_t sm[];
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(sm);
    constexpr int GROUPS = THREADS / L;
    const int c = threadIdx.x % L * V, hb = p.D;                   // hb: bytes of half a head
    const bool on = c < p.D / 2;
    const int slot = blockIdx.x, nq = (p.H[0] + HB - 1) / HB, nb = nq + (p.H[1] + HB - 1) / HB;
    const int b0 = blockIdx.z * nb / gridDim.z, b1 = (blockIdx.z + 1) * nb / gridDim.z;
    const int stride = gridDim.y * GROUPS, first = blockIdx.y * GROUPS + threadIdx.x / L, warp_off = threadIdx.x % 32 / L;
    const float inv_d = 1.f / (float)p.D;
    if (b0 == b1) return;
    int pos = on && first < p.T ? __ldg(p.pos + first) : 0;        // of the next token group to fetch
    auto fetch = [&](const Walk &k, int stage) {
        if (on && k.t < p.T) {
            const int w = k.b >= nq, h0 = (w ? k.b - nq : k.b) * HB;
            const Heads &x = p.x[w];
            const char *const src = x.base + slot * x.slot + k.t * x.token + h0 * x.head + c * 2;
#pragma unroll
            for (int i = 0; i < HB; ++i)
                if (h0 + i < p.H[w]) {
                    copy<2 * V>(S::chunk(base, stage, 2 * i), src + i * x.head);
                    copy<2 * V>(S::chunk(base, stage, 2 * i + 1), src + i * x.head + hb);
                }
            if (k.b == b0) {                                       // the first batch brings the token's angles
                fetch_angles<V, 2 * HB, PAIRS>(p, base, stage, pos, c);
                if (k.t + stride < p.T) pos = __ldg(p.pos + k.t + stride);
            }
        }
        copies_done();
    };
    Walk ahead{first, b0}, now{first, b0};
    for (int s = 0; s < STAGES - 1; ++s) fetch(ahead, s), ahead.next(b0, b1, stride);
    f32x2 cs[V], sn[V];
    for (int stage = 0; now.t - warp_off < p.T; now.next(b0, b1, stride)) {
        wait_oldest();
        const bool live = on && now.t < p.T;
        const int w = now.b >= nq, h0 = (w ? now.b - nq : now.b) * HB, heads = min(HB, p.H[w] - h0);
        const Heads &z = p.z[w];
        char *const dst = z.base + slot * z.slot + now.t * z.token + h0 * z.head + c * 2;
        f32x2 a[V], b[V];
        if (live) {
            f32x2 g[V], gp[V];
            ldf<V>(p.g[w] + c, p.D / 2, g);
            if (now.b == b0) angles<V, 2 * HB, PAIRS>(base, stage, cs, sn);
            partners<V, PAIRS>(g, gp);
#pragma unroll
            for (int i = 0; i < V; ++i) a[i] = mul2(cs[i], g[i]), b[i] = mul2(sn[i], gp[i]);
        }
#pragma unroll
        for (int k = 0; k < HB; ++k) {
            const bool here = live && k < heads;
            f32x2 f[V], q[V], ss = 0;
            if (here) {
                take<V>(S::chunk(base, stage, 2 * k), S::chunk(base, stage, 2 * k + 1), f);
#pragma unroll
                for (int i = 0; i < V; ++i) ss = fma2(f[i], f[i], ss);
            }
            const float sum = group_sum<L>(hsum(ss));
            if (!here) continue;
            const float r = rsqrtf(fmaf(sum, inv_d, p.eps));
            const f32x2 r2 = f2(r, r);
            partners<V, PAIRS>(f, q);
#pragma unroll
            for (int i = 0; i < V; ++i) q[i] = mul2(fma2(f[i], a[i], mul2(q[i], b[i])), r2);
            st<V>(dst + k * z.head, hb, q);
        }
        // the slot of the step before this one is free
        const int into = stage == 0 ? STAGES - 1 : stage - 1;
        fetch(ahead, into);
        ahead.next(b0, b1, stride);
        stage = stage == STAGES - 1 ? 0 : stage + 1;
    }
}

// The gradient.  A block stays within one slot and one share of its heads; its
// threads keep the weight gradients of their columns over all their rows, and
// the block's sums go to one row of `part`, added up by k_qk_norm_dg in block
// order.
template <int V, int L, bool PAIRS>
__global__ void __launch_bounds__(THREADS, 3) k_qk_norm_bwd(const Params p)
{
    using S = Stage<V, 4 * GB>;
    extern __shared__ __align__(16) uint8_t sm[];
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(sm);
    float *const red = (float *)sm;                                 // [warps][2][D], once the staging is done with
    constexpr int GROUPS = THREADS / L;
    const int c = threadIdx.x % L * V, hb = p.D;
    const bool on = c < p.D / 2;
    const int slot = blockIdx.x, share = blockIdx.z, shares = gridDim.z;
    const int stride = gridDim.y * GROUPS, first = blockIdx.y * GROUPS + threadIdx.x / L, warp_off = threadIdx.x % 32 / L;
    const float inv_d = 1.f / (float)p.D;
    f32x2 acc[2][V] = {};
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int nb = (p.H[w] + GB - 1) / GB, b0 = share * nb / shares, b1 = (share + 1) * nb / shares;
        if (b0 == b1) continue;
        f32x2 g[V] = {}, cs[V], sn[V];
        if (on) ldf<V>(p.g[w] + c, p.D / 2, g);
        const Heads &x = p.x[w], &z = p.z[w], &d = p.dx[w];
        int pos = on && first < p.T ? __ldg(p.pos + first) : 0;
        auto fetch = [&](const Walk &k, int stage) {
            if (on && k.t < p.T) {
                const char *const xs = x.base + slot * x.slot + k.t * x.token + k.b * GB * x.head + c * 2;
                const char *const zs = z.base + slot * z.slot + k.t * z.token + k.b * GB * z.head + c * 2;
#pragma unroll
                for (int i = 0; i < GB; ++i)
                    if (k.b * GB + i < p.H[w]) {
                        copy<2 * V>(S::chunk(base, stage, 4 * i), xs + i * x.head);
                        copy<2 * V>(S::chunk(base, stage, 4 * i + 1), xs + i * x.head + hb);
                        copy<2 * V>(S::chunk(base, stage, 4 * i + 2), zs + i * z.head);
                        copy<2 * V>(S::chunk(base, stage, 4 * i + 3), zs + i * z.head + hb);
                    }
                if (k.b == b0) {
                    fetch_angles<V, 4 * GB, PAIRS>(p, base, stage, pos, c);
                    if (k.t + stride < p.T) pos = __ldg(p.pos + k.t + stride);
                }
            }
            copies_done();
        };
        Walk ahead{first, b0}, now{first, b0};
        for (int s = 0; s < STAGES - 1; ++s) fetch(ahead, s), ahead.next(b0, b1, stride);
        for (int stage = 0; now.t - warp_off < p.T; now.next(b0, b1, stride)) {
            wait_oldest();
            const bool live = on && now.t < p.T;
            char *const ds = d.base + slot * d.slot + now.t * d.token + now.b * GB * d.head + c * 2;
            if (live && now.b == b0) angles<V, 4 * GB, PAIRS>(base, stage, cs, sn);
#pragma unroll
            for (int k = 0; k < GB; ++k) {
                const bool here = live && now.b * GB + k < p.H[w];
                f32x2 f[V], u[V], q[V], ss = 0, tt = 0;
                if (here) {
                    take<V>(S::chunk(base, stage, 4 * k), S::chunk(base, stage, 4 * k + 1), f);
                    take<V>(S::chunk(base, stage, 4 * k + 2), S::chunk(base, stage, 4 * k + 3), u);
                    partners<V, PAIRS>(u, q);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        // turned back: the partner's sine changes sign
                        float s0, s1;
                        unf2(sn[i], s0, s1);
                        u[i] = fma2(u[i], cs[i], mul2(q[i], f2(-s0, -s1)));    // dy
                        q[i] = mul2(u[i], g[i]);                             // t
                        ss = fma2(f[i], f[i], ss);
                        tt = fma2(q[i], f[i], tt);
                    }
                }
                const float sum = group_sum<L>(hsum(ss)), dot = group_sum<L>(hsum(tt));
                if (!here) continue;
                const float r = rsqrtf(fmaf(sum, inv_d, p.eps));
                const float m = -dot * inv_d * r * r * r;      // dx = r t - x r^3 mean(t x)
                const f32x2 r2 = f2(r, r), m2 = f2(m, m);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    acc[w][i] = fma2(u[i], mul2(f[i], r2), acc[w][i]);
                    q[i] = fma2(q[i], r2, mul2(f[i], m2));
                }
                st<V>(ds + k * d.head, hb, q);
            }
            const int into = stage == 0 ? STAGES - 1 : stage - 1;
            fetch(ahead, into);
            ahead.next(b0, b1, stride);
            stage = stage == STAGES - 1 ? 0 : stage + 1;
        }
    }
    // sum the groups of the warp, then the warps
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float s0, s1;
            unf2(acc[w][i], s0, s1);
#pragma unroll
            for (int o = 16; o >= L; o >>= 1) {
                s0 += __shfl_xor_sync(0xFFFFFFFFu, s0, o);
                s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, o);
            }
            if (on && (threadIdx.x & 31) < L) {
                const int at = (threadIdx.x / 32 * 2 + w) * p.D + (i < V / 2 ? 0 : p.D / 2) + c + 2 * (i % (V / 2));
                red[at] = s0;
                red[at + 1] = s1;
            }
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.D; i += THREADS) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < THREADS / 32; ++k) s += red[k * 2 * p.D + i];
        p.part[((size_t)(blockIdx.y * shares + share) * p.P + slot) * 2 * p.D + i] = s;
    }
}

// dg[w][slot][d]: the sum over the rows of `part`.  A lane owns an output, warp k
// adds rows k, k + 32, ... and the warps' sums are added in order.  CLEAR: in a
// caller's workspace the rows are zeroed once read, because other calls keep signal
// words there and almost any other number reads as a signal given.
constexpr int DG_WARPS = 32;

template <bool CLEAR>
__global__ void __launch_bounds__(32 * DG_WARPS) k_qk_norm_dg(const Params p)
{
    __shared__ float red[DG_WARPS][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, width = p.P * 2 * p.D;
    const int i = blockIdx.x * 32 + lane;                  // the width is a multiple of 16
    asm volatile("griddepcontrol.wait;" ::: "memory");     // the rows are written
    float s = 0.f;
    if (i < width)
#pragma unroll 8
        for (int b = warp; b < p.blocks; b += DG_WARPS) s += p.part[(size_t)b * width + i];
    if (CLEAR && i < width)                                // in a loop of its own: stores would hold up the loads
        for (int b = warp; b < p.blocks; b += DG_WARPS) p.part[(size_t)b * width + i] = 0.f;
    red[warp][lane] = s;
    __syncthreads();
    if (warp || i >= width) return;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < DG_WARPS; ++k) s += red[k][lane];
    const int slot = i / (2 * p.D), k = i % (2 * p.D);
    p.dg[k >= p.D][slot * p.D + (k >= p.D ? k - p.D : k)] = s;
}

template <auto KERNEL, int SMEM>
static cudaError_t start(dim3 blocks, const Params &p, cudaStream_t st)
{
    static OncePerDevice once;
    const cudaError_t e = once([] { return cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM); });
    if (e != cudaSuccess) return e;
    KERNEL<<<blocks, THREADS, SMEM, st>>>(p);
    return cudaGetLastError();
}

template <int V, int L>
static cudaError_t launch(const Params &p, bool grad, dim3 blocks, cudaStream_t st)
{
    if (!grad) {
        constexpr int smem = Stage<V, 2 * HB>::TOTAL;
        return p.pairs ? start<k_qk_norm<V, L, true>, smem>(blocks, p, st) : start<k_qk_norm<V, L, false>, smem>(blocks, p, st);
    }
    constexpr int smem = Stage<V, 4 * GB>::TOTAL;
    static_assert(smem >= THREADS / 32 * 2 * 2 * V * L * 4, "the block's sums fit the staging area");
    const cudaError_t e = p.pairs ? start<k_qk_norm_bwd<V, L, true>, smem>(blocks, p, st)
                                  : start<k_qk_norm_bwd<V, L, false>, smem>(blocks, p, st);
    if (e != cudaSuccess) return e;
    // set up while the gradient runs; its blocks start when that has ended
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((p.P * 2 * p.D + 31) / 32));
    cfg.blockDim = dim3(32 * DG_WARPS);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return p.clear ? cudaLaunchKernelEx(&cfg, k_qk_norm_dg<true>, p) : cudaLaunchKernelEx(&cfg, k_qk_norm_dg<false>, p);
}

// Lanes of a group for a head of D: D / 2V rounded up to a power of two.
static int group_lanes(int D, int V)
{
    int l = 1;
    while (l * V < D / 2) l *= 2;
    return l;
}

static cudaError_t launch_any(const Params &p, bool grad, dim3 blocks, cudaStream_t st)
{
    // V = 8 needs both halves of a head on 16-byte boundaries
    if (p.D % 16 == 0) {
        switch (group_lanes(p.D, 8)) {
        case 1: return launch<8, 1>(p, grad, blocks, st);
        case 2: return launch<8, 2>(p, grad, blocks, st);
        case 4: return launch<8, 4>(p, grad, blocks, st);
        case 8: return launch<8, 8>(p, grad, blocks, st);
        default: return launch<8, 16>(p, grad, blocks, st);
        }
    }
    switch (group_lanes(p.D, 4)) {
    case 1: return launch<4, 1>(p, grad, blocks, st);
    case 2: return launch<4, 2>(p, grad, blocks, st);
    case 4: return launch<4, 4>(p, grad, blocks, st);
    case 8: return launch<4, 8>(p, grad, blocks, st);
    case 16: return launch<4, 16>(p, grad, blocks, st);
    default: return launch<4, 32>(p, grad, blocks, st);
    }
}

static int take_heads(const rc_heads &in, Heads &h, const char *name, int P, int T, int H, int D)
{
    rc_heads x = in;
    const int rc_ = check_heads(x, name, P, T, H, D);
    h = Heads{(char *)x.base, x.slot, x.token, x.head};
    return rc_;
}

// Blocks of a launch: for each slot three per SM over all slots, or one per
// group of tokens where that is less; then batches of heads are shared out too.
static void grid_of(const rc_qk_norm_args &a, int sms, int most_shares, int &blocks, int &shares)
{
    const int groups = THREADS / group_lanes(a.D, a.D % 16 ? 4 : 8);
    const long long n = ((long long)a.T + groups - 1) / groups, most = (3ll * sms + a.P - 1) / a.P;
    blocks = (int)(n > most ? most : n < 1 ? 1 : n);
    shares = (int)(most / blocks);
    shares = shares > most_shares ? most_shares : shares < 1 ? 1 : shares;
}

static int batches(const rc_qk_norm_args &a, int n) { return (a.Hq + n - 1) / n + (a.Hkv + n - 1) / n; }

// Tokens: blocks step past the last one by up to their stride, in 32 bits.
constexpr int kMostTokens = INT_MAX - (1 << 20);

static int check_sizes(const rc_qk_norm_args &a)
{
    if (a.P < 1 || a.P > RC_MAX_P) return set_error(RC_ERR_INVALID, "P=%d outside 1..%d", a.P, RC_MAX_P);
    if (a.T < 0 || a.Hq < 1 || a.Hkv < 1 || a.Hq > 65536 || a.Hkv > 65536 || a.npos < 1)
        return set_error(RC_ERR_INVALID, "need T >= 0, 1 <= Hq, Hkv <= 65536 and npos >= 1 (got %d, %d, %d, %d)", a.T, a.Hq, a.Hkv, a.npos);
    if (a.T > kMostTokens) return set_error(RC_ERR_INVALID, "T=%d is above %d", a.T, kMostTokens);
    if (a.D < 8 || a.D > 256 || a.D % 8) return set_error(RC_ERR_INVALID, "D=%d is not a multiple of 8 up to 256", a.D);
    if (a.layout != RC_ROPE_HALF && a.layout != RC_ROPE_PAIRS) return set_error(RC_ERR_INVALID, "unknown rotation layout %d", a.layout);
    if (!(a.eps >= 0.f) || !std::isfinite(a.eps)) return set_error(RC_ERR_INVALID, "eps must be finite and not negative");
    return RC_OK;
}

// Results apart from the inputs.  A thread has read its share of a head before it
// writes there, so q_out may be q, dq may be q or dq_out, and k alike.
static int check_places(const rc_qk_norm_args &a, const Params &p, const char *const (&zname)[2], bool grad)
{
    auto at = [&](const char *name, const Heads &h, int H) {
        return heads_at(name, a.T ? rc_heads{h.base, h.slot, h.token, h.head} : rc_heads{}, a.P, a.T, H, a.D);
    };
    const Operand q = at("q", p.x[0], a.Hq), k = at("k", p.x[1], a.Hkv), zq = at(zname[0], p.z[0], a.Hq),
                  zk = at(zname[1], p.z[1], a.Hkv);
    if (!grad) {
        const Operand res[] = {zq, zk}, in[] = {q, k};
        const unsigned whole[] = {1, 2};
        return check_apart(res, 2, in, 2, whole);
    }
    const size_t bytes = (size_t)a.P * a.D * 4;
    const Operand res[] = {at("dq", p.dx[0], a.Hq), at("dk", p.dx[1], a.Hkv), bytes_at("dgamma_q", a.dgamma_q, bytes),
                           bytes_at("dgamma_k", a.dgamma_k, bytes)};
    const Operand in[] = {q, k, zq, zk};
    const unsigned whole[] = {1 | 4, 2 | 8, 0, 0};
    return check_apart(res, 4, in, 4, whole);
}

static int run(const rc_qk_norm_args *args, bool grad, void *stream)
{
    if (!args) return set_error(RC_ERR_INVALID, "null args");
    const rc_qk_norm_args &a = *args;
    int rc_ = check_sizes(a);
    if (rc_) return rc_;
    if (a.T == 0 && !grad) return RC_OK;
    Params p{};
    const char *const zname[] = {grad ? "dq_out" : "q_out", grad ? "dk_out" : "k_out"};
    if (a.T && ((rc_ = take_heads(a.q, p.x[0], "q", a.P, a.T, a.Hq, a.D)) || (rc_ = take_heads(a.k, p.x[1], "k", a.P, a.T, a.Hkv, a.D)) ||
                (rc_ = take_heads(a.q_out, p.z[0], zname[0], a.P, a.T, a.Hq, a.D)) ||
                (rc_ = take_heads(a.k_out, p.z[1], zname[1], a.P, a.T, a.Hkv, a.D))))
        return rc_;
    if (a.T && grad && ((rc_ = take_heads(a.dq, p.dx[0], "dq", a.P, a.T, a.Hq, a.D)) || (rc_ = take_heads(a.dk, p.dx[1], "dk", a.P, a.T, a.Hkv, a.D))))
        return rc_;
    if (!a.gamma_q || !a.gamma_k || !a.cos || !a.sin || (a.T && !a.pos)) return set_error(RC_ERR_INVALID, "null pointer");
    if (((uintptr_t)a.gamma_q | (uintptr_t)a.gamma_k | (uintptr_t)a.cos | (uintptr_t)a.sin) & 15u)
        return set_error(RC_ERR_INVALID, "gamma, cos and sin must be 16-byte aligned");
    if (grad && (!a.dgamma_q || !a.dgamma_k)) return set_error(RC_ERR_INVALID, "dgamma_q or dgamma_k is null");
    if ((rc_ = check_places(a, p, zname, grad))) return rc_;
    int sms = 0;
    if ((rc_ = device_sms(&sms))) return rc_;
    p.g[0] = a.gamma_q;
    p.g[1] = a.gamma_k;
    p.cos = a.cos;
    p.sin = a.sin;
    p.pos = a.pos;
    p.P = a.P;
    p.T = a.T;
    p.H[0] = a.Hq;
    p.H[1] = a.Hkv;
    p.D = a.D;
    p.npos = a.npos;
    p.pairs = a.layout == RC_ROPE_PAIRS;
    p.eps = a.eps;
    dim3 blocks(1);
    if (grad) {
        p.dg[0] = a.dgamma_q;
        p.dg[1] = a.dgamma_k;
        int per_slot, shares;
        grid_of(a, sms, batches(a, GB), per_slot, shares);
        p.blocks = per_slot * shares;
        blocks = dim3((unsigned)a.P, (unsigned)per_slot, (unsigned)shares);
        const size_t bytes = (size_t)p.blocks * a.P * 2 * a.D * 4;
        void *s = a.workspace;
        if (a.workspace && ((uintptr_t)a.workspace & 255u)) return set_error(RC_ERR_INVALID, "workspace must be 256-byte aligned");
        if (a.workspace && a.ws_bytes < kWsHead + bytes)
            return set_error(RC_ERR_INVALID, "workspace of %zu bytes is below the %zu this call needs", a.ws_bytes, kWsHead + bytes);
        if (a.workspace) s = (char *)s + kWsHead, p.clear = 1;
        else if ((rc_ = prepare_scratch(bytes, &s))) return rc_;
        p.part = (float *)s;
    } else {
        int per_slot, shares;
        grid_of(a, sms, batches(a, HB), per_slot, shares);
        blocks = dim3((unsigned)a.P, (unsigned)per_slot, (unsigned)shares);
    }
    const cudaError_t e = launch_any(p, grad, blocks, (cudaStream_t)stream);
    if (e != cudaSuccess) return set_error(RC_ERR_CUDA, "qk_norm_rope launch: %s", cudaGetErrorString(e));
    return RC_OK;
}

} // namespace qkn
} // namespace rc

extern "C" int qk_norm_rope(const rc_qk_norm_args *args, void *stream) { return rc::qkn::run(args, false, stream); }

extern "C" int qk_norm_rope_bwd(const rc_qk_norm_args *args, void *stream) { return rc::qkn::run(args, true, stream); }

extern "C" size_t qk_norm_rope_bwd_workspace_bytes(const rc_qk_norm_args *args)
{
    using namespace rc::qkn;
    int sms = 0;
    if (!args || check_sizes(*args) || rc::device_sms(&sms)) return 0;
    int blocks, shares;
    grid_of(*args, sms, batches(*args, GB), blocks, shares);
    return rc::kWsHead + (size_t)blocks * shares * args->P * 2 * args->D * 4;
}
