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
#include <cmath>
#include <cuda_bf16.h>

#include "internal.h"
#include "ringcoll.h"
#include "dev.cuh"

namespace rc {
namespace qkn {

constexpr int THREADS = 256;     // of qk_norm_rope
constexpr int BTHREADS = 128;    // of its gradient: up to 168 registers at three blocks per SM
constexpr int HB = 4;            // heads of a run in qk_norm_rope: all loaded before the first is used
constexpr int GB = 2;            // heads in flight in its gradient

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
    int runs[2], blocks;         // runs of HB heads of either kind; gradient: rows of `part`
    float eps;
};

// ------------------------------------------------------------ pairs of binary32
typedef uint64_t f32x2;
__device__ __forceinline__ f32x2 mk(float a, float b)
{
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void un(f32x2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f32x2 swap(f32x2 v)
{
    float a, b;
    un(v, a, b);
    return mk(b, a);
}
__device__ __forceinline__ f32x2 mul(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float hsum(f32x2 v)
{
    float a, b;
    un(v, a, b);
    return a + b;
}

// A thread's share of a head as loaded: V elements from c and V from c + D/2.
template <int V>
struct Raw {
    uint32_t w[V];               // V / 2 words of the first chunk, then of the second
};

template <int V>
__device__ __forceinline__ void ld(Raw<V> &r, const char *p, int half_bytes)
{
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (V == 8) {
            const uint4 v = __ldcs((const uint4 *)(p + k * half_bytes));
            r.w[4 * k] = v.x, r.w[4 * k + 1] = v.y, r.w[4 * k + 2] = v.z, r.w[4 * k + 3] = v.w;
        } else {
            const uint2 v = __ldcs((const uint2 *)(p + k * half_bytes));
            r.w[2 * k] = v.x, r.w[2 * k + 1] = v.y;
        }
}

template <int V>
__device__ __forceinline__ void unpack(const Raw<V> &r, f32x2 (&f)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = mk(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t pack(f32x2 v)
{
    float a, b;
    uint32_t r;
    un(v, a, b);
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
            f[k * V / 2 + i / 2] = mk(v.x, v.y);
            f[k * V / 2 + i / 2 + 1] = mk(v.z, v.w);
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

// cos of every element's angle, and sin with the sign it has on the element's
// partner in the forward rotation: z = x cs + x' sn.  Position t's row of the
// table; one outside the table gives NaN.
template <int V, bool PAIRS>
__device__ __forceinline__ void angles(const Params &p, int t, int c, f32x2 (&cs)[V], f32x2 (&sn)[V])
{
    const int pos = __ldg(p.pos + t);
    if (pos < 0 || pos >= p.npos) {
        const float nan = __int_as_float(0x7FC00000);
#pragma unroll
        for (int i = 0; i < V; ++i) cs[i] = sn[i] = mk(nan, nan);
        return;
    }
    const float *const ct = p.cos + (size_t)pos * (p.D / 2), *const st_ = p.sin + (size_t)pos * (p.D / 2);
    if (!PAIRS) {
        // both chunks turn by angles c .. c + V - 1
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 a = __ldg((const float4 *)(ct + c + i)), b = __ldg((const float4 *)(st_ + c + i));
            cs[i / 2] = cs[V / 2 + i / 2] = mk(a.x, a.y);
            cs[i / 2 + 1] = cs[V / 2 + i / 2 + 1] = mk(a.z, a.w);
            sn[i / 2] = mk(-b.x, -b.y);
            sn[i / 2 + 1] = mk(-b.z, -b.w);
            sn[V / 2 + i / 2] = mk(b.x, b.y);
            sn[V / 2 + i / 2 + 1] = mk(b.z, b.w);
        }
    } else {
        // word i of either chunk is a pair; the chunks' angles start at c / 2 and D / 4 + c / 2
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int k = (i < V / 2 ? 0 : p.D / 4) + c / 2 + i % (V / 2);
            const float a = __ldg(ct + k), b = __ldg(st_ + k);
            cs[i] = mk(a, a);
            sn[i] = mk(-b, b);
        }
    }
}

// Block (x, y): tokens y * groups.. of slot x / runs, run x % runs of heads (the
// runs of query heads, then those of key heads).  Blocks that run together
// then cover whole tokens, which lie together in memory.
template <int V, int L, bool PAIRS>
__global__ void __launch_bounds__(THREADS, 2) k_qk_norm(const Params p)
{
    const int lane = threadIdx.x % L, c = lane * V, hb = p.D;      // hb: bytes of half a head
    const bool on = c < p.D / 2;
    const int runs = p.runs[0] + p.runs[1], slot = blockIdx.x / runs, run = blockIdx.x % runs;
    const int w = run >= p.runs[0];
    const int h0 = (w ? run - p.runs[0] : run) * HB, heads = min(HB, p.H[w] - h0);
    const Heads x = p.x[w], z = p.z[w];
    const char *const src = x.base + slot * x.slot + h0 * x.head + c * 2;
    char *const dst = z.base + slot * z.slot + h0 * z.head + c * 2;
    const float inv_d = 1.f / (float)p.D;
    // every lane of a warp stays in the loop: the sums are warp-wide shuffles
    for (int t0 = blockIdx.y * (THREADS / L); t0 < p.T; t0 += gridDim.y * (THREADS / L)) {
        const int t = t0 + threadIdx.x / L;
        const bool live = on && t < p.T;
        Raw<V> raw[HB];
#pragma unroll
        for (int k = 0; k < HB; ++k)
            if (live && k < heads) ld<V>(raw[k], src + t * x.token + k * x.head, hb);
        f32x2 a[V], b[V];
        if (live) {
            f32x2 g[V], gp[V];
            ldf<V>(p.g[w] + c, p.D / 2, g);
            angles<V, PAIRS>(p, t, c, a, b);
            partners<V, PAIRS>(g, gp);
#pragma unroll
            for (int i = 0; i < V; ++i) a[i] = mul(a[i], g[i]), b[i] = mul(b[i], gp[i]);
        }
#pragma unroll
        for (int k = 0; k < HB; ++k) {
            const bool here = live && k < heads;
            f32x2 f[V], q[V], ss = 0;
            if (here) {
                unpack<V>(raw[k], f);
#pragma unroll
                for (int i = 0; i < V; ++i) ss = fma(f[i], f[i], ss);
            }
            const float sum = group_sum<L>(hsum(ss));
            if (!here) continue;
            const float r = rsqrtf(fmaf(sum, inv_d, p.eps));
            const f32x2 r2 = mk(r, r);
            partners<V, PAIRS>(f, q);
#pragma unroll
            for (int i = 0; i < V; ++i) q[i] = mul(fma(f[i], a[i], mul(q[i], b[i])), r2);
            st<V>(dst + t * z.token + k * z.head, hb, q);
        }
    }
}

// The gradient.  A block stays within one slot and one share of its heads; its threads keep the weight
// gradients of their columns over all their rows, and the block's sums go to
// one row of `part`, added up by k_qk_norm_dg in block order.
template <int V, int L, bool PAIRS>
__global__ void __launch_bounds__(BTHREADS, 3) k_qk_norm_bwd(const Params p)
{
    __shared__ float red[BTHREADS / 32][2][256];
    const int lane = threadIdx.x % L, c = lane * V, hb = p.D;
    const bool on = c < p.D / 2;
    const int slot = blockIdx.x, blk = blockIdx.y, share = blockIdx.z, shares = gridDim.z;
    const float inv_d = 1.f / (float)p.D;
#pragma unroll 1
    for (int w = 0; w < 2; ++w) {
        f32x2 acc[V] = {}, g[V] = {};
        if (on) ldf<V>(p.g[w] + c, p.D / 2, g);
        const Heads x = p.x[w], z = p.z[w], d = p.dx[w];
        const char *const xs = x.base + slot * x.slot + c * 2, *const zs = z.base + slot * z.slot + c * 2;
        char *const ds = d.base + slot * d.slot + c * 2;
        const int h0 = share * p.H[w] / shares, h1 = (share + 1) * p.H[w] / shares;
        for (int t0 = blk * (BTHREADS / L); t0 < p.T && h0 < h1; t0 += gridDim.y * (BTHREADS / L)) {
            const int t = t0 + threadIdx.x / L;
            const bool live = on && t < p.T;
            f32x2 cs[V], sn[V];
            for (int h = h0; h < h1; h += GB) {
                Raw<V> xr[GB], zr[GB];
#pragma unroll
                for (int k = 0; k < GB; ++k)
                    if (live && h + k < h1) {
                        ld<V>(xr[k], xs + t * x.token + (h + k) * x.head, hb);
                        ld<V>(zr[k], zs + t * z.token + (h + k) * z.head, hb);
                    }
                if (live && h == h0) angles<V, PAIRS>(p, t, c, cs, sn);
#pragma unroll
                for (int k = 0; k < GB; ++k) {
                    const bool here = live && h + k < h1;
                    f32x2 f[V], u[V], q[V], ss = 0, tt = 0;
                    if (here) {
                        unpack<V>(xr[k], f);
                        unpack<V>(zr[k], u);
                        partners<V, PAIRS>(u, q);
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            // turned back: the partner's sine changes sign
                            float s0, s1;
                            un(sn[i], s0, s1);
                            u[i] = fma(u[i], cs[i], mul(q[i], mk(-s0, -s1)));    // dy
                            q[i] = mul(u[i], g[i]);                             // t
                            ss = fma(f[i], f[i], ss);
                            tt = fma(q[i], f[i], tt);
                        }
                    }
                    const float sum = group_sum<L>(hsum(ss)), dot = group_sum<L>(hsum(tt));
                    if (!here) continue;
                    const float r = rsqrtf(fmaf(sum, inv_d, p.eps));
                    const float m = -dot * inv_d * r * r * r;      // dx = r t - x r^3 mean(t x)
                    const f32x2 r2 = mk(r, r), m2 = mk(m, m);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        acc[i] = fma(u[i], mul(f[i], r2), acc[i]);
                        q[i] = fma(q[i], r2, mul(f[i], m2));
                    }
                    st<V>(ds + t * d.token + (h + k) * d.head, hb, q);
                }
            }
        }
        // sum the groups of the warp, then the warps
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float s0, s1;
            un(acc[i], s0, s1);
#pragma unroll
            for (int o = 16; o >= L; o >>= 1) {
                s0 += __shfl_xor_sync(0xFFFFFFFFu, s0, o);
                s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, o);
            }
            if (on && (threadIdx.x & 31) < L) {
                const int at = (i < V / 2 ? 0 : p.D / 2) + c + 2 * (i % (V / 2));
                red[threadIdx.x >> 5][w][at] = s0;
                red[threadIdx.x >> 5][w][at + 1] = s1;
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.D; i += BTHREADS) {
        const int w = i >= p.D, d = w ? i - p.D : i;
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < BTHREADS / 32; ++k) s += red[k][w][d];
        p.part[((size_t)(blk * shares + share) * p.P + slot) * 2 * p.D + i] = s;
    }
}

// dg[w][slot][d]: the sum over blocks, one warp per output.
__global__ void __launch_bounds__(THREADS) k_qk_norm_dg(const Params p)
{
    const int i = blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (i >= p.P * 2 * p.D) return;
    float s = 0.f;
    for (int b = lane; b < p.blocks; b += 32) s += p.part[(size_t)b * p.P * 2 * p.D + i];
    s = group_sum<32>(s);
    const int slot = i / (2 * p.D), k = i % (2 * p.D);
    if (lane == 0) p.dg[k >= p.D][slot * p.D + (k >= p.D ? k - p.D : k)] = s;
}

template <int V, int L>
static void launch(const Params &p, bool grad, dim3 blocks, cudaStream_t st)
{
    if (grad) {
        if (p.pairs) k_qk_norm_bwd<V, L, true><<<blocks, BTHREADS, 0, st>>>(p);
        else k_qk_norm_bwd<V, L, false><<<blocks, BTHREADS, 0, st>>>(p);
        k_qk_norm_dg<<<(p.P * 2 * p.D + THREADS / 32 - 1) / (THREADS / 32), THREADS, 0, st>>>(p);
    } else {
        if (p.pairs) k_qk_norm<V, L, true><<<blocks, THREADS, 0, st>>>(p);
        else k_qk_norm<V, L, false><<<blocks, THREADS, 0, st>>>(p);
    }
}

// Lanes of a group for a head of D: D / 2V rounded up to a power of two.
static int group_lanes(int D, int V)
{
    int l = 1;
    while (l * V < D / 2) l *= 2;
    return l;
}

static void launch_any(const Params &p, bool grad, dim3 blocks, cudaStream_t st)
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

static int check_heads(const rc_heads &in, Heads &h, const char *name, int P, int T, int H, int D)
{
    const size_t least = (size_t)D * 2;
    h = Heads{(char *)in.base, in.slot, in.token, in.head};
    if (!h.base) return set_error(RC_ERR_INVALID, "%s is null", name);
    if (H == 1) h.head = least;
    if (T == 1) h.token = least;
    if (P == 1) h.slot = least;
    if (((uintptr_t)h.base | h.slot | h.token | h.head) & 15u)
        return set_error(RC_ERR_INVALID, "%s: base and strides must be multiples of 16 bytes", name);
    if (h.head < least || h.token < least || h.slot < least)
        return set_error(RC_ERR_INVALID, "%s: a stride is below the %zu bytes of a head", name, least);
    return RC_OK;
}

// The gradient's blocks: for each slot three per SM over all slots, or one per
// group of tokens where that is less; then the heads are shared out too.
static void bwd_blocks(const rc_qk_norm_args &a, int sms, int &blocks, int &shares)
{
    const int groups = BTHREADS / group_lanes(a.D, a.D % 16 ? 4 : 8);
    const long long n = ((long long)a.T + groups - 1) / groups, most = (3ll * sms + a.P - 1) / a.P;
    blocks = (int)(n > most ? most : n < 1 ? 1 : n);
    const int heads = ((a.Hq > a.Hkv ? a.Hq : a.Hkv) + GB - 1) / GB;
    shares = (int)(most / blocks);
    shares = shares > heads ? heads : shares < 1 ? 1 : shares;
}

static int check_sizes(const rc_qk_norm_args &a)
{
    if (a.P < 1 || a.P > RC_MAX_P) return set_error(RC_ERR_INVALID, "P=%d outside 1..%d", a.P, RC_MAX_P);
    if (a.T < 0 || a.Hq < 1 || a.Hkv < 1 || a.Hq > 65536 || a.Hkv > 65536 || a.npos < 1)
        return set_error(RC_ERR_INVALID, "need T >= 0, 1 <= Hq, Hkv <= 65536 and npos >= 1 (got %d, %d, %d, %d)", a.T, a.Hq, a.Hkv, a.npos);
    if (a.D < 8 || a.D > 256 || a.D % 8) return set_error(RC_ERR_INVALID, "D=%d is not a multiple of 8 up to 256", a.D);
    if (a.layout != RC_ROPE_HALF && a.layout != RC_ROPE_PAIRS) return set_error(RC_ERR_INVALID, "unknown rotation layout %d", a.layout);
    if (!(a.eps >= 0.f) || !std::isfinite(a.eps)) return set_error(RC_ERR_INVALID, "eps must be finite and not negative");
    return RC_OK;
}

static int run(const rc_qk_norm_args *args, bool grad, void *stream)
{
    if (!args) return set_error(RC_ERR_INVALID, "null args");
    const rc_qk_norm_args &a = *args;
    int rc_ = check_sizes(a);
    if (rc_) return rc_;
    if (a.T == 0 && !grad) return RC_OK;
    Params p{};
    const int T = a.T ? a.T : 1;
    if (a.T && ((rc_ = check_heads(a.q, p.x[0], "q", a.P, T, a.Hq, a.D)) || (rc_ = check_heads(a.k, p.x[1], "k", a.P, T, a.Hkv, a.D)) ||
                (rc_ = check_heads(a.q_out, p.z[0], grad ? "dq_out" : "q_out", a.P, T, a.Hq, a.D)) ||
                (rc_ = check_heads(a.k_out, p.z[1], grad ? "dk_out" : "k_out", a.P, T, a.Hkv, a.D))))
        return rc_;
    if (a.T && grad && ((rc_ = check_heads(a.dq, p.dx[0], "dq", a.P, T, a.Hq, a.D)) || (rc_ = check_heads(a.dk, p.dx[1], "dk", a.P, T, a.Hkv, a.D))))
        return rc_;
    if (!a.gamma_q || !a.gamma_k || !a.cos || !a.sin || (a.T && !a.pos)) return set_error(RC_ERR_INVALID, "null pointer");
    if (((uintptr_t)a.gamma_q | (uintptr_t)a.gamma_k | (uintptr_t)a.cos | (uintptr_t)a.sin) & 15u)
        return set_error(RC_ERR_INVALID, "gamma, cos and sin must be 16-byte aligned");
    if (grad && (!a.dgamma_q || !a.dgamma_k)) return set_error(RC_ERR_INVALID, "dgamma_q or dgamma_k is null");
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
        bwd_blocks(a, sms, per_slot, shares);
        p.blocks = per_slot * shares;
        blocks = dim3((unsigned)a.P, (unsigned)per_slot, (unsigned)shares);
        const size_t bytes = (size_t)p.blocks * a.P * 2 * a.D * 4;
        void *s = a.workspace;
        if (a.workspace && ((uintptr_t)a.workspace & 255u)) return set_error(RC_ERR_INVALID, "workspace must be 256-byte aligned");
        if (a.workspace && a.ws_bytes < bytes)
            return set_error(RC_ERR_INVALID, "workspace of %zu bytes is below the %zu this call needs", a.ws_bytes, bytes);
        if (!a.workspace && (rc_ = prepare_scratch(bytes, &s))) return rc_;
        p.part = (float *)s;
    } else {
        p.runs[0] = (a.Hq + HB - 1) / HB;
        p.runs[1] = (a.Hkv + HB - 1) / HB;
        const int groups = THREADS / group_lanes(a.D, a.D % 16 ? 4 : 8);
        const long long n = ((long long)a.T + groups - 1) / groups;
        blocks = dim3((unsigned)(a.P * (p.runs[0] + p.runs[1])), (unsigned)(n < 65535 ? n : 65535));
    }
    launch_any(p, grad, blocks, (cudaStream_t)stream);
    const cudaError_t e = cudaGetLastError();
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
    bwd_blocks(*args, sms, blocks, shares);
    return (size_t)blocks * shares * args->P * 2 * args->D * 4;
}
