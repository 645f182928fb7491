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
// gradient), the rows of cos and sin once per token and rank.  Lanes hold two
// chunks of V elements, c and c + D/2 further on, so both members of either
// kind of pair are in one thread and only the mean crosses lanes: a group of
// D / 2V lanes (rounded up to a power of two) covers a head.  A group keeps
// its token's angles in registers and takes up to 4 heads, all loads first.
#include <cmath>
#include <cuda_bf16.h>

#include "internal.h"
#include "ringcoll.h"
#include "dev.cuh"

namespace rc {
namespace qkn {

constexpr int THREADS = 256;
constexpr int HB = 4;            // heads in flight per group

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
    int P, T, H[2], D, npos, pairs, chunks, blocks;   // blocks: of one slot (gradient)
    float eps;
};

template <int V>
struct Vec;
template <>
struct Vec<8> {
    uint4 v;
    __device__ __forceinline__ uint32_t at(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
};
template <>
struct Vec<4> {
    uint2 v;
    __device__ __forceinline__ uint32_t at(int i) const { return i == 0 ? v.x : v.y; }
};

template <int V>
__device__ __forceinline__ Vec<V> ld(const char *p)
{
    Vec<V> r;
    if (V == 8) *(uint4 *)&r = __ldcs((const uint4 *)p);
    else *(uint2 *)&r = __ldcs((const uint2 *)p);
    return r;
}

template <int V>
__device__ __forceinline__ void unpack(const Vec<V> &v, float *f)
{
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        f[2 * i] = __uint_as_float(v.at(i) << 16);
        f[2 * i + 1] = __uint_as_float(v.at(i) & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint32_t pack(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int V>
__device__ __forceinline__ void st(char *p, const float *f)
{
    if (V == 8)
        __stcs((uint4 *)p, make_uint4(pack(f[0], f[1]), pack(f[2], f[3]), pack(f[V - 4], f[V - 3]), pack(f[V - 2], f[V - 1])));
    else
        __stcs((uint2 *)p, make_uint2(pack(f[0], f[1]), pack(f[2], f[3])));
}

template <int V>
__device__ __forceinline__ void ldf(const float *p, float *f)
{
#pragma unroll
    for (int i = 0; i < V; i += 4) *(float4 *)(f + i) = __ldg((const float4 *)(p + i));
}

// Sum over the L lanes of a group.
template <int L>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// The angles of this thread's V pairs, in the order its pairs are kept.
// Half layout: pair i is (lo[i], hi[i]), angle c + i.  Adjacent pairs: pair i is
// (lo[2i], lo[2i + 1]) for i < V/2, angle c/2 + i, then the same of hi, D/4 on.
// A position outside the table gives NaN.
template <int V>
__device__ __forceinline__ void angles(const Params &p, int t, int c, float (&cs)[V], float (&sn)[V])
{
    const int pos = __ldg(p.pos + t);
    if (pos < 0 || pos >= p.npos) {
#pragma unroll
        for (int i = 0; i < V; ++i) cs[i] = sn[i] = __int_as_float(0x7FC00000);
        return;
    }
    const float *const ct = p.cos + (size_t)pos * (p.D / 2), *const st_ = p.sin + (size_t)pos * (p.D / 2);
    if (!p.pairs) {
        ldf<V>(ct + c, cs);
        ldf<V>(st_ + c, sn);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            cs[i] = __ldg(ct + c / 2 + i);
            sn[i] = __ldg(st_ + c / 2 + i);
            cs[V / 2 + i] = __ldg(ct + p.D / 4 + c / 2 + i);
            sn[V / 2 + i] = __ldg(st_ + p.D / 4 + c / 2 + i);
        }
    }
}

// Rotates the thread's 2V elements f (lo then hi) in place; back: by the opposite angles.
template <int V>
__device__ __forceinline__ void rotate(float (&f)[2 * V], const float (&cs)[V], const float (&sn)[V], bool pairs, bool back)
{
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float s = back ? -sn[i] : sn[i];
        if (pairs) {
            const float a = f[2 * i], b = f[2 * i + 1];
            f[2 * i] = a * cs[i] - b * s;
            f[2 * i + 1] = a * s + b * cs[i];
        } else {
            const float a = f[i], b = f[V + i];
            f[i] = a * cs[i] - b * s;
            f[V + i] = a * s + b * cs[i];
        }
    }
}

// Work item: token, slot and one of `chunks` runs of heads (queries then keys).
template <int V, int L, bool PAIRS>
__global__ void __launch_bounds__(THREADS, 2) k_qk_norm(const Params p)
{
    const int lane = threadIdx.x % L, c = lane * V, h = p.D / 2, HT = p.H[0] + p.H[1];
    const bool on = c < h;
    const long long items = (long long)p.T * p.P * p.chunks;
    const float inv_d = 1.f / (float)p.D;
    // every lane of a warp stays in the loop: the sums are warp-wide shuffles
    const long long step = (long long)gridDim.x * (THREADS / L);
    for (long long i0 = (long long)blockIdx.x * (THREADS / L) + (threadIdx.x & ~31) / L; i0 < items; i0 += step) {
        const long long i = i0 + (threadIdx.x & 31) / L;
        const bool live = on && i < items;
        const int ch = (int)(i % p.chunks);
        const long long ts = i / p.chunks;
        const int slot = (int)(ts % p.P), t = (int)(ts / p.P);
        const int h0 = ch * HT / p.chunks, h1 = (ch + 1) * HT / p.chunks;
        Vec<V> lo[HB], hi[HB];
        float cs[V], sn[V];
#pragma unroll
        for (int k = 0; k < HB; ++k)
            if (live && h0 + k < h1) {
                const int w = h0 + k >= p.H[0];
                const Heads &x = p.x[w];
                const char *a = x.base + slot * x.slot + t * x.token + (h0 + k - (w ? p.H[0] : 0)) * x.head + c * 2;
                lo[k] = ld<V>(a);
                hi[k] = ld<V>(a + h * 2);
            }
        if (live) angles<V>(p, t, c, cs, sn);
#pragma unroll
        for (int k = 0; k < HB; ++k) {
            const bool here = live && h0 + k < h1;
            float f[2 * V], sum = 0.f;
            if (here) {
                unpack<V>(lo[k], f);
                unpack<V>(hi[k], f + V);
#pragma unroll
                for (int j = 0; j < 2 * V; ++j) sum = fmaf(f[j], f[j], sum);
            }
            sum = group_sum<L>(sum);
            if (!here) continue;
            const float r = rsqrtf(fmaf(sum, inv_d, p.eps));
            const int w = h0 + k >= p.H[0];
            float g[2 * V];
            ldf<V>(p.g[w] + c, g);
            ldf<V>(p.g[w] + h + c, g + V);
#pragma unroll
            for (int j = 0; j < 2 * V; ++j) f[j] = f[j] * r * g[j];
            rotate<V>(f, cs, sn, PAIRS, false);
            const Heads &z = p.z[w];
            char *a = z.base + slot * z.slot + t * z.token + (h0 + k - (w ? p.H[0] : 0)) * z.head + c * 2;
            st<V>(a, f);
            st<V>(a + h * 2, f + V);
        }
    }
}

// The gradient.  A block stays within one slot; its threads keep the weight
// gradients of their columns over all their rows, and the block's sums go to
// one row of `part`, added up by k_qk_norm_dg in block order.
template <int V, int L, bool PAIRS>
__global__ void __launch_bounds__(THREADS, 2) k_qk_norm_bwd(const Params p)
{
    __shared__ float red[THREADS / 32][2][512];
    const int lane = threadIdx.x % L, c = lane * V, h = p.D / 2;
    const bool on = c < h;
    const int slot = blockIdx.x / p.blocks, blk = blockIdx.x % p.blocks;
    const float inv_d = 1.f / (float)p.D;
    for (int w = 0; w < 2; ++w) {
        float acc[2 * V] = {};
        float g[2 * V] = {};
        if (on) {
            ldf<V>(p.g[w] + c, g);
            ldf<V>(p.g[w] + h + c, g + V);
        }
        const Heads &xh_ = p.x[w], &zh = p.z[w], &dh = p.dx[w];
        const int chunks = (p.H[w] + HB / 2 - 1) / (HB / 2);
        const long long items = (long long)p.T * chunks;
        for (long long i0 = (long long)blk * (THREADS / L) + (threadIdx.x & ~31) / L; i0 < items;
             i0 += (long long)p.blocks * (THREADS / L)) {
            const long long i = i0 + (threadIdx.x & 31) / L;
            const bool live = on && i < items;
            const int t = (int)(i / chunks), hb = (int)(i % chunks) * (HB / 2);
            Vec<V> xl[HB / 2], xu[HB / 2], zl[HB / 2], zu[HB / 2];
            float cs[V], sn[V];
#pragma unroll
            for (int k = 0; k < HB / 2; ++k)
                if (live && hb + k < p.H[w]) {
                    const char *a = xh_.base + slot * xh_.slot + t * xh_.token + (hb + k) * xh_.head + c * 2;
                    const char *b = zh.base + slot * zh.slot + t * zh.token + (hb + k) * zh.head + c * 2;
                    xl[k] = ld<V>(a);
                    xu[k] = ld<V>(a + h * 2);
                    zl[k] = ld<V>(b);
                    zu[k] = ld<V>(b + h * 2);
                }
            if (live) angles<V>(p, t, c, cs, sn);
#pragma unroll
            for (int k = 0; k < HB / 2; ++k) {
                const bool here = live && hb + k < p.H[w];
                float x[2 * V], d[2 * V], ss = 0.f, st_ = 0.f;
                if (here) {
                    unpack<V>(xl[k], x);
                    unpack<V>(xu[k], x + V);
                    unpack<V>(zl[k], d);
                    unpack<V>(zu[k], d + V);
                    rotate<V>(d, cs, sn, PAIRS, true);
#pragma unroll
                    for (int j = 0; j < 2 * V; ++j) {
                        ss = fmaf(x[j], x[j], ss);
                        st_ = fmaf(d[j] * g[j], x[j], st_);
                    }
                }
                ss = group_sum<L>(ss);
                st_ = group_sum<L>(st_);
                if (!here) continue;
                const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
                const float m = st_ * r * inv_d;            // mean of t xh
#pragma unroll
                for (int j = 0; j < 2 * V; ++j) {
                    const float xh = x[j] * r;
                    acc[j] = fmaf(d[j], xh, acc[j]);
                    d[j] = r * fmaf(-xh, m, d[j] * g[j]);
                }
                char *a = dh.base + slot * dh.slot + t * dh.token + (hb + k) * dh.head + c * 2;
                st<V>(a, d);
                st<V>(a + h * 2, d + V);
            }
        }
        // sum the groups of the warp, then the warps
#pragma unroll
        for (int j = 0; j < 2 * V; ++j)
#pragma unroll
            for (int o = 16; o >= L; o >>= 1) acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], o);
        if (on && (threadIdx.x & 31) < L)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                red[threadIdx.x >> 5][w][c + j] = acc[j];
                red[threadIdx.x >> 5][w][h + c + j] = acc[V + j];
            }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.D; i += THREADS) {
        const int w = i >= p.D, d = w ? i - p.D : i;
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < THREADS / 32; ++k) s += red[k][w][d];
        p.part[((size_t)blk * p.P + slot) * 2 * p.D + i] = s;
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
static void launch(const Params &p, bool grad, int blocks, cudaStream_t st)
{
    if (grad) {
        if (p.pairs) k_qk_norm_bwd<V, L, true><<<p.P * p.blocks, THREADS, 0, st>>>(p);
        else k_qk_norm_bwd<V, L, false><<<p.P * p.blocks, THREADS, 0, st>>>(p);
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

static void launch_any(const Params &p, bool grad, int blocks, cudaStream_t st)
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

// Blocks of one slot in the gradient: four per SM over all slots, or fewer
// when the rows do not fill them.
static int bwd_blocks(const rc_qk_norm_args &a, int sms)
{
    const long long per_block = THREADS / group_lanes(a.D, a.D % 16 ? 4 : 8);
    const long long rows = (long long)a.T * ((a.Hq > a.Hkv ? a.Hq : a.Hkv) + 1) / 2;
    long long n = (rows + per_block - 1) / per_block;
    const long long most = (4ll * sms + a.P - 1) / a.P;
    if (n > most) n = most;
    return n < 1 ? 1 : (int)n;
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
    long long blocks = 0;
    if (grad) {
        p.dg[0] = a.dgamma_q;
        p.dg[1] = a.dgamma_k;
        p.blocks = bwd_blocks(a, sms);
        const size_t bytes = (size_t)p.blocks * a.P * 2 * a.D * 4;
        void *s = a.workspace;
        if (a.workspace && ((uintptr_t)a.workspace & 255u)) return set_error(RC_ERR_INVALID, "workspace must be 256-byte aligned");
        if (a.workspace && a.ws_bytes < bytes)
            return set_error(RC_ERR_INVALID, "workspace of %zu bytes is below the %zu this call needs", a.ws_bytes, bytes);
        if (!a.workspace && (rc_ = prepare_scratch(bytes, &s))) return rc_;
        p.part = (float *)s;
    } else {
        p.chunks = (a.Hq + a.Hkv + HB - 1) / HB;
        const long long per_block = THREADS / group_lanes(a.D, a.D % 16 ? 4 : 8);
        blocks = ((long long)a.T * a.P * p.chunks + per_block - 1) / per_block;
        if (blocks > 64ll * sms) blocks = 64ll * sms;
    }
    launch_any(p, grad, (int)blocks, (cudaStream_t)stream);
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
    return (size_t)bwd_blocks(*args, sms) * args->P * 2 * args->D * 4;
}
