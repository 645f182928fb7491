// block_norm.cu -- between a block's last matmul and the next one's first, in one
// pass: norm of the block's output, gate and residual scale, residual sum, norm
// of the sum; and its gradient, from bf16 rows or from 8-bit checkpoints.
//
//   yh = y (mean y^2 + eps)^(-1/2),  w = alpha gate gamma_post,  h = res + w yh,
//   z = h q gamma_pre,  q = (mean h^2 + eps)^(-1/2).
// Gradient, with t = dz gamma_pre and v = w yh:
//   d = dh + q (t - h q^2 mean(t h)),  dres = d,  u = d w,
//   dy = p (u - yh mean(u yh)),  p = (mean y^2 + eps)^(-1/2),
//   dgamma_pre = sum_t dz h q,  dgate / (alpha gamma_post) = dgamma_post / (alpha gate) = sum_t d yh.
// mean(u yh) needs d, which needs sums over the whole row itself; taken apart,
//   sum u yh = sum v dh + q sum v t - q^3 mean(t h) sum v h,
// it joins the sums for d in one round, so a row takes two rounds (of sum y^2, then
// of the rest) instead of three.
//
// Bound by memory.  A block (for wide rows a pair) works on one row at a time and keeps it in registers;
// every thread copies its own share of the coming rows into its own shared-memory
// slots (cp.async) and reads it back, so no barrier stands between loads and use.
#include <cmath>

#include "act8.cuh"
#include "heads.h"
#include "internal.h"
#include "per_device.h"
#include "ringcoll.h"
#include "tc.cuh"

namespace rc {
namespace bn {

constexpr int kMostChannels = 16384;

// Where a thread keeps the weights of its channels.
enum Weights { IN_REGISTERS, IN_SHARED };

struct Params {
    Rows y, res, h, z, dh, dz, dy, dres;
    Act8 y8, res8, z8;
    const float *gpost, *gate, *gpre;
    float *dpost, *dgate, *dpre, *part;
    FastDiv tokens;                  // rows of a slot
    uint32_t rows, T, N, vecs;
    uint32_t y_chunk, dy_chunk;      // channels of a slot of y, dy (0: rows of all N)
    int stages, per, sums, clear;    // gradient: blocks of a slot; sums of a block's part; 1: zero `part` once read
    float alpha, eps, inv_n;
};

template <int B>
__device__ __forceinline__ void copy(uint32_t dst, const void *src)
{
    if (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void wait_oldest(int stages)
{
    if (stages == 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else if (stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else asm volatile("cp.async.wait_group 3;" ::: "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

// Sums of K values over a row's block, or pair of blocks (CL = 2), the same in every
// thread, always added in the same pattern.  In a warp the values are divided over the lanes
// while they are added (K values cost 9 exchanges in the place of 5 K), each group of
// 32 / PAD lanes ending with one of them; every warp leaves its sums in both blocks of a
// pair, and adds up all warps' sums alike.  Two areas take turns, so one barrier does; the
// places of warps that do not exist hold zeros.
constexpr int kAreaRow = 36;                            // floats of a value's row: 32 warps, and no bank twice
constexpr int kAreaBytes = 2 * 8 * kAreaRow * 4;

template <int K, int CL>
__device__ __forceinline__ void block_sum(float (&v)[K], float *area, int &turn)
{
    constexpr int PAD = K == 1 ? 1 : K == 2 ? 2 : 8, GROUP = 32 / PAD;
    const uint32_t lane = threadIdx.x & 31;
    float s[PAD];
#pragma unroll
    for (int k = 0; k < PAD; ++k) s[k] = k < K ? v[k] : 0.f;
#pragma unroll
    for (int n = PAD / 2, o = 16; n; n /= 2, o /= 2)
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const bool upper = lane & o;
            const float keep = upper ? s[k + n] : s[k], give = upper ? s[k] : s[k + n];
            s[k] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
        }
#pragma unroll
    for (int o = GROUP / 2; o; o /= 2) s[0] += __shfl_xor_sync(0xFFFFFFFFu, s[0], o);
    if (CL > 1 || blockDim.x > 32) {
        float *const row = area + turn * (8 * kAreaRow) + lane / GROUP * kAreaRow;
        turn ^= 1;
        if (CL == 1) {
            if (lane % GROUP == 0) row[threadIdx.x >> 5] = s[0];
            __syncthreads();
        } else {
            const uint32_t at = tc::smem_u32(row + tc::cluster_ctarank() * 16 + (threadIdx.x >> 5));
            if (lane % GROUP == 0)
#pragma unroll
                for (int c = 0; c < CL; ++c)
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(tc::mapa_shared(at, c)), "f"(s[0]) : "memory");
            __syncwarp();
            tc::cluster_sync_all();
        }
        if (PAD == 8) {
            const float4 a = *(const float4 *)(row + lane % 4 * 8), b = *(const float4 *)(row + lane % 4 * 8 + 4);
            s[0] = ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
        } else if (PAD == 2) {
            const float2 a = *(const float2 *)(row + lane % 16 * 2);
            s[0] = a.x + a.y;
        } else {
            s[0] = row[lane];
        }
#pragma unroll
        for (int o = GROUP / 2; o; o /= 2) s[0] += __shfl_xor_sync(0xFFFFFFFFu, s[0], o);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = PAD == 1 ? s[0] : __shfl_sync(0xFFFFFFFFu, s[0], k * GROUP);
}

template <int CL>
__device__ __forceinline__ void clear_area(float *area)
{
    for (int i = threadIdx.x; i < kAreaBytes / 4; i += blockDim.x) area[i] = 0.f;
    __syncthreads();
    if (CL > 1) tc::cluster_sync_all();
}

// The weights w and gamma_pre of vector v.  In shared memory the first and the last
// four channels of the vectors lie in planes, 16 bytes a lane.
__device__ __forceinline__ void ld8f(const float *p, f32x2 (&f)[4])
{
    const float4 a = __ldg((const float4 *)p), b = __ldg((const float4 *)p + 1);
    f[0] = f2(a.x, a.y);
    f[1] = f2(a.z, a.w);
    f[2] = f2(b.x, b.y);
    f[3] = f2(b.z, b.w);
}
__device__ __forceinline__ void scale_of(const Params &p, uint32_t v, f32x2 (&w)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = both(p.alpha);
    f32x2 g[4];
    if (p.gate) {
        ld8f(p.gate + v * 8, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = mul2(w[i], g[i]);
    }
    if (p.gpost) {
        ld8f(p.gpost + v * 8, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = mul2(w[i], g[i]);
    }
}
__device__ __forceinline__ void sts_plane(float *plane, uint32_t at, uint32_t vecs, const f32x2 (&f)[4])
{
    *(float4 *)(plane + at * 4) = make_float4(lo(f[0]), hi(f[0]), lo(f[1]), hi(f[1]));
    *(float4 *)(plane + (vecs + at) * 4) = make_float4(lo(f[2]), hi(f[2]), lo(f[3]), hi(f[3]));
}
__device__ __forceinline__ void lds_plane(const float *plane, uint32_t at, uint32_t vecs, f32x2 (&f)[4])
{
    const float4 a = *(const float4 *)(plane + at * 4), b = *(const float4 *)(plane + (vecs + at) * 4);
    f[0] = f2(a.x, a.y);
    f[1] = f2(a.z, a.w);
    f[2] = f2(b.x, b.y);
    f[3] = f2(b.z, b.w);
}

// Bytes that Scales keeps of shared memory.
__host__ __device__ __forceinline__ uint32_t scale_bytes(int vpt, uint32_t threads) { return 64u * vpt * threads; }

template <int VPT, Weights WHERE, bool PRE>
struct Scales {
    f32x2 w[WHERE == IN_REGISTERS ? VPT : 1][4], g[WHERE == IN_REGISTERS ? VPT : 1][4];
    float *plane;

    // first: the block's first vector
    __device__ __forceinline__ void init(const Params &p, float *shared, uint32_t first)
    {
        plane = shared;
        const uint32_t vecs = VPT * blockDim.x;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t at = i * blockDim.x + threadIdx.x, v = first + at;
            f32x2 a[4] = {}, b[4] = {};
            if (v < p.vecs) {
                scale_of(p, v, a);
                if (PRE) ld8f(p.gpre + v * 8, b);
            }
            if (WHERE == IN_SHARED) {               // read back by the thread that wrote them
                sts_plane(plane, at, vecs, a);
                if (PRE) sts_plane(plane + vecs * 8, at, vecs, b);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) w[i][k] = a[k], g[i][k] = b[k];
            }
        }
    }
    __device__ __forceinline__ void scale(int i, f32x2 (&f)[4]) const
    {
        if (WHERE == IN_SHARED) lds_plane(plane, i * blockDim.x + threadIdx.x, VPT * blockDim.x, f);
        else
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = w[i][k];
    }
    __device__ __forceinline__ void pre(int i, f32x2 (&f)[4]) const
    {
        if (WHERE == IN_SHARED) lds_plane(plane + VPT * blockDim.x * 8, i * blockDim.x + threadIdx.x, VPT * blockDim.x, f);
        else
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = g[i][k];
    }
};

// y or dy, whose slots hold `chunk` channels of all rows (0: rows of all channels): the start
// of row `row` (t of slot r), and behind it vector v.
__device__ __forceinline__ char *row_of(const Rows &o, uint32_t chunk, uint32_t row, uint32_t r, uint32_t t) { return chunk ? o.at(0, row) : o.at(r, t); }
__device__ __forceinline__ size_t behind(const Rows &o, uint32_t chunk, uint32_t v)
{
    if (!chunk) return (size_t)v * 16;
    const uint32_t s = v * 8 / chunk;
    return s * o.slot + (v * 8 - s * chunk) * 2;
}

// ------------------------------------------------------------ forward
template <int VPT, int MAXT, int CL, Weights WHERE, bool POST, bool PRE>
__global__ void __launch_bounds__(MAXT, 1) k_block_norm(const Params p)
{
    extern __shared__ __align__(16) uint8_t sm[];
    float *const area = (float *)sm;
    uint8_t *const after = sm + kAreaBytes;
    const uint32_t threads = blockDim.x, stage_bytes = 2 * VPT * 16 * threads;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(after + (WHERE == IN_SHARED ? scale_bytes(VPT, threads) : 0)) + threadIdx.x * 16;
    Scales<VPT, WHERE, PRE> ws;
    const uint32_t first_vec = CL > 1 ? tc::cluster_ctarank() * (VPT * threads) : 0, block = blockIdx.x / CL, blocks = gridDim.x / CL;
    ws.init(p, (float *)after, first_vec);
    clear_area<CL>(area);
    int turn = 0;
    size_t yoff[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) yoff[i] = behind(p.y, p.y_chunk, first_vec + i * threads + threadIdx.x);
    auto fetch = [&](uint32_t row, int stage) {
        if (row < p.rows) {
            const uint32_t r = p.tokens(row), t = row - r * p.T;
            const char *const yrow = row_of(p.y, p.y_chunk, row, r, t), *const rrow = p.res.at(r, t);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const uint32_t v = first_vec + i * threads + threadIdx.x;
                if (v >= p.vecs) continue;
                copy<16>(ring + stage * stage_bytes + i * 16 * threads, yrow + yoff[i]);
                copy<16>(ring + stage * stage_bytes + (VPT + i) * 16 * threads, rrow + v * 16);
            }
        }
        copies_done();
    };
    uint32_t ahead = block;                        // rows stay below 2^31 - 2^20, and a grid below 2^16
    for (int s = 0; s < p.stages; ++s, ahead += blocks) fetch(ahead, s);
    int stage = 0;
    for (uint32_t row = block; row < p.rows; row += blocks, ahead += blocks) {
        wait_oldest(p.stages);
        const uint32_t r = p.tokens(row), t = row - r * p.T;
        uint4 yw[VPT], rw[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            yw[i] = rw[i] = make_uint4(0, 0, 0, 0);
            if (first_vec + i * threads + threadIdx.x >= p.vecs) continue;
            yw[i] = lds16(ring + stage * stage_bytes + i * 16 * threads);
            rw[i] = lds16(ring + stage * stage_bytes + (VPT + i) * 16 * threads);
        }
        fetch(ahead, stage);
        stage = stage + 1 == p.stages ? 0 : stage + 1;
        float rp = 1.f;
        if (POST) {
            f32x2 ss = 0;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                f32x2 y[4];
                wide8(yw[i], y);
#pragma unroll
                for (int k = 0; k < 4; ++k) ss = fma2(y[k], y[k], ss);
            }
            float sum[1] = {hsum(ss)};
            block_sum<1, CL>(sum, area, turn);
            rp = rsqrtf(fmaf(sum[0], p.inv_n, p.eps));
        }
        f32x2 h[VPT][4], hh = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t v = first_vec + i * threads + threadIdx.x;
            const bool on = v < p.vecs;
            f32x2 y[4], w[4];
            wide8(yw[i], y);
            wide8(rw[i], h[i]);
            if (on) ws.scale(i, w);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (on) h[i][k] = fma2(w[k], mul2(y[k], both(rp)), h[i][k]);
                hh = fma2(h[i][k], h[i][k], hh);
            }
            if (on) __stcs((uint4 *)(p.h.at(r, t) + v * 16), narrow8(h[i]));
            if (p.y8.q.base) put8(p.y8, r, t, v, on, yw[i]);
            if (p.res8.q.base) put8(p.res8, r, t, v, on, rw[i]);
        }
        if (!PRE) continue;
        float sum[1] = {hsum(hh)};
        block_sum<1, CL>(sum, area, turn);
        const float q = rsqrtf(fmaf(sum[0], p.inv_n, p.eps));
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t v = first_vec + i * threads + threadIdx.x;
            const bool on = v < p.vecs;
            f32x2 g[4];
            uint4 zw = make_uint4(0, 0, 0, 0);
            if (on) {
                ws.pre(i, g);
#pragma unroll
                for (int k = 0; k < 4; ++k) h[i][k] = mul2(mul2(h[i][k], both(q)), g[k]);
                zw = narrow8(h[i]);
                __stcs((uint4 *)(p.z.at(r, t) + v * 16), zw);
            }
            if (p.z8.q.base) put8(p.z8, r, t, v, on, zw);
        }
    }
}

// ------------------------------------------------------------ gradient
// A block takes rows j, j + per, ... of one slot.  Its threads keep the sums of
// their channels over all its rows, and leave them in the block's part, which
// k_block_sums adds up in block order.
template <int VPT, int MAXT, int CL, bool FULL, Weights WHERE, bool HELD, bool POST, bool PRE>
__global__ void __launch_bounds__(MAXT, 1) k_block_norm_bwd(const Params p)
{
    extern __shared__ __align__(16) uint8_t sm[];
    constexpr int YB = HELD ? 8 : 16;                   // staged bytes of 8 channels of y and of res
    float *const area = (float *)sm;
    uint8_t *const after = sm + kAreaBytes;
    const uint32_t threads = blockDim.x, in_bytes = VPT * YB * threads, d_bytes = VPT * 16 * threads;
    const uint32_t stage_bytes = 2 * in_bytes + (PRE ? 2 : 1) * d_bytes;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(after + (WHERE == IN_SHARED ? scale_bytes(VPT, threads) : 0));
    Scales<VPT, WHERE, PRE> ws;
    const uint32_t first_vec = CL > 1 ? tc::cluster_ctarank() * (VPT * threads) : 0, block = blockIdx.x / CL;
    ws.init(p, (float *)after, first_vec);
    clear_area<CL>(area);
    const uint32_t r = block / p.per, first = block - r * p.per;
    int turn = 0;
    size_t yoff[HELD ? 1 : VPT], dyoff[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (!HELD) yoff[i] = behind(p.y, p.y_chunk, first_vec + i * threads + threadIdx.x);
        dyoff[i] = behind(p.dy, p.dy_chunk, first_vec + i * threads + threadIdx.x);
    }
    auto fetch = [&](uint32_t t, int stage) {
        if (t < p.T) {
            const uint32_t at = ring + stage * stage_bytes + threadIdx.x * YB, dat = ring + stage * stage_bytes + 2 * in_bytes + threadIdx.x * 16;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const uint32_t v = first_vec + i * threads + threadIdx.x;
                if (!FULL && v >= p.vecs) continue;
                if (HELD) {
                    copy<8>(at + i * YB * threads, p.y8.q.at(r, t) + v * 8);
                    copy<8>(at + in_bytes + i * YB * threads, p.res8.q.at(r, t) + v * 8);
                } else {
                    copy<16>(at + i * YB * threads, row_of(p.y, p.y_chunk, r * p.T + t, r, t) + yoff[i]);
                    copy<16>(at + in_bytes + i * YB * threads, p.res.at(r, t) + v * 16);
                }
                if (p.dh.base) copy<16>(dat + i * 16 * threads, p.dh.at(r, t) + v * 16);
                if (PRE) copy<16>(dat + d_bytes + i * 16 * threads, p.dz.at(r, t) + v * 16);
            }
        }
        copies_done();
    };
    uint32_t ey[HELD ? VPT : 1], er[HELD ? VPT : 1];     // the groups' bytes of the next row
    auto fetch_groups = [&](uint32_t t) {
        if (HELD && t < p.T)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const uint32_t v = first_vec + i * threads + threadIdx.x;
                if (!FULL && v >= p.vecs) continue;
                ey[i] = __ldcs((const uint8_t *)p.y8.e.at(r, t) + v / 4);
                er[i] = __ldcs((const uint8_t *)p.res8.e.at(r, t) + v / 4);
            }
    };
    f32x2 acc_d[VPT][4] = {}, acc_z[VPT][4] = {};
    uint32_t ahead = first;
    fetch_groups(first);
    for (int s = 0; s < p.stages; ++s, ahead += p.per) fetch(ahead, s);
    int stage = 0;
    for (uint32_t t = first; t < p.T; t += p.per, ahead += p.per) {
        wait_oldest(p.stages);
        const uint32_t at = ring + stage * stage_bytes + threadIdx.x * YB, dat = ring + stage * stage_bytes + 2 * in_bytes + threadIdx.x * 16;
        f32x2 y[VPT][4], h[VPT][4];
        uint4 dh[VPT], dz[VPT];
        f32x2 ss = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            dh[i] = dz[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[i][k] = h[i][k] = 0;
            if (!FULL && first_vec + i * threads + threadIdx.x >= p.vecs) continue;
            if (HELD) {
                held8(lds8(at + i * YB * threads), ey[i], y[i]);
                held8(lds8(at + in_bytes + i * YB * threads), er[i], h[i]);
            } else {
                wide8(lds16(at + i * YB * threads), y[i]);
                wide8(lds16(at + in_bytes + i * YB * threads), h[i]);
            }
            if (p.dh.base) dh[i] = lds16(dat + i * 16 * threads);
            if (PRE) dz[i] = lds16(dat + d_bytes + i * 16 * threads);
#pragma unroll
            for (int k = 0; k < 4; ++k) ss = fma2(y[i][k], y[i][k], ss);
        }
        fetch(ahead, stage);
        fetch_groups(t + p.per);
        stage = stage + 1 == p.stages ? 0 : stage + 1;
        float rp = 1.f;
        if (POST) {
            float sum[1] = {hsum(ss)};
            block_sum<1, CL>(sum, area, turn);
            rp = rsqrtf(fmaf(sum[0], p.inv_n, p.eps));
        }
        f32x2 hh = 0, th = 0, vd = 0, vt = 0, vh = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t v = first_vec + i * threads + threadIdx.x;
            if (!FULL && v >= p.vecs) continue;
            f32x2 w[4], g[4], d[4], z[4];
            ws.scale(i, w);
            if (PRE) ws.pre(i, g), wide8(dz[i], z);
            if (POST) wide8(dh[i], d);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                y[i][k] = mul2(y[i][k], both(rp));
                const f32x2 x = mul2(w[k], y[i][k]);
                h[i][k] = add2(h[i][k], x);
                if (POST) vd = fma2(x, d[k], vd);
                if (PRE) {
                    const f32x2 tt = mul2(z[k], g[k]);
                    hh = fma2(h[i][k], h[i][k], hh);
                    th = fma2(tt, h[i][k], th);
                    if (POST) vt = fma2(x, tt, vt), vh = fma2(x, h[i][k], vh);
                }
            }
        }
        float q = 0.f, c = 0.f, m = 0.f;                // d = dh + q t - c h;  dy = rp (d w - yh m)
        if (PRE && POST) {
            float s[5] = {hsum(hh), hsum(th), hsum(vd), hsum(vt), hsum(vh)};
            block_sum<5, CL>(s, area, turn);
            q = rsqrtf(fmaf(s[0], p.inv_n, p.eps));
            c = q * q * q * (s[1] * p.inv_n);
            m = (s[2] + q * s[3] - c * s[4]) * p.inv_n;
        } else if (PRE) {
            float s[2] = {hsum(hh), hsum(th)};
            block_sum<2, CL>(s, area, turn);
            q = rsqrtf(fmaf(s[0], p.inv_n, p.eps));
            c = q * q * q * (s[1] * p.inv_n);
        } else if (POST) {
            float s[1] = {hsum(vd)};
            block_sum<1, CL>(s, area, turn);
            m = s[0] * p.inv_n;
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t v = first_vec + i * threads + threadIdx.x;
            if (!FULL && v >= p.vecs) continue;
            f32x2 w[4], g[4], d[4], z[4];
            ws.scale(i, w);
            wide8(dh[i], d);
            if (PRE) ws.pre(i, g), wide8(dz[i], z);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (PRE) {
                    acc_z[i][k] = fma2(z[k], mul2(h[i][k], both(q)), acc_z[i][k]);
                    d[k] = fma2(mul2(z[k], g[k]), both(q), d[k]);
                    d[k] = fma2(h[i][k], both(-c), d[k]);
                }
                acc_d[i][k] = fma2(d[k], y[i][k], acc_d[i][k]);
                w[k] = mul2(d[k], w[k]);
                if (POST) w[k] = mul2(fma2(y[i][k], both(-m), w[k]), both(rp));
            }
            __stcs((uint4 *)(p.dres.at(r, t) + v * 16), narrow8(d));
            __stcs((uint4 *)(row_of(p.dy, p.dy_chunk, r * p.T + t, r, t) + dyoff[i]), narrow8(w));
        }
    }
    if (!p.sums) return;
    float *part = p.part + (size_t)block * p.sums * p.N;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (k == 0 ? !(p.gpost || p.gate) : !PRE) continue;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t v = first_vec + i * threads + threadIdx.x;
            if (!FULL && v >= p.vecs) continue;
            const f32x2(&f)[4] = k ? acc_z[i] : acc_d[i];
            ((float4 *)(part + v * 8))[0] = make_float4(lo(f[0]), hi(f[0]), lo(f[1]), hi(f[1]));
            ((float4 *)(part + v * 8))[1] = make_float4(lo(f[2]), hi(f[2]), lo(f[3]), hi(f[3]));
        }
        part += p.N;
    }
}

// Sum z of slot y over the blocks of the slot, four channels a lane: warp k adds parts k,
// k + SUM_WARPS, ... and the warps' sums are added in order.  CLEAR: in a caller's workspace
// the parts are zeroed once read, because other calls keep signal words there.
template <bool CLEAR, int SUM_WARPS>
__global__ void __launch_bounds__(32 * SUM_WARPS) k_block_sums(const Params p)
{
    __shared__ float4 red[SUM_WARPS][32];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = (blockIdx.x * 32 + lane) * 4, slot = blockIdx.y, which = blockIdx.z;
    asm volatile("griddepcontrol.wait;" ::: "memory");     // the parts are written
    const size_t step = (size_t)p.sums * p.N;
    float *const part = p.part + (size_t)slot * p.per * step + (size_t)which * p.N + c;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < p.N)
#pragma unroll 8
        for (uint32_t b = warp; b < (uint32_t)p.per; b += SUM_WARPS) {
            const float4 v = *(const float4 *)(part + b * step);
            s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
        }
    if (CLEAR && c < p.N)                                  // in a loop of its own: stores would hold up the loads
        for (uint32_t b = warp; b < (uint32_t)p.per; b += SUM_WARPS) *(float4 *)(part + b * step) = make_float4(0.f, 0.f, 0.f, 0.f);
    red[warp][lane] = s;
    __syncthreads();
    if (warp || c >= p.N) return;
#pragma unroll
    for (int k = 1; k < SUM_WARPS; ++k) {
        const float4 v = red[k][lane];
        s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
    }
    auto put = [&](float *to, float f, const float *g) {
        const float4 w = g ? __ldg((const float4 *)(g + c)) : make_float4(1.f, 1.f, 1.f, 1.f);
        to += (size_t)slot * p.N + c;                      // a caller's [P][N] floats, perhaps not on 16 bytes
        to[0] = f * s.x * w.x;
        to[1] = f * s.y * w.y;
        to[2] = f * s.z * w.z;
        to[3] = f * s.w * w.w;
    };
    if (which == 0 && (p.gpost || p.gate)) {
        if (p.gpost) put(p.dpost, p.alpha, p.gate);
        if (p.gate) put(p.dgate, p.alpha, p.gpost);
    } else {
        put(p.dpre, 1.f, nullptr);
    }
}

// ------------------------------------------------------------ host
// Vectors of 8 channels a thread.  Two halve what a row costs besides its channels (the
// sums over the block above all): 8192 x 4096 forward with checkpoints 58 us against 67
// with one, the gradient 72 against 100.  Where no SM gets a second row only its latency
// counts, and one is quicker (8 rows 4.1 us against 4.5).  Rows above 8192 channels are
// divided over a pair of blocks, which leave their sums in one another's shared memory.
struct Shape {
    int vpt, cl, threads, stages, regs;
    bool full;                       // every thread has all its vectors
    size_t smem;
};

static Shape shape_of(const rc_block_norm_args &a, bool grad, int sms)
{
    const int vecs = a.N / 8;
    Shape s{};
    s.cl = vecs > 1024 ? 2 : 1;
    s.vpt = s.cl == 1 && (long long)a.P * a.T <= sms ? 1 : 2;
    s.regs = s.vpt == 1 ? 64 : 128;                      // what the launch bounds leave a thread
    s.threads = ((vecs + s.vpt * s.cl - 1) / (s.vpt * s.cl) + 31) / 32 * 32;
    s.full = vecs == s.vpt * s.cl * s.threads;
    const bool held = grad && a.y8.q.base;
    const size_t lane = grad ? (held ? 16 : 32) + (a.gamma_pre ? 32 : 16) : 32;
    const size_t stage = lane * s.vpt * s.threads, fixed = kAreaBytes + (grad ? scale_bytes(s.vpt, s.threads) : 0);
    s.stages = 3;
    while (s.stages > 1 && fixed + s.stages * stage > (s.threads * s.regs > 32768 ? 220u : 110u) * 1024) --s.stages;
    s.smem = fixed + s.stages * stage;
    return s;
}

// Rows at once (blocks or pairs of them) that the GPU holds: by threads, registers (the
// launch bounds' share) and shared memory.
static int resident(const Shape &s, int sms)
{
    const int t = 2048 / s.threads, r = 65536 / (s.regs * s.threads), m = (int)(227 * 1024 / (s.smem + 1024));
    int n = t < r ? t : r;
    n = n < m ? n : m;
    n = n < 1 ? 1 : n > 32 ? 32 : n;
    return n * sms / s.cl;
}

static int blocks_of_slot(const rc_block_norm_args &a, const Shape &s, int sms)
{
    const int most = (resident(s, sms) + a.P - 1) / a.P;
    return a.T < most ? (a.T < 1 ? 1 : a.T) : most;
}

template <auto KERNEL>
static cudaError_t start(unsigned blocks, const Shape &s, const Params &p, cudaStream_t st)
{
    static OncePerDevice once;
    const cudaError_t e = once([] { return cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024); });
    if (e != cudaSuccess) return e;
    if (s.cl == 1) {
        KERNEL<<<blocks, s.threads, s.smem, st>>>(p);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks * s.cl);
    cfg.blockDim = dim3(s.threads);
    cfg.dynamicSmemBytes = s.smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = s.cl;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, KERNEL, p);
}

template <bool HELD, bool POST, bool PRE>
static cudaError_t launch_grad(unsigned blocks, const Shape &s, const Params &p, cudaStream_t st)
{
    if (s.vpt == 1) return start<k_block_norm_bwd<1, 1024, 1, false, IN_SHARED, HELD, POST, PRE>>(blocks, s, p, st);
    if (s.cl == 2) return start<k_block_norm_bwd<2, 512, 2, false, IN_SHARED, HELD, POST, PRE>>(blocks, s, p, st);
    if (s.full) return start<k_block_norm_bwd<2, 512, 1, true, IN_SHARED, HELD, POST, PRE>>(blocks, s, p, st);
    return start<k_block_norm_bwd<2, 512, 1, false, IN_SHARED, HELD, POST, PRE>>(blocks, s, p, st);
}

template <bool POST, bool PRE>
static cudaError_t launch(bool grad, bool held, unsigned blocks, const Shape &s, const Params &p, cudaStream_t st)
{
    if (grad) return held ? launch_grad<true, POST, PRE>(blocks, s, p, st) : launch_grad<false, POST, PRE>(blocks, s, p, st);
    if (s.vpt == 1) return start<k_block_norm<1, 1024, 1, IN_REGISTERS, POST, PRE>>(blocks, s, p, st);
    if (s.cl == 2) return start<k_block_norm<2, 512, 2, IN_REGISTERS, POST, PRE>>(blocks, s, p, st);
    return start<k_block_norm<2, 512, 1, IN_REGISTERS, POST, PRE>>(blocks, s, p, st);
}

static cudaError_t launch_any(bool grad, bool held, unsigned blocks, const Shape &s, const Params &p, cudaStream_t st)
{
    if (p.gpost) return p.gpre ? launch<true, true>(grad, held, blocks, s, p, st) : launch<true, false>(grad, held, blocks, s, p, st);
    return p.gpre ? launch<false, true>(grad, held, blocks, s, p, st) : launch<false, false>(grad, held, blocks, s, p, st);
}

static cudaError_t launch_sums(const Params &p, int P, cudaStream_t st)
{
    // set up while the gradient runs; its blocks start when that has ended
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((p.N + 127) / 128, (unsigned)P, (unsigned)p.sums);
    const bool few = cfg.gridDim.x * cfg.gridDim.y * cfg.gridDim.z < 128;      // blocks of 32 warps, if blocks are few
    cfg.blockDim = dim3(few ? 1024 : 256);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, p.clear ? (few ? k_block_sums<true, 32> : k_block_sums<true, 8>) : (few ? k_block_sums<false, 32> : k_block_sums<false, 8>), p);
}

static int sums_of(const rc_block_norm_args &a) { return (a.gamma_post || a.gate) + (a.gamma_pre ? 1 : 0); }

static int check_sizes(const rc_block_norm_args &a)
{
    const int rc_ = check_row_sizes(a.P, a.T, a.N, kMostChannels);
    if (rc_) return rc_;
    if ((a.y_cols | a.dy_cols) & ~1) return set_error(RC_ERR_INVALID, "y_cols and dy_cols are 0 or 1");
    if ((a.y_cols || a.dy_cols) && a.N % (8 * a.P)) return set_error(RC_ERR_INVALID, "N=%d channels in P=%d chunks: not multiples of 8", a.N, a.P);
    if (!std::isfinite(a.alpha)) return set_error(RC_ERR_INVALID, "alpha must be finite");
    if (!(a.eps >= 0.f) || !std::isfinite(a.eps)) return set_error(RC_ERR_INVALID, "eps must be finite and not negative");
    if (a.reserved) return set_error(RC_ERR_INVALID, "reserved is not 0");
    return RC_OK;
}

static int run(const rc_block_norm_args *args, bool grad, void *stream)
{
    if (!args) return set_error(RC_ERR_INVALID, "null args");
    rc_block_norm_args a = *args;
    int rc_ = check_sizes(a);
    if (rc_ || (a.T == 0 && !grad)) return rc_;
    const size_t bytes = (size_t)a.N * 2, chunk = bytes / a.P, groups = (size_t)(a.N + 31) / 32;
    const bool held = grad && a.y8.q.base, some = a.T > 0;
    if (((uintptr_t)a.gamma_post | (uintptr_t)a.gate | (uintptr_t)a.gamma_pre) & 15u)
        return set_error(RC_ERR_INVALID, "gamma_post, gate and gamma_pre must be 16-byte aligned");
    if (((uintptr_t)a.dgamma_post | (uintptr_t)a.dgate | (uintptr_t)a.dgamma_pre) & 3u)
        return set_error(RC_ERR_INVALID, "dgamma_post, dgate and dgamma_pre must be 4-byte aligned");
    if (grad && ((uintptr_t)a.workspace & 255u)) return set_error(RC_ERR_INVALID, "workspace must be 256-byte aligned");
    auto rows = [&](rc_rows &x, const char *name, bool cols) {
        return cols ? check_rows(x, name, a.P, a.P * a.T, chunk, 16) : check_rows(x, name, a.P, a.T, bytes, 16);
    };
    auto packed = [&](rc_act8 &x, const char *name) { return check_act8(x, name, a.P, a.T, a.N); };
    if (some && !held && ((rc_ = rows(a.y, "y", a.y_cols)) || (rc_ = rows(a.res, "res", false)))) return rc_;
    if (!grad) {
        if (!a.gamma_pre != !a.z.base) return set_error(RC_ERR_INVALID, "z goes with gamma_pre");
        if (a.z8.q.base && !a.z.base) return set_error(RC_ERR_INVALID, "z8 goes with z");
        if ((rc_ = rows(a.h, "h", false)) || (a.z.base && (rc_ = rows(a.z, "z", false))) || (a.y8.q.base && (rc_ = packed(a.y8, "y8"))) ||
            (a.res8.q.base && (rc_ = packed(a.res8, "res8"))) || (a.z8.q.base && (rc_ = packed(a.z8, "z8"))))
            return rc_;
    } else {
        if (!held && a.res8.q.base) return set_error(RC_ERR_INVALID, "res8 goes with y8");
        if (!a.gamma_post != !a.dgamma_post || !a.gate != !a.dgate || !a.gamma_pre != !a.dgamma_pre)
            return set_error(RC_ERR_INVALID, "dgamma_post, dgate and dgamma_pre go with gamma_post, gate and gamma_pre");
        if (some) {
            if (!a.gamma_pre != !a.dz.base) return set_error(RC_ERR_INVALID, "dz goes with gamma_pre");
            if ((held && ((rc_ = packed(a.y8, "y8")) || (rc_ = packed(a.res8, "res8")))) || (a.dh.base && (rc_ = rows(a.dh, "dh", false))) ||
                (a.dz.base && (rc_ = rows(a.dz, "dz", false))) || (rc_ = rows(a.dy, "dy", a.dy_cols)) || (rc_ = rows(a.dres, "dres", false)))
                return rc_;
        }
    }
    auto at = [&](const char *name, const rc_rows &x, bool cols = false) {
        const rc_rows o = some ? x : rc_rows{};
        return cols ? rows_at(name, o, a.P, a.P * a.T, chunk) : rows_at(name, o, a.P, a.T, bytes);
    };
    auto q8 = [&](const char *name, const rc_act8 &x, bool on) { return rows_at(name, on && some ? x.q : rc_rows{}, a.P, a.T, (size_t)a.N); };
    auto e8 = [&](const char *name, const rc_act8 &x, bool on) { return rows_at(name, on && some && x.q.base ? x.e : rc_rows{}, a.P, a.T, groups); };
    const Operand y = at("y", held ? rc_rows{} : a.y, a.y_cols), res_ = at("res", held ? rc_rows{} : a.res),
                  w0 = bytes_at("gamma_post", a.gamma_post, (size_t)a.N * 4), w1 = bytes_at("gate", a.gate, (size_t)a.N * 4),
                  w2 = bytes_at("gamma_pre", a.gamma_pre, (size_t)a.N * 4);
    if (!grad) {
        const Operand out[] = {at("h", a.h), at("z", a.z), q8("y8.q", a.y8, true), e8("y8.e", a.y8, true), q8("res8.q", a.res8, true),
                               e8("res8.e", a.res8, true), q8("z8.q", a.z8, true), e8("z8.e", a.z8, true)};
        const Operand in[] = {y, res_, w0, w1, w2};
        const unsigned whole[] = {2, 0, 0, 0, 0, 0, 0, 0};
        rc_ = check_apart(out, 8, in, 5, whole);
    } else {
        const size_t wb = (size_t)a.P * a.N * 4;
        const Operand out[] = {at("dy", a.dy, a.dy_cols), at("dres", a.dres), bytes_at("dgamma_post", a.dgamma_post, wb),
                               bytes_at("dgate", a.dgate, wb), bytes_at("dgamma_pre", a.dgamma_pre, wb)};
        const Operand in[] = {at("dh", a.dh), at("dz", a.dz), y, res_, q8("y8.q", a.y8, held), e8("y8.e", a.y8, held), q8("res8.q", a.res8, held),
                              e8("res8.e", a.res8, held), w0, w1, w2};
        const unsigned whole[] = {a.dy_cols ? 0u : 3u, 3, 0, 0, 0};
        rc_ = check_apart(out, 5, in, 11, whole);
    }
    if (rc_) return rc_;
    int sms = 0;
    if ((rc_ = device_sms(&sms))) return rc_;
    const Shape s = shape_of(a, grad, sms);
    Params p{};
    p.y = rows_of(a.y), p.res = rows_of(a.res), p.h = rows_of(a.h), p.z = rows_of(a.z);
    p.dh = rows_of(a.dh), p.dz = rows_of(a.dz), p.dy = rows_of(a.dy), p.dres = rows_of(a.dres);
    p.y8 = act8_of(a.y8), p.res8 = act8_of(a.res8), p.z8 = act8_of(a.z8);
    p.gpost = a.gamma_post, p.gate = a.gate, p.gpre = a.gamma_pre;
    p.dpost = a.dgamma_post, p.dgate = a.dgate, p.dpre = a.dgamma_pre;
    p.tokens = FastDiv::of(a.T ? (uint32_t)a.T : 1u);
    p.rows = (uint32_t)a.P * a.T;
    p.T = a.T;
    p.N = a.N;
    p.vecs = a.N / 8;
    p.y_chunk = a.y_cols ? a.N / a.P : 0;
    p.dy_chunk = a.dy_cols ? a.N / a.P : 0;
    p.stages = s.stages;
    p.alpha = a.alpha;
    p.eps = a.eps;
    p.inv_n = 1.f / (float)a.N;
    unsigned blocks;
    if (!grad) {
        const uint32_t most = (uint32_t)resident(s, sms);
        blocks = p.rows < most ? p.rows : most;
    } else {
        p.per = blocks_of_slot(a, s, sms);
        p.sums = sums_of(a);
        blocks = (unsigned)(p.per * a.P);
        const size_t need = (size_t)blocks * p.sums * a.N * 4;
        void *space = a.workspace;
        if (a.workspace && a.ws_bytes < kWsHead + need)
            return set_error(RC_ERR_INVALID, "workspace of %zu bytes is below the %zu this call needs", a.ws_bytes, kWsHead + need);
        if (a.workspace) space = (char *)space + kWsHead, p.clear = 1;
        else if (need && (rc_ = prepare_scratch(need, &space))) return rc_;
        p.part = (float *)space;
    }
    cudaError_t e = launch_any(grad, held, blocks, s, p, (cudaStream_t)stream);
    if (e == cudaSuccess && grad && p.sums) e = launch_sums(p, a.P, (cudaStream_t)stream);
    if (e != cudaSuccess) return set_error(RC_ERR_CUDA, "block_norm launch: %s", cudaGetErrorString(e));
    return RC_OK;
}

} // namespace bn
} // namespace rc

extern "C" int block_norm(const rc_block_norm_args *args, void *stream) { return rc::bn::run(args, false, stream); }

extern "C" int block_norm_bwd(const rc_block_norm_args *args, void *stream) { return rc::bn::run(args, true, stream); }

extern "C" size_t block_norm_bwd_workspace_bytes(const rc_block_norm_args *args)
{
    using namespace rc::bn;
    int sms = 0;
    if (!args || check_sizes(*args) || rc::device_sms(&sms)) return 0;
    const Shape s = shape_of(*args, true, sms);
    return rc::kWsHead + (size_t)blocks_of_slot(*args, s, sms) * args->P * sums_of(*args) * args->N * 4;
}
