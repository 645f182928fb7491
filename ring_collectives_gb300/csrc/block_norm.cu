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
// Bound by memory forward.  A block (for wide rows several) works on one row at a time
// and keeps it in registers; every thread copies its own share of the coming rows into its own
// shared-memory slots (cp.async) and reads it back, so no barrier stands between loads and
// use.  Channels past the end of a row arrive as zeros, with weights of zero, and only the
// stores leave them out.  The gradient is bound by what a row costs in instructions at 16
// warps an SM, which its sums of the weights' gradients (32 registers a thread) hold it to:
// issue slots 56 % busy, the shared-memory pipe 57 % (the weights are read from there twice).
//
// Measured on 8192 x 4096 with all weights: forward 47 us (5.7 TB/s, 84 % of the copy rate), with
// checkpoints of y and res 58 us (86 %); the gradient from the checkpoints 67 + 4 us (4.8 TB/s, 70 %).
// A row's sum y^2 taken with the sums of the row before, one round a row, changed little there (70.8 to
// 69.8 us) and cost rows that do not fill their threads 7 %.
#include <cmath>

#include "act8.cuh"
#include "heads.h"
#include "internal.h"
#include "per_device.h"
#include "ringcoll.h"
#include "warp.cuh"

namespace rc {
namespace bn {

constexpr int kMostChannels = 16384;

// Where a thread keeps the weights of its channels.
enum Weights { IN_REGISTERS, IN_SHARED };

// An operand [P][T][N], or in column chunks: slot s holds channels [s chunk, (s + 1) chunk) of
// all P * T rows, `skip` bytes further from one chunk to the next than in a row of all.
struct Side {
    bool cols;
    size_t skip;                     // 0 for rows
};

struct Params {
    Rows y, res, h, z, dh, dz, dy, dres;
    Act8 y8, res8, z8;
    const float *gpost, *gate, *gpre;
    float *dpost, *dgate, *dpre, *part;
    FastDiv tokens;                  // rows of a slot
    uint32_t rows, T, N, vecs;
    Side ys, dys, dzs;               // how y, dy and dz lie
    uint32_t chunk;                  // channels of a slot of those that lie in column chunks
    int stages;                      // of rows on their way
    int per, sums, clear;            // gradient: blocks of a slot; sums of a block's part; 1: zero `part` once read
    float alpha, eps, inv_n;
    WsHeader *hdr;                   // clusters: where a wait that ran out is recorded
    unsigned long long timeout_ns;
};

// Copies B bytes; for `on` false nothing is read and zeros are written.
template <int B>
__device__ __forceinline__ void copy(uint32_t dst, const void *src, bool on)
{
    if (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(on ? 8 : 0) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void wait_oldest(int stages)
{
    if (stages == 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else if (stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else asm volatile("cp.async.wait_group 3;" ::: "memory");
}
// Every copy of this thread has landed, those of rows that do not exist (zeros) among them.
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_all;" ::: "memory"); }
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

// Sums of K values over the threads of a row, the same in every one, always added in the
// same pattern.  In a warp the values are divided over the lanes while they are added
// (K values cost 9 exchanges in the place of 5 K), each group of 32 / PAD lanes ending with
// one of them.  GL > 0: a row has GL lanes, and that is all.  Else every warp leaves its
// sums in shared memory (for a cluster of blocks in all of them) and adds up all warps' sums alike.
// Two areas take turns, so one barrier does; the places of warps that do not exist hold zeros.
//
// Between a cluster's blocks sums travel with st.async, which counts their bytes on an
// mbarrier of the block that they go to.  (A cluster barrier would have to release, and so
// wait for the row's stores to memory: 2048 rows of 16384 took 200 us for the gradient.)
constexpr int kAreaRow = 36;                            // floats of a value's row: 32 warps, and no bank twice
constexpr int kAreaBytes = 2 * 8 * kAreaRow * 4 + 32;   // two areas; two mbarriers, the abort flag

template <int GL, int CL>
struct Sums {
    const Params &p;
    float *const area;
    uint32_t uses = 0;
    bool ok = true;

    __device__ __forceinline__ uint32_t bars() const { return tc::smem_u32(area + 2 * 8 * kAreaRow); }
    __device__ __forceinline__ int *flag() const { return (int *)(area + 2 * 8 * kAreaRow + 4); }
    __device__ __forceinline__ Sums(const Params &p_, uint8_t *at) : p(p_), area((float *)at)
    {
        if constexpr (GL == 0) {
            for (int i = threadIdx.x; i < kAreaBytes / 4; i += blockDim.x) area[i] = 0.f;
            __syncthreads();
        }
        if constexpr (CL > 1) {
            if (threadIdx.x == 0) {
                tc::mbar_init(bars(), 1);
                tc::mbar_init(bars() + 8, 1);
                asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            }
            __syncthreads();
            tc::cluster_sync_all();
        }
    }

    template <int K>
    __device__ __forceinline__ void operator()(float (&v)[K])
    {
        if (GL && GL < 32) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int o = GL / 2; o; o /= 2) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
            return;
        }
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
        if (!GL) {
            const uint32_t turn = uses & 1;
            float *const row = area + turn * (8 * kAreaRow) + lane / GROUP * kAreaRow;
            if (CL == 1) {
                if (lane % GROUP == 0) row[threadIdx.x >> 5] = s[0];
                __syncthreads();
            } else {
                const uint32_t at = tc::smem_u32(row + tc::cluster_ctarank() * (32 / CL) + (threadIdx.x >> 5)), bar = bars() + 8 * turn;
                if (threadIdx.x == 0) tc::mbar_expect_tx(bar, CL * (blockDim.x >> 5) * PAD * 4);
                if (lane % GROUP == 0)
#pragma unroll
                    for (int c = 0; c < CL; ++c)
                        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(tc::mapa_shared(at, c)),
                                     "r"(__float_as_uint(s[0])), "r"(tc::mapa_shared(bar, c))
                                     : "memory");
                __syncwarp();
                const tc::Abort ab{flag(), p.hdr, p.timeout_ns, 0xD0u, tc::mapa_shared(tc::smem_u32(flag()), tc::cluster_ctarank() ^ 1u)};
                if (ok) ok = tc::wait_all<true>(bar, (uses >> 1) & 1, ab, 1);
            }
            ++uses;
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

    // No block leaves while another may still write to it.
    __device__ __forceinline__ void leave() const
    {
        if (CL == 1) return;
        __syncthreads();
        tc::cluster_sync_all();
    }
};

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

// What a thread takes of a row: vectors first + i * lanes + id, i < VPT.  GL > 0: blocks of
// several rows, GL lanes each; else a row has the block's threads, or a cluster's (CL > 1).
template <int VPT, int GL, int CL>
struct Share {
    uint32_t lanes, id, group, groups, first;
    __device__ __forceinline__ Share()
        : lanes(GL ? GL : blockDim.x), id(GL ? threadIdx.x % (GL ? GL : 1) : threadIdx.x), group(GL ? threadIdx.x / (GL ? GL : 1) : 0),
          groups(GL ? blockDim.x / (GL ? GL : 1) : 1), first(CL > 1 ? tc::cluster_ctarank() * (VPT * blockDim.x) : 0)
    {
    }
    __device__ __forceinline__ uint32_t vec(int i) const { return first + i * lanes + id; }
};

// The weights of a thread's vectors.  In shared memory (scale_bytes) the first and the last
// four channels of the vectors lie in planes, 16 bytes a lane.
__host__ __device__ __forceinline__ uint32_t scale_bytes(int vpt, uint32_t lanes) { return 64u * vpt * lanes; }

template <int VPT, int GL, int CL, Weights WHERE>
struct Scales {
    f32x2 w[WHERE == IN_REGISTERS ? VPT : 1][4], g[WHERE == IN_REGISTERS ? VPT : 1][4];
    float *plane;
    uint32_t lanes, id;

    // A barrier has to follow.
    __device__ __forceinline__ Scales(const Params &p, float *shared, const Share<VPT, GL, CL> &me) : plane(shared), lanes(me.lanes), id(me.id)
    {
        if (WHERE == IN_SHARED && me.group) return;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t v = me.vec(i), at = i * lanes + id;
            f32x2 a[4] = {}, b[4] = {};
            if (v < p.vecs) {
                scale_of(p, v, a);
                if (p.gpre) ld8f(p.gpre + v * 8, b);
            }
            if (WHERE == IN_SHARED) {
                sts_plane(plane, at, VPT * lanes, a);
                sts_plane(plane + VPT * lanes * 8, at, VPT * lanes, b);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) w[i][k] = a[k], g[i][k] = b[k];
            }
        }
    }
    __device__ __forceinline__ void scale(int i, f32x2 (&f)[4]) const
    {
        if (WHERE == IN_SHARED) lds_plane(plane, i * lanes + id, VPT * lanes, f);
        else
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = w[i][k];
    }
    __device__ __forceinline__ void pre(int i, f32x2 (&f)[4]) const
    {
        if (WHERE == IN_SHARED) lds_plane(plane + VPT * lanes * 8, i * lanes + id, VPT * lanes, f);
        else
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = g[i][k];
    }
};

// Vector v, in column chunk s, of row `row` (t of slot r).
__device__ __forceinline__ char *place(const Rows &o, const Side &d, uint32_t row, uint32_t r, uint32_t t, uint32_t v, uint32_t s)
{
    return (d.cols ? o.at(0, row) : o.at(r, t)) + (size_t)v * 16 + s * d.skip;
}

// ------------------------------------------------------------ forward
// Which norms there are.  Known at compile time: looked up, they cost the gradient spilled
// registers (777 x 1544 without the first norm 12.3 us in the place of 8.6).
enum Kind { NONE = 0, POST = 1, PRE = 2, BOTH = 3 };

template <int VPT, int GL, int MAXT, int MINB, int CL, Weights WHERE, Kind KIND>
__global__ void __launch_bounds__(MAXT, MINB) k_block_norm(const Params p)
{
    extern __shared__ __align__(16) uint8_t sm[];
    constexpr bool post = KIND & POST, pre = KIND & PRE;
    const Share<VPT, GL, CL> me;
    const uint32_t threads = blockDim.x, stage_bytes = 2 * VPT * 16 * threads;
    uint8_t *const after = sm + (GL ? 0 : kAreaBytes);
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(after + (WHERE == IN_SHARED ? scale_bytes(VPT, me.lanes) : 0)) + threadIdx.x * 16;
    const Scales<VPT, GL, CL, WHERE> ws(p, (float *)after, me);
    Sums<GL, CL> total(p, sm);
    uint32_t chunk[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) chunk[i] = me.vec(i) * 8 / p.chunk;
    auto fetch = [&](uint32_t row, int stage) {
        if (GL || row < p.rows) {
            const uint32_t r = p.tokens(row), t = row - r * p.T;
            const char *const rrow = p.res.at(r, t);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const bool on = row < p.rows && me.vec(i) < p.vecs;
                copy<16>(ring + stage * stage_bytes + i * 16 * threads, place(p.y, p.ys, row, r, t, me.vec(i), chunk[i]), on);
                copy<16>(ring + stage * stage_bytes + (VPT + i) * 16 * threads, rrow + me.vec(i) * 16, on);
            }
        }
        copies_done();
    };
    const uint32_t step = gridDim.x / CL * me.groups;   // rows stay below 2^31 - 2^20, and a step below 2^18
    uint32_t row = blockIdx.x / CL * me.groups + me.group, ahead = row;
    for (int s = 0; s < p.stages; ++s, ahead += step) fetch(ahead, s);
    // a warp's lanes take part in its sums as long as one of its rows exists
    for (int stage = 0; row - (GL ? me.group % (32 / (GL ? GL : 32)) : 0) < p.rows; row += step, ahead += step) {
        wait_oldest(p.stages);
        const bool live = !GL || row < p.rows;
        const uint32_t r = p.tokens(row), t = row - r * p.T;
        uint4 yw[VPT], rw[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            yw[i] = lds16(ring + stage * stage_bytes + i * 16 * threads);
            rw[i] = lds16(ring + stage * stage_bytes + (VPT + i) * 16 * threads);
        }
        fetch(ahead, stage);
        stage = stage + 1 == p.stages ? 0 : stage + 1;
        float rp = 1.f;
        if (post) {
            f32x2 ss = 0;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                f32x2 y[4];
                wide8(yw[i], y);
#pragma unroll
                for (int k = 0; k < 4; ++k) ss = fma2(y[k], y[k], ss);
            }
            float sum[1] = {hsum(ss)};
            total(sum);
            rp = rsqrtf(fmaf(sum[0], p.inv_n, p.eps));
        }
        f32x2 h[VPT][4], hh = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t v = me.vec(i);
            const bool on = live && v < p.vecs;
            f32x2 y[4], w[4];
            wide8(yw[i], y);
            wide8(rw[i], h[i]);
            ws.scale(i, w);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                h[i][k] = fma2(w[k], mul2(y[k], both(rp)), h[i][k]);
                hh = fma2(h[i][k], h[i][k], hh);
            }
            if (on) __stcs((uint4 *)(p.h.at(r, t) + v * 16), narrow8(h[i]));
            if (p.y8.q.base) put8(p.y8, r, t, v, on, yw[i]);
            if (p.res8.q.base) put8(p.res8, r, t, v, on, rw[i]);
        }
        if (pre) {
            float sum[1] = {hsum(hh)};
            total(sum);
            const float q = rsqrtf(fmaf(sum[0], p.inv_n, p.eps));
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const uint32_t v = me.vec(i);
                const bool on = live && v < p.vecs;
                f32x2 g[4];
                ws.pre(i, g);
#pragma unroll
                for (int k = 0; k < 4; ++k) h[i][k] = mul2(mul2(h[i][k], both(q)), g[k]);
                const uint4 zw = narrow8(h[i]);
                if (on) __stcs((uint4 *)(p.z.at(r, t) + v * 16), zw);
                if (p.z8.q.base) put8(p.z8, r, t, v, on, on ? zw : make_uint4(0, 0, 0, 0));
            }
        }
        if (CL > 1 && !total.ok) break;
    }
    wait_copies();
    total.leave();
}

// ------------------------------------------------------------ gradient
// A block takes rows j, j + per, ... of one slot (with several rows at a time: runs of
// them).  Its threads keep the sums of their channels over all their rows, and the block
// leaves them in its part, which k_block_sums adds up in block order.
template <int VPT, int GL, int MAXT, int MINB, int CL, bool FULL, bool HELD, Kind KIND>
__global__ void __launch_bounds__(MAXT, MINB) k_block_norm_bwd(const Params p)
{
    extern __shared__ __align__(16) uint8_t sm[];
    constexpr int YB = HELD ? 8 : 16;                   // staged bytes of 8 channels of y and of res
    // sum y^2 from the bytes' exact dot products: 69 -> 67 us (8192 x 4096); rows that do not fill their
    // threads lose by it, for registers (4096 x 7000: 69 -> 75 us)
    constexpr bool SQUARES = HELD && FULL && (KIND & POST);
    constexpr bool post = KIND & POST, pre = KIND & PRE;
    const Share<VPT, GL, CL> me;
    uint8_t *const after = sm + (GL ? 0 : kAreaBytes);
    const uint32_t threads = blockDim.x, in_bytes = VPT * YB * threads, d_bytes = VPT * 16 * threads;
    const uint32_t stage_bytes = 2 * in_bytes + (pre ? 2 : 1) * d_bytes;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(after + scale_bytes(VPT, me.lanes));
    const Scales<VPT, GL, CL, IN_SHARED> ws(p, (float *)after, me);
    if (GL) __syncthreads();
    Sums<GL, CL> total(p, sm);
    const uint32_t block = blockIdx.x / CL, r = block / p.per, step = p.per * me.groups;
    uint32_t chunk[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) chunk[i] = me.vec(i) * 8 / p.chunk;
    auto fetch = [&](uint32_t t, int stage) {
        if (GL || t < p.T) {
            const uint32_t at = ring + stage * stage_bytes + threadIdx.x * YB, dat = ring + stage * stage_bytes + 2 * in_bytes + threadIdx.x * 16;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const uint32_t v = me.vec(i);
                const bool on = FULL || (t < p.T && v < p.vecs);
                if (HELD) {
                    copy<8>(at + i * YB * threads, p.y8.q.at(r, t) + v * 8, on);
                    copy<8>(at + in_bytes + i * YB * threads, p.res8.q.at(r, t) + v * 8, on);
                } else {
                    copy<16>(at + i * YB * threads, place(p.y, p.ys, r * p.T + t, r, t, v, chunk[i]), on);
                    copy<16>(at + in_bytes + i * YB * threads, p.res.at(r, t) + v * 16, on);
                }
                copy<16>(dat + i * 16 * threads, (p.dh.base ? p.dh : p.dres).at(r, t) + v * 16, on && p.dh.base);
                if (pre) copy<16>(dat + d_bytes + i * 16 * threads, place(p.dz, p.dzs, r * p.T + t, r, t, v, chunk[i]), on);
            }
        }
        copies_done();
    };
    uint32_t ey[HELD ? VPT : 1], er[HELD ? VPT : 1];     // the groups' bytes of the next row
    auto fetch_groups = [&](uint32_t t) {
        if (HELD)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const uint32_t v = me.vec(i);
                ey[i] = er[i] = 1;                       // where nothing is: 0 times a number
                if (t >= p.T || (!FULL && v >= p.vecs)) continue;
                ey[i] = __ldcs((const uint8_t *)p.y8.e.at(r, t) + v / 4);
                er[i] = __ldcs((const uint8_t *)p.res8.e.at(r, t) + v / 4);
            }
    };
    f32x2 acc_d[VPT][4] = {}, acc_z[VPT][4] = {};
    uint32_t t = (block - r * p.per) * me.groups + me.group, ahead = t;
    fetch_groups(t);
    for (int s = 0; s < p.stages; ++s, ahead += step) fetch(ahead, s);
    // a warp's lanes take part in its sums as long as one of its rows exists
    for (int stage = 0; t - (GL ? me.group % (32 / (GL ? GL : 32)) : 0) < p.T; t += step, ahead += step) {
        wait_oldest(p.stages);
        const bool live = !GL || t < p.T;
        const uint32_t at = ring + stage * stage_bytes + threadIdx.x * YB, dat = ring + stage * stage_bytes + 2 * in_bytes + threadIdx.x * 16;
        f32x2 y[VPT][4], h[VPT][4];
        uint4 dh[VPT], dz[VPT];
        f32x2 ss = 0;
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (HELD) {
                const uint2 b = lds8(at + i * YB * threads);
                held8(b, ey[i], y[i]);
                if (SQUARES) {
                    const float s = __uint_as_float(ey[i] << 23);
                    sq = fmaf((float)__dp4a((int)b.x, (int)b.x, __dp4a((int)b.y, (int)b.y, 0)) * s, s, sq);
                }
                held8(lds8(at + in_bytes + i * YB * threads), er[i], h[i]);
            } else {
                wide8(lds16(at + i * YB * threads), y[i]);
                wide8(lds16(at + in_bytes + i * YB * threads), h[i]);
            }
            dh[i] = lds16(dat + i * 16 * threads);
            if (pre) dz[i] = lds16(dat + d_bytes + i * 16 * threads);
            if (post && !SQUARES)
#pragma unroll
                for (int k = 0; k < 4; ++k) ss = fma2(y[i][k], y[i][k], ss);
        }
        fetch(ahead, stage);
        fetch_groups(t + step);
        stage = stage + 1 == p.stages ? 0 : stage + 1;
        float rp = 1.f;
        if (post) {
            float sum[1] = {SQUARES ? sq : hsum(ss)};
            total(sum);
            rp = live ? rsqrtf(fmaf(sum[0], p.inv_n, p.eps)) : 0.f;
        }
        f32x2 hh = 0, th = 0, vd = 0, vt = 0, vh = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            f32x2 w[4], g[4], d[4], z[4];
            ws.scale(i, w);
            if (pre) ws.pre(i, g), wide8(dz[i], z);
            if (post) wide8(dh[i], d);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (post) y[i][k] = mul2(y[i][k], both(rp));
                const f32x2 x = mul2(w[k], y[i][k]);
                h[i][k] = add2(h[i][k], x);
                if (post) vd = fma2(x, d[k], vd);
                if (pre) {
                    const f32x2 tt = mul2(z[k], g[k]);
                    hh = fma2(h[i][k], h[i][k], hh);
                    th = fma2(tt, h[i][k], th);
                    if (post) vt = fma2(x, tt, vt), vh = fma2(x, h[i][k], vh);
                }
            }
        }
        float q = 0.f, c = 0.f, m = 0.f;                // d = dh + q t - c h;  dy = rp (d w - yh m)
        if (KIND == BOTH) {
            float s[5] = {hsum(hh), hsum(th), hsum(vd), hsum(vt), hsum(vh)};
            total(s);
            q = live ? rsqrtf(fmaf(s[0], p.inv_n, p.eps)) : 0.f;         // a row that is not there adds zeros
            c = q * (q * (q * (s[1] * p.inv_n)));       // no cube of q by itself: it leaves the range where c does not
            m = (s[2] + q * s[3] - c * s[4]) * p.inv_n;
        } else if (KIND == PRE) {
            float s[2] = {hsum(hh), hsum(th)};
            total(s);
            q = live ? rsqrtf(fmaf(s[0], p.inv_n, p.eps)) : 0.f;
            c = q * (q * (q * (s[1] * p.inv_n)));
        } else if (KIND == POST) {
            float s[1] = {hsum(vd)};
            total(s);
            m = s[0] * p.inv_n;
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t v = me.vec(i);
            f32x2 w[4], g[4], d[4], z[4];
            ws.scale(i, w);
            wide8(dh[i], d);
            if (pre) ws.pre(i, g), wide8(dz[i], z);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (pre) {
                    if (HELD) {                         // one product less: 71 -> 69 us (8192 x 4096); from bf16 72 -> 75
                        z[k] = mul2(z[k], both(q));
                        acc_z[i][k] = fma2(z[k], h[i][k], acc_z[i][k]);
                        d[k] = fma2(z[k], g[k], d[k]);
                    } else {
                        acc_z[i][k] = fma2(z[k], mul2(h[i][k], both(q)), acc_z[i][k]);
                        d[k] = fma2(mul2(z[k], g[k]), both(q), d[k]);
                    }
                    d[k] = fma2(h[i][k], both(-c), d[k]);
                }
                acc_d[i][k] = fma2(d[k], y[i][k], acc_d[i][k]);
                w[k] = mul2(d[k], w[k]);
                if (post) w[k] = mul2(fma2(y[i][k], both(-m), w[k]), both(rp));
            }
            if (!FULL && (!live || v >= p.vecs)) continue;
            __stcs((uint4 *)(p.dres.at(r, t) + v * 16), narrow8(d));
            __stcs((uint4 *)place(p.dy, p.dys, r * p.T + t, r, t, v, chunk[i]), narrow8(w));
        }
        if (CL > 1 && !total.ok) break;
    }
    wait_copies();                                      // before the staging is written otherwise or given up
    total.leave();
    if (!p.sums) return;
    // the sums that are wanted, one after the other; with several rows a block those of all its groups
    float *part = p.part + (size_t)block * p.sums * p.N;
    float *const red = (float *)sm;                     // [group][N]
    if (GL) __syncthreads();                            // the staging is done with, by every warp and every copy
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (k == 0 ? !(p.gpost || p.gate) : !pre) continue;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint32_t v = me.vec(i);
            if (v >= p.vecs) continue;
            const f32x2(&f)[4] = k ? acc_z[i] : acc_d[i];
            float *const to = (GL ? red + me.group * p.N : part) + v * 8;
            ((float4 *)to)[0] = make_float4(lo(f[0]), hi(f[0]), lo(f[1]), hi(f[1]));
            ((float4 *)to)[1] = make_float4(lo(f[2]), hi(f[2]), lo(f[3]), hi(f[3]));
        }
        if (GL) {
            __syncthreads();
            for (uint32_t i = threadIdx.x; i < p.N; i += threads) {
                float s = 0.f;
                for (uint32_t g = 0; g < me.groups; ++g) s += red[g * p.N + i];
                part[i] = s;
            }
            __syncthreads();
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
// How rows are divided.  Up to 512 channels a row has 8, 16 or 32 lanes of a warp, and no
// barrier (240000 rows of 64 took 96 us with a warp each).  Wider rows have a block with two
// vectors of 8 channels a thread: two halve what a row costs besides its channels, the sums
// above all (8192 x 4096 forward with checkpoints 58 us against 67 with one, the gradient 72
// against 100).  Where no SM gets a second row only its latency counts, and one is quicker (8
// rows of 4096 4.1 us against 4.5).  Rows above 8192 channels have a cluster: in the gradient of four blocks,
// so that each SM works on parts of two rows (2048 x 16384: 89 us; 152 with two blocks of twice the
// size); forward of two (68 us with checkpoints).
struct Shape {
    int vpt, gl, cl, threads, stages, rows;   // rows: at once, in the blocks that the GPU holds
    int groups;                               // rows of a block at once
    int sms;
    bool full;                                // every thread has all its vectors
    bool lean;                                // forward: weights in shared memory, so that an SM holds two blocks
                                              // of 257 to 384 threads (6211 x 5064 with checkpoints: 75 -> 62 us)
    size_t smem;
};

static void cluster_of(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&at)[1], const Shape &s, unsigned clusters)
{
    cfg.gridDim = dim3(clusters * s.cl);
    cfg.blockDim = dim3(s.threads);
    cfg.dynamicSmemBytes = s.smem;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = s.cl;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
}

// How many clusters of the gradient's the current device holds at once: fewer than its SMs would,
// because a cluster stays inside one of their groups, and these are not all multiples of it (74
// clusters of four blocks, two an SM, on 152 SMs).  A launch of more would start the last ones when
// the first have ended, and last longer for it (2048 x 16384: 76 clusters 128 us, 74 of them 89).
// The blocks of several slots are rounded down to what the GPU holds for the same reason.
static int clusters_held(const Shape &s, const rc_block_norm_args &a, int fallback)
{
    static std::atomic<int> known[64][8][2][2];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return fallback;
    std::atomic<int> &n = known[dev][s.threads / 32 - 1][a.y8.q.base != nullptr][a.gamma_pre != nullptr];
    int held = n.load(std::memory_order_relaxed);
    if (held) return held;
    const auto kernel = k_block_norm_bwd<2, 0, 256, 2, 4, false, true, BOTH>;      // as any of them
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[1];
    cluster_of(cfg, at, s, (unsigned)fallback);
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&held, kernel, &cfg) != cudaSuccess || held < 1) {
        (void)cudaGetLastError();
        return fallback;
    }
    n.store(held, std::memory_order_relaxed);
    return held;
}

static Shape shape_of(const rc_block_norm_args &a, bool grad, int sms)
{
    const int vecs = a.N / 8;
    Shape s{};
    s.sms = sms;
    s.cl = vecs > 1024 ? (grad ? 4 : 2) : 1;
    s.gl = vecs <= 16 ? 8 : vecs <= 32 ? 16 : vecs <= 64 ? 32 : 0;
    s.vpt = s.gl ? (vecs > 8 ? 2 : 1) : s.cl == 1 && (long long)a.P * a.T <= sms ? 1 : 2;
    s.threads = s.gl ? 128 : ((vecs + s.vpt * s.cl - 1) / (s.vpt * s.cl) + 31) / 32 * 32;
    s.groups = s.gl ? s.threads / s.gl : 1;
    s.full = !s.gl && vecs == s.vpt * s.cl * s.threads;
    // registers: what the launch bounds leave a thread
    s.lean = !grad && !s.gl && s.cl == 1 && s.vpt == 2 && s.threads > 256 && s.threads <= 384;
    const int regs = s.gl ? (grad && s.vpt == 2 ? 168 : 128) : s.vpt == 1 ? 64 : s.lean ? 80 : 128, by_regs = 65536 / (regs * s.threads);
    const bool held = grad && a.y8.q.base;
    const size_t lane = grad ? (held ? 16 : 32) + (a.gamma_pre ? 32 : 16) : 32, stage = lane * s.vpt * s.threads;
    const size_t fixed = (s.gl ? 0 : kAreaBytes) + (grad || s.lean ? scale_bytes(s.vpt, s.gl ? s.gl : s.threads) : 0);
    const size_t room = (size_t)227 * 1024 / by_regs - 1024;
    s.stages = 3;
    while (s.stages > 1 && fixed + s.stages * stage > room) --s.stages;
    s.smem = fixed + s.stages * stage;
    if (grad && s.gl && s.smem < (size_t)s.groups * a.N * 4) s.smem = (size_t)s.groups * a.N * 4;   // the groups' sums
    const int by_smem = (int)(227 * 1024 / (s.smem + 1024)), blocks = by_regs < by_smem ? by_regs : by_smem;
    s.rows = (blocks < 1 ? 1 : blocks) * sms / s.cl * s.groups;
    if (grad && s.cl > 1) s.rows = clusters_held(s, a, s.rows);
    return s;
}

// No more than the GPU holds at once, and no more than end in as many turns, because every block's
// part is written and read again.  For the same reason a block has up to three rows before an SM
// gets another block (777 x 1544 without the first norm: 9 + 6 us with a block for every row or two, 8.4 + 3.7;
// 400 x 4096 10.8 + 4.6, 10.5 + 3.8); rows within a warp, of which a block has several anyway, do not.
static int blocks_of_slot(const rc_block_norm_args &a, const Shape &s)
{
    const int held = s.rows / s.groups / a.P, most = held < 1 ? 1 : held, need = (a.T + s.groups - 1) / s.groups;
    const long long rounds = ((long long)need * a.P * s.cl + s.sms - 1) / s.sms;
    const int least = s.gl || s.vpt == 1 ? 1 : rounds < 3 ? (int)rounds : 3, balanced = (need + most - 1) / most;
    const int turns = balanced > least ? balanced : least;
    return need < 1 ? 1 : (need + turns - 1) / turns;
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
    cudaLaunchAttribute at[1];
    cluster_of(cfg, at, s, blocks);
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, KERNEL, p);
}

template <Kind KIND>
static cudaError_t launch_forward(unsigned n, const Shape &s, const Params &p, cudaStream_t st)
{
    if (s.gl == 8) return s.vpt == 1 ? start<k_block_norm<1, 8, 128, 4, 1, IN_REGISTERS, KIND>>(n, s, p, st) : start<k_block_norm<2, 8, 128, 4, 1, IN_REGISTERS, KIND>>(n, s, p, st);
    if (s.gl == 16) return start<k_block_norm<2, 16, 128, 4, 1, IN_REGISTERS, KIND>>(n, s, p, st);
    if (s.gl) return start<k_block_norm<2, 32, 128, 4, 1, IN_REGISTERS, KIND>>(n, s, p, st);
    if (s.vpt == 1) return start<k_block_norm<1, 0, 1024, 1, 1, IN_REGISTERS, KIND>>(n, s, p, st);
    if (s.cl == 2) return start<k_block_norm<2, 0, 512, 1, 2, IN_REGISTERS, KIND>>(n, s, p, st);
    if (s.lean) return start<k_block_norm<2, 0, 384, 2, 1, IN_SHARED, KIND>>(n, s, p, st);
    return start<k_block_norm<2, 0, 512, 1, 1, IN_REGISTERS, KIND>>(n, s, p, st);
}

template <bool HELD, Kind KIND>
static cudaError_t launch_gradient(unsigned n, const Shape &s, const Params &p, cudaStream_t st)
{
    if (s.gl == 8 && s.vpt == 1) return start<k_block_norm_bwd<1, 8, 128, 4, 1, false, HELD, KIND>>(n, s, p, st);
    if (s.gl == 8) return start<k_block_norm_bwd<2, 8, 128, 3, 1, false, HELD, KIND>>(n, s, p, st);
    if (s.gl == 16) return start<k_block_norm_bwd<2, 16, 128, 3, 1, false, HELD, KIND>>(n, s, p, st);
    if (s.gl) return start<k_block_norm_bwd<2, 32, 128, 3, 1, false, HELD, KIND>>(n, s, p, st);
    if (s.vpt == 1) return start<k_block_norm_bwd<1, 0, 1024, 1, 1, false, HELD, KIND>>(n, s, p, st);
    if (s.cl == 4 && s.full) return start<k_block_norm_bwd<2, 0, 256, 2, 4, true, HELD, KIND>>(n, s, p, st);
    if (s.cl == 4) return start<k_block_norm_bwd<2, 0, 256, 2, 4, false, HELD, KIND>>(n, s, p, st);
    if (s.full) return start<k_block_norm_bwd<2, 0, 512, 1, 1, true, HELD, KIND>>(n, s, p, st);
    return start<k_block_norm_bwd<2, 0, 512, 1, 1, false, HELD, KIND>>(n, s, p, st);
}

template <Kind KIND>
static cudaError_t launch_kind(bool grad, bool held, unsigned n, const Shape &s, const Params &p, cudaStream_t st)
{
    if (!grad) return launch_forward<KIND>(n, s, p, st);
    return held ? launch_gradient<true, KIND>(n, s, p, st) : launch_gradient<false, KIND>(n, s, p, st);
}

static cudaError_t launch(bool grad, bool held, unsigned n, const Shape &s, const Params &p, cudaStream_t st)
{
    const auto go = p.gpre ? (p.gpost ? launch_kind<BOTH> : launch_kind<PRE>) : p.gpost ? launch_kind<POST> : launch_kind<NONE>;
    return go(grad, held, n, s, p, st);
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
    if ((a.y_cols | a.dy_cols | a.dz_cols) & ~1) return set_error(RC_ERR_INVALID, "y_cols, dy_cols and dz_cols are 0 or 1");
    if ((a.y_cols || a.dy_cols || a.dz_cols) && a.N % (8 * a.P)) return set_error(RC_ERR_INVALID, "N=%d channels in P=%d chunks: not multiples of 8", a.N, a.P);
    if (!std::isfinite(a.alpha)) return set_error(RC_ERR_INVALID, "alpha must be finite");
    if (!(a.eps >= 0.f) || !std::isfinite(a.eps)) return set_error(RC_ERR_INVALID, "eps must be finite and not negative");
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
                (a.dz.base && (rc_ = rows(a.dz, "dz", a.dz_cols))) || (rc_ = rows(a.dy, "dy", a.dy_cols)) || (rc_ = rows(a.dres, "dres", false)))
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
        const Operand in[] = {at("dh", a.dh), at("dz", a.dz, a.dz_cols), y, res_, q8("y8.q", a.y8, held), e8("y8.e", a.y8, held), q8("res8.q", a.res8, held),
                              e8("res8.e", a.res8, held), w0, w1, w2};
        const unsigned whole[] = {(a.dy_cols ? 0u : 1u) | (a.dy_cols == a.dz_cols ? 2u : 0u), 1u | (a.dz_cols ? 0u : 2u), 0, 0, 0};
        rc_ = check_apart(out, 5, in, 11, whole);
    }
    if (rc_) return rc_;
    int sms = 0;
    if ((rc_ = device_sms(&sms))) return rc_;
    const Shape s = shape_of(a, grad, sms);
    Params p{};
    uint32_t *unused = nullptr;
    // a caller's workspace has arbitrary contents here, so the library's own header takes what a wait reports
    if (s.cl > 1 && (rc_ = prepare_workspace_ext(nullptr, 0, 0, &p.hdr, &unused, &sms, &p.timeout_ns))) return rc_;
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
    p.chunk = a.y_cols || a.dy_cols || a.dz_cols ? a.N / a.P : a.N;
    auto side = [&](int cols, const rc_rows &o) { return Side{cols != 0, cols ? o.slot - chunk : 0}; };
    p.ys = side(a.y_cols, a.y), p.dys = side(a.dy_cols, a.dy), p.dzs = side(a.dz_cols, a.dz);
    p.stages = s.stages;
    p.alpha = a.alpha;
    p.eps = a.eps;
    p.inv_n = 1.f / (float)a.N;
    unsigned blocks;
    if (!grad) {
        const uint32_t most = (uint32_t)s.rows, all = p.rows < most ? p.rows : most;
        blocks = (all + s.groups - 1) / s.groups;
    } else {
        p.per = blocks_of_slot(a, s);
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
    cudaError_t e = launch(grad, held, blocks, s, p, (cudaStream_t)stream);
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
    return rc::kWsHead + (size_t)blocks_of_slot(*args, s) * args->P * sums_of(*args) * args->N * 4;
}
