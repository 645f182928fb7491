// glu.cu -- the gated activation between an MLP's matmuls, h = act(a) b, with 8-bit
// checkpoints of what it reads and writes, and its gradient from either form.
//
// Both activations are x s(c(x)), s the logistic function: c(x) = x, or for the tanh
// form of gelu 2 sqrt(2/pi) (x + 0.044715 x^3), because (1 + tanh y) / 2 = s(2 y).
// So act'(x) = s + x c'(x) s (1 - s), with s and 1 - s = s(-c) each from an exponential
// of its own sign: neither loses its small values by cancellation.
//
// Bound by memory: 6 bytes an element forward and up to 5 more for checkpoints, 10
// to 13 in the gradient.
#include "act8.cuh"
#include "heads.h"
#include "internal.h"
#include "ringcoll.h"

namespace rc {
namespace gl {

constexpr int THREADS = 256;

struct Params {
    Rows a, b, h, dh, da, db;        // h.base null: not wanted (gradient)
    Act8 a8, b8, h8;                 // q.base null: not given
    Flat f;
};

// rcp.approx keeps subnormal results, is exact to one unit in the last place, and takes
// an infinity to 0.
__device__ __forceinline__ float rcp(float x)
{
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kRoot = 1.5957691216057308f;     // 2 sqrt(2 / pi)

template <int ACT>
__device__ __forceinline__ float arg(float x)
{
    return ACT == RC_GLU_SILU ? x : kRoot * x * fmaf(0.044715f * x, x, 1.f);
}

template <int ACT>
__device__ __forceinline__ float act(float x)
{
    return x * rcp(1.f + __expf(-arg<ACT>(x)));
}

// act(x), and act'(x) in d.
template <int ACT>
__device__ __forceinline__ float act_grad(float x, float &d)
{
    const float c = arg<ACT>(x), s = rcp(1.f + __expf(-c)), t = rcp(1.f + __expf(c));
    const float slope = ACT == RC_GLU_SILU ? x : kRoot * x * fmaf(0.134145f * x, x, 1.f);
    d = s * fmaf(slope, t, 1.f);
    return x * s;
}

template <int ACT, int U>
__global__ void __launch_bounds__(THREADS) k_glu(const Params p)
{
    const uint64_t first = (uint64_t)blockIdx.x * (THREADS * U);
    const uint32_t row0 = (uint32_t)(first / p.f.lanes.d), rem0 = (uint32_t)(first - (uint64_t)row0 * p.f.lanes.d);
    uint4 wa[U], wb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Spot s(p.f, row0, rem0, u * THREADS + threadIdx.x);
        wa[u] = wb[u] = make_uint4(0, 0, 0, 0);
        if (s.on) {
            wa[u] = __ldcs((const uint4 *)(p.a.at(s.r, s.t) + s.v * 16));
            wb[u] = __ldcs((const uint4 *)(p.b.at(s.r, s.t) + s.v * 16));
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Spot s(p.f, row0, rem0, u * THREADS + threadIdx.x);
        f32x2 a[4], b[4];
        wide8(wa[u], a);
        wide8(wb[u], b);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = mul2(f2(act<ACT>(lo(a[i])), act<ACT>(hi(a[i]))), b[i]);
        const uint4 h = narrow8(a);
        if (s.on) __stcs((uint4 *)(p.h.at(s.r, s.t) + s.v * 16), h);
        if (p.a8.q.base) put8(p.a8, s.r, s.t, s.v, s.on, wa[u]);
        if (p.b8.q.base) put8(p.b8, s.r, s.t, s.v, s.on, wb[u]);
        if (p.h8.q.base) put8(p.h8, s.r, s.t, s.v, s.on, h);
    }
}

template <int ACT, bool HELD, int U>
__global__ void __launch_bounds__(THREADS) k_glu_bwd(const Params p)
{
    const uint64_t first = (uint64_t)blockIdx.x * (THREADS * U);
    const uint32_t row0 = (uint32_t)(first / p.f.lanes.d), rem0 = (uint32_t)(first - (uint64_t)row0 * p.f.lanes.d);
    uint4 wd[U], wa[U], wb[U];
    uint2 qa[U], qb[U];
    uint32_t ea[U], eb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Spot s(p.f, row0, rem0, u * THREADS + threadIdx.x);
        wd[u] = wa[u] = wb[u] = make_uint4(0, 0, 0, 0);
        qa[u] = qb[u] = make_uint2(0, 0);
        ea[u] = eb[u] = 0;
        if (!s.on) continue;
        wd[u] = __ldcs((const uint4 *)(p.dh.at(s.r, s.t) + s.v * 16));
        if (HELD) {
            qa[u] = __ldcs((const uint2 *)(p.a8.q.at(s.r, s.t) + s.v * 8));
            qb[u] = __ldcs((const uint2 *)(p.b8.q.at(s.r, s.t) + s.v * 8));
            ea[u] = *(const uint8_t *)(p.a8.e.at(s.r, s.t) + s.v / 4);
            eb[u] = *(const uint8_t *)(p.b8.e.at(s.r, s.t) + s.v / 4);
        } else {
            wa[u] = __ldcs((const uint4 *)(p.a.at(s.r, s.t) + s.v * 16));
            wb[u] = __ldcs((const uint4 *)(p.b.at(s.r, s.t) + s.v * 16));
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Spot s(p.f, row0, rem0, u * THREADS + threadIdx.x);
        f32x2 a[4], b[4], d[4];
        if (HELD) {
            held8(qa[u], ea[u], a);
            held8(qb[u], eb[u], b);
        } else {
            wide8(wa[u], a);
            wide8(wb[u], b);
        }
        wide8(wd[u], d);
        f32x2 da[4], db[4], h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float d0, d1;
            const float f0 = act_grad<ACT>(lo(a[i]), d0), f1 = act_grad<ACT>(hi(a[i]), d1);
            const f32x2 f = f2(f0, f1);
            h[i] = mul2(f, b[i]);
            db[i] = mul2(d[i], f);
            da[i] = mul2(mul2(d[i], b[i]), f2(d0, d1));
        }
        const uint4 hw = narrow8(h);
        if (s.on) {
            __stcs((uint4 *)(p.da.at(s.r, s.t) + s.v * 16), narrow8(da));
            __stcs((uint4 *)(p.db.at(s.r, s.t) + s.v * 16), narrow8(db));
            if (p.h.base) __stcs((uint4 *)(p.h.at(s.r, s.t) + s.v * 16), hw);
        }
        if (p.h8.q.base) put8(p.h8, s.r, s.t, s.v, s.on, hw);
    }
}

template <int ACT>
static void launch(const Params &p, bool grad, cudaStream_t st)
{
    constexpr int U = 2;
    const unsigned blocks = (unsigned)p.f.blocks(THREADS * U);
    if (!grad) k_glu<ACT, U><<<blocks, THREADS, 0, st>>>(p);
    else if (p.a8.q.base) k_glu_bwd<ACT, true, U><<<blocks, THREADS, 0, st>>>(p);
    else k_glu_bwd<ACT, false, U><<<blocks, THREADS, 0, st>>>(p);
}

static int run(const rc_glu_args *args, bool grad, void *stream)
{
    if (!args) return set_error(RC_ERR_INVALID, "null args");
    rc_glu_args g = *args;
    if (g.reserved[0] || g.reserved[1]) return set_error(RC_ERR_INVALID, "reserved is not 0");
    if (g.act != RC_GLU_SILU && g.act != RC_GLU_GELU) return set_error(RC_ERR_INVALID, "unknown activation %d", g.act);
    int rc_ = check_row_sizes(g.P, g.T, g.N, 1 << 20);
    if (rc_ || g.T == 0) return rc_;
    const size_t bytes = (size_t)g.N * 2, groups = (size_t)(g.N + 31) / 32;
    const bool held = grad && g.a8.q.base, a8 = g.a8.q.base, b8 = g.b8.q.base, h8 = g.h8.q.base;
    auto rows = [&](rc_rows &x, const char *name) { return check_rows(x, name, g.P, g.T, bytes, 16); };
    auto packed = [&](rc_act8 &x, const char *name) { return check_act8(x, name, g.P, g.T, g.N); };
    if ((!held && ((rc_ = rows(g.a, "a")) || (rc_ = rows(g.b, "b")))) ||
        ((held || (!grad && a8)) && (rc_ = packed(g.a8, "a8"))) || ((held || (!grad && b8)) && (rc_ = packed(g.b8, "b8"))) ||
        (h8 && (rc_ = packed(g.h8, "h8"))) || ((!grad || g.h.base) && (rc_ = rows(g.h, "h"))))
        return rc_;
    if (grad && ((rc_ = rows(g.dh, "dh")) || (rc_ = rows(g.da, "da")) || (rc_ = rows(g.db, "db")))) return rc_;
    auto at = [&](const char *name, const rc_rows &x) { return rows_at(name, x, g.P, g.T, bytes); };
    auto q = [&](const char *name, const rc_act8 &x, bool on) { return rows_at(name, on ? x.q : rc_rows{}, g.P, g.T, (size_t)g.N); };
    auto e = [&](const char *name, const rc_act8 &x, bool on) { return rows_at(name, on ? x.e : rc_rows{}, g.P, g.T, groups); };
    if (!grad) {
        const Operand res[] = {at("h", g.h), q("a8.q", g.a8, a8), e("a8.e", g.a8, a8), q("b8.q", g.b8, b8), e("b8.e", g.b8, b8),
                               q("h8.q", g.h8, h8), e("h8.e", g.h8, h8)};
        const Operand in[] = {at("a", g.a), at("b", g.b)};
        const unsigned whole[] = {3, 0, 0, 0, 0, 0, 0};
        rc_ = check_apart(res, 7, in, 2, whole);
    } else {
        const Operand res[] = {at("da", g.da), at("db", g.db), at("h", g.h), q("h8.q", g.h8, h8), e("h8.e", g.h8, h8)};
        const Operand in[] = {at("dh", g.dh), at("a", held ? rc_rows{} : g.a), at("b", held ? rc_rows{} : g.b), q("a8.q", g.a8, held),
                              e("a8.e", g.a8, held), q("b8.q", g.b8, held), e("b8.e", g.b8, held)};
        const unsigned whole[] = {7, 7, 0, 0, 0};
        rc_ = check_apart(res, 5, in, 7, whole);
    }
    if (rc_) return rc_;
    int sms = 0;
    if ((rc_ = device_sms(&sms))) return rc_;
    Params p{rows_of(g.a), rows_of(g.b), rows_of(g.h), rows_of(g.dh), rows_of(g.da), rows_of(g.db), act8_of(g.a8), act8_of(g.b8),
             act8_of(g.h8), Flat::of(g.P, g.T, g.N)};
    if (p.f.blocks(THREADS) > 0x7FFFFFFFull) return set_error(RC_ERR_INVALID, "P*T rows of N=%d channels are too many", g.N);
    if (g.act == RC_GLU_SILU) launch<RC_GLU_SILU>(p, grad, (cudaStream_t)stream);
    else launch<RC_GLU_GELU>(p, grad, (cudaStream_t)stream);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return set_error(RC_ERR_CUDA, "glu launch: %s", cudaGetErrorString(err));
    return RC_OK;
}

} // namespace gl
} // namespace rc

extern "C" int glu(const rc_glu_args *args, void *stream) { return rc::gl::run(args, false, stream); }

extern "C" int glu_bwd(const rc_glu_args *args, void *stream) { return rc::gl::run(args, true, stream); }
