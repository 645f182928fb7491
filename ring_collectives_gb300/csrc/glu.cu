// glu.cu -- the gated activation between an MLP's matmuls, h = act(a) b, with 8-bit
// checkpoints of what it reads and writes, and its gradient from either form.
//
// Both activations are x s(c(x)), s the logistic function: c(x) = x, or for the tanh
// form of gelu 2 sqrt(2/pi) (x + 0.044715 x^3), because (1 + tanh y) / 2 = s(2 y).
// So act'(x) = s + x c'(x) s (1 - s).  With e = exp(-|c|) and g = 1 / (1 + e), s and 1 - s
// are g and e g, in the order of c's sign: one exponential and one reciprocal for both, and no
// cancellation.  A c that passes the range is an infinity, whose logistic is 1 or 0; x c'(x), which would
// meet the 0 in a product, is left out there.
//
// Bound by memory: 6 bytes an element forward and 1 + 1/32 more for each checkpoint, 10
// to 13 in the gradient.  Measured on 8 x 8192 x 1792: with two checkpoints 148 us (6.4 TB/s,
// 94 % of the copy rate), the gradient from them with h again 173 us (101 %).  Blocks of 128
// threads, one run of 16 channels each: with 256 threads 165 and 180 us, with 512 220 and 190.
#include <cfloat>

#include "act8.cuh"
#include "heads.h"
#include "internal.h"
#include "ringcoll.h"

namespace rc {
namespace gl {

constexpr int THREADS = 128;

struct Params {
    Rows a, b, h, dh, da, db;        // h.base null: not wanted (gradient)
    Act8 a8, b8, h8;                 // q.base null: not given
    Flat f;
};

constexpr float kRoot = 1.5957691216057308f;     // 2 sqrt(2 / pi)

// s(c), and 1 - s(c) in t.  Both approximations are within two units in the last place (of
// the exponent's, 1.17 |c| more); an exponential below the normal numbers is 0.
__device__ __forceinline__ float logistic(float c, float &t)
{
    float e, g;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fabsf(c) * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(g) : "f"(1.f + e));
    const float l = e * g;
    t = c < 0.f ? g : l;
    return c < 0.f ? l : g;
}

template <int ACT>
__device__ __forceinline__ float arg(float x)
{
    return ACT == RC_GLU_SILU ? x : kRoot * x * fmaf(0.044715f * x, x, 1.f);
}

template <int ACT>
__device__ __forceinline__ float act(float x)
{
    float t;
    return x * logistic(arg<ACT>(x), t);
}

// act(x), and act'(x) in d.
template <int ACT>
__device__ __forceinline__ float act_grad(float x, float &d)
{
    float t;
    const float s = logistic(arg<ACT>(x), t);
    float slope = ACT == RC_GLU_SILU ? x : kRoot * x * fmaf(0.134145f * x, x, 1.f);
    // beyond 64 one of s and t is 0 and the other 1, and any number does; the cube is none from 1.2e13 on
    if (ACT == RC_GLU_GELU && fabsf(x) > 64.f && fabsf(x) <= FLT_MAX) slope = 0.f;
    d = s * fmaf(slope, t, 1.f);
    return x * s;
}

template <int ACT, bool WIDE>
__global__ void __launch_bounds__(THREADS) k_glu(const Params p)
{
    const uint64_t first = (uint64_t)blockIdx.x * THREADS;
    const uint32_t row0 = (uint32_t)(first / p.f.lanes.d), rem0 = (uint32_t)(first - (uint64_t)row0 * p.f.lanes.d);
    const Spot s(p.f, row0, rem0, threadIdx.x);
    uint4 wa[2], wb[2], wh[2];
    get16<WIDE>(p.a, s, wa);
    get16<WIDE>(p.b, s, wb);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        f32x2 a[4], b[4];
        wide8(wa[u], a);
        wide8(wb[u], b);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = mul2(f2(act<ACT>(lo(a[i])), act<ACT>(hi(a[i]))), b[i]);
        wh[u] = narrow8(a);
    }
    set16<WIDE>(p.h, s, wh[0], wh[1]);
    if (p.a8.q.base) set16<WIDE>(p.a8, s, wa);
    if (p.b8.q.base) set16<WIDE>(p.b8, s, wb);
    if (p.h8.q.base) set16<WIDE>(p.h8, s, wh);
}

template <int ACT, bool HELD, bool WIDE>
__global__ void __launch_bounds__(THREADS) k_glu_bwd(const Params p)
{
    const uint64_t first = (uint64_t)blockIdx.x * THREADS;
    const uint32_t row0 = (uint32_t)(first / p.f.lanes.d), rem0 = (uint32_t)(first - (uint64_t)row0 * p.f.lanes.d);
    const Spot s(p.f, row0, rem0, threadIdx.x);
    uint4 wd[2], wa[2], wb[2], wh[2], qa, qb;
    uint32_t ea, eb;
    if (HELD) {
        get16<WIDE>(p.a8, s, qa, ea);
        get16<WIDE>(p.b8, s, qb, eb);
    } else {
        get16<WIDE>(p.a, s, wa);
        get16<WIDE>(p.b, s, wb);
    }
    get16<WIDE>(p.dh, s, wd);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        f32x2 a[4], b[4], d[4], h[4];
        if (HELD) {
            held8(u ? make_uint2(qa.z, qa.w) : make_uint2(qa.x, qa.y), ea, a);
            held8(u ? make_uint2(qb.z, qb.w) : make_uint2(qb.x, qb.y), eb, b);
        } else {
            wide8(wa[u], a);
            wide8(wb[u], b);
        }
        wide8(wd[u], d);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float d0, d1;
            const float f0 = act_grad<ACT>(lo(a[i]), d0), f1 = act_grad<ACT>(hi(a[i]), d1);
            const f32x2 f = f2(f0, f1);
            h[i] = mul2(f, b[i]);
            a[i] = mul2(mul2(d[i], b[i]), f2(d0, d1));
            b[i] = mul2(d[i], f);
        }
        wa[u] = narrow8(a);
        wb[u] = narrow8(b);
        wh[u] = narrow8(h);
    }
    set16<WIDE>(p.da, s, wa[0], wa[1]);
    set16<WIDE>(p.db, s, wb[0], wb[1]);
    if (p.h.base) set16<WIDE>(p.h, s, wh[0], wh[1]);
    if (p.h8.q.base) set16<WIDE>(p.h8, s, wh);
}

template <int ACT, bool WIDE>
static void launch(const Params &p, bool grad, unsigned blocks, cudaStream_t st)
{
    if (!grad) k_glu<ACT, WIDE><<<blocks, THREADS, 0, st>>>(p);
    else if (p.a8.q.base) k_glu_bwd<ACT, true, WIDE><<<blocks, THREADS, 0, st>>>(p);
    else k_glu_bwd<ACT, false, WIDE><<<blocks, THREADS, 0, st>>>(p);
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
    if (grad && !held && b8) return set_error(RC_ERR_INVALID, "b8 goes with a8");
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
    const unsigned blocks = (unsigned)p.f.blocks(THREADS);
    // operands that are not given have null bases, and strides that a caller may leave as they are
    auto wide_if = [](const rc_rows &r, size_t b) { return !r.base || wide_of(r, b); };
    const bool wide = g.N % 16 == 0 && wide_if(g.a, 32) && wide_if(g.b, 32) && wide_if(g.h, 32) && (!grad || (wide_of(g.dh, 32) && wide_of(g.da, 32) && wide_of(g.db, 32))) &&
                      wide_if(g.a8.q, 16) && wide_if(g.b8.q, 16) && wide_if(g.h8.q, 16);
    const auto go = g.act == RC_GLU_SILU ? (wide ? launch<RC_GLU_SILU, true> : launch<RC_GLU_SILU, false>)
                                         : (wide ? launch<RC_GLU_GELU, true> : launch<RC_GLU_GELU, false>);
    go(p, grad, blocks, (cudaStream_t)stream);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return set_error(RC_ERR_CUDA, "glu launch: %s", cudaGetErrorString(err));
    return RC_OK;
}

} // namespace gl
} // namespace rc

extern "C" int glu(const rc_glu_args *args, void *stream) { return rc::gl::run(args, false, stream); }

extern "C" int glu_bwd(const rc_glu_args *args, void *stream) { return rc::gl::run(args, true, stream); }
