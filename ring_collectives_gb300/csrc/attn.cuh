// attn.cuh -- what the attention kernels share: the arguments of a launch,
// the mapping of work units to packed sequences, TMEM stores, the MMA whose
// A operand lies in TMEM, and the tensor maps of head-strided operands.
//
// Rows.  The G = Hq / Hkv query heads that share a key head are packed with
// the tokens: row r of a 128-row tile is token r / G, head r % G of the
// group.  A tile holds TT = 128 / G whole tokens (G * TT rows; the other rows
// stay masked), so one key tile serves all heads of the group, a single token
// fills G rows, and the gradients of a shared key head sum inside one tile.
#pragma once
#include <cuda.h>
#include <stdint.h>

#include "f32x2.cuh"
#include "internal.h"
#include "ringcoll.h"
#include "warp.cuh"

namespace rc {
namespace attn {

using namespace tc;

constexpr int KT = 128;                    // keys per tile, and rows per query tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Strided {
    char *base;
    size_t slot, token, head;              // bytes
};

struct Params {
    Strided q, out, dout, dq, dk, dv;      // operands that are also accessed without TMA
    const char *v;                         // values, for the non-finite path of the forward pass
    size_t v_slot, v_token, v_head;
    const char *o;                         // forward output (backward)
    size_t o_slot, o_token, o_head;
    float *lse;                            // [P][Tq][Hq], or null (forward)
    float *delta;                          // [P][Tq][Hq] rowsum(dO * O) (backward)
    float *part_o, *part_lse;              // partial results of split sequences
    const int32_t *cu_q, *cu_k, *used_k;
    WsHeader *hdr;
    int P, B, Tq, Tk, Hq, Hkv, G, D, causal;
    int TT;                                // tokens per 128-row tile
    int TPU;                               // query tokens per work unit
    int sms, part_rows, max_units;         // max_units: units that partial results have room for
    int out32;                             // 1: rows of out are whole 32-byte vectors
    int may_split;                         // 1: key ranges may be split (part_o / part_lse are there)
    int clear;                             // 1: partial results are zeroed once read (a caller's workspace)
    float scale;
    unsigned long long timeout_ns;
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w,
                                            uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
                 ::"r"(dst), "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, int u,
                                            uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
                 ::"r"(dst), "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(u), "r"(bar)
                 : "memory");
}

// ------------------------------------------------------------ MMA issue
// An MMA of these shapes runs for 64 clocks, so its issue has to be cheap.  The
// whole MMA warp walks the loops with warp-uniform values (uniform()) and one
// elected lane issues: descriptors then stay in uniform registers.  With all of
// it under one lane's branch, issuing took longer than executing: at 4096
// tokens x 32 heads of 128 the forward pass spent 2300 clocks of issue on each
// tile's 1024 clocks of MMA.
//
// Descriptors (smem_desc_sw128, smem_desc_mn_sw128) as a varying low word -- the
// address in 16-byte units, and the block step of an MN-major tile -- and this high word.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr int BLK = KT * 128;              // a 64-column block of a 128-row tile: 16 KiB
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) { return addr >> 4; }
__device__ __forceinline__ uint32_t desc_mn(uint32_t addr) { return (addr >> 4) | ((uint32_t)(BLK >> 4) << 16); }

__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kDescHi)
                 : "memory");
}

// A in TMEM as packed bf16
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 y, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kDescHi)
                 : "memory");
}

// Head sizes come in three classes, KS steps of 16 columns that the MMAs do: 4
// (D <= 64), 6 (D <= 96) and 8 (D <= 128).  Tiles lie in 64-column blocks, filled
// with zeros past D.  With the steps as a run-time bound every size paid 2 %.
constexpr int tile_cols(int ks) { return ks <= 4 ? 64 : 128; }

// D = A B^T over 16 KS columns, both tiles K-major in shared memory.
template <int KS>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t a, uint32_t b)
{
    constexpr uint32_t id = idesc_bf16_f32(KT, KT);
    const uint32_t ad = desc_k(a), bd = desc_k(b);
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
        const uint32_t off = (kk >> 2) * (BLK >> 4) + 2 * (kk & 3);
        mma_ss(d, ad + off, bd + off, id, kk != 0);
    }
}

// D (+)= A B over the 128 rows of B, its first 16 KS columns; A in TMEM, the second
// 64 of its columns (of bf16) `half` TMEM columns from the first.
template <int KS>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b, bool first, int half)
{
    constexpr uint32_t id = idesc_bf16_f32(KT, 16 * KS) | kIdescBMnMajor;
    const uint32_t bd = desc_mn(b);
#pragma unroll
    for (int kk = 0; kk < KT / 16; ++kk)
        mma_ts(d, a + (kk >> 2) * half + (kk & 3) * 8, bd + 128 * kk, id, kk ? 1u : (first ? 0u : 1u));
}

// Stores 16 / 32 columns of this thread's TMEM lane; tmem_wait_st() ends them.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *v)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                 "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
                 ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                 "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
                 "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
                 "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
                 : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The larger of three; NaN only when all are.
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    return pack_bf16x2(__float_as_uint(lo), __float_as_uint(hi));
}

// 128 threads of a warpgroup (named barrier 1 + wg).
__device__ __forceinline__ void wg_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

// ------------------------------------------------------------ sequences
// Offsets and lengths come from device memory and are clamped to the
// tensors, so no value of theirs reaches outside an operand.
struct Seq {
    int q0, ql, k0, kl;
};

__device__ __forceinline__ Seq seq_of(const Params &p, int b)
{
    Seq s;
    const int qa = min(max(__ldg(p.cu_q + b), 0), p.Tq), qb = min(max(__ldg(p.cu_q + b + 1), qa), p.Tq);
    const int ka = min(max(__ldg(p.cu_k + b), 0), p.Tk), kb = min(max(__ldg(p.cu_k + b + 1), ka), p.Tk);
    s.q0 = qa;
    s.ql = qb - qa;
    s.k0 = ka;
    s.kl = kb - ka;
    if (p.used_k) s.kl = min(max(__ldg(p.used_k + b), 0), s.kl);
    return s;
}

// Keys that query token i of the sequence sees (possibly none).  The causal
// mask is aligned to the end: the last query sees every key.
__device__ __forceinline__ int seen(const Params &p, const Seq &s, int i)
{
    if (!p.causal) return s.kl;
    return min(max(i + 1 + (s.kl - s.ql), 0), s.kl);
}

__device__ __forceinline__ int warp_incl_scan(int v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Finds the sequence that holds item x when sequence b holds count(b) items;
// every lane of the warp gets (b, x - items before b).
template <class F>
__device__ __forceinline__ void locate(int B, int x, int lane, F count, int &b_out, int &local)
{
    int before = 0;
    b_out = B - 1;
    local = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
        const int b = b0 + lane;
        const int n = b < B ? count(b) : 0;
        const int inc = warp_incl_scan(n, lane);
        const int total = __shfl_sync(0xFFFFFFFFu, inc, 31);
        if (x < before + total) {
            const unsigned hit = __ballot_sync(0xFFFFFFFFu, x < before + inc);
            const int l = __ffs(hit) - 1;
            b_out = b0 + l;
            local = x - before - __shfl_sync(0xFFFFFFFFu, inc - n, l);
            return;
        }
        before += total;
    }
}

__device__ __forceinline__ long long warp_sum(long long v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

constexpr int kNoSplit = 1 << 28;          // key tiles of a part when keys are not split

// Key ranges up to this many tiles are never split.  Measured in graphs, 8 heads,
// split / whole: a token on 8 tiles 16.0 / 13.9 us, on 12 tiles 16.0 / 16.7 us; 64
// tokens on 8 tiles 21.6 / 20.1, on 12 tiles 21.5 / 25.4 us; and the join's launch is
// about 4 us of host time.  (Asked on the host of what the tensors could hold and
// on the device of what they hold, so the room in a cache changes no result.)
constexpr int kWholeTiles = 10;

// Units that a split adds at most: parts are no smaller than 4 rounds of units need.
constexpr long long split_units(int sms) { return 4ll * sms; }

// Units go to blocks as they come free: block i starts with unit i and takes
// the next one from a counter.  Two words of the status header that nothing
// else uses hold the counter and the blocks that are done; the last block
// clears both, also in a launch that gave up (every block reaches its end).
// Which block runs a unit changes no result.  SET: the words of this kernel
// (the dK/dV launch may begin before the dQ launch has quite ended).
template <int SET>
__device__ __forceinline__ int claim_unit(const Params &p, int lane)
{
    int u = 0;
    if (lane == 0) u = (int)(gridDim.x + atomicAdd(&p.hdr->pad[2 + 2 * SET], 1u));
    return __shfl_sync(0xFFFFFFFFu, u, 0);
}

template <int SET>
__device__ __forceinline__ void units_done(const Params &p)
{
    __threadfence();
    if (atomicAdd(&p.hdr->pad[3 + 2 * SET], 1u) == gridDim.x - 1) {
        atomicExch(&p.hdr->pad[2 + 2 * SET], 0u);
        atomicExch(&p.hdr->pad[3 + 2 * SET], 0u);
    }
}

// Host helpers (attn_api.cu).
int head_map5(CUtensorMap *map, const rc_heads &h, int P, int T, int Hkv, int G, int D, int box_tokens);
int head_map4(CUtensorMap *map, const rc_heads &h, int P, int T, int Hkv, int D);
cudaError_t launch_attn_fwd(const Params &p, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                            bool split, cudaStream_t st);
cudaError_t launch_attn_bwd(const Params &p, const CUtensorMap &mq, const CUtensorMap &mdo, const CUtensorMap &mk,
                            const CUtensorMap &mv, cudaStream_t st);

} // namespace attn
} // namespace rc
