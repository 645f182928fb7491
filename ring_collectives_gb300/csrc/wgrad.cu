// wgrad.cu -- the weight gradient of a matmul from an activation held in 8 bits,
// on the 5th-generation tensor cores:
//     dw[n][k] (+)= sum_t dy[t][n] x[t][k],   x = q 2^(e - 127) by groups of 32 k.
//
// x's values are bf16 numbers, so it is widened on the way to the tensor cores and
// nothing is rounded but the sums.  Both operands have the tokens, the dimension that
// is summed over, as their slow one: both are MN-major tiles, 64 channels (128
// swizzled bytes) by 64 tokens a block.
//
// One persistent launch of CTA pairs.  A pair owns a 256 x 256 tile of dw, each CTA
// 128 rows n of it in TMEM, and steps over the tokens by 64:
//   warp 0       copies its 128 n of dy by TMA (tokens and channels past the end
//                arrive as zeros);
//   warps 2, 3   copy 128 k of q ahead (rows on 16 bytes by TMA; rows of an odd number of 8
//                bytes by TMA too, the even ones and the odd ones each; others by cp.async),
//                and the groups' bytes;
//   warps 8-15   widen them into the swizzled tile, groups of four warps taking steps in
//                turn.  A group converts in registers before it waits for a stage, so
//                the stage is held for the stores and the fence only;
//   warp 1       (even CTA) issues the MMAs of the pair, M = N = 256;
//   warps 1, 16-19 (odd CTA) announce its widened steps to the even one;
//   warps 4-7    take finished tiles from TMEM, while the next one is summed.
// Whole tiles are dealt out in rounds; the tokens of those that are left over are
// divided evenly over all pairs, and k_wgrad_join adds the parts in order.
//
// Bound by shared memory, and by what a step's way to the tensor cores takes in all: a step's MMAs last 512
// clocks, in which a CTA's shared memory takes in 16 KB of dy, 8 KB of q and 16 KB of widened x, and gives out
// the q again and 32 KB to the tensor cores, 80 KB or 640 clocks; and of the five stages some three are
// taken by steps that wait for their announcement.  Measured: 8 ranks x 768x4096 over 8192
// tokens 270 + 7 us (412 GFLOP, 1.49 PFLOP/s; the MMAs by themselves take 195 us, with dy's
// copies 219), one rank's 4096x4096 188 + 7 us (1.41 PFLOP/s), 4096x4104 198 + 8 us (rows of an
// odd number of 8 bytes; by cp.async 286 before announcements were releases).  Three groups of widening warps in
// the place of two: 271, 190 and 198 us, and registers spilled in the additions to dw.  Over a few tokens
// the tiles' stores bound it, a row a lane: 8 x 2816x3456 over 4 tokens 37 us (4.2 TB/s), 2736x3448 with every
// other row off whole sectors 43 us (73 with 16-byte stores), in binary32 64 us, added to what is there 186.
#include <cudaTypedefs.h>

#include <mutex>

#include "act8.cuh"
#include "heads.h"
#include "per_device.h"
#include "warp.cuh"

namespace rc {
namespace wg {

using namespace tc;

constexpr int TILE = 256, HALF = 128;         // a pair's tile of dw; a CTA's rows n, and its columns k to widen
constexpr int STEP = 64;                      // tokens a step
constexpr int STAGES = 5;
constexpr int BLOCK = 64 * STEP * 2;          // 64 channels x 64 tokens of bf16
constexpr int OPERAND = 2 * BLOCK;            // a CTA's half of an operand's stage
constexpr int GROUPS = 2, GROUP = 128;        // groups of threads that widen steps in turn
constexpr int DEEP = 6;                       // steps of q on their way or waiting to be widened
constexpr int TOKENS = GROUP / 8;             // a group takes 128 k of as many tokens at a time,
constexpr int PIECES = STEP / TOKENS;         // so often in a step
constexpr int STEP_BYTES = STEP * HALF;
constexpr int ODD_ROW = HALF + 16;            // bytes of an odd row in the slot of a step (TWINS)
constexpr int EVEN_BYTES = STEP / 2 * HALF, SLOT = EVEN_BYTES + STEP / 2 * ODD_ROW;
// How rows of q come: by cp.async, by TMA, or the even and the odd ones each by TMA.  Looked up
// at run time the choice cost 4 % of the whole launch: the widening warps are that busy.
enum Mode { COPIES, ROWS, TWINS };
constexpr int EPILOGUE = 4;                   // warps that store
// Warps that announce the odd CTA's widened steps to the even one, a stage each: warp 1 and those from
// FIRST_HERALD on.  A release at cluster scope takes about 2000 clocks while copies are on their way, so one warp for all
// stages made the whole launch last 720 us in the place of 271, two 340, three 280.  One fence for all steps that are
// ready, before relaxed arrivals, took 373 us with one warp.
constexpr int HERALDS = STAGES;
constexpr int FIRST_HERALD = (256 + GROUPS * GROUP) / 32;
constexpr int THREADS = 256 + GROUPS * GROUP + (HERALDS - 1) * 32;
constexpr int ESLOT = STEP * 4 + 16;          // a step's groups' bytes, and whether its first row is an odd one
constexpr int SLOTS = DEEP * SLOT, ESLOTS = DEEP * ESLOT;
constexpr int TMEM_COLS = 512;                // two accumulators
constexpr int SMEM = STAGES * 2 * OPERAND + SLOTS + ESLOTS + 1024 + 512;
static_assert(SMEM <= 227 * 1024 && TOKENS % 8 == 0, "the stages and slots fit; a thread's tokens share a swizzle");
// A group waits for a slot's or stage's next phase by its parity, so the phase before must be
// known to be over: a slot's last step is the group's own (its copies may end in any order),
// and a stage's last MMAs come before those that the group's last stage was freed by.
static_assert(DEEP % GROUPS == 0 && DEEP % 2 == 0 && STAGES >= GROUPS, "a slot has one loading warp and one group");
constexpr uint32_t kIdesc = idesc_bf16_f32(TILE, TILE) | (1u << 15) | kIdescBMnMajor;   // both MN-major

struct Params {
    Act8 x8;
    Rows dw;
    float *part;                              // [pair][2][64 of four k][256 n][4]
    WsHeader *hdr;
    int P, T, N, K;
    int n_tiles, k_tiles, whole, left;        // tiles dealt out whole; left over
    int pairs, sharers;                       // pairs of the launch; those that share the tiles left over
    uint32_t steps;
    int dy_shared, q_shared, f32, accumulate, st32, clear;
    unsigned long long timeout_ns;
};

// A pair's share of the steps of the tiles left over: [first(i), first(i + 1)), never empty
// for i < sharers.
__device__ __forceinline__ uint64_t first_step(const Params &p, int pair)
{
    const uint64_t all = (uint64_t)p.left * p.steps;
    if (pair >= p.sharers) return all;
    if (all >> 25) return all * (uint32_t)pair / (uint32_t)p.sharers;
    return (uint32_t)all * (uint32_t)pair / (uint32_t)p.sharers;      // fewer than 128 pairs: 32 bits do
}

// What a pair does one after the other: whole tiles, then parts of at most two.
struct Walk {
    int tile, part;                           // part: -1 whole, else its slot (2 pair + i); tile < 0: done
    uint32_t step, end;
    int r, n, k;                              // of the tile: rank, first n and k
    uint64_t at, stop;                        // steps of the tiles left over
    __device__ __forceinline__ void place(const Params &p)
    {
        const int per = p.n_tiles * p.k_tiles, rest = tile % per;
        r = tile / per;
        n = rest / p.k_tiles * TILE;
        k = rest % p.k_tiles * TILE;
    }
    __device__ __forceinline__ void parts(const Params &p)
    {
        if (at >= stop) {
            tile = -1;
            return;
        }
        const uint32_t i = (uint32_t)(at / p.steps);
        step = (uint32_t)(at - (uint64_t)i * p.steps);
        end = (uint32_t)(stop - at < p.steps - step ? step + (stop - at) : p.steps);
        at += end - step;
        tile = p.whole + (int)i;
        ++part;
        place(p);
    }
    __device__ __forceinline__ void start(const Params &p, int pair)
    {
        tile = pair;
        part = -1;
        at = first_step(p, pair);
        stop = first_step(p, pair + 1);
        if (tile < p.whole) step = 0, end = p.steps, place(p);
        else part = 2 * pair - 1, parts(p);
    }
    __device__ __forceinline__ void next_tile(const Params &p, int pair)
    {
        if (part < 0 && tile + p.pairs < p.whole) {
            tile += p.pairs;
            step = 0;
            place(p);
            return;
        }
        if (part < 0) part = 2 * pair - 1;
        parts(p);
    }
    __device__ __forceinline__ void next(const Params &p, int pair)
    {
        if (++step == end) next_tile(p, pair);
    }
};

// Steps of a pair, of all its tiles and parts.
__device__ __forceinline__ uint32_t steps_of(const Params &p, int pair)
{
    uint32_t n = 0;
    Walk w;
    for (w.start(p, pair); w.tile >= 0; w.next_tile(p, pair)) n += w.end - w.step;
    return n;
}

// Descriptors of MN-major tiles in blocks of BLOCK bytes (smem_desc_mn_sw128): a varying low
// word, and this high word.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_mn(uint32_t addr) { return (addr >> 4) | ((uint32_t)(BLOCK >> 4) << 16); }
__device__ __forceinline__ void mma_pair(uint32_t d, uint32_t a, uint32_t b, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "r"(b), "r"(kIdesc), "r"(acc), "r"(kDescHi)
                 : "memory");
}

// Hands back an accumulator: its TMEM loads have completed, and nothing is published.  What another
// CTA reads is announced with mbar_arrive_remote, a release.
__device__ __forceinline__ void arrive_remote_relaxed(uint32_t bar_cluster)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

// Copies 8 bytes of q; for `on` false nothing is read and zeros are written.
__device__ __forceinline__ void copy(uint32_t dst, const void *src, bool on)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(on ? 8 : 0) : "memory");
}

// A row of a tile in units of 16 bytes, as far as it exists; ADD: what is there is added, 32 columns of it on
// their way at once and with those from TMEM.  (Unit by unit 8 x 2816x3456 in binary32 over 4 tokens took
// 432 us in the place of 184; the next 32 as well, while these are stored, 141 there but 337 instead of 132
// us in bf16: a line's store waits for loads of its other half.)  Each way of storing has a loop of its own,
// because few instructions matter: by one loop with all of them the same without ADD took 132 us
// instead of 64, and in bf16 40 instead of 35.
template <bool F32, bool ADD>
__device__ __forceinline__ void store_row(const Params &p, uint32_t from, char *row, int k, bool mine)
{
    constexpr int UNITS = F32 ? 8 : 4, WIDTH = F32 ? 4 : 8;
    uint4 *o = (uint4 *)row + k / WIDTH;
    uint4 old[UNITS] = {};
    auto load = [&](int k, const uint4 *o) {
        if (p.st32 && k + 32 <= p.K) {
#pragma unroll
            for (int u = 0; u < UNITS; u += 2) ld8_ef_if(o + u, mine, old[u], old[u + 1]);
        } else {
#pragma unroll
            for (int u = 0; u < UNITS; ++u)
                if (mine && k + u * WIDTH < p.K) old[u] = __ldcs(o + u);
        }
    };
#pragma unroll 1
    for (int col = 0; col < TILE; col += 32, k += 32, o += UNITS) {
        uint32_t v[32];
        if (ADD) load(k, o);
        tmem_ld32(from + col, v);
        uint4 x[UNITS];
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            f32x2 f[WIDTH / 2];
#pragma unroll
            for (int j = 0; j < WIDTH / 2; ++j) f[j] = f2(__uint_as_float(v[u * WIDTH + 2 * j]), __uint_as_float(v[u * WIDTH + 2 * j + 1]));
            if constexpr (F32) {
                if (ADD) f[0] = add2(f2(__uint_as_float(old[u].x), __uint_as_float(old[u].y)), f[0]);
                if (ADD) f[1] = add2(f2(__uint_as_float(old[u].z), __uint_as_float(old[u].w)), f[1]);
                x[u] = make_uint4(__float_as_uint(lo(f[0])), __float_as_uint(hi(f[0])), __float_as_uint(lo(f[1])), __float_as_uint(hi(f[1])));
            } else {
                f32x2 b[4];
                wide8(old[u], b);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (ADD) f[j] = add2(b[j], f[j]);
                x[u] = narrow8(f);
            }
        }
        if (!mine) continue;
        if (p.st32 && k + 32 <= p.K) {
#pragma unroll
            for (int u = 0; u < UNITS; u += 2) st8<kStEvictFirst>(o + u, x[u], x[u + 1]);
        } else {
#pragma unroll
            for (int u = 0; u < UNITS; ++u)
                if (k + u * WIDTH < p.K) st_v4(o + u, x[u]);
        }
    }
}

// 32 columns of a row of a whole tile in bf16, by whole sectors of 32 bytes.  A row that lies off them (`off`;
// every other one where K is an odd multiple of 8) keeps its last 16 bytes in `carry` for the next 32.
__device__ __forceinline__ void store32_whole(const Params &p, uint4 *o, bool first, const uint32_t (&v)[32], bool off, uint4 &carry)
{
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]), pack_bf16x2(v[8 * i + 4], v[8 * i + 5]),
                          pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
    if (!p.st32) {
        if (off) {
            const uint4 last = w[3];
            if (first) st_v4(o, w[0]);
            w[3] = w[2], w[2] = w[1], w[1] = w[0], w[0] = carry;
            carry = last;
            --o;
        }
        if (!off || !first) st8<kStEvictFirst>(o, w[0], w[1]);
    } else {
        st8<kStEvictFirst>(o, w[0], w[1]);
    }
    st8<kStEvictFirst>(o + 2, w[2], w[3]);
}

template <Mode MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1) k_wgrad(const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap map_q,
                                                                            const __grid_constant__ CUtensorMap map_o, const Params p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *const gbase = smem_raw + (base - raw);
    const uint32_t sA = base, sB = sA + STAGES * OPERAND, sQ = sB + STAGES * OPERAND, sE = sQ + SLOTS, bars = sE + ESLOTS;
    uint8_t *const bars_g = gbase + STAGES * 2 * OPERAND + SLOTS + ESLOTS;
    const uint32_t full_a = bars, full_b = bars + 8 * STAGES, empty = bars + 16 * STAGES, tfull = bars + 24 * STAGES, tempty = tfull + 16,
                   drained = tempty + 16, qfull = drained + 16, qempty = qfull + 8 * DEEP;
    constexpr int WORDS = 24 * STAGES + 48 + 16 * DEEP;
    uint32_t *const tmem_slot = (uint32_t *)(bars_g + WORDS);
    int *const abort_flag = (int *)(bars_g + WORDS + 4);
    static_assert(WORDS + 8 <= 512, "barriers fit behind the slots");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t cta = cluster_ctarank();
    const bool even = cta == 0;
    const int pair = (int)(blockIdx.x >> 1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_a + 8 * s, 1);                 // the even CTA's arm for the bytes of both
            mbar_init(full_b + 8 * s, GROUP / 32 + even);     // the group's warps; in the even CTA also the odd one's announcement
            mbar_init(empty + 8 * s, 1);                  // one commit of the pair's MMAs
        }
        for (int d = 0; d < DEEP; ++d) {
            mbar_init(qfull + 8 * d, MODE == COPIES ? 33 : 2);    // the arm for TMA's bytes or a warp's own copies; the groups' bytes
            mbar_init(qempty + 8 * d, GROUP / 32);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull + 8 * a, 1);
            mbar_init(tempty + 8 * a, 2 * EPILOGUE);
        }
        mbar_init(drained, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&map) : "memory");
        if (MODE != COPIES) asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&map_q) : "memory");
        if (MODE == TWINS) asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&map_o) : "memory");
    }
    __syncthreads();
    cluster_sync_all();
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Abort ab{abort_flag, p.hdr, p.timeout_ns, 0xACu, mapa_shared(smem_u32(abort_flag), cta ^ 1u)};

    if (warp == 0) {
        // ---------------- dy by TMA (both CTAs; the bytes are counted on the even one's barrier)
        const uint32_t full_a_even = mapa_shared(full_a, 0);
        uint32_t stage = 0, phase = 0;
        int steps = 0;
        Walk w;
        for (w.start(p, pair); w.tile >= 0; w.next(p, pair), ++steps) {
            if (!wait_all(empty + 8 * stage, phase ^ 1u, ab, 2)) break;
            if (elect_one()) {
                if (even) mbar_expect_tx(full_a + 8 * stage, 2 * OPERAND);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    tma_load_3d_pair(sA + stage * OPERAND + i * BLOCK, &map, w.n + (int)cta * HALF + 64 * i, (int)(w.step * STEP),
                                     p.dy_shared ? 0 : w.r, full_a_even + 8 * stage);
            }
            if (++stage == STAGES) stage = 0, phase ^= 1u;
        }
        if (even && *(volatile int *)abort_flag)          // no copy of either CTA stays in flight
            for (int s = steps > STAGES ? steps - STAGES : 0; s < steps; ++s) wait_bar(full_a + 8 * (s % STAGES), (uint32_t)(s / STAGES & 1), ab, 9, true);
    } else if (warp == 1 && even) {
        // ---------------- MMAs of the pair (the whole warp, one elected lane issues)
        uint32_t stage = 0, phase = 0;
        int it = 0;
        bool ok = true;
        Walk w;
        for (w.start(p, pair); w.tile >= 0 && ok; ++it, w.next_tile(p, pair)) {
            const uint32_t acc = it & 1, d = tmem + acc * TILE;
            if (!wait_all<true>(tempty + 8 * acc, ((it >> 1) & 1) ^ 1u, ab, 3)) break;
            uint32_t more = 0;                            // 0: the first MMA overwrites the accumulator
            for (uint32_t s = w.step; s < w.end; ++s) {
                if (!wait_all<true>(full_a + 8 * stage, phase, ab, 4, full_b + 8 * stage)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t ad = desc_mn(sA + stage * OPERAND), bd = desc_mn(sB + stage * OPERAND);
#pragma unroll
                    for (int i = 0; i < STEP / 16; ++i) mma_pair(d, ad + 128 * i, bd + 128 * i, i ? 1u : more);   // 16 tokens: 2048 bytes
                    tc_commit_pair_mc(empty + 8 * stage, 3);
                    if (s + 1 == w.end) tc_commit_pair_mc(tfull + 8 * acc, 3);
                }
                more = 1;
                if (++stage == STAGES) stage = 0, phase ^= 1u;
            }
        }
        if (elect_one()) tc_commit_pair_mc(drained, 1);
        wait_bar(drained, 0, ab, 10, true);
    } else if (warp == 1 || warp >= FIRST_HERALD) {
        // ---------------- the odd CTA's widened steps, announced to the even one, whose MMAs read them: one release at
        // cluster scope for the four warps that wrote, after their own arrivals here, so that they never wait for
        // one.  A warp announces every step of its stage, so the stage's phase before is known to be over.
        const uint32_t stage = warp == 1 ? 0u : (uint32_t)(warp - FIRST_HERALD + 1), full_even = mapa_shared(full_b + 8 * stage, 0);
        const uint32_t total = even ? 0u : steps_of(p, pair);
        uint32_t phase = 0;
        for (uint32_t n = stage; n < total; n += STAGES, phase ^= 1u) {
            if (!wait_all(full_b + 8 * stage, phase, ab, 13)) break;
            if (elect_one()) mbar_arrive_remote(full_even);
        }
    } else if (warp == 2 || warp == 3) {
        // ---------------- q and e ahead, a warp every other step.  q by TMA where its rows start on 16 bytes or
        // every other one does; else by cp.async, eight lanes a token's 128 bytes.  The
        // four groups' bytes of two tokens a lane are loaded two steps of the warp ahead, because a byte
        // cannot be copied so.  Past the last token or channel: zeros.
        const int c = lane & 7, t0 = lane >> 3, mine = warp - 2;
        Walk w{}, far{};                                  // the step to copy, and the one whose groups' bytes to load
        auto skip = [&](Walk &x, int n) {
            for (; n && x.tile >= 0; --n) x.next(p, pair);
        };
        uint32_t e[2][2][4] = {};                         // as loaded: nothing waits for them before they are stored
        auto groups = [&](uint32_t (&b)[2][4]) {
            if (far.tile < 0) return;
            const int first = (far.k + (int)cta * HALF) >> 5, all = (p.K + 31) >> 5;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t t = far.step * STEP + lane + 32 * i;
                const bool here = t < (uint32_t)p.T;
                const uint8_t *const at = (const uint8_t *)p.x8.e.at(far.r, t) + first;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    b[i][g] = 1;
                    if (here && first + g < all) b[i][g] = __ldg(at + g);
                }
            }
            skip(far, 2);
        };
        w.start(p, pair);
        skip(w, mine);
        far = w;
        groups(e[0]);
        groups(e[1]);
        uint32_t slot = (uint32_t)mine, phase = 0;
        uint32_t n = (uint32_t)mine;                      // steps of the pair before w
        bool ok = true;
        while (ok && w.tile >= 0) {
#pragma unroll
            for (int turn = 0; turn < 2; ++turn) {
                if (w.tile < 0) break;
                if (!(ok = wait_all(qempty + 8 * slot, phase ^ 1u, ab, 8))) break;
                const uint32_t row = (p.q_shared ? 0u : (uint32_t)w.r * (uint32_t)p.T) + w.step * STEP;   // of all ranks' (TWINS)
                if (MODE != COPIES) {
                    if (elect_one()) {
                        const uint32_t dst = sQ + slot * SLOT, bar = qfull + 8 * slot;
                        const int k = w.k + (int)cta * HALF;
                        if (MODE == ROWS) {
                            mbar_expect_tx(bar, STEP_BYTES);
                            tma_load_3d(dst, &map_q, k, (int)(w.step * STEP), p.q_shared ? 0 : w.r, bar);
                        } else {
                            mbar_expect_tx(bar, SLOT);
                            tma_load_2d(dst, &map_q, k, (int)((row + 1) / 2), bar);
                            tma_load_2d(dst + EVEN_BYTES, &map_o, k, (int)(row / 2), bar);
                        }
                    }
                } else {
                    const int k = w.k + (int)cta * HALF + c * 16;
                    const bool on = k < p.K, more = k + 8 < p.K;
                    const uint32_t dst = sQ + slot * SLOT + t0 * HALF + c * 16;
                    const char *src = p.x8.q.at(w.r, w.step * STEP + t0) + k;
#pragma unroll 4
                    for (int i = 0; i < STEP; i += 4, src += 4 * p.x8.q.row) {
                        const bool here = on && w.step * STEP + t0 + i < (uint32_t)p.T;
                        copy(dst + i * HALF, here ? src : p.x8.q.base, here);
                        copy(dst + i * HALF + 8, here && more ? src + 8 : p.x8.q.base, here && more);
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(qfull + 8 * slot) : "memory");
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(sE + slot * ESLOT + (lane + 32 * i) * 4),
                                 "r"(e[turn][i][0] | e[turn][i][1] << 8 | e[turn][i][2] << 16 | e[turn][i][3] << 24)
                                 : "memory");
                if (MODE == TWINS && lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(sE + slot * ESLOT + STEP * 4), "r"(row & 1u) : "memory");
                arrive_warp(qfull + 8 * slot, lane);
                skip(w, 2);
                groups(e[turn]);
                n += 2;
                slot += 2;
                if (slot >= DEEP) slot -= DEEP, phase ^= 1u;
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");  // no copy stays in flight, also after a wait that ran out
        if (MODE != COPIES && *(volatile int *)abort_flag)
            for (uint32_t i = n > DEEP ? n - DEEP : (uint32_t)mine; i < n; i += 2) wait_bar(qfull + 8 * (i % DEEP), i / DEEP & 1u, ab, 12, true);
    } else if (warp >= 8) {
        // ---------------- q to bf16.  The steps are dealt out to groups of warps in turn.  A thread takes 16 k
        // of every 16th token of a step.  Of a swizzled row of 128 bytes (64 k) a lane writes two 16-byte
        // chunks; lanes 4-7 write the other block's, in the other order: no bank twice.
        const int group = (warp - 8) / (GROUP / 32), j = threadIdx.x & (GROUP - 1), c = j & 7, t0 = j >> 3;
        const uint32_t in = sQ + t0 * HALF + c * 16, ein = sE + t0 * 4 + (c >> 1), out = sB + (c >> 2) * BLOCK + t0 * 128;
        const uint32_t ch = ((c & 3) * 2 + (c >> 2)) ^ (t0 & 7);        // of the first chunk written; the other: ^ 1
        const bool flip = c >= 4;
        const uint32_t total = steps_of(p, pair);         // this group's: group, group + GROUPS, ...
        uint32_t stage = (uint32_t)group, phase = 0, slot = (uint32_t)group, qphase = 0;
        for (uint32_t n = (uint32_t)group; n < total; n += GROUPS) {
            if (!wait_all(qfull + 8 * slot, qphase, ab, 7)) break;
            uint32_t odd = 0;                             // of this thread's rows: its tokens are all even or all odd
            if (MODE == TWINS) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(odd) : "r"(sE + slot * ESLOT + STEP * 4) : "memory");
            odd = (odd ^ t0) & 1u;
            uint4 q[PIECES], x[PIECES][2];
            uint32_t e[PIECES], high = 0;
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                if (MODE != TWINS) {
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(q[i].x), "=r"(q[i].y), "=r"(q[i].z), "=r"(q[i].w)
                                 : "r"(in + slot * SLOT + i * (TOKENS * HALF))
                                 : "memory");
                } else {
                    const uint32_t at = sQ + slot * SLOT + c * 16 + (odd ? EVEN_BYTES + 8 + ((t0 >> 1) + i * (TOKENS / 2)) * ODD_ROW : ((t0 >> 1) + i * (TOKENS / 2)) * HALF);
                    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(q[i].x), "=r"(q[i].y) : "r"(at) : "memory");
                    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(q[i].z), "=r"(q[i].w) : "r"(at + 8) : "memory");
                }
                asm volatile("ld.shared.u8 %0, [%1];" : "=r"(e[i]) : "r"(ein + slot * ESLOT + i * (TOKENS * 4)) : "memory");
                high = max(high, e[i]);
            }
            auto widen = [&](auto held) {
#pragma unroll
                for (int i = 0; i < PIECES; ++i) {
                    f32x2 f[4], g[4];
                    held(flip ? make_uint2(q[i].z, q[i].w) : make_uint2(q[i].x, q[i].y), e[i], f);
                    held(flip ? make_uint2(q[i].x, q[i].y) : make_uint2(q[i].z, q[i].w), e[i], g);
                    x[i][0] = narrow8(f);
                    x[i][1] = narrow8(g);
                }
            };
            if (__any_sync(0xFFFFFFFFu, high > kLowMost)) widen([](const uint2 &w, uint32_t b, f32x2 (&f)[4]) { held8(w, b, f); });
            else widen([](const uint2 &w, uint32_t b, f32x2 (&f)[4]) { held8_low(w, b, f); });
            arrive_warp(qempty + 8 * slot, lane);
            if (!wait_all(empty + 8 * stage, phase ^ 1u, ab, 11)) break;
#pragma unroll
            for (int i = 0; i < PIECES; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(out + stage * OPERAND + i * (TOKENS * 128) + ((ch ^ k) << 4)),
                                 "r"(x[i][k].x), "r"(x[i][k].y), "r"(x[i][k].z), "r"(x[i][k].w)
                                 : "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            arrive_warp(full_b + 8 * stage, lane);
            stage += GROUPS;
            if (stage >= STAGES) stage -= STAGES, phase ^= 1u;
            slot += GROUPS;
            if (slot >= DEEP) slot -= DEEP, qphase ^= 1u;
        }
    } else if (warp >= 4) {
        // ---------------- finished tiles: this CTA's 128 rows, warp 4 + i the TMEM lanes 32 i..
        const int i = warp & 3;
        const uint32_t tempty_even = mapa_shared(tempty, 0);
        int it = 0;
        Walk w;
        for (w.start(p, pair); w.tile >= 0; ++it, w.next_tile(p, pair)) {
            const uint32_t acc = it & 1;
            const int local = (int)cta * HALF + i * 32 + lane, n = w.n + local;
            if (!wait_idle(tfull + 8 * acc, (it >> 1) & 1, ab, 6)) break;
            tc_fence_after();
            const uint32_t from = tmem + ((uint32_t)(i * 32) << 16) + acc * TILE;
            float *const part = w.part < 0 ? nullptr : p.part + ((size_t)w.part * TILE * TILE + local * 4);
            char *const row = p.dw.at(w.r, n);
            if (!part && !p.f32 && !p.accumulate && w.k + TILE <= p.K) {
                const bool off = (uintptr_t)row & 16;
                uint4 *const o = (uint4 *)(row + (size_t)w.k * 2);
                uint4 carry = make_uint4(0, 0, 0, 0);
#pragma unroll 1
                for (int col = 0; col < TILE; col += 32) {
                    uint32_t v[32];
                    tmem_ld32(from + col, v);
                    if (n < p.N) store32_whole(p, o + col / 8, col == 0, v, off, carry);
                }
                if (off && n < p.N) st_v4(o + TILE / 8 - 1, carry);
            } else if (part) {
#pragma unroll 1
                for (int col = 0; col < TILE; col += 32) {
                    uint32_t v[32];
                    tmem_ld32(from + col, v);
#pragma unroll
                    for (int x = 0; x < 8; ++x)           // four columns of 32 rows side by side
                        st_v4(part + (col / 4 + x) * (TILE * 4), make_uint4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]));
                }
            } else if (p.f32) {
                if (p.accumulate) store_row<true, true>(p, from, row, w.k, n < p.N);
                else store_row<true, false>(p, from, row, w.k, n < p.N);
            } else {
                if (p.accumulate) store_row<false, true>(p, from, row, w.k, n < p.N);
                else store_row<false, false>(p, from, row, w.k, n < p.N);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (even) mbar_arrive(tempty + 8 * acc);
                else arrive_remote_relaxed(tempty_even + 8 * acc);
            }
        }
    }

    // no MMA of the pair is in flight and no epilogue still reads TMEM once both CTAs meet
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
}

// Tile y of those left over, 8 columns from 8 x: the sum of its parts in the order of
// their tokens, a row a thread.  CLEAR: in a caller's workspace the parts are zeroed once
// read, because other calls keep signal words there.
template <bool CLEAR>
__global__ void __launch_bounds__(TILE) k_wgrad_join(const Params p)
{
    const int i = blockIdx.y, per = p.n_tiles * p.k_tiles, tile = p.whole + i, rest = tile % per;
    const int n = rest / p.k_tiles * TILE + (int)threadIdx.x, k = rest % p.k_tiles * TILE + (int)blockIdx.x * 8;
    // the sharers whose shares meet the tile's steps [from, to): the first may have begun in the tile
    // before, which is then its part 0 and this tile its part 1
    const uint64_t from = (uint64_t)i * p.steps, to = from + p.steps;
    int first = (int)(from * (uint32_t)p.sharers / ((uint64_t)p.left * p.steps));
    while (first_step(p, first + 1) <= from) ++first;
    while (first_step(p, first) > from) --first;
    int end = first + 1;
    while (end < p.sharers && first_step(p, end) < to) ++end;
    const bool second = first_step(p, first) < from;
    const size_t step = (size_t)2 * TILE * TILE / 4;
    float4 *part = (float4 *)p.part + first * step + (size_t)blockIdx.x * 2 * TILE + threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");     // the parts are written
    float4 *const own = part + (second ? step / 2 : 0);
    float4 s[2] = {own[0], own[TILE]};
    if (CLEAR) own[0] = own[TILE] = make_float4(0.f, 0.f, 0.f, 0.f);
    part += step;
#pragma unroll 8
    for (int j = 0; j < end - first - 1; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 v = part[j * step + h * TILE];
            s[h] = make_float4(s[h].x + v.x, s[h].y + v.y, s[h].z + v.z, s[h].w + v.w);
        }
    if (CLEAR)                                             // in a loop of its own: stores would hold up the loads
        for (int j = 0; j < end - first - 1; ++j) part[j * step] = part[j * step + TILE] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (n >= p.N || k >= p.K) return;
    char *const row = p.dw.at(tile / per, n);
    if (p.f32) {
        float4 *const o = (float4 *)(row + (size_t)k * 4);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (p.accumulate) {
                const float4 old = o[h];
                s[h] = make_float4(old.x + s[h].x, old.y + s[h].y, old.z + s[h].z, old.w + s[h].w);
            }
            o[h] = s[h];
        }
    } else {
        uint4 *const o = (uint4 *)(row + (size_t)k * 2);
        f32x2 f[4] = {f2(s[0].x, s[0].y), f2(s[0].z, s[0].w), f2(s[1].x, s[1].y), f2(s[1].z, s[1].w)};
        if (p.accumulate) {
            f32x2 old[4];
            wide8(*o, old);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = add2(old[j], f[j]);
        }
        *o = narrow8(f);
    }
}

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &qr) == cudaSuccess &&
            qr == cudaDriverEntryPointSuccess)
            fn = (PFN_cuTensorMapEncodeTiled_v12000)f;
    });
    return fn;
}

static int encode(CUtensorMap *map, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, uint32_t rank, const void *base, const cuuint64_t *dims,
                  const cuuint64_t *strides, const cuuint32_t *box)
{
    auto fn = encode_fn();
    if (!fn) return set_error(RC_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(map, type, rank, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return set_error(RC_ERR_INVALID, "tensor map encoding failed (CUresult %d)", (int)r);
    return RC_OK;
}

// [P][T][channels] in boxes of `width` channels x 64 tokens.
static int make_map(CUtensorMap *map, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const rc_rows &o, int P, int T, int channels, uint32_t width)
{
    const bool one = P == 1 || o.slot == 0;
    const cuuint64_t dims[3] = {(cuuint64_t)channels, (cuuint64_t)T, one ? 1u : (cuuint64_t)P};
    const cuuint64_t strides[2] = {(cuuint64_t)o.row, one ? (cuuint64_t)o.row : (cuuint64_t)o.slot};
    const cuuint32_t box[3] = {width, STEP, 1};
    return encode(map, type, swizzle, 3, o.base, dims, strides, box);
}

// Rows of an odd number of 8 bytes, every other of which starts 8 bytes off a boundary of 16:
// the even rows by one map, and the odd ones by another that starts 8 bytes before the first.
static int make_twins(CUtensorMap *even, CUtensorMap *odd, const rc_rows &q, uint64_t rows, int K)
{
    const cuuint64_t stride[1] = {2 * (cuuint64_t)q.row}, de[2] = {(cuuint64_t)K, (rows + 1) / 2}, dodd[2] = {(cuuint64_t)K + 8, rows / 2};
    const cuuint32_t be[2] = {HALF, STEP / 2}, bo[2] = {ODD_ROW, STEP / 2};
    const int rc_ = encode(even, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_NONE, 2, q.base, de, stride, be);
    return rc_ ? rc_ : encode(odd, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_NONE, 2, (const char *)q.base + q.row - 8, dodd, stride, bo);
}

// Tiles that fill whole rounds of the pairs are dealt out whole.  The tokens of the rest are
// divided over all pairs where that saves more steps than parts cost: they are written and
// read again, and joined by a second launch.
constexpr uint32_t kPartSteps = 24;           // steps saved from which on tokens are divided
constexpr uint32_t kShareSteps = 4;           // steps of a share, at least

static void plan(const rc_wgrad_args &a, int sms, Params &p)
{
    p.P = a.P;
    p.T = a.T;
    p.N = a.N;
    p.K = a.K;
    p.n_tiles = (a.N + TILE - 1) / TILE;
    p.k_tiles = (a.K + TILE - 1) / TILE;
    p.steps = ((uint32_t)a.T + STEP - 1) / STEP;
    const int tiles = a.P * p.n_tiles * p.k_tiles;
    p.pairs = sms / 2;
    p.left = tiles % p.pairs;
    const uint64_t saved = (uint64_t)p.steps * (uint32_t)(p.pairs - p.left) / (uint32_t)p.pairs;
    if (p.left && saved < kPartSteps) p.left = 0;
    p.whole = tiles - p.left;
    const uint64_t shares = (uint64_t)p.left * p.steps / kShareSteps;
    p.sharers = p.left ? (int)(shares < (uint64_t)p.left ? (uint64_t)p.left : shares < (uint64_t)p.pairs ? shares : (uint64_t)p.pairs) : 0;
    if (p.whole < p.pairs) p.pairs = p.whole > p.sharers ? p.whole : p.sharers;
}
static size_t part_bytes(const Params &p) { return (size_t)p.sharers * 2 * TILE * TILE * 4; }

template <Mode MODE>
static cudaError_t start(const CUtensorMap &map, const CUtensorMap &map_q, const CUtensorMap &map_o, const Params &p, cudaStream_t st)
{
    static OncePerDevice once;
    const cudaError_t e = once([] { return cudaFuncSetAttribute(k_wgrad<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM); });
    if (e != cudaSuccess) return e;
    k_wgrad<MODE><<<2 * p.pairs, THREADS, SMEM, st>>>(map, map_q, map_o, p);
    return cudaGetLastError();
}

static int check_sizes(const rc_wgrad_args &a)
{
    int rc_ = check_row_sizes(a.P, 0, a.N, 1 << 20);
    if (!rc_) rc_ = check_row_sizes(a.P, 0, a.K, 1 << 20);
    if (rc_) return rc_;
    if (a.T < 0 || a.T >= 0x7FFFFFFF - (1 << 20)) return set_error(RC_ERR_INVALID, "T=%d is not in 0 <= T < 2^31 - 2^20", a.T);
    const long long tiles = (long long)a.P * ((a.N + TILE - 1) / TILE) * ((a.K + TILE - 1) / TILE);
    if (tiles > 1 << 24) return set_error(RC_ERR_INVALID, "%lld tiles of dw are more than 2^24", tiles);
    if (a.dw_type != RC_BF16 && a.dw_type != RC_F32) return set_error(RC_ERR_INVALID, "dw_type is RC_BF16 or RC_F32");
    if (a.accumulate & ~1) return set_error(RC_ERR_INVALID, "accumulate is 0 or 1");
    if (a.reserved[0] || a.reserved[1]) return set_error(RC_ERR_INVALID, "reserved is not 0");
    return RC_OK;
}

static int run(const rc_wgrad_args *args, void *stream)
{
    if (!args) return set_error(RC_ERR_INVALID, "null args");
    rc_wgrad_args a = *args;
    int rc_ = check_sizes(a);
    if (rc_) return rc_;
    const size_t row = (size_t)a.K * (a.dw_type == RC_F32 ? 4 : 2);
    if ((rc_ = check_rows(a.dw, "dw", a.P, a.N, row, 16))) return rc_;
    if ((uintptr_t)a.workspace & 255u) return set_error(RC_ERR_INVALID, "workspace must be 256-byte aligned");
    const cudaStream_t st = (cudaStream_t)stream;
    if (a.T && ((rc_ = check_rows(a.dy, "dy", a.P, a.T, (size_t)a.N * 2, 16, true)) || (rc_ = check_act8(a.x8, "x8", a.P, a.T, a.K, true)))) return rc_;
    const Operand res[] = {rows_at("dw", a.dw, a.P, a.N, row)};
    auto in_of = [&](const char *name, const rc_rows &o, size_t bytes) { return rows_at(name, a.T ? o : rc_rows{}, o.slot ? a.P : 1, a.T, bytes); };
    const Operand in[] = {in_of("dy", a.dy, (size_t)a.N * 2), in_of("x8.q", a.x8.q, (size_t)a.K), in_of("x8.e", a.x8.e, (size_t)(a.K + 31) / 32)};
    if ((rc_ = check_apart(res, 1, in, 3))) return rc_;
    int sms = 0;
    if ((rc_ = device_sms(&sms))) return rc_;
    if (a.T == 0) {
        cudaError_t e = cudaSuccess;
        for (int r = 0; r < a.P && !a.accumulate && e == cudaSuccess; ++r)
            e = cudaMemset2DAsync((char *)a.dw.base + r * a.dw.slot, a.dw.row, 0, row, (size_t)a.N, st);
        return e == cudaSuccess ? RC_OK : set_error(RC_ERR_CUDA, "gemm_wgrad: %s", cudaGetErrorString(e));
    }
    if (sms < 2) return set_error(RC_ERR_UNSUPPORTED, "gemm_wgrad needs two SMs");
    Params p{};
    plan(a, sms, p);
    p.x8 = act8_of(a.x8);
    p.dw = rows_of(a.dw);
    p.dy_shared = a.P == 1 || a.dy.slot == 0;
    p.q_shared = a.P == 1 || a.x8.q.slot == 0;
    const rc_rows &q = a.x8.q;
    const uint64_t rows = p.q_shared ? (uint64_t)a.T : (uint64_t)a.P * a.T;
    Mode mode = COPIES;
    if (!(((uintptr_t)q.base | (a.P > 1 ? q.slot : 0) | q.row) & 15u)) mode = ROWS;
    else if (!((uintptr_t)q.base & 15u) && q.row % 16 == 8 && rows > 1 && rows < 0x7FFFFFFFu && (p.q_shared || q.slot == q.row * (size_t)a.T)) mode = TWINS;
    p.f32 = a.dw_type == RC_F32;
    p.accumulate = a.accumulate;
    p.st32 = !(((uintptr_t)a.dw.base | a.dw.slot | a.dw.row) & 31u);
    const size_t bytes = part_bytes(p);
    uint32_t *unused = nullptr;
    if ((rc_ = prepare_workspace_ext(a.workspace, a.ws_bytes, a.workspace ? (kWsHead - sizeof(WsHeader) + bytes) / 4 : 0, &p.hdr, &unused, &sms,
                                     &p.timeout_ns)))
        return rc_;
    void *space = (char *)a.workspace + kWsHead;
    if (!a.workspace && bytes && (rc_ = prepare_scratch(bytes, &space))) return rc_;
    p.clear = a.workspace != nullptr;
    p.part = (float *)space;
    CUtensorMap map, map_q, map_o;
    if ((rc_ = make_map(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, a.dy, a.P, a.T, a.N, 64))) return rc_;
    map_q = map_o = map;                      // where they are not used
    if (mode == ROWS) rc_ = make_map(&map_q, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_NONE, q, a.P, a.T, a.K, HALF);
    if (mode == TWINS) rc_ = make_twins(&map_q, &map_o, q, rows, a.K);
    if (rc_) return rc_;
    const auto go = mode == ROWS ? start<ROWS> : mode == TWINS ? start<TWINS> : start<COPIES>;
    cudaError_t e = go(map, map_q, map_o, p, st);
    if (e == cudaSuccess && p.left) {
        // set up while the tiles are summed; its blocks start when that has ended
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(TILE / 8, (unsigned)p.left);
        cfg.blockDim = dim3(TILE);
        cfg.stream = st;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        e = p.clear ? cudaLaunchKernelEx(&cfg, k_wgrad_join<true>, p) : cudaLaunchKernelEx(&cfg, k_wgrad_join<false>, p);
    }
    if (e != cudaSuccess) return set_error(RC_ERR_CUDA, "gemm_wgrad launch: %s", cudaGetErrorString(e));
    return RC_OK;
}

} // namespace wg
} // namespace rc

extern "C" int gemm_wgrad(const rc_wgrad_args *args, void *stream) { return rc::wg::run(args, stream); }

extern "C" size_t gemm_wgrad_workspace_bytes(const rc_wgrad_args *args)
{
    using namespace rc::wg;
    int sms = 0;
    if (!args || check_sizes(*args) || rc::device_sms(&sms) || sms < 2) return 0;
    Params p{};
    if (args->T) plan(*args, sms, p);
    return rc::kWsHead + part_bytes(p);
}
