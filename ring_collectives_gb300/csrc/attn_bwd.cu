// attn_bwd.cu -- gradients of attention over packed sequences, on the
// 5th-generation tensor cores.  With p_ij = exp(s_ij - lse_i) recomputed from
// the forward pass's log-sums and delta_i = dO_i . O_i:
//   dV_j = sum_i p_ij dO_i,   dS_ij = p_ij (dO_i . V_j - delta_i),
//   dQ_i = scale sum_j dS_ij K_j,   dK_j = scale sum_i dS_ij Q_i.
//
// One kernel in two forms, launched one after the other, each owning its
// outputs: k_attn_bwd<., false> (dQ) keeps 128 query rows and runs over the key
// tiles; k_attn_bwd<., true> (dK, dV) keeps 128 keys and runs over the query
// row tiles of all heads of the group, so the gradients of a shared key head
// add up in one accumulator.  Recomputing S and dO V^T in both costs 7 instead
// of 5 products per tile pair; in exchange no sum crosses blocks: no atomics,
// no binary32 dQ in memory, and results that do not depend on timing.
//
// Blocks of 12 warps, one per SM: warps 0-7 do the elementwise work (two
// warpgroups, 64 columns of a 128x128 tile each, a thread a row), warp 8 the
// units and TMA loads, warp 9 the MMAs, and for dK and dV warps 10-11 bring
// the row statistics.  P and dS are rounded to bf16 -- the tensor cores'
// input type -- and written to TMEM over the scores they came from, where they
// are the A operands of the second products; all sums are binary32.  delta takes
// the output as the forward pass left it, in bf16 (nothing else is kept), and sums
// in binary32.  exp2 takes weights below 2^-126 for 0.  All of it together leaves
// the gradients off by 1.3 times what bf16 in and out costs anyway.
//
// Bounds: tensor cores, 3 products a tile pair for dQ and 4 for dK and dV.  8192
// tokens, 32 heads of 128: dQ 559 us, 1474 TFLOP/s; dK and dV 653 us, 1685
// TFLOP/s.  dQ is further from the peak; giving its products more buffers or its
// warpgroups separate halves of a tile made it no faster.  Units of dK and dV are
// not divided, so with few key heads a few blocks work and the rest idle: 4096
// tokens, 8 heads of 128 on 1 key head (32 units), 412 us for the whole gradient,
// whose 5 products would be 46 us at the measured peak.  The two-kernel form was
// taken for its fixed order of sums; 8192 tokens at the peak would be 742 us.
#include "attn.cuh"
#include "per_device.h"

namespace rc {
namespace attn {

constexpr int BWD_THREADS = 384;
constexpr int BUNITS = 4;

struct BUnit {
    Seq s;
    int hk, slot;
    int first;      // dq: first query token of the tile; dkv: first key
    int count;      // dq: valid tokens; dkv: valid keys
    int from, n;    // first inner tile and their number
    int index;      // -1: no more units
};

// dq: one unit per 128-row query tile, the ones that see most keys first.
// dkv: one unit per key tile in order, so those seen by most queries first.
template <bool DKV>
__device__ __forceinline__ int bunits(const Params &p, const Seq &s)
{
    return DKV ? (s.kl + KT - 1) / KT : (s.ql + p.TT - 1) / p.TT;
}

template <bool DKV>
__device__ int bunits_total(const Params &p, int lane)
{
    long long n = 0;
    for (int b = lane; b < p.B; b += 32) n += bunits<DKV>(p, seq_of(p, b));
    return (int)warp_sum(n);
}

template <bool DKV>
__device__ BUnit bunit_of(const Params &p, int u, int lane)
{
    BUnit w;
    const int HP = p.P * p.Hkv, hp = u % HP;
    w.index = u;
    w.hk = hp % p.Hkv;
    w.slot = hp / p.Hkv;
    int b, local;
    locate(p.B, u / HP, lane, [&](int bb) { return bunits<DKV>(p, seq_of(p, bb)); }, b, local);
    w.s = seq_of(p, b);
    if (DKV) {
        w.first = local * KT;
        w.count = min(KT, w.s.kl - w.first);
        // the first query token that sees key `first`
        const int i0 = p.causal ? max(0, w.first - (w.s.kl - w.s.ql)) : 0;
        w.from = min(i0, w.s.ql) / p.TT;
        w.n = i0 < w.s.ql ? (w.s.ql + p.TT - 1) / p.TT - w.from : 0;
    } else {
        w.first = (bunits<false>(p, w.s) - 1 - local) * p.TT;
        w.count = min(p.TT, w.s.ql - w.first);
        w.from = 0;
        w.n = (seen(p, w.s, w.first + w.count - 1) + KT - 1) / KT;
    }
    return w;
}

// One 64-column block after another of a 128-row tile.
template <int DP>
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap *map, int token, int hk, int slot, uint32_t bar)
{
    for (int d = 0; d < DP / 64; ++d) tma_load_5d(dst + d * BLK, map, d * 64, 0, token, hk, slot, bar);
}

template <int DP>
__device__ __forceinline__ void load_keys(uint32_t dst, const CUtensorMap *map, int token, int hk, int slot, uint32_t bar)
{
    for (int d = 0; d < DP / 64; ++d) tma_load_4d(dst + d * BLK, map, d * 64, token, hk, slot, bar);
}

// Clears rows [r0, 128) of a tile of DP columns; `tid` of `n` threads.
template <int DP>
__device__ __forceinline__ void clear_rows(uint8_t *tile, int r0, int tid, int n)
{
    for (int i = tid; i < (KT - r0) * 8 * (DP / 64); i += n) {
        const int blk = i / ((KT - r0) * 8), k = i % ((KT - r0) * 8);
        *(uint4 *)(tile + blk * BLK + r0 * 128 + k * 16) = make_uint4(0, 0, 0, 0);
    }
}

__device__ __forceinline__ void fence_smem_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 64 accumulator columns of this thread's row, times f, as bf16 at dst (columns
// [c0, c0 + 64) of a head of D).
__device__ __forceinline__ void store_acc(uint32_t t, char *dst, int c0, int D, float f, bool valid, bool zero)
{
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        uint32_t o[32];
        if (!zero) {
            tmem_ld32(t + q * 32, o);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
        if (!valid) continue;
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            const int c = c0 + q * 32 + i;
            if (c < D)
                st_v4(dst + c * 2, make_uint4(pack2(__uint_as_float(o[i]) * f, __uint_as_float(o[i + 1]) * f),
                                              pack2(__uint_as_float(o[i + 2]) * f, __uint_as_float(o[i + 3]) * f),
                                              pack2(__uint_as_float(o[i + 4]) * f, __uint_as_float(o[i + 5]) * f),
                                              pack2(__uint_as_float(o[i + 6]) * f, __uint_as_float(o[i + 7]) * f)));
        }
    }
}

// Shared-memory plan.  Two resident tiles (dq: Q, dO; dkv: K, V), a ring of
// NA tiles (dq: K; dkv: Q) and one of NB tiles (dq: V; dkv: dO).  The first
// ring is deeper because its tiles serve two products an iteration apart.
template <int DP>
struct BwdCfg {
    static constexpr int TILE = KT * DP * 2;
    static constexpr int NA = 3, NB = 2;
    static constexpr int CTL = 3072;      // with 32 KiB tiles exactly the 227 KiB of a block
    static constexpr int SMEM = (2 + NA + NB) * TILE + CTL;
};

// Barriers of both kernels, in the control area.
struct Bars {
    uint32_t res_full, res_empty, a_full, a_empty, b_full, b_empty, s_full, dp_full, p_ready, ds_ready, acc_full,
        stat_full, stat_empty, u_full, u_empty, drain;
};

template <int NA, int NB>
__device__ __forceinline__ Bars bars_at(uint32_t x)
{
    Bars b;
    b.res_full = x;
    b.res_empty = x + 8;
    b.a_full = x + 16;
    b.a_empty = b.a_full + 8 * NA;
    b.b_full = b.a_empty + 8 * NA;
    b.b_empty = b.b_full + 8 * NB;
    b.s_full = b.b_empty + 8 * NB;      // two
    b.dp_full = b.s_full + 16;
    b.p_ready = b.dp_full + 8;
    b.ds_ready = b.p_ready + 8;
    b.acc_full = b.ds_ready + 8;
    b.stat_full = b.acc_full + 8;       // two
    b.stat_empty = b.stat_full + 16;    // two
    b.u_full = b.stat_empty + 16;
    b.u_empty = b.u_full + 8 * BUNITS;
    b.drain = b.u_empty + 8 * BUNITS;
    return b;
}

template <int KS, bool DKV>
__global__ void __launch_bounds__(BWD_THREADS, 1)
    k_attn_bwd(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_do,
               const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const Params p)
{
    constexpr int DP = tile_cols(KS);
    using C = BwdCfg<DP>;
    constexpr int TILE = C::TILE, NA = C::NA, NB = C::NB;
    constexpr int READERS = DKV ? 11 : 9;     // warps that release a unit
    extern __shared__ __align__(1024) uint8_t gbase[];   // swizzled tiles start on 1024 bytes
    const uint32_t base = smem_u32(gbase);
    const uint32_t sR0 = base, sR1 = base + TILE, sA = base + 2 * TILE, sB = sA + NA * TILE;
    uint8_t *const gA = gbase + 2 * TILE, *const gB = gA + NA * TILE;
    uint8_t *const ctl = gB + NB * TILE;
    const Bars bar = bars_at<NA, NB>(smem_u32(ctl));
    BUnit *const units = (BUnit *)(ctl + 512);
    uint32_t *const tmem_slot = (uint32_t *)(ctl + 1000);
    int *const abort_flag = (int *)(ctl + 1004);
    float *const stats = (float *)(ctl + 1024);       // dkv: [2 stages][-lse log2 e, -delta][128 rows]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(bar.res_full, 1);
        mbar_init(bar.res_empty, 1);
        for (int s = 0; s < NA; ++s) mbar_init(bar.a_full + 8 * s, 1), mbar_init(bar.a_empty + 8 * s, 1);
        for (int s = 0; s < NB; ++s) mbar_init(bar.b_full + 8 * s, 1), mbar_init(bar.b_empty + 8 * s, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar.s_full + 8 * s, 1);
            mbar_init(bar.stat_full + 8 * s, 2);
            mbar_init(bar.stat_empty + 8 * s, 8);
        }
        mbar_init(bar.dp_full, 1);
        mbar_init(bar.p_ready, 8);
        mbar_init(bar.ds_ready, 8);
        mbar_init(bar.acc_full, 1);
        for (int i = 0; i < BUNITS; ++i) mbar_init(bar.u_full + 8 * i, 1), mbar_init(bar.u_empty + 8 * i, READERS);
        mbar_init(bar.drain, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&map_q) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&map_do) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&map_k) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&map_v) : "memory");
    }
    // Rows past G * TT are never loaded; as rows of a B operand they must be finite.
    if (DKV && p.G * p.TT < KT)
        for (int s = 0; s < NA + NB; ++s) clear_rows<DP>(gA + s * TILE, p.G * p.TT, threadIdx.x, BWD_THREADS);
    fence_smem_async();
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // dq:  S buffers 0 and 128, dP 256, dQ 384.  dkv: dV 0, dK 128, S 256, dP 384.
    const Abort ab{abort_flag, p.hdr, p.timeout_ns, DKV ? 0xB3u : 0xB2u, 0};

    auto next_unit = [&](uint32_t it) -> const BUnit * {
        if (!wait_all(bar.u_full + 8 * (it % BUNITS), (it / BUNITS) & 1, ab, 12)) return nullptr;
        const BUnit *w = units + it % BUNITS;
        return w->index < 0 ? nullptr : w;
    };
    auto release_unit = [&](uint32_t it) {
        arrive_warp(bar.u_empty + 8 * (it % BUNITS), lane);
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 8) {
            // ---------------- units and TMA loads (the whole warp, one elected lane issues)
            const int total = bunits_total<DKV>(p, lane) * p.P * p.Hkv;
            const uint32_t rows = (uint32_t)(p.G * p.TT) * 128u * (DP / 64);
            uint32_t ea = 0, eb = 0, nr = 0, it = 0;
            bool ok = true;
            BUnit next;
            // Makes unit u (or the end of all units) the block's next one.
            auto publish = [&](int u) {
                if (u < total) next = bunit_of<DKV>(p, u, lane);
                else next.index = -1;
                if (!(ok = wait_all(bar.u_empty + 8 * (it % BUNITS), ((it / BUNITS) & 1) ^ 1u, ab, 13))) return;
                if (lane == 0) {
                    units[it % BUNITS] = next;
                    mbar_arrive(bar.u_full + 8 * (it % BUNITS));
                }
                __syncwarp();
                ++it;
            };
            publish(blockIdx.x);
            while (ok && next.index >= 0) {
                const BUnit w = next;
                if (w.n > 0) {
                    if (!(ok = wait_all(bar.res_empty, (nr & 1) ^ 1u, ab, 1))) break;
                    if (elect_one()) {
                        mbar_expect_tx(bar.res_full, DKV ? 2 * TILE : 2 * rows);
                        if (DKV) {
                            load_keys<DP>(sR0, &map_k, w.s.k0 + w.first, w.hk, w.slot, bar.res_full);
                            load_keys<DP>(sR1, &map_v, w.s.k0 + w.first, w.hk, w.slot, bar.res_full);
                        } else {
                            load_rows<DP>(sR0, &map_q, w.s.q0 + w.first, w.hk, w.slot, bar.res_full);
                            load_rows<DP>(sR1, &map_do, w.s.q0 + w.first, w.hk, w.slot, bar.res_full);
                        }
                    }
                    ++nr;
                }
                for (int j = 0; j < w.n && ok; ++j) {
                    // the next unit is worked out once this one has two tiles to go on with
                    if (j == 2) publish(claim_unit<DKV ? 1 : 0>(p, lane));
                    const uint32_t st = ea % NA, su = eb % NB;
                    const int at = DKV ? w.s.q0 + (w.from + j) * p.TT : w.s.k0 + j * KT;
                    if (!ok || !(ok = wait_all(bar.a_empty + 8 * st, ((ea / NA) & 1) ^ 1u, ab, 2))) break;
                    if (elect_one()) {
                        mbar_expect_tx(bar.a_full + 8 * st, DKV ? rows : TILE);
                        if (DKV) load_rows<DP>(sA + st * TILE, &map_q, at, w.hk, w.slot, bar.a_full + 8 * st);
                        else load_keys<DP>(sA + st * TILE, &map_k, at, w.hk, w.slot, bar.a_full + 8 * st);
                    }
                    ++ea;
                    if (!(ok = wait_all(bar.b_empty + 8 * su, ((eb / NB) & 1) ^ 1u, ab, 2))) break;
                    if (elect_one()) {
                        mbar_expect_tx(bar.b_full + 8 * su, DKV ? rows : TILE);
                        if (DKV) load_rows<DP>(sB + su * TILE, &map_do, at, w.hk, w.slot, bar.b_full + 8 * su);
                        else load_keys<DP>(sB + su * TILE, &map_v, at, w.hk, w.slot, bar.b_full + 8 * su);
                    }
                    ++eb;
                }
                if (ok && w.n <= 2) publish(claim_unit<DKV ? 1 : 0>(p, lane));
            }
            if (lane == 0) units_done<DKV ? 1 : 0>(p);
            if (lane == 0 && *(volatile int *)abort_flag) {
                // let the copies in flight land before the block gives up its shared memory
                for (uint32_t s = 0; s < NA; ++s)
                    if (ea > s) wait_bar(bar.a_full + 8 * s, ((ea - 1 - s) / NA) & 1, ab, 9, true);
                for (uint32_t s = 0; s < NB; ++s)
                    if (eb > s) wait_bar(bar.b_full + 8 * s, ((eb - 1 - s) / NB) & 1, ab, 9, true);
                if (nr) wait_bar(bar.res_full, (nr - 1) & 1, ab, 9, true);
            }
            __syncwarp();
        } else if (warp == 9) {
            // ---------------- MMA issuer (the whole warp, one elected lane issues)
            uint32_t sa = 0, pa = 0, sb = 0, pb = 0;     // ring positions: stage and phase
            uint32_t nr = 0, nt = 0;                     // nt: tiles done, the phase of p_ready and ds_ready
            bool ok = true;
            const uint32_t tm = (uint32_t)uniform((int)tmem);
            const BUnit *wp;
            auto commit = [&](uint32_t b) {
                if (elect_one()) tc_commit(b);
            };
            // Scores of tile A (first ring) or B (second ring) against a resident tile.
            auto scores_a = [&](uint32_t d, uint32_t full) {
                if (!wait_all(bar.a_full + 8 * sa, pa, ab, 4)) return false;
                tc_fence_after();
                if (elect_one()) {
                    mma_scores<KS>(d, sR0, sA + sa * TILE);
                    tc_commit(full);
                }
                if (++sa == NA) sa = 0, pa ^= 1u;
                return true;
            };
            auto scores_b = [&](uint32_t d) {
                if (!wait_all(bar.b_full + 8 * sb, pb, ab, 5)) return false;
                tc_fence_after();
                if (elect_one()) {
                    mma_scores<KS>(d, sR1, sB + sb * TILE);
                    tc_commit(bar.dp_full);
                    if (!DKV) tc_commit(bar.b_empty + 8 * sb);
                }
                if (++sb == NB) sb = 0, pb ^= 1u;
                return true;
            };
            uint32_t ra = 0, rb = 0;                     // stages of the tile whose second products come next
            auto rows_a = [&](uint32_t d, uint32_t a, bool first) {
                tc_fence_after();
                if (elect_one()) {
                    mma_rows<KS>(d, a, sA + ra * TILE, first, 64);
                    tc_commit(bar.a_empty + 8 * ra);
                }
                if (++ra == NA) ra = 0;
            };
            for (uint32_t it = 0; ok && (wp = next_unit(it)); release_unit(it++)) {
                const int n = uniform(wp->n);
                if (n == 0) continue;
                if (!(ok = wait_all(bar.res_full, nr & 1, ab, 3))) break;
                ++nr;
                if (DKV) {
                    // S^T = K Q^T, dP^T = V dO^T; dV += P^T dO, dK += dS^T Q.  S of the next
                    // tile is issued behind dV (it takes P's place), dP behind dK.
                    ok = scores_a(tm + 256, bar.s_full) && scores_b(tm + 384);
                    auto rows_b = [&](bool first) {
                        if (!wait_all(bar.p_ready, nt & 1, ab, 6)) return false;
                        tc_fence_after();
                        if (elect_one()) {
                            mma_rows<KS>(tm, tm + 256, sB + rb * TILE, first, 64);
                            tc_commit(bar.b_empty + 8 * rb);
                        }
                        if (++rb == NB) rb = 0;
                        return true;
                    };
                    // Tiles with another after them, without a condition more than that takes.
                    for (int j = 0; j < n - 1 && ok; ++j, ++nt) {
                        if (!(ok = rows_b(j == 0) && scores_a(tm + 256, bar.s_full))) break;
                        if (!(ok = wait_all(bar.ds_ready, nt & 1, ab, 7))) break;
                        rows_a(tm + 128, tm + 384, j == 0);
                        ok = scores_b(tm + 384);
                    }
                    if (!ok || !(ok = rows_b(n == 1) && wait_all(bar.ds_ready, nt & 1, ab, 7))) break;
                    rows_a(tm + 128, tm + 384, n == 1);
                    ++nt;
                } else {
                    // S = Q K^T, dP = dO V^T; dQ += dS K.  Scores run two tiles ahead in two
                    // buffers; dP of the next tile goes first once dS of this one is out.
                    ok = scores_a(tm, bar.s_full) && scores_b(tm + 256);
                    if (ok && n > 1) ok = scores_a(tm + 128, bar.s_full + 8);
                    int j = 0;
                    for (; j < n - 2 && ok; ++j, ++nt) {
                        const uint32_t buf = j & 1;
                        if (!(ok = wait_all(bar.ds_ready, nt & 1, ab, 7) && scores_b(tm + 256))) break;
                        rows_a(tm + 384, tm + buf * 128, j == 0);
                        ok = scores_a(tm + buf * 128, bar.s_full + 8 * buf);
                    }
                    for (; j < n && ok; ++j, ++nt) {
                        const uint32_t buf = j & 1;
                        if (!(ok = wait_all(bar.ds_ready, nt & 1, ab, 7))) break;
                        if (j + 1 < n && !(ok = scores_b(tm + 256))) break;
                        rows_a(tm + 384, tm + buf * 128, j == 0);
                    }
                }
                commit(bar.acc_full);
                commit(bar.res_empty);
            }
            commit(bar.drain);
            if (lane == 0) wait_bar(bar.drain, 0, ab, 10, true);
            __syncwarp();
        } else if (DKV) {
            // ---------------- row statistics: 64 rows of a tile per warp
            asm volatile("griddepcontrol.wait;" ::: "memory");      // the dQ launch has written delta
            uint32_t e = 0;
            bool ok = true;
            const BUnit *wp;
            for (uint32_t it = 0; ok && (wp = next_unit(it)); release_unit(it++)) {
                const BUnit &w = *wp;
                for (int j = 0; j < w.n && ok; ++j, ++e) {
                    const uint32_t st = e & 1;
                    float l2[2], dl[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = (warp - 10) * 64 + h * 32 + lane;
                        const int tok = (w.from + j) * p.TT + r / p.G;
                        l2[h] = INFINITY;      // exp2(s - inf) = 0: rows that do not exist or see nothing
                        dl[h] = 0.f;
                        if (r < p.G * p.TT && tok < w.s.ql) {
                            const size_t at = ((size_t)w.slot * p.Tq + w.s.q0 + tok) * p.Hq + w.hk * p.G + r % p.G;
                            const float x = p.lse[at];
                            if (x != -INFINITY) l2[h] = x * kLog2e;
                            dl[h] = p.delta[at];
                        }
                    }
                    if (!(ok = wait_all(bar.stat_empty + 8 * st, ((e >> 1) & 1) ^ 1u, ab, 14))) break;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = (warp - 10) * 64 + h * 32 + lane;
                        stats[st * 256 + r] = -l2[h];
                        stats[st * 256 + 128 + r] = -dl[h];
                    }
                    arrive_warp(bar.stat_full + 8 * st, lane);
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int wg = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tm = tmem + lane_off;
        const uint64_t c2 = f2(p.scale * kLog2e, p.scale * kLog2e);
        uint32_t ns = 0, nu = 0, nsb[2] = {0, 0};
        bool ok = true;
        const BUnit *wp;
        for (uint32_t it = 0; ok && (wp = next_unit(it)); release_unit(it++)) {
            const BUnit &w = *wp;
            const int n = w.n;
            if (DKV) {
                // ---------------- thread: key first + r, query rows [64 wg, 64 wg + 64) of each tile
                const int key = w.first + r;
                const bool valid = r < w.count;
                for (int j = 0; j < n; ++j, ++ns) {
                    const uint32_t st = ns & 1;
                    const int tok0 = (w.from + j) * p.TT;
                    const int rows = p.G * min(p.TT, w.s.ql - tok0);
                    if (!(ok = wait_all(bar.s_full, ns & 1, ab, 8))) break;
                    tc_fence_after();
                    uint32_t s[2][32];
                    tmem_ld32_async(tm + 256 + wg * 64, s[0]);
                    tmem_ld32_async(tm + 256 + wg * 64 + 32, s[1]);
                    if (!(ok = wait_all(bar.stat_full + 8 * st, (ns >> 1) & 1, ab, 15))) break;
                    tmem_wait_ld32(s[0]);
                    tmem_wait_ld32(s[1]);
                    const float *const sl = stats + st * 256 + wg * 64, *const sd = sl + 128;
                    // rows [lo, hi) of the tile see this key; the tokens are limited to the tile's
                    // before they become rows, or few tokens on a long key range would pass 32 bits
                    int lo = p.causal ? min(max(key - (w.s.kl - w.s.ql) - tok0, 0), p.TT) * p.G : 0;
                    int hi = rows;
                    if (!valid) lo = KT;
                    lo -= wg * 64;
                    hi -= wg * 64;
                    const bool mask = __any_sync(0xFFFFFFFFu, lo > 0 || hi < 64);
                    float pr[64];
                    uint32_t pk[2][16];
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const ulonglong2 l4 = *(const ulonglong2 *)(sl + q * 32 + i);   // minus the row's log-sum
                            float *const x = pr + q * 32 + i;
                            unf2(fma2(f2(__uint_as_float(s[q][i]), __uint_as_float(s[q][i + 1])), c2, l4.x), x[0], x[1]);
                            unf2(fma2(f2(__uint_as_float(s[q][i + 2]), __uint_as_float(s[q][i + 3])), c2, l4.y), x[2], x[3]);
#pragma unroll
                            for (int h = 0; h < 4; ++h) x[h] = ex2(x[h]);
                        }
                    if (mask) {
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            if (i < lo || i >= hi) pr[i] = 0.f;
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) pk[q][i] = pack2(pr[q * 32 + 2 * i], pr[q * 32 + 2 * i + 1]);
                        tmem_st16(tm + 256 + wg * 64 + q * 16, pk[q]);
                    }
                    tmem_wait_st();
                    const bool tail = rows < p.G * p.TT;
                    if (tail) {
                        // rows of the next sequence in this tile: cleared in both operands, which have landed
                        // once S and dP are complete
                        if (!(ok = wait_all(bar.dp_full, ns & 1, ab, 16))) break;
                        // ring entry ns holds this tile in both rings
                        clear_rows<DP>(gA + (ns % NA) * TILE, rows, threadIdx.x, 256);
                        clear_rows<DP>(gB + (ns % NB) * TILE, rows, threadIdx.x, 256);
                        fence_smem_async();
                    }
                    tc_fence_before();
                    arrive_warp(bar.p_ready, lane);
                    if (!(ok = wait_all(bar.dp_full, ns & 1, ab, 16))) break;
                    tc_fence_after();
                    tmem_ld32_async(tm + 384 + wg * 64, s[0]);
                    tmem_ld32_async(tm + 384 + wg * 64 + 32, s[1]);
                    tmem_wait_ld32(s[0]);
                    tmem_wait_ld32(s[1]);
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const ulonglong2 d4 = *(const ulonglong2 *)(sd + q * 32 + i);   // minus the row's delta
                            float *const x = pr + q * 32 + i;
                            unf2(mul2(f2(x[0], x[1]), add2(f2(__uint_as_float(s[q][i]), __uint_as_float(s[q][i + 1])), d4.x)),
                                 x[0], x[1]);
                            unf2(mul2(f2(x[2], x[3]), add2(f2(__uint_as_float(s[q][i + 2]), __uint_as_float(s[q][i + 3])), d4.y)),
                                 x[2], x[3]);
                        }
                    if (mask) {
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            if (i < lo || i >= hi) pr[i] = 0.f;
                    }
                    arrive_warp(bar.stat_empty + 8 * st, lane);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) pk[q][i] = pack2(pr[q * 32 + 2 * i], pr[q * 32 + 2 * i + 1]);
                        tmem_st16(tm + 384 + wg * 64 + q * 16, pk[q]);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    arrive_warp(bar.ds_ready, lane);
                }
                if (!ok) break;
                if (n > 0) {
                    if (!(ok = wait_all(bar.acc_full, nu & 1, ab, 11))) break;
                    ++nu;
                    tc_fence_after();
                }
                if (wg * 64 < DP) {
                    const size_t at = (size_t)w.s.k0 + key;
                    store_acc(tm + wg * 64, p.dv.base + w.slot * p.dv.slot + at * p.dv.token + w.hk * p.dv.head, wg * 64,
                              p.D, 1.f, valid, n == 0);
                    store_acc(tm + 128 + wg * 64, p.dk.base + w.slot * p.dk.slot + at * p.dk.token + w.hk * p.dk.head,
                              wg * 64, p.D, p.scale, valid, n == 0);
                }
            } else {
                // ---------------- thread: query row r of the tile, keys [64 wg, 64 wg + 64) of each tile
                const int ti = r / p.G, head = w.hk * p.G + r % p.G;
                const bool valid = ti < w.count;
                const size_t qi = (size_t)w.s.q0 + w.first + ti;
                const size_t at = ((size_t)w.slot * p.Tq + qi) * p.Hq + head;
                int here = (valid ? seen(p, w.s, w.first + ti) : 0) - wg * 64;   // keys seen from this tile's half on
                float l2 = INFINITY, delta = 0.f;
                if (valid) {
                    // both warpgroups sum the whole row: cheaper than a barrier between them
                    const float x = p.lse[at];
                    if (x != -INFINITY) l2 = x * kLog2e;
                    const char *o = p.o + w.slot * p.o_slot + qi * p.o_token + head * p.o_head;
                    const char *g = p.dout.base + w.slot * p.dout.slot + qi * p.dout.token + head * p.dout.head;
#pragma unroll 4
                    for (int i = 0; i < p.D; i += 8) {
                        const uint4 a = *(const uint4 *)(o + i * 2), b = *(const uint4 *)(g + i * 2);
                        const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            delta = fmaf(__uint_as_float(av[h] << 16), __uint_as_float(bv[h] << 16), delta);
                            delta = fmaf(__uint_as_float(av[h] & 0xFFFF0000u), __uint_as_float(bv[h] & 0xFFFF0000u), delta);
                        }
                    }
                    if (wg == 0) p.delta[at] = delta;
                }
                for (int j = 0; j < n; ++j, ++ns, here -= KT) {
                    const int sb = j & 1;
                    if (!(ok = wait_all(bar.s_full + 8 * sb, nsb[sb] & 1, ab, 8))) break;
                    ++nsb[sb];
                    tc_fence_after();
                    uint32_t s[2][32];
                    float pr[64];
                    tmem_ld32_async(tm + sb * 128 + wg * 64, s[0]);
                    tmem_ld32_async(tm + sb * 128 + wg * 64 + 32, s[1]);
                    tmem_wait_ld32(s[0]);
                    tmem_wait_ld32(s[1]);
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float *const x = pr + q * 32 + i;
                            unf2(fma2(f2(__uint_as_float(s[q][i]), __uint_as_float(s[q][i + 1])), c2, f2(-l2, -l2)), x[0], x[1]);
                            x[0] = ex2(x[0]);
                            x[1] = ex2(x[1]);
                        }
                    if (!(ok = wait_all(bar.dp_full, ns & 1, ab, 16))) break;
                    tc_fence_after();
                    tmem_ld32_async(tm + 256 + wg * 64, s[0]);
                    tmem_ld32_async(tm + 256 + wg * 64 + 32, s[1]);
                    tmem_wait_ld32(s[0]);
                    tmem_wait_ld32(s[1]);
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float *const x = pr + q * 32 + i;
                            const uint64_t d = add2(f2(__uint_as_float(s[q][i]), __uint_as_float(s[q][i + 1])), f2(-delta, -delta));
                            unf2(mul2(f2(x[0], x[1]), d), x[0], x[1]);
                        }
                    if (__any_sync(0xFFFFFFFFu, here < 64)) {
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            if (i >= here) pr[i] = 0.f;
                    }
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) pk[i] = pack2(pr[q * 32 + 2 * i], pr[q * 32 + 2 * i + 1]);
                        tmem_st16(tm + sb * 128 + wg * 64 + q * 16, pk);
                    }
                    tmem_wait_st();
                    const int left = w.s.kl - j * KT;
                    if (left < KT) {     // keys past the end, as rows of dQ's B operand
                        clear_rows<DP>(gA + (ns % NA) * TILE, left, threadIdx.x, 256);
                        fence_smem_async();
                    }
                    tc_fence_before();
                    arrive_warp(bar.ds_ready, lane);
                }
                if (!ok) break;
                if (n > 0) {
                    if (!(ok = wait_all(bar.acc_full, nu & 1, ab, 11))) break;
                    ++nu;
                    tc_fence_after();
                }
                if (wg * 64 < DP)
                    store_acc(tm + 384 + wg * 64, p.dq.base + w.slot * p.dq.slot + qi * p.dq.token + head * p.dq.head,
                              wg * 64, p.D, p.scale, valid, n == 0);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;");
    if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <int KS>
static cudaError_t launch(const Params &p, const CUtensorMap &mq, const CUtensorMap &mdo, const CUtensorMap &mk,
                          const CUtensorMap &mv, cudaStream_t st)
{
    constexpr int DP = tile_cols(KS);
    static OncePerDevice once;
    cudaError_t e = once([] {
        const cudaError_t x = cudaFuncSetAttribute(k_attn_bwd<KS, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   BwdCfg<DP>::SMEM);
        return x != cudaSuccess ? x : cudaFuncSetAttribute(k_attn_bwd<KS, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                           BwdCfg<DP>::SMEM);
    });
    if (e != cudaSuccess) return e;
    if (p.Tq) {
        k_attn_bwd<KS, false><<<p.sms, BWD_THREADS, BwdCfg<DP>::SMEM, st>>>(mq, mdo, mk, mv, p);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess && p.Tk) {
        // Set up while the dQ launch runs: blocks start once every block of it has come to its
        // end, which hides the launch's latency and no more, and wait before the first use of delta.
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)p.sms);
        cfg.blockDim = dim3(BWD_THREADS);
        cfg.dynamicSmemBytes = BwdCfg<DP>::SMEM;
        cfg.stream = st;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = p.Tq ? 1 : 0;
        e = cudaLaunchKernelEx(&cfg, k_attn_bwd<KS, true>, mq, mdo, mk, mv, p);
    }
    return e;
}

cudaError_t launch_attn_bwd(const Params &p, const CUtensorMap &mq, const CUtensorMap &mdo, const CUtensorMap &mk,
                            const CUtensorMap &mv, cudaStream_t st)
{
    return p.D <= 64 ? launch<4>(p, mq, mdo, mk, mv, st) : p.D <= 96 ? launch<6>(p, mq, mdo, mk, mv, st) : launch<8>(p, mq, mdo, mk, mv, st);
}

} // namespace attn
} // namespace rc
