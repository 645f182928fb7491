// attn_fwd.cu -- attention over packed sequences on the 5th-generation tensor
// cores, forward.
//
//   s_ij = scale q_i . k_j over the keys j that token i sees,
//   o_i = sum_j exp(s_ij - m_i) v_j / l_i,  l_i = sum_j exp(s_ij - m_i),
//   lse_i = m_i + ln l_i
// in one pass over the keys: a running maximum m and sum l for each row, both
// in binary32, and an accumulator O that is rescaled when m moves.  m is only
// moved when it would grow by more than 2^8 (any m gives the same quotient;
// the sums stay far inside binary32), which almost never happens after the
// first tile, so the accumulator stays in TMEM.  The weights exp(s - m) are
// rounded to bf16 for the second product -- the tensor cores' input type --
// while l sums them unrounded: the result is off by 1.2 to 1.4 times what bf16 in
// and out costs anyway.  exp2 takes weights below 2^-126 for 0.
//
// One persistent block per SM, 12 warps:
//   warps 0-3, 4-7  softmax of row tile 0 / 1: one thread a row, so maxima and
//                   sums need no shuffles; S arrives in TMEM, P goes back to
//                   TMEM over S and is the A operand of the second product
//   warp 8          units (claimed as blocks come free) and TMA loads: query
//                   tiles, then key and value tiles through one ring of stages
//                   in the order the MMAs consume them
//   warp 9          MMA issue: S_t = Q_t K^T, O_t += P_t V for the two tiles in
//                   turn, so one tile's softmax runs under the other's MMAs
//   warps 10-11     guard: clears non-finite values from the value rows that some
//                   row does not see, because 0 x inf would reach it; rows that
//                   do see one add it in the epilogue
// Two forms.  PAIR: the two row tiles are 256 consecutive rows and share every
// key tile.  SPLIT (few rows per sequence, single tokens above all): both are
// the same rows, over two halves of a key range, so the loads of one hide the
// latency of the other and the kernel runs at the rate of the key cache.  Warps
// w and w + 4 then hold the same rows in the same TMEM lanes: they exchange
// maxima and sums and each joins half of the columns.
// When there are too few units to fill the GPU, key ranges are split over
// units and k_attn_join adds the partial results in a fixed order.
//
// Bounds.  PAIR: 4 products of 128 x 128 x 128 a pair of tiles are 2048 clocks of
// tensor cores; the chain scores - softmax - weights of one tile, half hidden by
// the other's, makes it about 2700.  16384 tokens, 32 heads of 128: 1.22 ms,
// 1810 TFLOP/s as a single launch (called back to back, at the power limit, 1.31 to
// 1.37 ms).  A unit's ends cost 2 to 3 tiles, so six prompts of 1 to 4097 tokens, 32
// heads: 214 us, 1334 TFLOP/s.  SPLIT: memory; 64 tokens on caches of 200 to 7982 keys, 8 key heads:
// 183 us, 5.8 TB/s with the join; one token on 32768 keys of 8 heads: 34 us, 3.9
// TB/s, because the plan, the first loads and the join run one after the other.
#include "attn.cuh"
#include "per_device.h"

namespace rc {
namespace attn {

constexpr int FWD_THREADS = 384;

template <int DP, bool SPLIT>
struct FwdCfg {
    static constexpr int KV_STAGE = KT * DP * 2;
    static constexpr int NQ = SPLIT ? 1 : 2;
    static constexpr int STAGES = DP == 128 ? (SPLIT ? 6 : 5) : 8;
    static constexpr int CTL = 3072;      // barriers and units; maxima and sums of the halves.  With 32 KiB
                                          // tiles this is exactly the 227 KiB of a block
    static constexpr int SMEM = (NQ + STAGES) * KV_STAGE + CTL;
};

// The split of this launch's keys, the same in every warp and kernel of it.
struct Plan {
    int cs;        // key tiles per part (kNoSplit: no key range is split)
    int units;     // units of one key head
};

__device__ __forceinline__ int parts_of(int kt, int cs)
{
    return max(1, (kt + cs - 1) / cs);
}

// How far keys are split (p.may_split: the host found too few unsplit units to
// fill the GPU and made room for partial results).  Each lane tries a part
// size -- 1 to 4 rounds of units over the SMs, with 0 to 7 sixteenths of slack,
// and in the last lane no split -- and the one that ends first is taken.  With t
// the tiles that a unit's row tiles run through and the cost of its ends, in
// tiles, all units are done after `rounds` x t at the latest, and as they go to
// free blocks, also after the blocks' mean share + t; the join comes on top.
// Measured against the best fixed part size of 5 to 64 tiles: token 1 x 32768 keys
// 34.6 (36.0) us, prompt pieces 49.9 (54.6) us, 64 ragged tokens 183.2 (181.6) us.
template <bool SPLIT>
__device__ Plan make_plan(const Params &p, int lane)
{
    constexpr int kEnds = SPLIT ? 2 : 3, kJoin = 4;
    const int HP = p.P * p.Hkv;
    Plan pl;
    pl.cs = kNoSplit;
    if (p.may_split) {
        long long work = 0;
        int most = 0;
        for (int b = lane; b < p.B; b += 32) {
            const Seq s = seq_of(p, b);
            const int kt = (s.kl + KT - 1) / KT;
            work += (long long)((s.ql + p.TPU - 1) / p.TPU) * kt;
            most = max(most, kt);
        }
        work = warp_sum(work) * HP;
        most = max(1, __reduce_max_sync(0xFFFFFFFFu, most));
        const long long per = (long long)p.sms * (1 + (lane >> 3)) * 16;
        const long long c = max((work * (16 + (lane & 7)) + per - 1) / per, 4ll);
        const int cs = c >= most || lane == 31 || most <= kWholeTiles ? most : (int)c;
        int units = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            int nt = 0, kt = 0;
            if (b0 + lane < p.B) {
                const Seq s = seq_of(p, b0 + lane);
                nt = (s.ql + p.TPU - 1) / p.TPU;
                kt = (s.kl + KT - 1) / KT;
            }
            for (int i = 0; i < min(32, p.B - b0); ++i)
                units += __shfl_sync(0xFFFFFFFFu, nt, i) * parts_of(__shfl_sync(0xFFFFFFFFu, kt, i), cs);
        }
        const long long n = (long long)units * HP, t = (SPLIT ? (cs + 1) / 2 : cs) + kEnds;
        const long long cost = min((n + p.sms - 1) / p.sms * t, ((SPLIT ? work / 2 : work) + n * kEnds) / p.sms + t) +
                               (cs < most ? kJoin : 0);
        // More units than there is room for: only where offsets decrease, so that sequences overlap.
        const bool fits = cs == most || n <= p.max_units;
        const unsigned mine = fits ? (unsigned)min(cost, 0x7FFFFFFFll) : 0xFFFFFFFFu, least = __reduce_min_sync(0xFFFFFFFFu, mine);
        const int pick = 31 - __clz(__ballot_sync(0xFFFFFFFFu, mine == least));   // the largest of the best
        pl.cs = __shfl_sync(0xFFFFFFFFu, cs < most ? cs : kNoSplit, pick);
        pl.units = __shfl_sync(0xFFFFFFFFu, units, pick);
        return pl;
    }
    long long u = 0;
    for (int b = lane; b < p.B; b += 32) u += (seq_of(p, b).ql + p.TPU - 1) / p.TPU;
    pl.units = (int)warp_sum(u);
    return pl;
}

struct Unit {
    Seq s;
    int hk, slot;
    int tok;         // first query token of row tile 0, within the sequence
    int ntok[2];     // valid tokens of the row tiles
    int jb[2], n[2]; // first key tile and number of key tiles of each row tile
    int guard;       // keys from here on are not seen by every row
    int nparts;      // parts of this unit's rows (1: results are final)
    int index;       // unit number (partial results); -1: no more units
    int poison;      // set by the guard when it cleared a value of this unit
};
constexpr int UNITS = 4;            // units in the block's ring
constexpr int UNIT_READERS = 11;    // warps that release one: MMA, guard, softmax

template <bool SPLIT>
__device__ Unit unit_of(const Params &p, const Plan &pl, int u, int lane)
{
    Unit w;
    const int HP = p.P * p.Hkv;
    const int x = u / HP, hp = u % HP;
    w.index = u;
    w.hk = hp % p.Hkv;
    w.slot = hp / p.Hkv;
    int b, local;
    locate(p.B, x, lane,
           [&](int bb) {
               const Seq s = seq_of(p, bb);
               return ((s.ql + p.TPU - 1) / p.TPU) * parts_of((s.kl + KT - 1) / KT, pl.cs);
           },
           b, local);
    w.s = seq_of(p, b);
    const int kt = (w.s.kl + KT - 1) / KT, cs = pl.cs;
    w.nparts = parts_of(kt, cs);
    const int nt = (w.s.ql + p.TPU - 1) / p.TPU;
    const int tile = nt - 1 - local / w.nparts, c = local % w.nparts;   // the tiles that see most keys first
    w.tok = tile * p.TPU;
    const int left = w.s.ql - w.tok;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int first = SPLIT ? w.tok : w.tok + t * p.TT;
        w.ntok[t] = SPLIT ? min(left, p.TT) : min(max(left - t * p.TT, 0), p.TT);
        const int see = w.ntok[t] > 0 ? seen(p, w.s, first + w.ntok[t] - 1) : 0;
        const int je = min((see + KT - 1) / KT, cs >= kNoSplit ? kNoSplit : (c + 1) * cs);
        w.jb[t] = c * (cs >= kNoSplit ? 0 : cs);
        w.n[t] = max(0, je - w.jb[t]);
    }
    if (SPLIT) {
        w.n[0] = (w.n[0] + 1) / 2;
        w.n[1] -= w.n[0];
        w.jb[1] += w.n[0];
    }
    w.guard = seen(p, w.s, w.tok);
    w.poison = 0;
    return w;
}

// Ring entries in the order the MMAs consume them.  PAIR: K_0, V_0, K_1, V_1,
// ... (each serves both row tiles).  SPLIT: K0_0 K1_0 | V0_0 K0_1 | V1_0 K1_1 |
// V0_1 ... with the entries of finished halves left out.  f(is_v, t, j).
template <bool SPLIT, class F>
__device__ __forceinline__ void for_entries(const Unit &w, F f)
{
    if (!SPLIT) {
        const int n = max(w.n[0], w.n[1]);
        if (n > 0 && !f(false, 0, 0)) return;
        for (int j = 0; j < n; ++j) {
            if (!f(true, 0, j)) return;
            if (j + 1 < n && !f(false, 0, j + 1)) return;
        }
    } else {
        const int n = max(w.n[0], w.n[1]);
        for (int t = 0; t < 2; ++t)
            if (w.n[t] > 0 && !f(false, t, 0)) return;
        for (int j = 0; j < n; ++j)
            for (int t = 0; t < 2; ++t) {
                if (j < w.n[t] && !f(true, t, j)) return;
                if (j + 1 < w.n[t] && !f(false, t, j + 1)) return;
            }
    }
}

// a * 0 + c on pairs of bf16
__device__ __forceinline__ uint32_t fma0_bf16x2(uint32_t a, uint32_t c)
{
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(0u), "r"(c));
    return d;
}

__device__ __forceinline__ bool nonfinite_bf16(uint32_t bits16) { return (bits16 & 0x7F80u) == 0x7F80u; }

template <int KS, bool SPLIT>
__global__ void __launch_bounds__(FWD_THREADS, 1)
    k_attn_fwd(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
               const __grid_constant__ CUtensorMap map_v, const Params p)
{
    constexpr int DP = tile_cols(KS);
    using C = FwdCfg<DP, SPLIT>;
    constexpr int NST = C::STAGES, STAGE = C::KV_STAGE;
    extern __shared__ __align__(1024) uint8_t gbase[];   // swizzled tiles start on 1024 bytes
    const uint32_t base = smem_u32(gbase), sQ = base, sKV = base + C::NQ * STAGE;
    uint8_t *const gKV = gbase + C::NQ * STAGE;
    uint8_t *const ctl = gKV + NST * STAGE;
    const uint32_t bars = smem_u32(ctl);
    const uint32_t full_bar = bars, empty_bar = bars + 8 * NST, guard_bar = bars + 16 * NST;
    const uint32_t q_full = bars + 24 * NST, q_empty = q_full + 8;
    const uint32_t s_full = q_full + 16, p_ready = q_full + 32, o_full = q_full + 48, drain_bar = q_full + 64;
    uint32_t *const tmem_slot = (uint32_t *)(ctl + 24 * NST + 72);
    int *const abort_flag = (int *)(ctl + 24 * NST + 76);
    const uint32_t u_full = q_full + 80, u_empty = u_full + 8 * UNITS;
    const uint32_t swap_bar = u_empty + 8 * UNITS, joined_bar = swap_bar + 32;   // SPLIT: of warps w and w + 4
    Unit *const units = (Unit *)(ctl + 24 * NST + 80 + 16 * UNITS + 64);
    static_assert(24 * NST + 80 + 16 * UNITS + 64 + UNITS * sizeof(Unit) <= 1024, "control area");
    float2 *const half_stats = (float2 *)(ctl + 1024);                           // SPLIT: [half][row] maximum, sum

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(full_bar + 8 * s, 1);
            mbar_init(empty_bar + 8 * s, 3);     // the MMAs' commit and the two guard warps
            mbar_init(guard_bar + 8 * s, 2);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full + 8 * t, 1);
            mbar_init(p_ready + 8 * t, 4);
            mbar_init(o_full + 8 * t, 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(swap_bar + 8 * i, 2);
            mbar_init(joined_bar + 8 * i, 2);
        }
        mbar_init(drain_bar, 1);
        for (int i = 0; i < UNITS; ++i) {
            mbar_init(u_full + 8 * i, 1);
            mbar_init(u_empty + 8 * i, UNIT_READERS);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&map_q) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&map_k) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&map_v) : "memory");
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;        // S/P tiles at columns 0 and 128, O tiles at 256 and 384
    const Abort ab{abort_flag, p.hdr, p.timeout_ns, 0xB1u, 0};

    // The next unit of the block's ring; null when there is none or the block gave up.
    auto next_unit = [&](uint32_t it) -> const Unit * {
        if (!wait_all(u_full + 8 * (it % UNITS), (it / UNITS) & 1, ab, 12)) return nullptr;
        const Unit *w = units + it % UNITS;
        return w->index < 0 ? nullptr : w;
    };
    auto release_unit = [&](uint32_t it) {
        arrive_warp(u_empty + 8 * (it % UNITS), lane);
    };

    // 384 x 168 registers at launch = 256 x 216 + 128 x 72.  Set inside
    // the branches: ptxas allocates the code that a setmaxnreg dominates by it.
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 8) {
            // ---------------- units and TMA loads (the whole warp, one elected lane issues)
            const Plan pl = make_plan<SPLIT>(p, lane);
            const int total = pl.units * p.P * p.Hkv;
            if (p.may_split && blockIdx.x == 0 && lane == 0) p.hdr->pad[6] = (uint32_t)pl.cs;   // for the join
            uint32_t e = 0, nq = 0, it = 0;
            bool ok = true;
            Unit next;
            // Makes unit u (or the end of all units) the block's next one.
            auto publish = [&](int u) {
                if (u < total) next = unit_of<SPLIT>(p, pl, u, lane);
                else next.index = -1;
                if (!(ok = wait_all(u_empty + 8 * (it % UNITS), ((it / UNITS) & 1) ^ 1u, ab, 13))) return false;
                if (lane == 0) {
                    units[it % UNITS] = next;
                    mbar_arrive(u_full + 8 * (it % UNITS));
                }
                __syncwarp();
                ++it;
                return true;
            };
            const uint32_t q_bytes = (uint32_t)(p.G * p.TT) * 128u * (DP / 64);
            publish(blockIdx.x);
            while (ok && next.index >= 0) {
                const Unit w = next;
                const uint32_t e0 = e;
                // The query tiles wait for the previous unit's last scores; the first key and
                // value tiles do not, and go ahead of them.  The next unit is worked out with
                // those on the way: that takes about 2000 clocks.
                const uint32_t ahead = nq == 0 ? 1 : NST - 2;
                bool begun = max(w.n[0], w.n[1]) == 0;
                auto begin = [&]() {
                    begun = true;
                    if (!(ok = wait_all(q_empty, (nq & 1) ^ 1u, ab, 1))) return false;
                    if (elect_one()) {
                        const int tiles = !SPLIT && w.ntok[1] > 0 ? 2 : 1;
                        mbar_expect_tx(q_full, q_bytes * tiles);
                        for (int t = 0; t < tiles; ++t)
                            for (int d = 0; d < DP / 64; ++d)
                                tma_load_5d(sQ + t * STAGE + d * BLK, &map_q, d * 64, 0, w.s.q0 + w.tok + t * p.TT, w.hk,
                                            w.slot, q_full);
                    }
                    ++nq;
                    return publish(claim_unit<0>(p, lane));
                };
                for_entries<SPLIT>(w, [&](bool is_v, int t, int j) {
                    if (!begun && e - e0 == ahead && !begin()) return false;
                    const uint32_t st = e % NST;
                    if (!(ok = wait_all(empty_bar + 8 * st, ((e / NST) & 1) ^ 1u, ab, 2))) return false;
                    if (elect_one()) {
                        mbar_expect_tx(full_bar + 8 * st, STAGE);
                        for (int d = 0; d < DP / 64; ++d)
                            tma_load_4d(sKV + st * STAGE + d * BLK, is_v ? &map_v : &map_k, d * 64,
                                        w.s.k0 + (w.jb[t] + j) * KT, w.hk, w.slot, full_bar + 8 * st);
                    }
                    ++e;
                    return true;
                });
                if (max(w.n[0], w.n[1]) == 0) publish(claim_unit<0>(p, lane));
                else if (ok && !begun) begin();
            }
            if (lane == 0) units_done<0>(p);
            if (lane == 0 && *(volatile int *)abort_flag) {
                // let the copies in flight land before the block gives up its shared memory
                for (uint32_t s = 0; s < NST; ++s)
                    if (e > s) wait_bar(full_bar + 8 * s, ((e - 1 - s) / NST) & 1, ab, 9, true);
                if (nq) wait_bar(q_full, (nq - 1) & 1, ab, 9, true);
            }
            __syncwarp();
        } else if (warp == 9) {
            // ---------------- MMA issuer (the whole warp, one elected lane issues)
            uint32_t st = 0, ph = 0;                       // ring position: stage and phase
            uint32_t nq = 0, guard_phase = 0, np0 = 0, np1 = 0;
            bool ok = true;
            const uint32_t tm = (uint32_t)uniform((int)tmem);
            const Unit *wp;
            auto advance = [&]() {
                if (++st == NST) st = 0, ph ^= 1u;
            };
            // The ring's current entry has landed (and been looked over, if guarded).
            auto take = [&](bool guarded) {
                if (guarded) {
                    if (!wait_all(guard_bar + 8 * st, (guard_phase >> st) & 1, ab, 5)) return false;
                    guard_phase ^= 1u << st;
                    return true;
                }
                return wait_all(full_bar + 8 * st, ph, ab, 4);
            };
            auto weights = [&](int t) {
                const bool got = wait_all(p_ready + 8 * t, (t ? np1 : np0) & 1, ab, 6);
                if (t) ++np1;
                else ++np0;
                return got;
            };
            // S_t = Q_t K^T with the keys of stage s
            auto score = [&](int t, uint32_t s) {
                tc_fence_after();
                if (elect_one()) {
                    mma_scores<KS>(tm + t * KT, sQ + (SPLIT ? 0 : t * STAGE), sKV + s * STAGE);
                    tc_commit(s_full + 8 * t);
                }
            };
            // O_t += P_t V with the values of stage s
            auto weigh = [&](int t, uint32_t s, bool first, bool last) {
                tc_fence_after();
                if (elect_one()) {
                    mma_rows<KS>(tm + 256 + t * KT, tm + t * KT, sKV + s * STAGE, first, 32);
                    if (last) tc_commit(o_full + 8 * t);
                }
            };
            auto commit = [&](uint32_t bar) {
                if (elect_one()) tc_commit(bar);
            };
            for (uint32_t it = 0; ok && (wp = next_unit(it)); release_unit(it++)) {
                const int n0 = uniform(wp->n[0]), n1 = uniform(wp->n[1]);
                const int gt = uniform(wp->guard) / KT, g0 = gt - uniform(wp->jb[0]), g1 = gt - uniform(wp->jb[1]);   // first guarded tile
                const int n = max(n0, n1);
                if (n == 0) continue;
                if (!(ok = wait_all(q_full, nq & 1, ab, 3))) break;
                ++nq;
                if (!SPLIT) {
                    if (!(ok = take(false))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        if (n0 > 0) mma_scores<KS>(tm, sQ, sKV + st * STAGE), tc_commit(s_full);
                        if (n1 > 0) mma_scores<KS>(tm + KT, sQ + STAGE, sKV + st * STAGE), tc_commit(s_full + 8);
                        tc_commit(empty_bar + 8 * st);
                        if (n == 1) tc_commit(q_empty);
                    }
                    advance();
                    int j = 0;
                    // Tiles that both row tiles have, and another after them.  Written without a
                    // condition more than it needs: this loop's issue is on the critical path.
                    for (const int both = n0 == n1 ? n - 1 : 0; j < both; ++j) {
                        const uint32_t sv = st;
                        if (!(ok = take(j >= g0))) break;
                        advance();
                        const uint32_t sk = st;
                        if (!(ok = take(false))) break;
                        advance();
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (!(ok = weights(t))) break;
                            tc_fence_after();
                            if (elect_one()) {
                                mma_rows<KS>(tm + 256 + t * KT, tm + t * KT, sKV + sv * STAGE, j == 0, 32);
                                if (t == 1) tc_commit(empty_bar + 8 * sv);
                            }
                            if (elect_one()) {
                                mma_scores<KS>(tm + t * KT, sQ + t * STAGE, sKV + sk * STAGE);
                                tc_commit(s_full + 8 * t);
                                if (t == 1) tc_commit(empty_bar + 8 * sk);
                                if (t == 1 && j + 2 == n) tc_commit(q_empty);
                            }
                        }
                        if (!ok) break;
                    }
                    for (; ok && j < n; ++j) {
                        // The values of this tile and the keys of the next are there before the
                        // weights are waited for, so nothing stands between the two products.
                        const uint32_t sv = st;
                        if (!(ok = take(j >= g0))) break;
                        advance();
                        const uint32_t sk = st;
                        const bool more = j + 1 < n;
                        if (more) {
                            if (!(ok = take(false))) break;
                            advance();
                        }
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const int nt = t ? n1 : n0;
                            if (j >= nt) continue;
                            if (!(ok = weights(t))) break;
                            tc_fence_after();
                            const bool last_v = t == 1 || j >= n1;                   // the tile's last use here
                            const bool last_k = t == 1 || j + 1 >= n1;
                            if (elect_one()) {
                                mma_rows<KS>(tm + 256 + t * KT, tm + t * KT, sKV + sv * STAGE, j == 0, 32);
                                if (last_v) tc_commit(empty_bar + 8 * sv);
                            }
                            if (elect_one()) {
                                if (j + 1 < nt) {
                                    mma_scores<KS>(tm + t * KT, sQ + t * STAGE, sKV + sk * STAGE);
                                    tc_commit(s_full + 8 * t);
                                    if (last_k) {
                                        tc_commit(empty_bar + 8 * sk);
                                        if (j + 2 == n) tc_commit(q_empty);
                                    }
                                } else {
                                    tc_commit(o_full + 8 * t);
                                }
                            }
                        }
                        if (!ok) break;
                    }
                } else {
                    int left = n0 + n1;                    // scores to issue with this unit's queries
                    auto scored = [&](int t) {
                        if (!take(false)) return false;
                        score(t, st);
                        commit(empty_bar + 8 * st);
                        advance();
                        if (--left == 0) commit(q_empty);
                        return true;
                    };
                    if (n0 > 0) ok = scored(0);
                    if (ok && n1 > 0) ok = scored(1);
                    for (int j = 0; j < n && ok; ++j) {
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const int nt = t ? n1 : n0;
                            if (j >= nt || !ok) continue;
                            if (!(ok = take(j >= (t ? g1 : g0)) && weights(t))) continue;
                            weigh(t, st, j == 0, j + 1 == nt);
                            commit(empty_bar + 8 * st);
                            advance();
                            if (j + 1 < nt) ok = scored(t);
                        }
                    }
                }
            }
            commit(drain_bar);
            if (lane == 0) wait_bar(drain_bar, 0, ab, 10, true);
            __syncwarp();
        } else {
            // ---------------- guard: every other group of 32 16-byte pieces of a value tile
            const int g = warp - 10;
            uint32_t e = 0;
            bool ok = true;
            const Unit *wp;
            for (uint32_t it = 0; ok && (wp = next_unit(it)); release_unit(it++)) {
                const Unit &w = *wp;
                for_entries<SPLIT>(w, [&](bool is_v, int t, int j) {
                    // Every entry is waited for and released, in order: a guard that
                    // only looked at its own entries could meet a stage's barrier one
                    // whole round early or late, where the phase parity says nothing.
                    const uint32_t en = e++, st = en % NST;
                    const int jt = w.jb[t] + j;
                    if (!(ok = wait_idle(full_bar + 8 * st, (en / NST) & 1, ab, 7))) return false;
                    if (!is_v || jt < w.guard / KT) {
                        arrive_warp(empty_bar + 8 * st, lane);
                        return true;
                    }
                    // The rows from here on, 16 bytes a lane at a time: x * 0 is NaN for x
                    // infinite or NaN, and stays in the sum.  Values to clear are rare,
                    // so they are looked for again.
                    const int lo = max(w.guard - jt * KT, 0), n16 = (KT - lo) * 8;
                    uint8_t *const rows = gKV + st * STAGE + lo * 128;
                    uint32_t sum[4] = {0, 0, 0, 0};
#pragma unroll 4
                    for (int i = g * 32 + lane; i < n16; i += 64)
#pragma unroll
                        for (int b = 0; b < DP / 64; ++b) {
                            const uint4 x = *(const uint4 *)(rows + b * BLK + i * 16);
                            sum[0] = fma0_bf16x2(x.x, sum[0]);
                            sum[1] = fma0_bf16x2(x.y, sum[1]);
                            sum[2] = fma0_bf16x2(x.z, sum[2]);
                            sum[3] = fma0_bf16x2(x.w, sum[3]);
                        }
                    uint32_t all = fma0_bf16x2(sum[0], sum[1]);
                    all = fma0_bf16x2(all, fma0_bf16x2(sum[2], sum[3]));
                    if (__any_sync(0xFFFFFFFFu, nonfinite_bf16(all) || nonfinite_bf16(all >> 16))) {
                        const int valid = w.s.kl - jt * KT - lo;    // rows from here on are past the end
                        // the same pieces that this warp looked at: the other may have found nothing
#pragma unroll 1
                        for (int i = g * 32 + lane; i < n16; i += 64)
#pragma unroll 1
                            for (int h = 0; h < 4 * (DP / 64); ++h) {
                                uint32_t *const a = (uint32_t *)(rows + (h >> 2) * BLK + i * 16) + (h & 3);
                                const uint32_t x = *a;
                                const uint32_t keep = (nonfinite_bf16(x) ? 0u : 0xFFFFu) | (nonfinite_bf16(x >> 16) ? 0u : 0xFFFF0000u);
                                if (keep == 0xFFFFFFFFu) continue;
                                *a = x & keep;
                                if (i / 8 < valid) *(volatile int *)&units[it % UNITS].poison = 1;
                            }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    }
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(guard_bar + 8 * st);
                        mbar_arrive(empty_bar + 8 * st);
                    }
                    return true;
                });
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // ---------------- softmax and epilogue of row tile t
        const int t = warp >> 2;
        const int r = threadIdx.x & 127;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + t * KT, tO = tmem + lane_off + 256 + t * KT;
        const float c = p.scale * kLog2e;
        uint32_t ns = 0, no[2] = {0, 0}, nswap = 0;
        bool ok = true;
        const Unit *wp;
        for (uint32_t it = 0; ok && (wp = next_unit(it)); release_unit(it++)) {
            const Unit &w = *wp;
            const int n = w.n[t];
            const int ti = r / p.G;                                    // token of this row within the tile
            const int tok = (SPLIT ? w.tok : w.tok + t * p.TT) + ti;   // and within the sequence
            const bool valid = ti < w.ntok[t];
            const int lim = valid ? seen(p, w.s, tok) : 0;             // keys this row sees
            int here = lim - w.jb[t] * KT;                             // and from this key tile on
            // From this tile on some row of the warp does not see every key.
            const bool any = __any_sync(0xFFFFFFFFu, valid);
            const int mask_from = __reduce_min_sync(0xFFFFFFFFu, valid ? max(here, 0) : kNoSplit) / KT;
            float m = -INFINITY, mc = 0.f, l = 0.f;                    // mc = c * m, 0 while nothing was seen
            for (int j = 0; j < n; ++j, here -= KT) {
                if (!(ok = wait_all(s_full + 8 * t, ns & 1, ab, 8))) break;
                ++ns;
                tc_fence_after();
                if (SPLIT && !any) {      // no row of this warp is in use: whatever P holds is not read
                    arrive_warp(p_ready + 8 * t, lane);
                    continue;
                }
                uint32_t v[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_ld32_async(tS + q * 32, v[q]);
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_wait_ld32(v[q]);
                if (j >= mask_from) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (q * 32 + i >= here) v[q][i] = 0xFF800000u;
                }
                // 32 weights and their share of the row sum
                uint64_t sum = 0;
                auto weights32 = [&](const uint32_t (&x)[32], uint32_t (&pk)[16], uint64_t acc) {
                    const uint64_t c2 = f2(c, c), m2 = f2(-mc, -mc);
                    uint64_t s0 = acc, s1 = 0;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float a, b;
                        unf2(fma2(f2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), c2, m2), a, b);
                        a = ex2(a);
                        b = ex2(b);
                        if (i & 1) s1 = add2(s1, f2(a, b));
                        else s0 = add2(s0, f2(a, b));
                        pk[i] = pack2(a, b);
                    }
                    return add2(s0, s1);
                };
                // The first 32 weights are taken with the maximum so far, under the search for
                // the new one, and taken again in the rare case that it has to move.
                uint32_t p0[16];
                uint64_t w0 = weights32(v[0], p0, 0);
                float mx[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    mx[q] = fmaxf(__uint_as_float(v[q][0]), __uint_as_float(v[q][1]));
#pragma unroll
                    for (int i = 2; i < 32; i += 2) mx[q] = max3(mx[q], __uint_as_float(v[q][i]), __uint_as_float(v[q][i + 1]));
                }
                const float mt = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
                // Move m when it would grow by more than 8 / c, or off -inf.
                const bool move = mt > m && (m == -INFINITY || (mt - m) * c > 8.f);
                if (__any_sync(0xFFFFFFFFu, move)) {
                    const float f = !move ? 1.f : (m == -INFINITY ? 0.f : ex2((m - mt) * c));
                    if (move) {
                        m = mt;
                        mc = mt * c;
                    }
                    l *= f;
                    if (j > 0) {
                        uint32_t o[32];
#pragma unroll 1
                        for (int q = 0; q < DP / 32; ++q) {
                            tmem_ld32(tO + q * 32, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st32(tO + q * 32, o);
                        }
                    }
                    w0 = weights32(v[0], p0, 0);
                }
                sum = w0;
                tmem_st16(tS, p0);
#pragma unroll
                for (int q = 1; q < 4; ++q) {
                    uint32_t pk[16];
                    sum = weights32(v[q], pk, sum);
                    tmem_st16(tS + q * 16, pk);
                }
                float sa, sb;
                unf2(sum, sa, sb);
                l += sa + sb;
                tmem_wait_st();
                tc_fence_before();
                arrive_warp(p_ready + 8 * t, lane);
            }
            if (!ok) break;
            // The accumulators: this row tile's, or in the SPLIT form those of both halves.
            float mcs[2] = {mc, mc}, ls[2] = {l, 0.f};
            if (SPLIT && any) {
                const uint32_t pair = 8 * (warp & 3);
                half_stats[t * KT + r] = make_float2(mc, l);
                arrive_warp(swap_bar + pair, lane);
                if (!(ok = wait_all(swap_bar + pair, nswap & 1, ab, 14))) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 x = half_stats[h * KT + r];
                    mcs[h] = x.x;
                    ls[h] = x.y;
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!SPLIT && h != t) continue;
                if (w.n[h] > 0) {
                    if (!(SPLIT && !any) && !(ok = wait_all(o_full + 8 * h, no[h] & 1, ab, 11))) break;
                    ++no[h];
                }
            }
            if (!ok) break;
            if (SPLIT && !any) continue;                               // nor in the other half's warp
            tc_fence_after();
            float fac[2];
            if (SPLIT) {
                // a half without keys for this row has the sum 0, whatever its maximum
                mc = ls[0] == 0.f ? mcs[1] : ls[1] == 0.f ? mcs[0] : fmaxf(mcs[0], mcs[1]);
                fac[0] = ls[0] == 0.f ? 0.f : ex2(mcs[0] - mc);
                fac[1] = ls[1] == 0.f ? 0.f : ex2(mcs[1] - mc);
                l = ls[0] * fac[0] + ls[1] * fac[1];
            } else {
                fac[0] = 1.f;
            }
            const int head = w.hk * p.G + r % p.G;
            const bool final_ = w.nparts == 1;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const size_t qi = (size_t)w.s.q0 + tok;
            const bool add_back = *(volatile const int *)&w.poison != 0;
            char *const dst = p.out.base + w.slot * p.out.slot + qi * p.out.token + head * p.out.head;
            const size_t part_row = (size_t)(SPLIT ? w.index : 2 * w.index + t) * p.part_rows + r;
            float *const part = p.part_o + part_row * DP;
            const int end = SPLIT ? w.jb[1] + w.n[1] : w.jb[t] + n;    // of the unit's key tiles
            constexpr int QN = SPLIT ? DP / 64 : DP / 32;              // blocks of 32 columns of a warp
            // Not unrolled: run once a unit, its instructions are fetched anew each time (unrolled,
            // ragged prompts took 219.5 us for 214.4, one token on 32768 keys 35.5 for 34.1).
#pragma unroll 1
            for (int q_ = 0; q_ < QN; ++q_) {
                const int q = SPLIT ? t * QN + q_ : q_;
                float f[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) f[i] = 0.f;
#pragma unroll
                for (int h = 0; h < (SPLIT ? 2 : 1); ++h) {
                    if ((SPLIT ? w.n[h] : n) == 0) continue;
                    const float fh = fac[h] * inv;
                    uint32_t o[32];
                    tmem_ld32((SPLIT ? tmem + lane_off + 256 + h * KT : tO) + q * 32, o);
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] = fmaf(__uint_as_float(o[i]), fh, f[i]);
                }
                if (!valid) continue;
                if (add_back) {
                    // non-finite values that this row does see, taken out by the guard
                    const int k1 = min(lim, end * KT);
                    for (int k = max(w.guard, w.jb[SPLIT ? 0 : t] * KT); k < k1; ++k) {
                        const uint16_t *vr = (const uint16_t *)(p.v + w.slot * p.v_slot +
                                                                ((size_t)w.s.k0 + k) * p.v_token + w.hk * p.v_head);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (q * 32 + i < p.D) {
                                const uint32_t x = vr[q * 32 + i];
                                if (nonfinite_bf16(x)) f[i] += __uint_as_float(x << 16);
                            }
                    }
                }
                if (final_ && p.out32) {
#pragma unroll
                    for (int i = 0; i < 32; i += 16)
                        if (q * 32 + i < p.D)
                            st8<kStNormal>(dst + (q * 32 + i) * 2,
                                           make_uint4(pack2(f[i], f[i + 1]), pack2(f[i + 2], f[i + 3]),
                                                      pack2(f[i + 4], f[i + 5]), pack2(f[i + 6], f[i + 7])),
                                           make_uint4(pack2(f[i + 8], f[i + 9]), pack2(f[i + 10], f[i + 11]),
                                                      pack2(f[i + 12], f[i + 13]), pack2(f[i + 14], f[i + 15])));
                } else if (final_) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        if (q * 32 + i < p.D)
                            st_v4(dst + (q * 32 + i) * 2, make_uint4(pack2(f[i], f[i + 1]), pack2(f[i + 2], f[i + 3]),
                                                                     pack2(f[i + 4], f[i + 5]), pack2(f[i + 6], f[i + 7])));
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        st8<kStNormal>(part + q * 32 + i,
                                       make_uint4(__float_as_uint(f[i]), __float_as_uint(f[i + 1]),
                                                  __float_as_uint(f[i + 2]), __float_as_uint(f[i + 3])),
                                       make_uint4(__float_as_uint(f[i + 4]), __float_as_uint(f[i + 5]),
                                                  __float_as_uint(f[i + 6]), __float_as_uint(f[i + 7])));
                }
            }
            if (SPLIT) {
                // the accumulators are overwritten when this warp and its partner hand over new weights
                const uint32_t pair = 8 * (warp & 3);
                tc_fence_before();
                arrive_warp(joined_bar + pair, lane);
                if (!(ok = wait_all(joined_bar + pair, nswap & 1, ab, 15))) break;
                tc_fence_after();
                ++nswap;
            }
            if (valid && !(SPLIT && t == 1)) {
                const float lse = l == 0.f ? -INFINITY : (mc + log2f(l)) * kLn2;
                if (!final_)
                    p.part_lse[part_row] = lse;
                else if (p.lse)
                    p.lse[((size_t)w.slot * p.Tq + qi) * p.Hq + head] = lse;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;");
    if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Joins the parts of split rows in part order:
//   lse = m + ln sum_c exp(lse_c - m),  o = sum_c exp(lse_c - lse) o_c.
// In a caller's workspace (CLEAR) each part is zeroed once it is read: other calls
// keep signal words there, which must not find a number that looks like a signal.
// That costs 1.7 us (one token on 32768 keys, 33.9 -> 35.6) to 4 us (two pieces of
// prompts, 50 -> 54) and nothing where the library's own space is used.
// Few rows have up to hundreds of parts: a block of 8 warps takes a row, warp w
// adds parts w, w + 8, ..., and the warps' sums are added in warp order.  Many
// rows (kJoinRows a multiprocessor on average) have few parts: a warp takes a row.
constexpr int JOIN_WARPS = 8;

constexpr int kJoinRows = 8;

template <int DP, bool SPLIT, bool WIDE, bool CLEAR>
__global__ void __launch_bounds__(32 * JOIN_WARPS) k_attn_join(const Params p)
{
    constexpr int W = WIDE ? JOIN_WARPS : 1;               // warps of a row
    constexpr int ROWS = JOIN_WARPS / W;                   // rows of a block at a time
    __shared__ float acc_s[W][DP + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");     // the parts are written, and their size
    Plan pl;
    pl.cs = (int)ld_relaxed_gpu(&p.hdr->pad[6]);
    if (pl.cs >= kNoSplit) return;
    const int HP = p.P * p.Hkv;
    // Split launches have few rows (well below 2^31), so 32-bit divisions do; with 64-bit ones
    // they were most of the kernel.
    const unsigned rows = (unsigned)p.P * p.Tq * p.Hq;
    for (unsigned row = blockIdx.x * ROWS + warp / W; row < rows; row += gridDim.x * ROWS) {
        const unsigned tok = row / p.Hq;
        const int head = (int)(row - tok * p.Hq), slot = (int)(tok / p.Tq), qi = (int)(tok - slot * p.Tq);
        // the sequence of token qi, and the units before it
        int units = 0, b_hit = -1;
        for (int b0 = 0; b0 < p.B && b_hit < 0; b0 += 32) {
            const int b = b0 + lane;
            Seq sb{};
            int n = 0;
            if (b < p.B) {
                sb = seq_of(p, b);
                n = ((sb.ql + p.TPU - 1) / p.TPU) * parts_of((sb.kl + KT - 1) / KT, pl.cs);
            }
            const int inc = warp_incl_scan(n, lane);
            const unsigned hit = __ballot_sync(0xFFFFFFFFu, b < p.B && qi >= sb.q0 && qi < sb.q0 + sb.ql);
            const int src = hit ? __ffs(hit) - 1 : 31;
            units += __shfl_sync(0xFFFFFFFFu, hit ? inc - n : inc, src);
            if (hit) b_hit = b0 + src;
        }
        if (b_hit < 0) continue;
        const Seq s = seq_of(p, b_hit);
        const int kt = (s.kl + KT - 1) / KT;
        const int np = parts_of(kt, pl.cs);
        if (np == 1) continue;
        const int i = qi - s.q0, tile = i / p.TPU, nt = (s.ql + p.TPU - 1) / p.TPU;
        const int in_tile = i - tile * p.TPU, t_pair = in_tile / p.TT;
        const int r = (in_tile % p.TT) * p.G + head % p.G;
        const int x0 = units + (nt - 1 - tile) * np, hp = slot * p.Hkv + head / p.G;
        auto slot_of = [&](int c) {
            const size_t u = (size_t)(x0 + c) * HP + hp;
            return (SPLIT ? u : 2 * u + t_pair) * p.part_rows + r;
        };
        float m = -INFINITY;
        for (int c = lane; c < np; c += 32) m = fmaxf(m, p.part_lse[slot_of(c)]);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float base = m == -INFINITY ? 0.f : m;
        constexpr int E = DP / 32;                         // elements of a lane, next to each other
        float acc[E] = {}, sum = 0.f;
        for (int c0 = warp % W; c0 < np; c0 += 4 * W) {    // four parts' loads at a time
            float x[4][E], wgt[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int c = c0 + k * W;
                const size_t sl = slot_of(c < np ? c : c0);
                wgt[k] = c < np ? p.part_lse[sl] : -INFINITY;
                float *const part = p.part_o + sl * DP + lane * E;
                if (E == 4) *(float4 *)x[k] = *(const float4 *)part;
                else *(float2 *)x[k] = *(const float2 *)part;
            }
            if (CLEAR) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (c0 + k * W < np) {
                        float *const part = p.part_o + slot_of(c0 + k * W) * DP + lane * E;
                        if (E == 4) *(float4 *)part = make_float4(0.f, 0.f, 0.f, 0.f);
                        else *(float2 *)part = make_float2(0.f, 0.f);
                    }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c0 + k * W < np) {
                    wgt[k] = expf(wgt[k] - base);
                    sum += wgt[k];
#pragma unroll
                    for (int d = 0; d < E; ++d) acc[d] = fmaf(wgt[k], x[k][d], acc[d]);
                }
        }
        char *const dst = p.out.base + slot * p.out.slot + (size_t)qi * p.out.token + head * p.out.head;
        if (WIDE) {
#pragma unroll
            for (int d = 0; d < E; ++d) acc_s[warp][lane * E + d] = acc[d];
            if (lane == 0) acc_s[warp][DP] = sum;
            __syncthreads();                               // the row is the whole block's
            sum = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) sum += acc_s[w][DP];
            const int d = threadIdx.x;
            if (d < p.D) {
                float o = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) o += acc_s[w][d];
                st_u16(dst + d * 2, (uint16_t)pack2(sum == 0.f ? 0.f : o / sum, 0.f));
            }
            __syncthreads();                               // and every warp is done with the row's log-sums
        } else if (lane * E < p.D) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int d = 0; d < E; d += 2) st_u32(dst + (lane * E + d) * 2, pack2(acc[d] * inv, acc[d + 1] * inv));
        }
        if (lane == 0 && warp % W == 0 && p.lse) p.lse[row] = sum == 0.f ? -INFINITY : base + logf(sum);
        if (CLEAR && warp % W == 0) {
            __syncwarp();
            for (int c = lane; c < np; c += 32) p.part_lse[slot_of(c)] = 0.f;
        }
    }
}

template <int KS, bool SPLIT>
static cudaError_t launch(const Params &p, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                          cudaStream_t st)
{
    constexpr int DP = tile_cols(KS);
    static OncePerDevice once;
    cudaError_t e = once([] {
        return cudaFuncSetAttribute(k_attn_fwd<KS, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    FwdCfg<DP, SPLIT>::SMEM);
    });
    if (e != cudaSuccess) return e;
    k_attn_fwd<KS, SPLIT><<<p.sms, FWD_THREADS, FwdCfg<DP, SPLIT>::SMEM, st>>>(mq, mk, mv, p);
    e = cudaGetLastError();
    if (e != cudaSuccess || !p.may_split) return e;
    // Set up while the units run: the join's blocks start once every block has come to its end,
    // which hides the launch's latency.
    cudaLaunchConfig_t cfg{};
    const long long rows = (long long)p.P * p.Tq * p.Hq;
    const bool wide = rows < (long long)kJoinRows * p.sms;
    const long long blocks = wide ? rows : (rows + JOIN_WARPS - 1) / JOIN_WARPS;
    cfg.gridDim = dim3((unsigned)(blocks < 8ll * p.sms ? blocks : 8ll * p.sms));
    cfg.blockDim = dim3(32 * JOIN_WARPS);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (p.clear)
        return wide ? cudaLaunchKernelEx(&cfg, k_attn_join<DP, SPLIT, true, true>, p)
                    : cudaLaunchKernelEx(&cfg, k_attn_join<DP, SPLIT, false, true>, p);
    return wide ? cudaLaunchKernelEx(&cfg, k_attn_join<DP, SPLIT, true, false>, p)
                : cudaLaunchKernelEx(&cfg, k_attn_join<DP, SPLIT, false, false>, p);
}

cudaError_t launch_attn_fwd(const Params &p, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                            bool split, cudaStream_t st)
{
    if (p.D <= 64) return split ? launch<4, true>(p, mq, mk, mv, st) : launch<4, false>(p, mq, mk, mv, st);
    if (p.D <= 96) return split ? launch<6, true>(p, mq, mk, mv, st) : launch<6, false>(p, mq, mk, mv, st);
    return split ? launch<8, true>(p, mq, mk, mv, st) : launch<8, false>(p, mq, mk, mv, st);
}

} // namespace attn
} // namespace rc
