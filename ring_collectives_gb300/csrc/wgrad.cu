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
//   warps 8-15   copy their pieces of 128 k of q ahead with cp.async, each thread into
//                slots of its own, widen them and write the swizzled tile;
//   warp 1       (even CTA) issues the MMAs of the pair, M = N = 256;
//   warps 4-7    take finished tiles from TMEM, while the next one is summed.
// Whole tiles are dealt out in rounds; the tokens of those that are left over are
// divided evenly over all pairs, and k_wgrad_join adds the parts in order.
#include <cudaTypedefs.h>

#include <mutex>

#include "act8.cuh"
#include "heads.h"
#include "per_device.h"
#include "tc.cuh"

namespace rc {
namespace wg {

using namespace tc;

constexpr int TILE = 256, HALF = 128;         // a pair's tile of dw; a CTA's rows n, and its columns k to widen
constexpr int STEP = 64;                      // tokens a step
constexpr int STAGES = 5;
constexpr int BLOCK = 64 * STEP * 2;          // 64 channels x 64 tokens of bf16
constexpr int OPERAND = 2 * BLOCK;            // a CTA's half of an operand's stage
constexpr int DEEP = 5;                       // steps of q that a thread's slots hold
constexpr int WIDEN = 256, EPILOGUE = 4;      // threads that widen; warps that store
constexpr int THREADS = 256 + WIDEN;
constexpr int SLOTS = DEEP * WIDEN * 32;      // 32 bytes of q a thread and step
constexpr int TMEM_COLS = 512;                // two accumulators
constexpr int SMEM = STAGES * 2 * OPERAND + SLOTS + 1024 + 256;
constexpr uint32_t kIdesc = idesc_bf16_f32(TILE, TILE) | (1u << 15) | kIdescBMnMajor;   // both MN-major

struct Params {
    Act8 x8;
    Rows dw;
    float *part;                              // [pair][2][256][256]
    WsHeader *hdr;
    int P, T, N, K;
    int n_tiles, k_tiles, whole, left, pairs; // tiles dealt out whole; left over; pairs of the launch
    uint32_t steps;
    int dy_shared, wide, f32, accumulate, st32, clear;
    unsigned long long timeout_ns;
};

// A pair's share of the steps of the tiles left over: [first(i), first(i + 1)).
__host__ __device__ __forceinline__ uint64_t first_step(const Params &p, int pair)
{
    return (uint64_t)p.left * p.steps * (uint32_t)pair / (uint32_t)p.pairs;
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

__device__ __forceinline__ void arrive_remote_relaxed(uint32_t bar_cluster)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

// Copies of q into a thread's slot; nothing is read for `on` false, and the slot is zeroed.
template <int B>
__device__ __forceinline__ void copy(uint32_t dst, const void *src, bool on)
{
    if (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(on ? 8 : 0) : "memory");
}

// 32 columns of a row of dw from v, as far as they exist; k: the first of them.
template <bool F32>
__device__ __forceinline__ void store32(const Params &p, char *row, int k, uint32_t (&v)[32])
{
    if (F32) {
        float4 *const o = (float4 *)(row + (size_t)k * 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (k + 4 * i >= p.K) break;
            float4 f = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]), __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
            if (p.accumulate) {
                const float4 old = __ldcs(o + i);
                f = make_float4(old.x + f.x, old.y + f.y, old.z + f.z, old.w + f.w);
            }
            __stcs(o + i, f);
        }
        return;
    }
    uint4 *const o = (uint4 *)(row + (size_t)k * 2);
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (p.accumulate && k + 8 * i < p.K) {
            f32x2 old[4];
            wide8(__ldcs(o + i), old);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[8 * i + 2 * j] = __float_as_uint(__uint_as_float(v[8 * i + 2 * j]) + lo(old[j]));
                v[8 * i + 2 * j + 1] = __float_as_uint(__uint_as_float(v[8 * i + 2 * j + 1]) + hi(old[j]));
            }
        }
        w[i] = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]), pack_bf16x2(v[8 * i + 4], v[8 * i + 5]),
                          pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
    }
    if (p.st32 && k + 32 <= p.K) {
        st8<kStEvictFirst>(o, w[0], w[1]);
        st8<kStEvictFirst>(o + 2, w[2], w[3]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (k + 8 * i < p.K) st_v4(o + i, w[i]);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1) k_wgrad(const __grid_constant__ CUtensorMap map, const Params p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *const gbase = smem_raw + (base - raw);
    const uint32_t sA = base, sB = sA + STAGES * OPERAND, sQ = sB + STAGES * OPERAND, bars = sQ + SLOTS;
    uint8_t *const bars_g = gbase + STAGES * 2 * OPERAND + SLOTS;
    const uint32_t full_a = bars, full_b = bars + 8 * STAGES, empty = bars + 16 * STAGES, tfull = bars + 24 * STAGES, tempty = tfull + 16,
                   drained = tempty + 16;
    uint32_t *const tmem_slot = (uint32_t *)(bars_g + 24 * STAGES + 40);
    int *const abort_flag = (int *)(bars_g + 24 * STAGES + 44);
    static_assert(24 * STAGES + 48 <= 256, "barriers fit behind the slots");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t cta = cluster_ctarank();
    const bool even = cta == 0;
    const int pair = (int)(blockIdx.x >> 1);
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_a + 8 * s, 1);                 // the even CTA's arm for the bytes of both
            mbar_init(full_b + 8 * s, 2 * (WIDEN / 32));  // every widening warp of both CTAs
            mbar_init(empty + 8 * s, 1);                  // one commit of the pair's MMAs
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

    if (warp == 0 && lane == 0) {
        // ---------------- dy by TMA (both CTAs; the bytes are counted on the even one's barrier)
        const uint32_t full_even = mapa_shared(full_a, 0);
        uint32_t stage = 0, phase = 0;
        int issued[STAGES] = {};
        Walk w;
        for (w.start(p, pair); w.tile >= 0; w.next(p, pair)) {
            if (!wait_bar(empty + 8 * stage, phase ^ 1u, ab, 2)) break;
            if (even) mbar_expect_tx(full_a + 8 * stage, 2 * OPERAND);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                tma_load_3d_pair(sA + stage * OPERAND + i * BLOCK, &map, w.n + (int)cta * HALF + 64 * i, (int)(w.step * STEP),
                                 p.dy_shared ? 0 : w.r, full_even + 8 * stage);
            issued[stage]++;
            if (++stage == STAGES) stage = 0, phase ^= 1u;
        }
        if (even && *(volatile int *)abort_flag)          // no copy of either CTA stays in flight
            for (int s = 0; s < STAGES; ++s)
                if (issued[s] > 0) wait_bar(full_a + 8 * s, (uint32_t)((issued[s] - 1) & 1), ab, 9, true);
    } else if (warp == 1 && lane == 0 && even) {
        // ---------------- MMAs of the pair
        uint32_t stage = 0, phase = 0;
        int it = 0;
        bool ok = true;
        Walk w;
        for (w.start(p, pair); w.tile >= 0 && ok; ++it, w.next_tile(p, pair)) {
            const uint32_t acc = it & 1;
            if (!wait_bar<true>(tempty + 8 * acc, ((it >> 1) & 1) ^ 1u, ab, 3)) break;
            tc_fence_after();
            const uint32_t d = tmem + acc * TILE;
            for (uint32_t s = w.step; s < w.end; ++s) {
                if (!wait_bar(full_a + 8 * stage, phase, ab, 4) || !wait_bar<true>(full_b + 8 * stage, phase, ab, 5)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t ad = smem_desc_mn_sw128(sA + stage * OPERAND, BLOCK), bd = smem_desc_mn_sw128(sB + stage * OPERAND, BLOCK);
#pragma unroll
                for (int i = 0; i < STEP / 16; ++i)       // 16 tokens: 2048 bytes
                    tc_mma_pair(d, ad + (uint64_t)(128 * i), bd + (uint64_t)(128 * i), kIdesc, s != w.step || i != 0);
                tc_commit_pair_mc(empty + 8 * stage, 3);
                if (++stage == STAGES) stage = 0, phase ^= 1u;
            }
            tc_commit_pair_mc(tfull + 8 * acc, 3);
        }
        tc_commit_pair_mc(drained, 1);
        wait_bar(drained, 0, ab, 10, true);
    } else if (warp >= 8) {
        // ---------------- q to bf16.  A thread takes 16 k of the tokens t and t + 32 of a step: eight
        // lanes read the 128 bytes of a token.  Of a swizzled row of 128 bytes (64 k) a lane writes two
        // 16-byte chunks; lanes 4-7 write the other block's, in the other order: no bank twice.
        const int j = threadIdx.x - 256, c = j & 7, t0 = j >> 3;
        const uint32_t slot = sQ + j * 16;                // pieces of 16 bytes, threads side by side
        const uint32_t full_even = mapa_shared(full_b, 0);
        const uint32_t out = sB + (c >> 2) * BLOCK;
        Walk now, ahead;
        now.start(p, pair);
        ahead = now;
        uint32_t e[DEEP][2];
        auto fetch = [&](int d) {
            if (ahead.tile >= 0) {
                const int k = ahead.k + (int)cta * HALF + c * 16;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t t = ahead.step * STEP + t0 + 32 * i, dst = slot + (d * 2 + i) * (WIDEN * 16);
                    const bool on = t < (uint32_t)p.T && k < p.K, more = on && k + 8 < p.K;
                    const char *const src = on ? p.x8.q.at(ahead.r, t) + k : p.x8.q.base;
                    if (p.wide) copy<16>(dst, src, on);
                    else copy<8>(dst, src, on), copy<8>(dst + 8, more ? src + 8 : p.x8.q.base, more);
                    e[d][i] = 1;
                    if (on) e[d][i] = __ldg((const uint8_t *)p.x8.e.at(ahead.r, t) + (k >> 5));
                }
                ahead.next(p, pair);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int d = 0; d < DEEP; ++d) fetch(d);
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        while (ok && now.tile >= 0) {
#pragma unroll
            for (int d = 0; d < DEEP; ++d) {
                if (now.tile < 0) break;
                asm volatile("cp.async.wait_group %0;" ::"n"(DEEP - 1) : "memory");
                int got = lane == 0 ? (int)wait_bar(empty + 8 * stage, phase ^ 1u, ab, 7) : 0;
                got = __shfl_sync(0xFFFFFFFFu, got, 0);
                if (!got) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint4 q;
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                                 : "r"(slot + (d * 2 + i) * (WIDEN * 16))
                                 : "memory");
                    f32x2 f[4], g[4];
                    held8(make_uint2(q.x, q.y), e[d][i], f);
                    held8(make_uint2(q.z, q.w), e[d][i], g);
                    const uint4 a = narrow8(f), b = narrow8(g);
                    const uint32_t t = t0 + 32 * i, row = out + stage * OPERAND + t * 128, ch = (c & 3) * 2;
                    const bool flip = c >= 4;
                    const uint4 u = flip ? b : a, v = flip ? a : b;
                    const uint32_t cu = flip ? ch + 1 : ch, cv = flip ? ch : ch + 1;
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((cu ^ (t & 7)) << 4)), "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w) : "memory");
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((cv ^ (t & 7)) << 4)), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
                }
                asm volatile("fence.proxy.async.shared::cluster;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    if (even) mbar_arrive(full_b + 8 * stage);
                    else mbar_arrive_remote(full_even + 8 * stage);
                }
                fetch(d);
                now.next(p, pair);
                if (++stage == STAGES) stage = 0, phase ^= 1u;
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else if (warp >= 4) {
        // ---------------- finished tiles: this CTA's 128 rows, warp 4 + i the TMEM lanes 32 i..
        const int i = warp & 3;
        const uint32_t tempty_even = mapa_shared(tempty, 0);
        int it = 0;
        Walk w;
        for (w.start(p, pair); w.tile >= 0; ++it, w.next_tile(p, pair)) {
            const uint32_t acc = it & 1;
            int got = lane == 0 ? (int)wait_bar(tfull + 8 * acc, (it >> 1) & 1, ab, 6) : 0;
            got = __shfl_sync(0xFFFFFFFFu, got, 0);
            if (!got) break;
            tc_fence_after();
            const int local = (int)cta * HALF + i * 32 + lane, n = w.n + local;
            const uint32_t from = tmem + ((uint32_t)(i * 32) << 16) + acc * TILE;
            float *const part = w.part < 0 ? nullptr : p.part + ((size_t)w.part * TILE + local) * TILE;
            char *const row = p.dw.at(w.r, n);
#pragma unroll 1
            for (int col = 0; col < TILE; col += 32) {
                uint32_t v[32];
                tmem_ld32(from + col, v);
                if (part) {
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        *(float4 *)(part + col + 4 * x) = make_float4(__uint_as_float(v[4 * x]), __uint_as_float(v[4 * x + 1]),
                                                                      __uint_as_float(v[4 * x + 2]), __uint_as_float(v[4 * x + 3]));
                } else if (n < p.N) {
                    if (p.f32) store32<true>(p, row, w.k + col, v);
                    else store32<false>(p, row, w.k + col, v);
                }
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

// Tile y of those left over, rows 4 x..: the sum of its parts in the order of their
// tokens.  CLEAR: in a caller's workspace the parts are zeroed once read, because other
// calls keep signal words there.
template <bool CLEAR>
__global__ void __launch_bounds__(256) k_wgrad_join(const Params p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int i = blockIdx.y, per = p.n_tiles * p.k_tiles, tile = p.whole + i, rest = tile % per;
    const int local = blockIdx.x * 4 + (threadIdx.x >> 6), col = (threadIdx.x & 63) * 4;
    const int n = rest / p.k_tiles * TILE + local, k = rest % p.k_tiles * TILE + col;
    const uint64_t from = (uint64_t)i * p.steps, to = from + p.steps, all = (uint64_t)p.left * p.steps;
    // the pairs whose share reaches into [from, to): the last that starts at or before `from`, and on
    int pair = (int)(from * (uint32_t)p.pairs / all);
    while (first_step(p, pair + 1) <= from) ++pair;
    while (pair > 0 && first_step(p, pair) > from) --pair;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (; pair < p.pairs && first_step(p, pair) < to; ++pair) {
        const uint64_t begin = first_step(p, pair);
        if (first_step(p, pair + 1) == begin) continue;             // an empty share
        const int second = begin / p.steps != (uint64_t)i;          // the pair's first part is of the tile before
        float4 *const part = (float4 *)(p.part + ((size_t)(2 * pair + second) * TILE + local) * TILE + col);
        const float4 v = *part;
        s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
        if (CLEAR) *part = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (n >= p.N || k >= p.K) return;
    char *const row = p.dw.at(tile / per, n);
    if (p.f32) {
        float4 *const o = (float4 *)(row + (size_t)k * 4);
        if (p.accumulate) {
            const float4 old = *o;
            s = make_float4(old.x + s.x, old.y + s.y, old.z + s.z, old.w + s.w);
        }
        *o = s;
    } else {
        uint2 *const o = (uint2 *)(row + (size_t)k * 2);
        if (p.accumulate) {
            const uint2 old = *o;
            const f32x2 a = wide2(old.x), b = wide2(old.y);
            s = make_float4(lo(a) + s.x, hi(a) + s.y, lo(b) + s.z, hi(b) + s.w);
        }
        *o = make_uint2(narrow2(f2(s.x, s.y)), narrow2(f2(s.z, s.w)));
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

// dy as [P][T][N] in boxes of 64 channels x 64 tokens, 128-byte swizzle.
static int make_map(CUtensorMap *map, const rc_rows &dy, int P, int T, int N)
{
    auto fn = encode_fn();
    if (!fn) return set_error(RC_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled is not available from the driver");
    const bool one = P == 1 || dy.slot == 0;
    const cuuint64_t dims[3] = {(cuuint64_t)N, (cuuint64_t)T, one ? 1u : (cuuint64_t)P};
    const cuuint64_t strides[2] = {(cuuint64_t)dy.row, one ? (cuuint64_t)dy.row : (cuuint64_t)dy.slot};
    const cuuint32_t box[3] = {64, STEP, 1}, estr[3] = {1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, dy.base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return set_error(RC_ERR_INVALID, "tensor map encoding failed (CUresult %d)", (int)r);
    return RC_OK;
}

// Tiles that fill whole rounds of the pairs are dealt out whole.  The tokens of the rest are
// divided over all pairs where that saves more steps than parts cost: they are written and
// read again, and joined by a second launch.
constexpr uint32_t kPartSteps = 24;

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
    if (!p.left && p.whole < p.pairs) p.pairs = p.whole;
}
static size_t part_bytes(const Params &p) { return p.left ? (size_t)p.pairs * 2 * TILE * TILE * 4 : 0; }

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
    p.wide = !(((uintptr_t)a.x8.q.base | a.x8.q.slot | a.x8.q.row | (size_t)a.K) & 15u);
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
    CUtensorMap map;
    if ((rc_ = make_map(&map, a.dy, a.P, a.T, a.N))) return rc_;
    static OncePerDevice once;
    cudaError_t e = once([] { return cudaFuncSetAttribute(k_wgrad, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM); });
    if (e == cudaSuccess) {
        k_wgrad<<<2 * p.pairs, THREADS, SMEM, st>>>(map, p);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess && p.left) {
        // set up while the tiles are summed; its blocks start when that has ended
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(TILE / 4, (unsigned)p.left);
        cfg.blockDim = dim3(256);
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
