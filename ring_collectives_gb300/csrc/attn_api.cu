// attn_api.cu -- the C entry points of the attention operators: argument
// checks, tensor maps, the form and split of a launch, partial-result space.
#include <cudaTypedefs.h>

#include <climits>
#include <cmath>
#include <mutex>

#include "attn.cuh"
#include "heads.h"

namespace rc {
namespace attn {

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &qr) ==
                cudaSuccess &&
            qr == cudaDriverEntryPointSuccess)
            fn = (PFN_cuTensorMapEncodeTiled_v12000)f;
    });
    return fn;
}

static int encode(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                  const cuuint32_t *box)
{
    auto fn = encode_fn();
    if (!fn) return set_error(RC_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled is not available from the driver");
    cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(base), dims,
                          strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return set_error(RC_ERR_INVALID, "tensor map encoding failed (CUresult %d)", (int)r);
    return RC_OK;
}

// Query-side heads as [P][Hkv][T][G][D], a box of box_tokens tokens of one
// group.  Columns past D and tokens past T read as zero.
int head_map5(CUtensorMap *map, const rc_heads &h, int P, int T, int Hkv, int G, int D, int box_tokens)
{
    const cuuint64_t dims[5] = {(cuuint64_t)D, (cuuint64_t)G, (cuuint64_t)T, (cuuint64_t)Hkv, (cuuint64_t)P};
    const cuuint64_t strides[4] = {h.head, h.token, (cuuint64_t)G * h.head, h.slot};
    const cuuint32_t box[5] = {64, (cuuint32_t)G, (cuuint32_t)box_tokens, 1, 1};
    return encode(map, h.base, 5, dims, strides, box);
}

// Key-side heads as [P][Hkv][T][D], a box of 128 tokens.
int head_map4(CUtensorMap *map, const rc_heads &h, int P, int T, int Hkv, int D)
{
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)T, (cuuint64_t)Hkv, (cuuint64_t)P};
    const cuuint64_t strides[3] = {h.token, h.head, h.slot};
    const cuuint32_t box[4] = {64, KT, 1, 1};
    return encode(map, h.base, 4, dims, strides, box);
}

// Tokens: the kernels count up to a few tiles past them in 32 bits.
constexpr int kMostTokens = INT_MAX - (1 << 20);

// An upper bound of the row or key tiles of all sequences, ranks and key heads: one
// for every `tile` tokens and one more for each sequence that has any.
static long long most_tiles(const rc_attn_args &a, int tokens, int tile)
{
    return (long long)a.P * a.Hkv * (tokens / tile + (long long)(a.B < tokens ? a.B : tokens));
}

static int check_sizes(const rc_attn_args &a)
{
    if (a.P < 1 || a.P > RC_MAX_P) return set_error(RC_ERR_INVALID, "P=%d outside 1..%d", a.P, RC_MAX_P);
    if (a.B < 1 || a.Tq < 0 || a.Tk < 0) return set_error(RC_ERR_INVALID, "need B >= 1, Tq >= 0 and Tk >= 0 (got %d, %d, %d)", a.B, a.Tq, a.Tk);
    if (a.Hq < 1 || a.Hkv < 1 || a.Hq % a.Hkv || a.Hq / a.Hkv > KT || a.Hq > 65536)
        return set_error(RC_ERR_INVALID, "need Hq a multiple of Hkv and Hq/Hkv <= %d (got %d, %d)", KT, a.Hq, a.Hkv);
    if (a.Tq > kMostTokens || a.Tk > kMostTokens)
        return set_error(RC_ERR_INVALID, "Tq=%d or Tk=%d is above %d", a.Tq, a.Tk, kMostTokens);
    if (most_tiles(a, a.Tq, KT / (a.Hq / a.Hkv)) > kMostTokens || most_tiles(a, a.Tk, KT) > kMostTokens)
        return set_error(RC_ERR_INVALID, "more than %d tiles over all sequences, ranks and key heads", kMostTokens);
    if (a.D < 8 || a.D > 128 || a.D % 8) return set_error(RC_ERR_INVALID, "D=%d is not a multiple of 8 up to 128", a.D);
    if (!(a.scale > 0.f) || !std::isfinite(a.scale)) return set_error(RC_ERR_INVALID, "scale must be positive and finite");
    if (a.causal != 0 && a.causal != 1) return set_error(RC_ERR_INVALID, "causal must be 0 or 1");
    if (a.reserved) return set_error(RC_ERR_INVALID, "reserved must be 0");
    return RC_OK;
}

static Strided strided(const rc_heads &h) { return Strided{(char *)h.base, h.slot, h.token, h.head}; }

static void fill(Params &p, const rc_attn_args &a)
{
    p.lse = a.lse;
    p.cu_q = a.cu_q;
    p.cu_k = a.cu_k;
    p.used_k = a.used_k;
    p.P = a.P;
    p.B = a.B;
    p.Tq = a.Tq;
    p.Tk = a.Tk;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.D = a.D;
    p.causal = a.causal;
    p.scale = a.scale;
    p.TT = KT / p.G;
}

// The form of a forward launch and the bytes of its partial results.
struct FwdPlan {
    bool split;
    size_t units, rows, bytes;
};

// SPLIT when the queries of a sequence fill at most one row tile on average.
// Measured, SPLIT / PAIR: 1 sequence x 8 heads on 16384 keys, 4 rows 20.6 / 22.6 us,
// 128 rows 27.1 / 28.6 us, 160 rows 33.9 / 29.1 us; 64 sequences x 8 heads on 2048
// keys, 4 rows 102 / 109 us, 160 rows 145 / 124 us.
static FwdPlan plan_fwd(Params &p, int sms)
{
    FwdPlan f{};
    f.split = (long long)p.Tq * p.G <= (long long)KT * p.B;
    p.sms = sms;
    p.TPU = f.split ? p.TT : 2 * p.TT;
    const long long HP = (long long)p.P * p.Hkv, rows = (p.Tq + p.TPU - 1) / p.TPU;
    p.may_split = (rows > p.B ? rows : p.B) * HP < (f.split ? 4ll : 2ll) * sms;   // units, about
    if ((p.Tk + KT - 1) / KT <= kWholeTiles) p.may_split = 0;
    p.part_rows = p.G * (p.TT < p.Tq ? p.TT : p.Tq);
    if (p.may_split) {
        long long n0 = p.Tq / p.TPU + p.B;     // row tiles (pairs), at most
        if (n0 > p.Tq) n0 = p.Tq;
        f.units = (size_t)(n0 * HP + split_units(sms));
        p.max_units = (int)f.units;
        const size_t DP = p.D <= 64 ? 64 : 128;
        f.rows = (f.split ? 1 : 2) * f.units * (size_t)p.part_rows;
        f.bytes = f.rows * (DP + 1) * 4;
    }
    return f;
}

// The status header and `bytes` of space for intermediate results.  In a caller's
// workspace that space is where calls that signal keep words which they compare with the
// epoch in the header, and almost any other number there reads as a signal given.  So it
// is left zeroed (p.clear): a word that no launch has signalled yet.
static int take_workspace(const rc_attn_args &a, size_t bytes, Params &p, char **scratch)
{
    uint32_t *unused = nullptr;
    int sms = 0;
    if (a.workspace && ((uintptr_t)a.workspace & 255u))
        return set_error(RC_ERR_INVALID, "workspace must be 256-byte aligned");
    int rc_ = prepare_workspace_ext(a.workspace, a.ws_bytes, a.workspace ? (kWsHead - sizeof(WsHeader) + bytes + 3) / 4 : 0,
                                    &p.hdr, &unused, &sms, &p.timeout_ns);
    if (rc_) return rc_;
    if (a.workspace) {
        *scratch = (char *)a.workspace + kWsHead;
        p.clear = 1;
        return RC_OK;
    }
    void *s = nullptr;
    if (bytes && (rc_ = prepare_scratch(bytes, &s))) return rc_;
    *scratch = (char *)s;
    return RC_OK;
}

// Where operands lie; without tokens (and for no lse) nowhere.
static Operand of_queries(const char *name, const rc_heads &h, const rc_attn_args &a)
{
    return heads_at(name, a.Tq ? h : rc_heads{}, a.P, a.Tq, a.Hq, a.D);
}
static Operand of_keys(const char *name, const rc_heads &h, const rc_attn_args &a)
{
    return heads_at(name, a.Tk ? h : rc_heads{}, a.P, a.Tk, a.Hkv, a.D);
}
static Operand of_lse(const rc_attn_args &a) { return bytes_at("lse", a.Tq ? a.lse : nullptr, (size_t)a.P * a.Tq * a.Hq * 4); }

static int run_fwd(const rc_attn_args *args, void *stream)
{
    if (!args) return set_error(RC_ERR_INVALID, "null args");
    rc_attn_args a = *args;
    int rc_ = check_sizes(a);
    if (rc_) return rc_;
    if (a.Tq == 0) return RC_OK;
    if ((rc_ = check_heads(a.q, "q", a.P, a.Tq, a.Hq, a.D)) || (rc_ = check_heads(a.out, "out", a.P, a.Tq, a.Hq, a.D)))
        return rc_;
    if (a.Tk && ((rc_ = check_heads(a.k, "k", a.P, a.Tk, a.Hkv, a.D)) || (rc_ = check_heads(a.v, "v", a.P, a.Tk, a.Hkv, a.D))))
        return rc_;
    if (!a.cu_q || !a.cu_k) return set_error(RC_ERR_INVALID, "cu_q or cu_k is null");
    const Operand res[] = {of_queries("out", a.out, a), of_lse(a)};
    const Operand in[] = {of_queries("q", a.q, a), of_keys("k", a.k, a), of_keys("v", a.v, a)};
    if ((rc_ = check_apart(res, 2, in, 3))) return rc_;
    int sms = 0;
    if ((rc_ = device_sms(&sms))) return rc_;
    Params p{};
    fill(p, a);
    const FwdPlan f = plan_fwd(p, sms);
    char *scratch = nullptr;
    if ((rc_ = take_workspace(a, f.bytes, p, &scratch))) return rc_;
    p.part_o = (float *)scratch;
    p.part_lse = (float *)(scratch + f.rows * (p.D <= 64 ? 64 : 128) * 4);
    p.out = strided(a.out);
    p.out32 = !(((uintptr_t)a.out.base | a.out.slot | a.out.token | a.out.head) & 31u) && a.D % 16 == 0;
    p.v = (const char *)a.v.base;
    p.v_slot = a.v.slot;
    p.v_token = a.v.token;
    p.v_head = a.v.head;
    CUtensorMap mq, mk, mv;
    if ((rc_ = head_map5(&mq, a.q, a.P, a.Tq, a.Hkv, p.G, a.D, p.TT))) return rc_;
    if (a.Tk) {
        if ((rc_ = head_map4(&mk, a.k, a.P, a.Tk, a.Hkv, a.D)) || (rc_ = head_map4(&mv, a.v, a.P, a.Tk, a.Hkv, a.D)))
            return rc_;
    } else {
        mk = mv = mq;   // no key exists, so neither is read
    }
    const cudaError_t e = launch_attn_fwd(p, mq, mk, mv, f.split, (cudaStream_t)stream);
    if (e != cudaSuccess) return set_error(RC_ERR_CUDA, "attn_fwd launch: %s", cudaGetErrorString(e));
    return RC_OK;
}

static size_t delta_bytes(const rc_attn_args &a) { return (size_t)a.P * a.Tq * a.Hq * 4; }

static int run_bwd(const rc_attn_args *args, void *stream)
{
    if (!args) return set_error(RC_ERR_INVALID, "null args");
    rc_attn_args a = *args;
    int rc_ = check_sizes(a);
    if (rc_) return rc_;
    if (a.Tq == 0 && a.Tk == 0) return RC_OK;
    if (a.Tq && ((rc_ = check_heads(a.q, "q", a.P, a.Tq, a.Hq, a.D)) ||
                 (rc_ = check_heads(a.out, "out", a.P, a.Tq, a.Hq, a.D)) ||
                 (rc_ = check_heads(a.dout, "dout", a.P, a.Tq, a.Hq, a.D)) ||
                 (rc_ = check_heads(a.dq, "dq", a.P, a.Tq, a.Hq, a.D))))
        return rc_;
    if (a.Tk && ((rc_ = check_heads(a.k, "k", a.P, a.Tk, a.Hkv, a.D)) ||
                 (rc_ = check_heads(a.v, "v", a.P, a.Tk, a.Hkv, a.D)) ||
                 (rc_ = check_heads(a.dk, "dk", a.P, a.Tk, a.Hkv, a.D)) ||
                 (rc_ = check_heads(a.dv, "dv", a.P, a.Tk, a.Hkv, a.D))))
        return rc_;
    if (!a.cu_q || !a.cu_k) return set_error(RC_ERR_INVALID, "cu_q or cu_k is null");
    if (a.Tq && !a.lse) return set_error(RC_ERR_INVALID, "lse is null");
    const Operand res[] = {of_queries("dq", a.dq, a), of_keys("dk", a.dk, a), of_keys("dv", a.dv, a)};
    const Operand in[] = {of_queries("q", a.q, a),     of_keys("k", a.k, a),          of_keys("v", a.v, a),
                          of_queries("out", a.out, a), of_queries("dout", a.dout, a), of_lse(a)};
    if ((rc_ = check_apart(res, 3, in, 6))) return rc_;
    Params p{};
    fill(p, a);
    if ((rc_ = device_sms(&p.sms))) return rc_;
    char *scratch = nullptr;
    if ((rc_ = take_workspace(a, delta_bytes(a), p, &scratch))) return rc_;
    p.delta = (float *)scratch;
    p.o = (const char *)a.out.base;
    p.o_slot = a.out.slot;
    p.o_token = a.out.token;
    p.o_head = a.out.head;
    p.dout = strided(a.dout);
    p.dq = strided(a.dq);
    p.dk = strided(a.dk);
    p.dv = strided(a.dv);
    CUtensorMap mq{}, mdo{}, mk{}, mv{};
    if (a.Tq && ((rc_ = head_map5(&mq, a.q, a.P, a.Tq, a.Hkv, p.G, a.D, p.TT)) ||
                 (rc_ = head_map5(&mdo, a.dout, a.P, a.Tq, a.Hkv, p.G, a.D, p.TT))))
        return rc_;
    if (a.Tk && ((rc_ = head_map4(&mk, a.k, a.P, a.Tk, a.Hkv, a.D)) || (rc_ = head_map4(&mv, a.v, a.P, a.Tk, a.Hkv, a.D))))
        return rc_;
    if (!a.Tq) mq = mdo = mk;   // without queries (or keys) no tile of theirs is read
    if (!a.Tk) mk = mv = mq;
    cudaError_t e = launch_attn_bwd(p, mq, mdo, mk, mv, (cudaStream_t)stream);
    if (e == cudaSuccess && p.clear && a.Tq) e = cudaMemsetAsync(p.delta, 0, delta_bytes(a), (cudaStream_t)stream);
    if (e != cudaSuccess) return set_error(RC_ERR_CUDA, "attn_bwd launch: %s", cudaGetErrorString(e));
    return RC_OK;
}

} // namespace attn
} // namespace rc

extern "C" int attn_bwd(const rc_attn_args *args, void *stream) { return rc::attn::run_bwd(args, stream); }

extern "C" size_t attn_bwd_workspace_bytes(const rc_attn_args *args)
{
    using namespace rc::attn;
    int sms = 0;
    if (!args || check_sizes(*args) || rc::device_sms(&sms)) return 0;
    return rc::kWsHead + delta_bytes(*args);
}

extern "C" int attn_fwd(const rc_attn_args *args, void *stream) { return rc::attn::run_fwd(args, stream); }

extern "C" size_t attn_fwd_workspace_bytes(const rc_attn_args *args)
{
    using namespace rc::attn;
    int sms = 0;
    if (!args || check_sizes(*args) || rc::device_sms(&sms)) return 0;
    Params p{};
    fill(p, *args);
    return rc::kWsHead + plan_fwd(p, sms).bytes;
}
