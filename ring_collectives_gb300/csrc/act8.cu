// act8.cu -- activation checkpoints in 8 bits: bf16 rows to signed bytes with a
// power of two for every 32 channels, and back (the format is act8.cuh's).
//
// Bound by memory: 2 bytes of an element on one side, 1 + 1/32 on the other.  Measured:
// 8192 x 4096 to 8 bits 17.5 us and back 16.3 us (5.8 and 6.2 TB/s, 86 and 92 % of the copy
// rate); 65536 x 1792 back 53 us (99 %).  Blocks of 128 threads with one run of channels each:
// with 256 threads and two runs 18.5 and 17.8 us.
#include "act8.cuh"
#include "heads.h"
#include "internal.h"
#include "ringcoll.h"

namespace rc {
namespace a8 {

constexpr int THREADS = 128;

struct Params {
    Rows x;
    Act8 x8;
    Flat f;
};

template <bool PACK, bool WIDE>
__global__ void __launch_bounds__(THREADS) k_act8(const Params p)
{
    const uint64_t first = (uint64_t)blockIdx.x * THREADS;
    const uint32_t row0 = (uint32_t)(first / p.f.lanes.d), rem0 = (uint32_t)(first - (uint64_t)row0 * p.f.lanes.d);
    const Spot s(p.f, row0, rem0, threadIdx.x);
    if (PACK) {
        uint4 w[2];
        get16<WIDE>(p.x, s, w);
        set16<WIDE>(p.x8, s, w);
    } else {
        uint4 q;
        uint32_t e;
        get16<WIDE>(p.x8, s, q, e);
        f32x2 a[4], b[4];
        held8(make_uint2(q.x, q.y), e, a);
        held8(make_uint2(q.z, q.w), e, b);
        set16<WIDE>(p.x, s, narrow8(a), narrow8(b));
    }
}

static int run(const rc_act8_args *args, bool pack, void *stream)
{
    if (!args) return set_error(RC_ERR_INVALID, "null args");
    rc_act8_args a = *args;
    if (a.reserved) return set_error(RC_ERR_INVALID, "reserved is not 0");
    int rc_ = check_row_sizes(a.P, a.T, a.N, 1 << 20);
    if (rc_ || a.T == 0) return rc_;
    if ((rc_ = check_rows(a.x, "x", a.P, a.T, (size_t)a.N * 2, 16)) || (rc_ = check_act8(a.x8, "x8", a.P, a.T, a.N))) return rc_;
    const Operand x = rows_at("x", a.x, a.P, a.T, (size_t)a.N * 2), q = rows_at("x8.q", a.x8.q, a.P, a.T, (size_t)a.N),
                  e = rows_at("x8.e", a.x8.e, a.P, a.T, (size_t)(a.N + 31) / 32);
    const Operand bytes[] = {q, e}, values[] = {x};
    if ((rc_ = pack ? check_apart(bytes, 2, values, 1) : check_apart(values, 1, bytes, 2))) return rc_;
    int sms = 0;
    if ((rc_ = device_sms(&sms))) return rc_;
    const Params p{rows_of(a.x), act8_of(a.x8), Flat::of(a.P, a.T, a.N)};
    const uint64_t blocks = p.f.blocks(THREADS);
    if (blocks > 0x7FFFFFFFull) return set_error(RC_ERR_INVALID, "P*T rows of N=%d channels are too many", a.N);
    const bool wide = a.N % 16 == 0 && wide_of(a.x, 32) && wide_of(a.x8.q, 16);
    const auto kernel = pack ? (wide ? k_act8<true, true> : k_act8<true, false>) : (wide ? k_act8<false, true> : k_act8<false, false>);
    kernel<<<(unsigned)blocks, THREADS, 0, (cudaStream_t)stream>>>(p);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return set_error(RC_ERR_CUDA, "act8 launch: %s", cudaGetErrorString(err));
    return RC_OK;
}

} // namespace a8
} // namespace rc

extern "C" int act8_pack(const rc_act8_args *args, void *stream) { return rc::a8::run(args, true, stream); }

extern "C" int act8_unpack(const rc_act8_args *args, void *stream) { return rc::a8::run(args, false, stream); }
