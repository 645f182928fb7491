// heads.cu -- checks of operands in strided heads or rows, and whether two of them
// share bytes (host code only).
//
// Every call asks, so the usual answer is found with few operations and little
// code: operands whose spans do not meet, and results whose strides nest.  Only
// what that leaves open (heads interleaved in one fused buffer) is looked at
// element by element, in the sense of Meeting below.
#include <algorithm>

#include "heads.h"

namespace rc {

int check_heads(rc_heads &h, const char *name, int P, int T, int H, int D)
{
    if (!h.base) return set_error(RC_ERR_INVALID, "%s is null", name);
    const size_t least = (size_t)D * 2;
    if (H == 1) h.head = least;
    if (T == 1) h.token = least;
    if (P == 1) h.slot = least;
    if (((uintptr_t)h.base | h.slot | h.token | h.head) & 15u)
        return set_error(RC_ERR_INVALID, "%s: base and strides must be multiples of 16 bytes", name);
    if (h.head < least || h.token < least || h.slot < least)
        return set_error(RC_ERR_INVALID, "%s: a stride is below the %zu bytes of a head", name, least);
    if (h.slot >> 40 || h.token >> 40 || h.head >> 32)
        return set_error(RC_ERR_INVALID, "%s: a stride is too large", name);
    return RC_OK;
}

int check_rows(rc_rows &r, const char *name, int P, int T, size_t bytes, size_t align, bool shared)
{
    if (!r.base) return set_error(RC_ERR_INVALID, "%s is null", name);
    const size_t whole = (bytes + align - 1) / align * align;
    if (T <= 1) r.row = whole;
    if (P == 1) r.slot = whole;
    if (((uintptr_t)r.base | r.slot | r.row) & (align - 1))
        return set_error(RC_ERR_INVALID, "%s: base and strides must be multiples of %zu bytes", name, align);
    if (r.row < bytes || (r.slot < bytes && !(shared && r.slot == 0)))
        return set_error(RC_ERR_INVALID, "%s: a stride is below the %zu bytes of a row", name, bytes);
    if (r.slot >> 40 || r.row >> 32) return set_error(RC_ERR_INVALID, "%s: a stride is too large", name);
    return RC_OK;
}

int check_act8(rc_act8 &a, const char *name, int P, int T, int N, bool shared)
{
    if (!a.q.base || !a.e.base) return set_error(RC_ERR_INVALID, "%s: its bytes or exponents are null", name);
    const int rc_ = check_rows(a.q, name, P, T, (size_t)N, 8, shared);
    return rc_ ? rc_ : check_rows(a.e, name, P, T, (size_t)(N + 31) / 32, 1, shared);
}

int check_row_sizes(int P, int T, int N, int most_channels)
{
    if (P < 1 || P > RC_MAX_P) return set_error(RC_ERR_INVALID, "P=%d outside 1..%d", P, RC_MAX_P);
    if (N < 8 || N % 8 || N > most_channels) return set_error(RC_ERR_INVALID, "N=%d is not a multiple of 8 up to %d", N, most_channels);
    if (T < 0 || (long long)P * T >= (1ll << 31) - (1 << 20)) return set_error(RC_ERR_INVALID, "P=%d slots of T=%d rows: not 0 <= P*T < 2^31 - 2^20", P, T);
    return RC_OK;
}

namespace {

typedef __int128 wide;                     // 2^31 tokens at strides up to 2^40

// The bytes [base + sum_i c_i stride_i, + len) for all 0 <= c_i < n_i.  Dimensions of
// extent 1 are left out, the others lie in falling order of strides.
struct Region {
    wide base, len;
    int dims = 0;
    struct {
        wide stride;
        long long n;
    } dim[3];

    explicit Region(const Operand &o) : base((uintptr_t)o.h.base), len(o.bytes)
    {
        add(o.h.slot, o.P);
        add(o.h.token, o.T);
        add(o.h.head, o.H);
    }
    void add(size_t stride, long long n)
    {
        if (n < 2) return;
        int i = dims++;
        for (; i && dim[i - 1].stride < (wide)stride; --i) dim[i] = dim[i - 1];
        dim[i].stride = stride;
        dim[i].n = n;
    }
    bool same(const Region &o) const
    {
        if (base != o.base || len != o.len || dims != o.dims) return false;
        for (int i = 0; i < dims; ++i)
            if (dim[i].stride != o.dim[i].stride || dim[i].n != o.dim[i].n) return false;
        return true;
    }
};

// Looks for two elements, a of A and b of B, whose byte ranges meet: with d = b - a,
//     -len B < d < len A,   d = (base B - base A) + sum c_i s_i,  lo_i <= c_i <= hi_i,
// where dimensions of equal stride count as one (c their difference).  Strides are
// taken in falling order, and of each only the c that the smaller ones can still make
// up for: one or two in nested layouts.  Layouts that need more than kSteps choices
// to decide count as apart; overlap is refused where it is found.
class Meeting {
    struct Dim {
        wide s, lo, hi;
    } d[6];
    wide rest_lo[7], rest_hi[7], above, below, start;   // what dimensions i.. can add; the open range of d
    int n = 0, steps = 0;
    bool self;
    static constexpr int kSteps = 4096;

    void add(wide s, long long lo, long long hi)
    {
        for (int i = 0; i < n; ++i)
            if (d[i].s == s) {
                d[i].lo += lo;
                d[i].hi += hi;
                return;
            }
        int i = n++;
        for (; i && d[i - 1].s < s; --i) d[i] = d[i - 1];
        d[i] = Dim{s, lo, hi};
    }
    static wide floor_div(wide a, wide b) { return a / b - (a % b < 0); }
    bool look(int i, wide at, bool moved)
    {
        if (i == n) return (moved || !self) && at > above && at < below;
        // above < at + c s + [rest_lo, rest_hi] < below
        const wide lo = std::max(d[i].lo, floor_div(above - at - rest_hi[i + 1], d[i].s) + 1);
        const wide hi = std::min(d[i].hi, -floor_div(at + rest_lo[i + 1] - below, d[i].s) - 1);
        for (wide c = lo; c <= hi; ++c) {
            if (++steps > kSteps) return false;
            if (look(i + 1, at + c * d[i].s, moved || c != 0)) return true;
        }
        return false;
    }

public:
    // self: two different elements of one operand (a is b).
    Meeting(const Region &a, const Region &b, bool self_) : self(self_)
    {
        for (int i = 0; i < a.dims; ++i) add(a.dim[i].stride, 1 - a.dim[i].n, 0);
        for (int i = 0; i < b.dims; ++i) add(b.dim[i].stride, 0, b.dim[i].n - 1);
        rest_lo[n] = rest_hi[n] = 0;
        for (int i = n; i--;) {
            rest_lo[i] = rest_lo[i + 1] + d[i].lo * d[i].s;
            rest_hi[i] = rest_hi[i + 1] + d[i].hi * d[i].s;
        }
        above = -b.len;
        below = a.len;
        start = b.base - a.base;
    }
    bool found() { return look(0, start, false); }
};

// Operands whose spans meet share bytes; may_be_one: being the same heads is allowed.
__attribute__((noinline, cold)) bool share(const Operand &x, const Operand &y, bool may_be_one)
{
    const Region a(x), b(y);
    return !(may_be_one && a.same(b)) && Meeting(a, b, false).found();
}

// Two heads of one operand share bytes.
__attribute__((noinline, cold)) bool folded(const Operand &x)
{
    const Region a(x);
    for (int i = 1; i < a.dims; ++i)
        if (a.dim[i].stride == a.dim[i - 1].stride) return true;   // (1, 0) and (0, 1) are one place
    return Meeting(a, a, true).found();
}

// The first byte behind an operand.  In binary64: exact for real addresses (below
// 2^53), and strides that would pass 64 bits stay far above them.
double end_of(const Operand &o)
{
    return (double)(uintptr_t)o.h.base + (double)o.bytes + (o.P - 1) * (double)o.h.slot + (o.T - 1) * (double)o.h.token +
           (o.H - 1) * (double)o.h.head;
}

// Heads in a token (or the token's slot), and those in a slot or a token, as in
// [P][T][H][D] and in fused activations [T][P][H][D].
bool nested(const Operand &o)
{
    const double heads = o.bytes + (o.H - 1) * (double)o.h.head, token = o.T > 1 ? o.h.token : 1e30,
                 slot = o.P > 1 ? o.h.slot : 1e30;
    return (o.H == 1 || o.h.head >= o.bytes) && std::min(token, slot) >= heads &&
           (slot >= heads + (o.T - 1) * (double)o.h.token || token >= heads + (o.P - 1) * (double)o.h.slot);
}

} // namespace

int check_apart(const Operand *results, int nres, const Operand *inputs, int nin, const unsigned *whole)
{
    constexpr int kMost = 20;
    double ends[kMost];                    // of the results, then of the inputs
    for (int i = 0; i < nres + nin; ++i) ends[i] = end_of(i < nres ? results[i] : inputs[i - nres]);
    for (int i = 0; i < nres; ++i) {
        const Operand &r = results[i];
        if (!r.h.base) continue;
        if (!nested(r) && folded(r)) return set_error(RC_ERR_INVALID, "%s: its heads overlap", r.name);
        const double first = (double)(uintptr_t)r.h.base;
        for (int j = i + 1; j < nres + nin; ++j) {
            const Operand &o = j < nres ? results[j] : inputs[j - nres];
            if (ends[j] <= first || ends[i] <= (double)(uintptr_t)o.h.base || !o.h.base) continue;
            if (share(r, o, j >= nres && whole && whole[i] >> (j - nres) & 1u))
                return set_error(RC_ERR_INVALID, "%s and %s overlap", r.name, o.name);
        }
    }
    return RC_OK;
}

} // namespace rc
