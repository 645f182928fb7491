// heads.h -- checks of head-strided operands, and whether two of them share
// bytes (host code only).
#pragma once
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "internal.h"
#include "ringcoll.h"

namespace rc {

// The space of a caller's workspace starts here, behind the status header that
// calls sharing it keep at its start.
constexpr size_t kWsHead = 256;
static_assert(kWsHead >= sizeof(WsHeader), "the header lies in front of the space");

// Checks one operand [P][T][H][D] and gives the strides of extents of 1 a valid value.
inline int check_heads(rc_heads &h, const char *name, int P, int T, int H, int D)
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

// The bytes of an operand: [base + sum_i c_i stride_i, + len) for all 0 <= c_i < n_i.
// Dimensions of extent 1 are left out, the others lie in falling order of strides.
struct Region {
    typedef __int128 wide;               // 2^31 tokens at strides up to 2^40
    const char *name = nullptr;
    uintptr_t base = 0;
    size_t len = 0;
    int dims = 0;
    struct {
        size_t stride;
        long long n;
    } dim[3];
    wide end = 0;

    Region() = default;
    Region(const char *name_, const void *p, size_t bytes) : name(name_), base((uintptr_t)p), len(bytes), end((wide)base + bytes) {}
    Region(const char *name_, const rc_heads &h, int P, int T, int H, int D) : Region(name_, h.base, (size_t)D * 2)
    {
        add(h.slot, P);
        add(h.token, T);
        add(h.head, H);
    }
    void add(size_t stride, long long n)
    {
        if (n < 2) return;
        int i = dims++;
        for (; i && dim[i - 1].stride < stride; --i) dim[i] = dim[i - 1];
        dim[i].stride = stride;
        dim[i].n = n;
        end += (wide)stride * (n - 1);
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
    typedef Region::wide wide;
    struct Dim {
        wide s, lo, hi;
    } d[6];
    wide rest_lo[7], rest_hi[7], above, below;    // what dimensions i.. can add; the open range of d
    int n = 0, steps = 0;
    bool self;
    static constexpr int kSteps = 4096;

    void add(size_t s, long long lo, long long hi)
    {
        for (int i = 0; i < n; ++i)
            if (d[i].s == (wide)s) {
                d[i].lo += lo;
                d[i].hi += hi;
                return;
            }
        int i = n++;
        for (; i && d[i - 1].s < (wide)s; --i) d[i] = d[i - 1];
        d[i] = Dim{(wide)s, lo, hi};
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
        above = -(wide)b.len;
        below = (wide)a.len;
        start = (wide)b.base - (wide)a.base;
    }
    bool found() { return look(0, start, false); }

private:
    wide start;
};

inline bool overlap(const Region &a, const Region &b)
{
    if (a.end <= (Region::wide)b.base || b.end <= (Region::wide)a.base) return false;
    return Meeting(a, b, false).found();
}

// Two heads of one operand share bytes.
inline bool folded(const Region &a)
{
    for (int i = 1; i < a.dims; ++i)
        if (a.dim[i].stride == a.dim[i - 1].stride) return true;   // (1, 0) and (0, 1) are one place
    Region::wide inner = a.len;
    bool nested = true;
    for (int i = a.dims; i-- && nested;) {
        nested = (Region::wide)a.dim[i].stride >= inner;
        inner += (Region::wide)a.dim[i].stride * (a.dim[i].n - 1);
    }
    return !nested && Meeting(a, a, true).found();
}

// Results `out` may not share bytes with an input, with one another or within
// themselves.  in_place: a result may be an input as a whole, head for head.
template <int NOUT, int NIN>
inline int check_apart(const Region (&out)[NOUT], const Region (&in)[NIN], bool (*in_place)(int out, int in) = nullptr)
{
    for (int i = 0; i < NOUT; ++i) {
        if (!out[i].base) continue;
        if (folded(out[i])) return set_error(RC_ERR_INVALID, "%s: its heads overlap", out[i].name);
        for (int j = 0; j < i; ++j)
            if (out[j].base && overlap(out[i], out[j]))
                return set_error(RC_ERR_INVALID, "%s and %s overlap", out[j].name, out[i].name);
        for (int j = 0; j < NIN; ++j) {
            if (!in[j].base || (in_place && in_place(i, j) && out[i].same(in[j]))) continue;
            if (overlap(out[i], in[j])) return set_error(RC_ERR_INVALID, "%s overlaps %s", out[i].name, in[j].name);
        }
    }
    return RC_OK;
}

} // namespace rc
