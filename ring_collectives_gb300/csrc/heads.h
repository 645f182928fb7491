// heads.h -- checks of operands in strided heads or rows, and whether two of them
// share bytes (heads.cu; host code only).
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "internal.h"
#include "ringcoll.h"

namespace rc {

// The space of a caller's workspace starts here, behind the status header that
// calls sharing it keep at its start.
constexpr size_t kWsHead = 256;
static_assert(kWsHead >= sizeof(WsHeader), "the header lies in front of the space");

// Checks one operand [P][T][H][D] and gives the strides of extents of 1 a valid value.
int check_heads(rc_heads &h, const char *name, int P, int T, int H, int D);

// Where an operand lies: ranges of `bytes` bytes at h.base + r h.slot + t h.token + i h.head.
// No base: nowhere.
struct Operand {
    const char *name;
    rc_heads h;
    int P, T, H;
    size_t bytes;
};
inline Operand heads_at(const char *name, const rc_heads &h, int P, int T, int H, int D)
{
    return Operand{name, h, P, T, H, (size_t)D * 2};
}
// Checks rows [P][T] of `bytes` bytes each, aligned to `align`, and gives the strides of
// extents of 1 a valid value.  shared: a slot stride of 0 is one operand of all ranks.
int check_rows(rc_rows &r, const char *name, int P, int T, size_t bytes, size_t align, bool shared = false);
// The bytes of N channels and of their groups; and P, T, N of a call on rows.
int check_act8(rc_act8 &a, const char *name, int P, int T, int N, bool shared = false);
int check_row_sizes(int P, int T, int N, int most_channels);
inline Operand rows_at(const char *name, const rc_rows &r, int P, int T, size_t bytes)
{
    return Operand{name, rc_heads{r.base, r.slot, r.row, 0}, P, T, 1, bytes};
}
inline Operand bytes_at(const char *name, const void *p, size_t bytes)
{
    return Operand{name, rc_heads{const_cast<void *>(p), 0, 0, 0}, 1, 1, 1, bytes};
}

// Results may not share bytes with an input, with one another or within
// themselves.  whole[i]: a bit for each input that result i may be as a whole,
// head for head (null: none).
int check_apart(const Operand *results, int nres, const Operand *inputs, int nin, const unsigned *whole = nullptr);

} // namespace rc
