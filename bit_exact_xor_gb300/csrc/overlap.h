// Whether the memory of a call's operands overlaps: what is written may not be
// part of what other threads of the call still read.  Host code only.
#pragma once

#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <utility>

#include "../../include/dcr.h"

namespace dcr {

int set_error(int code, const char* fmt, ...);

// `rows` of `bytes` each, `step` bytes apart (no fewer than `bytes`).
struct Memory {
    uintptr_t at = 0;
    uint64_t rows = 0, bytes = 0, step = 0;
    const char* name = "";
    Memory() = default;
    Memory(const char* name_, const void* p, uint64_t bytes_) : at(uintptr_t(p)), rows(p && bytes_ ? 1 : 0), bytes(bytes_), step(bytes_), name(name_) {}
    Memory(const char* name_, const void* p, uint32_t size, uint64_t rows_, uint64_t cols, uint64_t stride)
        : at(uintptr_t(p)), rows(p && cols ? rows_ : 0), bytes(cols * size), step(stride * size), name(name_)
    {
        if (rows > 1 && step == bytes) bytes *= rows, step = bytes, rows = 1;
    }
    // behind the last byte
    uintptr_t end() const
    {
        const uintptr_t room = ~uintptr_t(0) - at - bytes;
        return rows > 1 && rows - 1 > room / step ? ~uintptr_t(0) : at + (rows - 1) * step + bytes;
    }
    // one of the rows has a byte from lo on that lies below hi
    bool hit(uintptr_t lo, uintptr_t hi) const
    {
        const uint64_t i = lo < at + bytes ? 0 : (lo - at - bytes) / step + 1;     // the first row that ends behind lo
        return i < rows && at + i * step < hi;
    }
};

// Exact, so that matrices side by side in the columns of one buffer do not
// overlap.
inline bool overlap(Memory a, Memory b)
{
    if (a.rows == 0 || b.rows == 0 || a.end() <= b.at || b.end() <= a.at) return false;
    if (a.at > b.at) std::swap(a, b);
    // of rows equally far apart, b's first one meets one of a's if any does
    if (b.rows == 1 || (a.rows > 1 && a.step == b.step)) return a.hit(b.at, b.at + b.bytes);
    if (a.rows > b.rows) std::swap(a, b);
    for (uint64_t i = 0; i < a.rows && a.at + i * a.step < b.end(); ++i)
        if (b.hit(a.at + i * a.step, a.at + i * a.step + a.bytes)) return true;
    return false;
}

// Refuses a call of which something written overlaps anything else.
inline int check_overlap(const char* what, std::initializer_list<Memory> written, std::initializer_list<Memory> read)
{
    for (const Memory* w = written.begin(); w != written.end(); ++w) {
        for (const Memory& r : read)
            if (overlap(*w, r)) return set_error(DCR_ERR_INVALID, "%s: %s overlaps %s", what, w->name, r.name);
        for (const Memory* o = w + 1; o != written.end(); ++o)
            if (overlap(*w, *o)) return set_error(DCR_ERR_INVALID, "%s: %s overlaps %s", what, w->name, o->name);
    }
    return DCR_OK;
}

}  // namespace dcr
