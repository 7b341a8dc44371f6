// ra_args.h -- what the entry points' checks of arguments share.
#pragma once

#include <cstdio>

#include "ra_internal.h"

namespace ra {

inline int refuse(int code, const char *msg) { return set_last_error(code, msg); }

template <typename... A>
int refuse(int code, const char *fmt, A... a)
{
    char msg[256];
    snprintf(msg, sizeof(msg), fmt, a...);
    return set_last_error(code, msg);
}

inline bool is_aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline bool overlap(const void *a, size_t an, const void *b, size_t bn)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bn && y < x + an;
}

} // namespace ra
