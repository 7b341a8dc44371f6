// ra_wide4.cuh -- e2m1 codes of a 4-bit cache widened to e4m3.
//
// Values are summed over tokens by products that take one power of two for a
// token, but a block of 32 codes has one of its own.  With the largest of a row's
// bytes as the row's, e, a code becomes the e4m3 code of code * 2^(6 - k),
// k = e - byte: at most 384, exact for k up to 14 (half a step of 2^-10, 2^-17 of
// the row's largest value, at the most below), and the row stands at 2^(e - 6).
// The eight magnitudes of a k are eight bytes, so that one byte permute with the
// codes as its selector widens four of them: nine integer instructions for eight
// codes with their signs, and with loads, stores and the table's entry some 50 for
// 32.
#pragma once

#include "ra_rows.cuh"

namespace ra {

// Entry k: the magnitudes' codes at 2^(6 - k), zeros from some k on; the last: a
// block without a value (a row's largest byte is below 255, so no k is that).
// From the first token on that some row of queries does not see, such blocks are zeros,
// as a product would carry their NaN to it; rows that do see them get theirs at the
// end, by the first of those tokens with such a block.
constexpr int kWide4Entries = 256, kWide4Nan = 255; // (254: zeros)
constexpr int kWide4Up = 6; // a row's byte is its largest less this, 0 at the least
constexpr int kNoToken = 0x7fffffff;

// Notes a token whose block of V has no value: `first`, of the block, in shared memory.
__device__ __forceinline__ void note_without(uint32_t first, int token)
{
    asm volatile("red.shared.min.s32 [%0], %1;" ::"r"(first), "r"(token) : "memory");
}

// The same of a row's blocks that have a bit set in their byte of `none`; end: behind
// the last token.  Rare, so kept out of the loop's code.
static __device__ __noinline__ void note_row(uint32_t firsts, uint32_t none, bool half, int token, int end)
{
    for (int b = 0; b < 4; ++b) {
        const int t = token + (half ? b >> 1 : 0);
        if ((none >> (8 * b) & 1u) && t < end) note_without(firsts + (half ? b & 1 : b) * 4, t);
    }
}

__device__ __forceinline__ void wide4_fill(uint2 *table, int k)
{
    const float s = k > 100 ? 0.f : __uint_as_float((uint32_t)(127 + kWide4Up - k) << 23);
    table[k] = k == kWide4Nan ? make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu)
                              : make_uint2(e4m3x4(0.f, 0.5f * s, s, 1.5f * s), e4m3x4(2.f * s, 3.f * s, 4.f * s, 6.f * s));
}

// From a row's scale bytes (four blocks, or two of each of two tokens: HALF) its
// byte -- at least kWide4Up, and not of blocks without a value -- and, as bytes, the
// blocks' entries.  token: the row's (first); from token `edge` to below `end` blocks
// without a value are zeros, and noted in `firsts`.
template <bool HALF>
__device__ __forceinline__ uint32_t wide4_rows(uint32_t w, uint32_t *top, uint32_t firsts, int token, int edge, int end)
{
    auto tops = [&](uint32_t x) {
        const uint32_t lo = max(x & 0xffu, x >> 8 & 0xffu), hi = max(x >> 16 & 0xffu, x >> 24);
        top[0] = max(HALF ? lo : max(lo, hi), (uint32_t)kWide4Up);
        top[1] = HALF ? max(hi, (uint32_t)kWide4Up) : top[0];
    };
    // (no byte of the difference borrows: a row's byte is none of its blocks' less)
    auto entries = [&](uint32_t x) { return top[0] * (HALF ? 0x0101u : 0x01010101u) + (HALF ? top[1] * 0x01010000u : 0u) - x; };
    tops(w);
    if (max(top[0], top[1]) < 255u) return entries(w);
    const uint32_t none = __vcmpeq4(w, 0xffffffffu); // rare
    tops(w & ~none);
    const uint32_t zero = HALF ? (token >= edge ? 0x0101u : 0u) | (token + 1 >= edge ? 0x01010000u : 0u) : token >= edge ? 0x01010101u : 0u;
    if (none & zero) note_row(firsts, none & zero, HALF, token, end); // (255 becomes 254)
    return (entries(w & ~none) & ~none) | (none & ~zero);
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel)
{
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}

// Eight codes, the first in the lowest four bits, as eight bytes.
__device__ __forceinline__ uint2 wide4(uint32_t w, const uint2 &t)
{
    const uint32_t m = w & 0x77777777u, s = w << 4; // signs: bit 7 of bytes of s and of w in turn
    return make_uint2(prmt(t.x, t.y, m) | (prmt(s, w, 0x5140u) & 0x80808080u),
                      prmt(t.x, t.y, m >> 16) | (prmt(s, w, 0x7362u) & 0x80808080u));
}

} // namespace ra
