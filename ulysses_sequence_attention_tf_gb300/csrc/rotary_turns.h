// rotary_turns.h -- a frequency in turns, exact to 64 bits behind the point.  Host code.
#pragma once

#include <cmath>
#include <cstdint>

namespace tfu {

// Frequencies, in radians a position, that turn_fraction takes.
constexpr double kMostFrequency = 0x1p60;

// frequency / 2 pi modulo 1, as the nearest multiple of 2^-64.  The frequency is a whole number m < 2^53 times a power of two, so the
// product of m with 1 / 2 pi's first 128 binary places is exact in 181 bits; what these places leave out, less than 2^-128,
// is below 2^-68 of a turn for the largest frequency.  A negative one is the other's complement, exact modulo a turn.
inline uint64_t turn_fraction(double frequency) {
    int e;
    const uint64_t m = uint64_t(std::ldexp(std::frexp(std::fabs(frequency), &e), 53));
    e -= 53;  // |frequency| = m 2^e, e <= 8
    // m / 2 pi = p 2^-128, p in three words from the lowest on
    constexpr uint64_t kHigh = 0x28be60db9391054aull, kLow = 0x7f09d5f47d4d3770ull;  // 1 / 2 pi
    const unsigned __int128 low = (unsigned __int128)m * kLow, high = (unsigned __int128)m * kHigh + uint64_t(low >> 64);
    const uint64_t p[4] = {uint64_t(low), uint64_t(high), uint64_t(high >> 64), 0};
    // p 2^(e - 128) in units of 2^-64: p shifted right by 64 - e, of which 64 bits are below the point of p's middle word
    const int shift = 64 - e;
    if (shift > 191) return 0;
    auto bits = [&](int from) {  // 64 of p's bits from this one on
        const int word = from / 64, by = from % 64;
        const uint64_t rest = word < 3 && by ? p[word + 1] << (64 - by) : 0;
        return (p[word] >> by) | rest;
    };
    const uint64_t turn = bits(shift) + (bits(shift - 1) & 1u);
    return frequency < 0 ? ~turn + 1 : turn;
}

}  // namespace tfu
