// ra_rotary.cuh -- the angles of the position rotation, in turns.
//
// Plain integer arithmetic callable from host and device (tests/rotary_probe.cu runs
// it on the CPU).  f / 2 pi is a 64-bit fraction of a turn, p times that modulo 2^64 the
// angle: whole turns fall away exactly.  The fraction has to be right to its last bits,
// since p multiplies its error.  f is m 2^e with a whole m of 24 bits, so the fraction is
// m times those 96 bits of 1 / 2 pi that 2^e brings behind the point (after Payne
// and Hanek), right to 2^-63 of a turn: 1e-9 of a radian at p = 2^29.  The top 32 bits
// of the angle go to fp32, off by 2^-32 of a turn and 2^-25 of half a turn (9.6e-8 of a
// radian): 1e-7 of a radian at most in all.  As a product in 64-bit floating point
// the angle was off by 1.7e-7 for f <= 1 and 7e-4 at f = 10^4, and 64 tokens (32 / 8 heads,
// d = 128) took 3.2 us instead of 3.1; as the sum of three such products 3.45.
#pragma once
#include <cstdint>
#include <cstring>

#include "ra_positions.cuh"

namespace ra {

// The turns of a frequency as a fraction of 2^64.  (Below 2^-73 they are 0, as far
// as any position can tell; from 2^56 on, infinities and NaN among them, any number.)
RA_HD unsigned long long turn_fraction(float f) {
    uint32_t bits;
    memcpy(&bits, &f, 4);
    const int exponent = (int)(bits >> 23) & 255;
    const uint32_t m = (bits & 0x7fffffu) | (exponent > 0 ? 0x800000u : 0u);
    const unsigned __int128 inverse = (unsigned __int128)0x28be60db9391054aull << 64 | 0x7f09d5f47d4d3770ull;      // 2^128 / 2 pi
    const int shift = exponent > 182 ? 0 : 182 - exponent;
    const unsigned long long turns = shift < 128 ? (unsigned long long)((inverse >> shift) * m >> 32) : 0ull;
    return bits >> 31 ? 0ull - turns : turns;
}

// The angle of position p in half turns, in [-1, 1].
RA_HD float half_turns(int p, unsigned long long fraction) {
    const unsigned long long phase = (unsigned long long)(long long)p * fraction;
    return (float)(int)(phase >> 32) * 0x1p-31f;
}

}  // namespace ra
