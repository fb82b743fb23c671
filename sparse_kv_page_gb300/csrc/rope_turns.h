// rope_turns.h - a rotary pair's angle per position in turns (host code).
#pragma once

#include <cmath>
#include <cstdint>

namespace locks {

// x / (2 pi) as a fraction of a turn in units of 2^-64, whole turns dropped. The quotient is
// formed as a double-double (1 / (2 pi) to 106 bits), so its fraction is good to half such a
// unit for any |x| up to thousands of radians per position. Formed for |x| and turned round
// (modulo 2^64) where x is negative: 1 - p of a small p would lose p's last bits.
inline uint64_t turn_fraction(double x) {
    constexpr double kHi = 0.15915494309189535, kLo = -9.8393378335251835e-18;   // 1 / (2 pi)
    const double size = std::fabs(x), p = size * kHi;
    const double err = std::fma(size, kHi, -p) + size * kLo;
    const double hi = p - std::floor(p);                    // exact: p >= 0, both multiples of p's last bit
    // hi in [0, 1) and err tiny: to 2^-64, in two exact 32-bit steps
    const double a = std::floor(hi * 4294967296.0);
    const double rest = (hi * 4294967296.0 - a) + err * 4294967296.0;   // in units of 2^-32
    const double b = std::nearbyint(rest * 4294967296.0);   // may be negative or 2^32: the sum wraps
    const uint64_t turns = (static_cast<uint64_t>(a) << 32) + static_cast<uint64_t>(static_cast<int64_t>(b));
    return x < 0.0 ? 0 - turns : turns;
}

}  // namespace locks
