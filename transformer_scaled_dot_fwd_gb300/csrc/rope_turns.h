// Rotary frequencies as fractions of a turn (host).
#pragma once

#include <cmath>
#include <cstdint>

namespace attn {

// w radians a position as a fraction of a turn, modulo one turn, in units of 2^-64;
// positions are whole numbers, so whole turns drop out.  Off by at most one unit for
// |w| < 2^40: 1 / 2 pi and the product w / 2 pi are held as sums of two doubles, whose
// fractional parts are taken exactly and added as integers.  No library calls on the
// GPU's hosts: a call turns up to 64 frequencies (with fmod, ldexp and llround 0.5 us).
inline uint64_t rope_turns(double w) {
    const double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;  // 1 / 2 pi
    const double p = w * hi;
    const double part[2] = {p, std::fma(w, lo, std::fma(w, hi, -p))};
    uint64_t units = 0;
    double rest = 0;
    for (double x : part) {
        const double m = std::fabs(x - std::trunc(x)) * 0x1p64, whole = std::floor(m);
        const uint64_t u = static_cast<uint64_t>(whole);
        units += x < 0 ? 0 - u : u;
        rest += x < 0 ? whole - m : m - whole;
    }
    return units + static_cast<uint64_t>(static_cast<int64_t>(std::floor(rest + 0.5)));
}

}  // namespace attn
