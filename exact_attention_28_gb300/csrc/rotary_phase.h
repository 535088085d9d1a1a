// Frequencies of the rotary positions as fractions of a turn, on the host.
#pragma once

#include <cmath>
#include <cstdint>

namespace fa {

// f / (2 pi) turns modulo 1, in units of 2^-64 of a turn, to the nearest: off
// by at most 2^-65 turns (and f 2^-160) for any finite f.
//
// 1 / (2 pi) is the sum of three doubles.  The first two products are taken as
// two doubles each (the second holds what the first rounds away), every part
// modulo 1 (exact, in [-1/2, 1/2]) and as an integer in units of 2^-96, so that
// the sum of all is rounded once.  The remainder is a call, not x minus
// nearbyint(x): a compiler may fuse that difference with the product in x.
inline uint64_t rotary_phase(double f) {
    constexpr double kTurn[3] = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57, -0x1.6447e493ad4cep-111};
    const auto fixed = [](double x) {
        const double y = std::ldexp(std::remainder(x, 1.0), 48), whole = std::trunc(y);
        return static_cast<__int128>(whole) * (int64_t{1} << 48) + std::llrint(std::ldexp(y - whole, 48));
    };
    __int128 sum = fixed(f * kTurn[2]);
    for (int i = 0; i < 2; ++i) {
        const double product = f * kTurn[i];
        sum += fixed(product) + fixed(std::fma(f, kTurn[i], -product));
    }
    return static_cast<uint64_t>((sum + (int64_t{1} << 31)) >> 32);
}

}  // namespace fa
