// Rotary positions: a pair (a, b) of a head's dimensions at position p becomes
//   gain (a cos t - b sin t),  gain (b cos t + a sin t),  t = 2 pi p turns,
// turns the pair's advance per position.  Pair m is (m, m + rot / 2) in the
// half layout, (2 m, 2 m + 1) in the pairs layout.
//
// Turns come as 64-bit fractions, so the product with the position, kept to 64
// bits, is the angle already brought into one turn, exact to 2^-32 turns at any
// position (in fp32, p = 10^6 at one radian a position is off by 0.06 rad).  Its leading word
// gives the quadrant and an angle within an eighth of a turn, where two short
// polynomials (least squares in the maximum norm, fitted for this) leave errors
// under 2^-23 of one: a 2^11th of the rounding of an fp16 result.
#pragma once

#include <type_traits>

#include "common.hpp"
#include "internal.hpp"

namespace pi {

__device__ __forceinline__ void rope_cos_sin(int pos, uint64_t turns, float gain, float& c, float& s) {
    const int t = (int)(uint32_t)(((uint64_t)(int64_t)pos * turns) >> 32);   // 2^-32 turns
    const uint32_t q = ((uint32_t)t + 0x20000000u) >> 30;                    // quadrant, to the nearest
    const float a = (float)(int)((uint32_t)t - (q << 30)) * 1.4629180792671596e-09f, x = a * a;   // 2 pi / 2^32
    const float sn = fmaf(a * x, fmaf(x, fmaf(x, -0x1.994eb4p-13f, 0x1.11076p-7f), -0x1.555546p-3f), a);
    const float cs = fmaf(x, fmaf(x, fmaf(x, fmaf(x, 0x1.9a025ap-16f, -0x1.6c0c8cp-10f), 0x1.55554ap-5f), -0.5f), 1.f);
    const float u = q & 1u ? sn : cs, v = q & 1u ? cs : sn;   // a quarter turn on: cos -> -sin, sin -> cos
    c = ((q + 1u) & 2u ? -u : u) * gain;
    s = (q & 2u ? -v : v) * gain;
}

// From so many units on, four heads share a thread's angles; below, the threads
// would be too few to fill the chip.  By the card, shared and not, heads of 128:
// half layout, 72 heads: 64 tokens (2^15 units) 3.6 and 3.1 us, 512 (2^18) 5.3 and
// 6.1, 2048 13.4 and 15.4, 8192 49.7 and 54; beside an append, 64 heads: 256 tokens
// (2^17) 6.8 and 7.0, 512 7.6 and 8.2, 8192 57 and 81.
constexpr long long kRopeShareFrom = 1 << 18;

constexpr int kRopePairs = 1;   // of pi_rope_layout; 0: half

// A thread's share of a head: 16 dimensions of the pairs layout (eight where rot or
// d does not divide into 16); of the half layout two runs of eight, rot / 2 apart, or
// eight that are not turned; where rot does not divide into these, one pair.
__host__ __device__ inline int rope_dims(const Rope& R, int d) {   // of a unit that is turned
    if (R.rot % 16 == 0 && (R.layout != kRopePairs || d % 16 == 0)) return 16;
    return R.rot % 8 == 0 && R.layout == kRopePairs ? 8 : 2;
}
__host__ __device__ inline int rope_units(const Rope& R, int d) {
    const int dims = rope_dims(R, d);
    return R.layout != kRopePairs && dims == 16 ? R.rot / 16 + (d - R.rot) / 8 : d / dims;
}

// Unit `slot % units` of heads slot / units, + groups, + 2 groups, ... (up to HPT of
// them, which share the angles) of one token: x and y its first heads, y == x or apart.
template <int HPT>
__device__ __forceinline__ void rotate_heads(const Rope& R, int d, int n_head, int groups, int units, int pos, const h16* x,
                                             h16* y, int slot) {
    const int g = slot / units, u = slot - g * units, half = R.rot / 2;
    auto turn = [&](f16 a, f16 b, float c, float s, f16& p, f16& q) __attribute__((always_inline)) {
        const float fa = (float)a, fb = (float)b;
        p = (f16)fmaf(fa, c, -(fb * s));   // one rounding to fp16, the result's
        q = (f16)fmaf(fb, c, fa * s);
    };
    const int dims = rope_dims(R, d);
    if (dims == 2) {
        const bool turned = u < half;
        if (!turned && x == y) return;
        const int i = !turned ? R.rot + 2 * (u - half) : R.layout == kRopePairs ? 2 * u : u;
        const int j = turned && R.layout != kRopePairs ? u + half : i + 1;
        f16 a[HPT], b[HPT];
#pragma unroll
        for (int k = 0; k < HPT; ++k) {
            const int h = g + k * groups;
            if (h < n_head) a[k] = x[(size_t)h * d + i], b[k] = x[(size_t)h * d + j];
        }
        float c = 0.f, s = 0.f;
        if (turned) rope_cos_sin(pos, R.turns[u], R.gain, c, s);
#pragma unroll
        for (int k = 0; k < HPT; ++k) {
            const int h = g + k * groups;
            if (h >= n_head) continue;
            if (turned) turn(a[k], b[k], c, s, a[k], b[k]);
            y[(size_t)h * d + i] = a[k];
            y[(size_t)h * d + j] = b[k];
        }
        return;
    }
    // VECS vectors of eight dimensions a head, the second `behind` dimensions after the
    // first; rotate: turns them, by the angles from pair m0 on.
    auto run = [&](auto vecs, int at, int behind, bool turned, int m0, auto rotate) __attribute__((always_inline)) {
        constexpr int VECS = decltype(vecs)::value;
        u32x4 v[HPT][VECS];
#pragma unroll
        for (int k = 0; k < HPT; ++k) {
            const int h = g + k * groups;
            if (h >= n_head) continue;
#pragma unroll
            for (int i = 0; i < VECS; ++i) v[k][i] = ld16(x + (size_t)h * d + at + i * behind);
        }
        float c[4 * VECS], s[4 * VECS];
        if (turned) {
#pragma unroll
            for (int m = 0; m < 4 * VECS; ++m) rope_cos_sin(pos, R.turns[m0 + m], R.gain, c[m], s[m]);
        }
#pragma unroll
        for (int k = 0; k < HPT; ++k) {
            const int h = g + k * groups;
            if (h >= n_head) continue;
            if (turned) rotate(v[k], c, s);
#pragma unroll
            for (int i = 0; i < VECS; ++i) *reinterpret_cast<u32x4*>(y + (size_t)h * d + at + i * behind) = v[k][i];
        }
    };
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    if (R.layout == kRopePairs) {
        const int at = dims * u;
        if (at >= R.rot && x == y) return;
        auto neighbours = [&](auto& v, auto& c, auto& s) __attribute__((always_inline)) {
#pragma unroll
            for (int m = 0; m < (int)(sizeof(c) / sizeof(c[0])); ++m) {
                const f16x2 w = as_h2(v[m / 4][m % 4]);
                f16 p, q;
                turn(w.x, w.y, c[m], s[m], p, q);
                v[m / 4][m % 4] = __builtin_bit_cast(uint32_t, f16x2{p, q});
            }
        };
        if (dims == 16) run(Two{}, at, 8, at < R.rot, at / 2, neighbours);
        else run(One{}, at, 0, at < R.rot, at / 2, neighbours);
        return;
    }
    if (u < R.rot / 16) {
        run(Two{}, 8 * u, half, true, 8 * u, [&](auto& v, auto& c, auto& s) __attribute__((always_inline)) {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const f16x2 a = as_h2(v[0][m]), b = as_h2(v[1][m]);
                f16 e0, e1, f0, f1;
                turn(a.x, b.x, c[2 * m], s[2 * m], e0, f0);
                turn(a.y, b.y, c[2 * m + 1], s[2 * m + 1], e1, f1);
                v[0][m] = __builtin_bit_cast(uint32_t, f16x2{e0, e1});
                v[1][m] = __builtin_bit_cast(uint32_t, f16x2{f0, f1});
            }
        });
    } else if (x != y) {
        run(One{}, R.rot + (u - R.rot / 16) * 8, 0, false, 0, [](auto&, auto&, auto&) {});
    }
}

}  // namespace pi
