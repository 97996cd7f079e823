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
// would be too few to fill the chip.
constexpr long long kRopeShareFrom = 1 << 19;

constexpr int kRopePairs = 1;   // of pi_rope_layout; 0: half

// A thread's share of a head: eight dimensions of the pairs layout; of the half
// layout two runs of eight, rot / 2 apart, or eight that are not turned; where
// those runs would not start at 16 bytes, one pair.
__host__ __device__ inline int rope_units(const Rope& R, int d) {
    if (R.layout == kRopePairs) return d / 8;
    return R.rot % 16 == 0 ? R.rot / 16 + (d - R.rot) / 8 : d / 2;
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
    if (R.layout != kRopePairs && R.rot % 16 != 0) {
        const bool turned = u < half;
        if (!turned && x == y) return;
        const int i = turned ? u : R.rot + 2 * (u - half), j = turned ? u + half : i + 1;
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
    const bool pairs = R.layout == kRopePairs, two = !pairs && u < R.rot / 16;
    const int at = pairs || two ? 8 * u : R.rot + (u - R.rot / 16) * 8;
    const bool turned = two || (pairs && at < R.rot);
    if (!turned && x == y) return;
    u32x4 a[HPT], b[HPT];
#pragma unroll
    for (int k = 0; k < HPT; ++k) {
        const int h = g + k * groups;
        if (h >= n_head) continue;
        a[k] = ld16(x + (size_t)h * d + at);
        if (two) b[k] = ld16(x + (size_t)h * d + at + half);
    }
    if (two) {
        float c[8], s[8];
#pragma unroll
        for (int m = 0; m < 8; ++m) rope_cos_sin(pos, R.turns[at + m], R.gain, c[m], s[m]);
#pragma unroll
        for (int k = 0; k < HPT; ++k) {
            const int h = g + k * groups;
            if (h >= n_head) continue;
            u32x4 p, q;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const f16x2 v = as_h2(a[k][m]), w = as_h2(b[k][m]);
                f16 e0, e1, f0, f1;
                turn(v.x, w.x, c[2 * m], s[2 * m], e0, f0);
                turn(v.y, w.y, c[2 * m + 1], s[2 * m + 1], e1, f1);
                p[m] = __builtin_bit_cast(uint32_t, f16x2{e0, e1});
                q[m] = __builtin_bit_cast(uint32_t, f16x2{f0, f1});
            }
            *reinterpret_cast<u32x4*>(y + (size_t)h * d + at) = p;
            *reinterpret_cast<u32x4*>(y + (size_t)h * d + at + half) = q;
        }
        return;
    }
    float c[4], s[4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
        if (turned && at / 2 + m < half) rope_cos_sin(pos, R.turns[at / 2 + m], R.gain, c[m], s[m]);
#pragma unroll
    for (int k = 0; k < HPT; ++k) {
        const int h = g + k * groups;
        if (h >= n_head) continue;
        u32x4 p = a[k];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            if (!turned || at / 2 + m >= half) continue;
            const f16x2 v = as_h2(a[k][m]);
            f16 e, f;
            turn(v.x, v.y, c[m], s[m], e, f);
            p[m] = __builtin_bit_cast(uint32_t, f16x2{e, f});
        }
        *reinterpret_cast<u32x4*>(y + (size_t)h * d + at) = p;
    }
}

}  // namespace pi
