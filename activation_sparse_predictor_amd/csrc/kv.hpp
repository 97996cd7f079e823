// Device helpers of the 8-bit paged cache (kv.hip, append.hip, attend.hip): code
// formats, byte order, rounding, and where a call's tokens lie.
#pragma once

#include "common.hpp"
#include "internal.hpp"

namespace pi {

// A page's bytes come in granules of 16 tokens, 16 d bytes for K and for V.
constexpr int kGran = 16;

// Inside a page and head, the byte of token t and dimension i is
//   K: (t / 4) * 4 d + (i / 16) * 64 + (t % 4) * 16 + i % 16
//   V: (t / 16) * 16 d + i * 16 + t % 16
// First byte of a page and head; pages * heads * bytes pass 32 bits.
__device__ __forceinline__ size_t page_base(const KvCache& c, int id, int h) {
    return ((size_t)id * c.n_kv + h) * (size_t)(c.page * c.d);
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __builtin_inff(); }

template <int FMT> struct Codes;

// int8: byte = code + 128.
template <> struct Codes<0> {
    static constexpr float kMax = 127.f;
    static constexpr uint32_t kZero4 = 0x80808080u;   // four zero codes
    // Four codes as fp16, exactly: each byte beneath 0x64 is the fp16 number
    // 1024 + byte, and 1024 + byte - 1152 = code.
    static __device__ __forceinline__ void to_f16(uint32_t w, f16x2& a, f16x2& b) {
        const f16x2 off = {(f16)1152.0f, (f16)1152.0f};
        a = as_h2(__builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) - off;
        b = as_h2(__builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) - off;
    }
    // round(clamp(x, -127, 127)) of two numbers as two bytes (rintf: ties to even)
    static __device__ __forceinline__ uint32_t encode2(float x, float y) {
        const int a = (int)rintf(fminf(fmaxf(x, -kMax), kMax)) + 128;
        const int b = (int)rintf(fminf(fmaxf(y, -kMax), kMax)) + 128;
        return (uint32_t)a | ((uint32_t)b << 8);
    }
};

// fp8: the byte is the OCP e4m3 number; the conversions round to nearest even.
template <> struct Codes<1> {
    static constexpr float kMax = 448.f;
    static constexpr uint32_t kZero4 = 0u;
    static __device__ __forceinline__ void to_f16(uint32_t w, f16x2& a, f16x2& b) {
        a = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
        b = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true));
    }
    static __device__ __forceinline__ uint32_t encode2(float x, float y) {
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(fminf(fmaxf(x, -kMax), kMax), fminf(fmaxf(y, -kMax), kMax), 0,
                                                         false) & 0xFFFFu;
    }
};

template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    return Codes<FMT>::encode2(a, b) | (Codes<FMT>::encode2(c, d) << 16);
}

// The scale and the quotient are rounded to nearest in fp32, as the definition
// has them.  A quotient that is a tie in exact arithmetic (fp16 values and
// largest values share few bits, so there are some: 3 in 10^5 codes) falls to
// the side that those two roundings leave it on, which another way of dividing
// by QMAX, or 64 bits, need not share.
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// Largest |x| of two fp16 pairs as bits: the order of the magnitudes' bits is
// that of the numbers, with infinity and then NaN above all of them.
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t x) {
    const u16x2 a = __builtin_bit_cast(u16x2, m), b = __builtin_bit_cast(u16x2, x & 0x7FFF7FFFu);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(a, b));
}

// x / s rounded to nearest, given inv = 1 / s rounded to nearest: one product
// and one residual step (Markstein's division).  With |x| in fp16's range and
// s = max|x| / QMAX at least 2^-24 / 448 > 2^-33 nothing here is subnormal.
__device__ __forceinline__ float quotient(float x, float s, float inv) {
    const float q = x * inv;
    return fmaf(fmaf(-q, s, x), inv, q);
}

template <int FMT>
__device__ __forceinline__ uint32_t encode4_f16(uint32_t lo, uint32_t hi, float s, float inv) {
    const f16x2 a = as_h2(lo), b = as_h2(hi);
    return encode4<FMT>(quotient((float)a.x, s, inv), quotient((float)a.y, s, inv), quotient((float)b.x, s, inv),
                        quotient((float)b.y, s, inv));
}

// Four codes rounded again after the scale grew by 1 / r.
template <int FMT>
__device__ __forceinline__ uint32_t requant4(uint32_t w, float r) {
    f16x2 a, b;
    Codes<FMT>::to_f16(w, a, b);
    return encode4<FMT>((float)a.x * r, (float)a.y * r, (float)b.x * r, (float)b.y * r);
}

// The codes of a block's V tokens [a, e), from the values x of MAXT tasks a thread
// (two dimensions of a granule's 16 tokens, a token's in one word), scale s and inv =
// 1 / s (zero: all codes are 0), the older codes times r if the scale grew.
template <int FMT, int kThreads, int MAXT>
__device__ __forceinline__ void store_v(uint8_t* dst, const uint32_t (&x)[MAXT][16], int tid, int dp, int a, int e, float s, float inv,
                                        float r, bool zero, bool grew) {
#pragma unroll
    for (int i = 0; i < MAXT; ++i) {
        const int u = tid + i * kThreads;
        const int g = u / dp * kGran;
        if (g >= e || (g + kGran <= a && !grew)) continue;
        u32x4* at = reinterpret_cast<u32x4*>(dst + (size_t)u * 32);
        // the granule's new codes for both dimensions, [a, e) of them to be used
        u32x4 n[2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t lo4 = Codes<FMT>::kZero4, hi4 = lo4;
            if (!zero && g + 4 * j + 3 >= a && g + 4 * j < e) {
                const uint32_t p = x[i][4 * j], y = x[i][4 * j + 1], z = x[i][4 * j + 2], w = x[i][4 * j + 3];
                lo4 = encode4_f16<FMT>((p & 0xFFFFu) | (y << 16), (z & 0xFFFFu) | (w << 16), s, inv);
                hi4 = encode4_f16<FMT>((p >> 16) | (y & 0xFFFF0000u), (z >> 16) | (w & 0xFFFF0000u), s, inv);
            }
            n[0][j] = lo4;
            n[1][j] = hi4;
        }
        if (g >= a && g + kGran <= e) {
            at[0] = n[0];
            at[1] = n[1];
        } else if (!grew) {   // single bytes, without waiting for what lies between them
            uint8_t* b = reinterpret_cast<uint8_t*>(at);
#pragma unroll
            for (int t = 0; t < kGran; ++t) {
                if (g + t < a || g + t >= e) continue;
                b[t] = (uint8_t)(n[0][t / 4] >> (t % 4 * 8));
                b[kGran + t] = (uint8_t)(n[1][t / 4] >> (t % 4 * 8));
            }
        } else {   // the older codes rounded again, and what lies behind the new ones kept
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const u32x4 o = at[k];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int t = g + 4 * j;
                    const uint32_t again = t < a ? requant4<FMT>(o[j], r) : 0u;
                    uint32_t keep = 0u;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint32_t by = 0xFFu << (8 * y);
                        keep |= (t + y < a ? again : t + y < e ? n[k][j] : o[j]) & by;
                    }
                    n[k][j] = keep;
                }
            }
            at[0] = n[0];
            at[1] = n[1];
        }
    }
}

// A sequence of the batch, with everything read from the device clamped so
// that no row and no table entry outside the arrays can follow from it.
struct Seq {
    int s, row0, n, ctx;   // its index, first row, rows and length
};
__device__ __forceinline__ Seq kv_seq(const KvBatch& b, int s) {
    const int a = b.q_start[s], e = b.q_start[s + 1], c = b.ctx[s];
    Seq q;
    q.s = s;
    q.row0 = a < 0 ? 0 : (a > b.n_tok ? b.n_tok : a);
    const int end = e > b.n_tok ? b.n_tok : e;
    q.n = end > q.row0 ? end - q.row0 : 0;
    const int cap = b.table_stride * b.page;
    q.ctx = c < 0 ? 0 : (c > cap ? cap : c);
    return q;
}

// Inclusive sum over the wave's lanes: shifts inside each 16-lane row, then
// the rows' last lanes broadcast to the rows behind them (DPP, no LDS).
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast 15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast 31 into rows 2 and 3
    return v;
}

// The sequence that item `item` of a list of count(seq) items per sequence
// belongs to, and the item's number inside it (wave-uniform; s = -1 past the
// list's end).  Every lane takes one sequence a round.
template <class F>
__device__ __forceinline__ Seq find_seq(const KvBatch& b, int item, int& inside, F count) {
    Seq none{-1, 0, 0, 0};
    int before = 0;
    for (int s0 = 0; s0 < b.n_seq; s0 += kWave) {
        const int s = s0 + lane_id();
        const Seq q = s < b.n_seq ? kv_seq(b, s) : Seq{-1, 0, 0, 0};
        const int n = s < b.n_seq ? count(q) : 0;
        const int upto = before + wave_scan(n);
        const uint64_t hit = __ballot(upto > item);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            Seq r;
            r.s = s0 + l;
            r.row0 = __builtin_amdgcn_readlane(q.row0, l);
            r.n = __builtin_amdgcn_readlane(q.n, l);
            r.ctx = __builtin_amdgcn_readlane(q.ctx, l);
            inside = item - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(n, l));
            return r;
        }
        before = __builtin_amdgcn_readlane(upto, kWave - 1);
    }
    inside = 0;
    return none;
}

// Upper bound of the blocks of `page` tokens that the batch's rows lie in:
// n rows touch at most (n + page - 2) / page + 1 of them, and at most n.
inline long long touched(const KvBatch& b, int page) {
    long long n = b.n_tok;
    const long long each = (long long)b.n_seq * ((b.max_q + page - 2) / page + 1);
    const long long all = (long long)b.n_tok / page + 2LL * b.n_seq;
    if (each < n) n = each;
    if (all < n) n = all;
    return n;
}

}  // namespace pi
