// Device helpers of the 8-bit paged cache (kv.hip, attend.hip): code formats,
// byte order, and where a call's tokens lie.
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

}  // namespace pi
