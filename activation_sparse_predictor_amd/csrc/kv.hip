// Writing the 8-bit paged cache and reading it back.
//
// Append: per block (page), head and matrix, with N the new and O the older
// tokens of the block, s = max(s0, max_N |x| / QMAX), codes of O rounded again
// by s0 / s when s grew, codes of N = round(x / s).  Read: fp16(code * s).
// Both are bound by memory: an append has to read 2 bytes and write 1 an
// element, a read the other way round.
//
// One group of 1 or 4 waves owns a (block, head, matrix) from its largest
// value to its codes, so the new tokens' values are read once and stay in
// registers while the scale is found, and nothing is shared between groups.
// Measured: 16384 tokens of 8 heads of 128 written in 25 us (4.0 TB/s) and read
// back in 20 (5.0 TB/s); 32 ragged sequences, 82 thousand tokens, read in 102-106
// us (4.8-5.0 TB/s; a large copy reaches 4.9).  One token a sequence is latency:
// the lengths, the table, the values and the scale, the codes, one after the
// other: 4.6 us a launch for one sequence, 7 for 64.
#include "kv.hpp"

namespace pi {

// WAVES waves a group, 2 MAXT K tasks (16 dimensions of a token) or MAXT V
// tasks (2 dimensions of a granule's 16 tokens) a thread, both covering a
// block of page * d <= 2048 * WAVES * MAXT elements.  A task's index is its
// place in the block's bytes, so the stores of a wave are contiguous.
template <int FMT, int WAVES, int MAXT>
__global__ __launch_bounds__(256) void k_kv_append(KvCache c, KvBatch b, const h16* __restrict__ ksrc,
                                                   long long k_stride, const h16* __restrict__ vsrc,
                                                   long long v_stride) {
    constexpr int kThreads = WAVES * kWave;
    __shared__ uint32_t s_max[4];
    const int wave = threadIdx.x / kWave, tid = threadIdx.x % kThreads;
    const int h = blockIdx.y >> 1;
    const bool is_v = blockIdx.y & 1;
    const int item = blockIdx.x * (4 / WAVES) + wave / WAVES;
    const int page = c.page, d = c.d;
    int inside;
    const Seq q = find_seq(b, item, inside, [page](const Seq& x) {
        const int lo = x.ctx > x.n ? x.ctx - x.n : 0;
        return x.n > 0 && x.ctx > 0 ? (x.ctx - 1) / page - lo / page + 1 : 0;
    });
    if (q.s < 0) return;
    const int first = q.ctx - q.n;   // position of the sequence's first row; rows before 0 have no place
    const int lo = first > 0 ? first : 0;
    const int blk = lo / page + inside, t0 = blk * page;
    const int id = b.table[(size_t)q.s * b.table_stride + blk];
    if (id < 0 || id >= c.n_pages) return;
    const int a = lo > t0 ? lo - t0 : 0;                      // the block's tokens [a, e) are new
    const int e = q.ctx - t0 < page ? q.ctx - t0 : page;
    const int row0 = q.row0 + t0 - first;                     // row of the block's token 0
    const long long stride = is_v ? v_stride : k_stride;
    const h16* src = (is_v ? vsrc : ksrc) + (size_t)h * d;
    uint8_t* dst = (is_v ? c.v : c.k) + page_base(c, id, h);
    float* scale = (is_v ? c.v_scale : c.k_scale) + (size_t)id * c.n_kv + h;
    const float s0 = a > 0 ? *scale : 0.f;

    // the new tokens' values, and the largest of them
    const int dc = d / 16, dp = d / 2;
    uint32_t x[MAXT][16];
    uint32_t m2 = 0u;
    if (!is_v) {
#pragma unroll
        for (int i = 0; i < 2 * MAXT; ++i) {
            const int u = tid + i * kThreads;
            const int t = u / (4 * dc) * 4 + (u & 3), ch = (u >> 2) % dc;
            uint32_t* w = &x[i / 2][i % 2 * 8];
            u32x4 p = {0u, 0u, 0u, 0u}, r = p;
            if (t >= a && t < e) {
                const h16* g = src + (size_t)(row0 + t) * stride + ch * 16;
                p = ld16_stream(g);
                r = ld16_stream(g + 8);
            }
            w[0] = p.x, w[1] = p.y, w[2] = p.z, w[3] = p.w, w[4] = r.x, w[5] = r.y, w[6] = r.z, w[7] = r.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < MAXT; ++i) {
            const int u = tid + i * kThreads;
            const int g = u / dp * kGran, p = u % dp;
#pragma unroll
            for (int t = 0; t < 16; ++t) {
                x[i][t] = 0u;
                if (g + t >= a && g + t < e)
                    x[i][t] = *reinterpret_cast<const uint32_t*>(src + (size_t)(row0 + g + t) * stride + 2 * p);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < MAXT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) m2 = max_abs2(m2, x[i][j]);
    uint32_t mb = (m2 & 0xFFFFu) > (m2 >> 16) ? (m2 & 0xFFFFu) : (m2 >> 16);
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const uint32_t o = __shfl_xor(mb, off, kWave);
        mb = o > mb ? o : mb;
    }
    if constexpr (WAVES > 1) {
        if (lane_id() == 0) s_max[wave] = mb;
        __syncthreads();
        for (int i = 0; i < WAVES; ++i) mb = s_max[i] > mb ? s_max[i] : mb;
    }
    const bool bad = mb >= 0x7C00u || !finite(s0);
    const float m = (float)__builtin_bit_cast(f16, (unsigned short)mb);
    const float s = bad ? __builtin_nanf("") : fmaxf(s0, m / Codes<FMT>::kMax);
    const bool grew = !bad && s > s0 && a > 0;
    const bool zero = bad || s == 0.f;
    const float inv = zero ? 0.f : 1.f / s, r = grew ? s0 / s : 1.f;
    if (tid == 0) *scale = s;

    if (!is_v) {
#pragma unroll
        for (int i = 0; i < 2 * MAXT; ++i) {
            const int u = tid + i * kThreads;
            const int t = u / (4 * dc) * 4 + (u & 3);
            const uint32_t* w = &x[i / 2][i % 2 * 8];
            u32x4* at = reinterpret_cast<u32x4*>(dst + (size_t)u * 16);
            if (t >= a && t < e) {
                u32x4 o = {Codes<FMT>::kZero4, Codes<FMT>::kZero4, Codes<FMT>::kZero4, Codes<FMT>::kZero4};
                if (!zero) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[j] = encode4_f16<FMT>(w[2 * j], w[2 * j + 1], s, inv);
                }
                *at = o;
            } else if (grew && t < a) {
                u32x4 o = *at;
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = requant4<FMT>(o[j], r);
                *at = o;
            }
        }
        return;
    }
    store_v<FMT, kThreads, MAXT>(dst, x, tid, dp, a, e, s, inv, r, zero, grew);
}

// One wave a (granule, head).  K: 16 dimensions of a token a task; V: 2
// dimensions of the granule's 16 tokens, so that a wave's fp16 stores of one
// token are contiguous.
template <int FMT>
__global__ __launch_bounds__(256) void k_kv_read(KvCache c, KvBatch b, h16* __restrict__ kout, h16* __restrict__ vout) {
    const int wave = threadIdx.x / kWave, lane = lane_id();
    const int h = blockIdx.y, d = c.d;
    int inside;
    const Seq q = find_seq(b, blockIdx.x * 4 + wave, inside, [](const Seq& x) {
        return x.n > 0 ? ((x.ctx - 1) >> 4) - ((x.ctx - x.n) >> 4) + 1 : 0;
    });
    if (q.s < 0) return;
    const int first = q.ctx - q.n;
    const int p0 = ((first >> 4) + inside) * kGran;           // the granule's first position
    const int a = first > p0 ? first - p0 : 0;                // its tokens [a, e) are wanted
    const int e = q.ctx - p0 < kGran ? q.ctx - p0 : kGran;
    const size_t row0 = (size_t)(q.row0 + p0 - first);        // row of its token 0; used for [a, e) only
    float ks = 0.f, vs = 0.f;                                 // before the sequence: zeros
    const uint8_t *kb = c.k, *vb = c.v;
    if (p0 >= 0) {
        int id = b.table[(size_t)q.s * b.table_stride + p0 / c.page];
        const bool known = id >= 0 && id < c.n_pages;
        id = known ? id : 0;
        const size_t at = page_base(c, id, h) + (size_t)(p0 & (c.page - 1)) * d;
        kb += at;
        vb += at;
        ks = known ? c.k_scale[(size_t)id * c.n_kv + h] : __builtin_nanf("");
        vs = known ? c.v_scale[(size_t)id * c.n_kv + h] : __builtin_nanf("");
    }
    const int dc = d / 16, dp = d / 2;
    const size_t ld = (size_t)c.n_kv * d;
    for (int u = lane; u < d; u += kWave) {
        const int t = u / (4 * dc) * 4 + (u & 3), ch = (u >> 2) % dc;
        if (t < a || t >= e) continue;
        u32x4 w = {0u, 0u, 0u, 0u};
        if (p0 >= 0) w = ld16_stream(kb + (size_t)u * 16);
        u32x4 o[2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f16x2 p, y;
            Codes<FMT>::to_f16(w[j], p, y);
            const f16x2 z = {(f16)((float)p.x * ks), (f16)((float)p.y * ks)};
            const f16x2 v = {(f16)((float)y.x * ks), (f16)((float)y.y * ks)};
            o[j / 2][j % 2 * 2] = p0 >= 0 ? __builtin_bit_cast(uint32_t, z) : 0u;
            o[j / 2][j % 2 * 2 + 1] = p0 >= 0 ? __builtin_bit_cast(uint32_t, v) : 0u;
        }
        u32x4* to = reinterpret_cast<u32x4*>(kout + (row0 + t) * ld + (size_t)h * d + ch * 16);
        to[0] = o[0];
        to[1] = o[1];
    }
    for (int u = lane; u < dp; u += kWave) {
        u32x4 w[2] = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
        if (p0 >= 0) {
            w[0] = ld16_stream(vb + (size_t)u * 32);
            w[1] = ld16_stream(vb + (size_t)u * 32 + 16);
        }
        h16* to = vout + row0 * ld + (size_t)h * d + 2 * u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f16x2 p[2], y[2];
            Codes<FMT>::to_f16(w[0][j], p[0], p[1]);
            Codes<FMT>::to_f16(w[1][j], y[0], y[1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 4 * j + i;
                const f16x2 z = {(f16)((float)p[i / 2][i % 2] * vs), (f16)((float)y[i / 2][i % 2] * vs)};
                if (t >= a && t < e)
                    *reinterpret_cast<uint32_t*>(to + (size_t)t * ld) = p0 >= 0 ? __builtin_bit_cast(uint32_t, z) : 0u;
            }
        }
    }
}

hipError_t launch_kv_append(const KvCache& c, const KvBatch& b, const h16* k, long long k_stride, const h16* v,
                            long long v_stride, hipStream_t s) {
    const long long items = touched(b, c.page);
    const int e = c.page * c.d;
#define PI_APPEND(F, W, T)                                                                                       \
    hipLaunchKernelGGL((k_kv_append<F, W, T>), dim3((unsigned)((items * (W) + 3) / 4), 2 * c.n_kv), dim3(256), 0, s, \
                       c, b, k, k_stride, v, v_stride)
#define PI_APPEND_E(F)                       \
    if (e <= 2048) PI_APPEND(F, 1, 1);       \
    else if (e <= 4096) PI_APPEND(F, 1, 2);  \
    else if (e <= 8192) PI_APPEND(F, 4, 1);  \
    else if (e <= 16384) PI_APPEND(F, 4, 2); \
    else if (e <= 32768) PI_APPEND(F, 4, 4); \
    else PI_APPEND(F, 4, 8)
    if (c.fmt == 0) { PI_APPEND_E(0); } else { PI_APPEND_E(1); }
#undef PI_APPEND_E
#undef PI_APPEND
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvCache& c, const KvBatch& b, h16* k, h16* v, hipStream_t s) {
    // rows before position 0 make granules too; they count like the others
    const dim3 grid((unsigned)((touched(b, kGran) + 3) / 4), c.n_kv);
    if (c.fmt == 0) hipLaunchKernelGGL(k_kv_read<0>, grid, dim3(256), 0, s, c, b, k, v);
    else hipLaunchKernelGGL(k_kv_read<1>, grid, dim3(256), 0, s, c, b, k, v);
    return hipGetLastError();
}

}  // namespace pi
