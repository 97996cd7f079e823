// Writing the 8-bit paged cache with the position rotation on the way
// (pi_kv_append_rope).
//
// The blocks' rules are kv.hip's; here the keys are first turned by their cache
// positions (rope.hpp) and stay in fp32 from there to their codes, so that the
// rotation adds no rounding of its own; the batch's row i may be any row of k and
// v (a list on the device: the drafted tokens that were accepted); and the
// queries' heads are turned by further workgroups of the same launch.
//
// Bytes bound the large calls: four prompts of 2048 tokens of 64 query and 8 kv
// heads of 128 move 319 MB (of which the queries 268) in 66.5 us, 4.8 TB/s, where a
// large copy reaches 5.1.  Small ones are a chain of dependent reads, lengths ->
// page -> scale beside list -> rows and angles, then the block's maximum and the codes:
// one token of 56 heads 6.7 us (without rotation and queries 5.0), 64 sequences of
// 64 query and 8 kv heads 8.9, the accepted rows of 48 trees 6.7.
//
// The half layout with rot not a multiple of 32 (heads of 80 turned whole) works out
// every angle twice and reads a pair's other half in single loads: keys and values of
// four prompts of 2048 tokens of 32 heads of 80 take 103 us, where the pairs layout
// takes 71, heads of 96 65 and heads that are not turned 50; single tokens take the same.
#include "kv.hpp"
#include "rope.hpp"

namespace pi {

constexpr int kAppThreads(int waves) { return waves > 4 ? waves * kWave : 256; }

struct AppendArgs {
    KvCache c;
    KvBatch b;
    Rope rope;          // rot 0: the keys are not turned
    const int32_t* rows;
    int n_src;
    const h16 *k, *v, *q;
    long long k_stride, v_stride, q_stride, out_stride;
    int n_head, groups, units;   // of the queries
    h16* q_out;
};

// |x| as bits, in the order of the magnitudes, infinity and NaN above them.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The queries' part of the launch: workgroups of four waves or more, a wave 64 slots of one token.
template <int HPT>
__device__ __forceinline__ void append_queries(const AppendArgs& A, long long wave) {
    const int slots = A.groups * A.units, each = (slots + kWave - 1) / kWave;
    const long long tok = wave / each;
    if (tok >= A.b.n_tok) return;
    int inside;
    const Seq q = find_seq(A.b, (int)tok, inside, [](const Seq& x) { return x.n; });
    const int slot = (int)(wave - tok * each) * kWave + lane_id();
    if (q.s < 0 || slot >= slots) return;
    const size_t row = (size_t)(q.row0 + inside);
    rotate_heads<HPT>(A.rope, A.c.d, A.n_head, A.groups, A.units, q.ctx - q.n + inside, A.q + row * A.q_stride,
                      A.q_out + row * A.out_stride, slot);
}

// WAVES waves a block (page), head and matrix, 2 MAXT K tasks (16 dimensions of
// a token) or MAXT V tasks (2 dimensions of a granule's 16 tokens) a thread, both
// covering page * d <= 2048 * WAVES * MAXT elements.  Grid rows: K and V of each
// head, then the queries.
template <int FMT, int WAVES, int MAXT, int HPT>
__global__ __launch_bounds__(kAppThreads(WAVES)) void k_kv_append_rope(AppendArgs A) {
    constexpr int kThreads = WAVES * kWave, kBlockWaves = kAppThreads(WAVES) / kWave, kTasks = 2 * MAXT;
    __shared__ uint32_t s_max[kBlockWaves];
    const KvCache& c = A.c;
    const KvBatch& b = A.b;
    const int wave = threadIdx.x / kWave, tid = threadIdx.x % kThreads;
    if ((int)blockIdx.y >= 2 * c.n_kv) {
        const long long block = (long long)((int)blockIdx.y - 2 * c.n_kv) * gridDim.x + blockIdx.x;
        append_queries<HPT>(A, block * kBlockWaves + wave);
        return;
    }
    const int h = blockIdx.y >> 1;
    const bool is_v = blockIdx.y & 1;
    const int item = blockIdx.x * (kBlockWaves / WAVES) + wave / WAVES;
    const int page = c.page, d = c.d;
    int inside;
    const Seq q = find_seq(b, item, inside, [page](const Seq& x) {
        const int lo = x.ctx > x.n ? x.ctx - x.n : 0;
        return x.n > 0 && x.ctx > 0 ? (x.ctx - 1) / page - lo / page + 1 : 0;
    });
    // (one wave a group: no barrier below; several: they share item and leave together)
    if (q.s < 0) return;
    const int first = q.ctx - q.n;   // position of the sequence's first row; rows before 0 have no place
    const int lo = first > 0 ? first : 0;
    const int blk = lo / page + inside, t0 = blk * page;
    const int id = b.table[(size_t)q.s * b.table_stride + blk];
    if (id < 0 || id >= c.n_pages) return;
    const int a = lo > t0 ? lo - t0 : 0;                      // the block's tokens [a, e) are new
    const int e = q.ctx - t0 < page ? q.ctx - t0 : page;
    const int row0 = q.row0 + t0 - first;                     // row of the block's token 0
    const long long stride = is_v ? A.v_stride : A.k_stride;
    const h16* src = (is_v ? A.v : A.k) + (size_t)h * d;
    uint8_t* dst = (is_v ? c.v : c.k) + page_base(c, id, h);
    float* scale = (is_v ? c.v_scale : c.k_scale) + (size_t)id * c.n_kv + h;
    const float s0 = a > 0 ? *scale : 0.f;
    // the row of token t, -1 if the list names none
    auto row_of = [&](int t) {
        const int r = row0 + t;
        if (!A.rows) return r;
        const int x = A.rows[r];
        return x >= 0 && x < A.n_src ? x : -1;
    };

    const int dc = d / 16, dp = d / 2, rot = A.rope.rot, half = rot / 2;
    // K tasks.  Where a pair's two runs of 16 dimensions are whole tasks, one thread
    // has both (its tasks 2 i and 2 i + 1) and works out the angles once.
    // (np tasks of two a token: with page * dc <= 128 WAVES MAXT, powers of two but dc,
    // page * np fits 64 WAVES MAXT for odd dc >= 3 too)
    const bool twin = rot > 0 && A.rope.layout != kRopePairs && rot % 32 == 0;
    const int np = twin ? (dc + 1) / 2 : dc;
    auto place = [&](int i, int& t, int& ch) {   // token and run of 16 of task i
        const int u = twin ? tid + i / 2 * kThreads : tid + i * kThreads;
        t = u / (4 * np) * 4 + (u & 3);
        const int p = (u >> 2) % np;
        ch = !twin ? p : p < rot / 32 ? p + (i & 1) * (rot / 32) : 2 * p + (i & 1);
        return t >= 0 && t < page && ch < dc;
    };
    float xk[kTasks][16];
    uint32_t xv[MAXT][16];
    uint32_t mb = 0u;
    if (!is_v) {
        auto load16 = [&](const h16* g, float* x) __attribute__((always_inline)) {
            const u32x4 p = ld16_stream(g), r = ld16_stream(g + 8);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f16x2 m = as_h2(p[j]), n = as_h2(r[j]);
                x[2 * j] = (float)m.x, x[2 * j + 1] = (float)m.y, x[8 + 2 * j] = (float)n.x, x[9 + 2 * j] = (float)n.y;
            }
        };
#pragma unroll
        for (int i = 0; i < kTasks; ++i) {
            int t, ch;
            const bool has = place(i, t, ch) && t >= a && t < e;
#pragma unroll
            for (int j = 0; j < 16; ++j) xk[i][j] = 0.f;
            if (!has) continue;
            const int r = row_of(t);
            if (r < 0) {
                xk[i][0] = __builtin_nanf("");
                continue;
            }
            const h16* g = src + (size_t)r * stride + ch * 16;
            load16(g, xk[i]);
            if (rot == 0 || twin || ch * 16 >= rot) continue;
            const int pos = t0 + t;
            if (A.rope.layout == kRopePairs) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (ch * 8 + j >= half) continue;
                    float cs, sn;
                    rope_cos_sin(pos, A.rope.turns[ch * 8 + j], A.rope.gain, cs, sn);
                    const float x = xk[i][2 * j], y = xk[i][2 * j + 1];
                    xk[i][2 * j] = fmaf(x, cs, -(y * sn));
                    xk[i][2 * j + 1] = fmaf(y, cs, x * sn);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int m = ch * 16 + j;
                    if (m >= rot) continue;
                    const bool low = m < half;
                    const float other = (float)g[j + (low ? half : -half)];
                    float cs, sn;
                    rope_cos_sin(pos, A.rope.turns[low ? m : m - half], A.rope.gain, cs, sn);
                    xk[i][j] = low ? fmaf(xk[i][j], cs, -(other * sn)) : fmaf(xk[i][j], cs, other * sn);
                }
            }
        }
        if (twin) {
#pragma unroll
            for (int i = 0; i < kTasks; i += 2) {
                int t, ch;
                if (!place(i, t, ch) || t < a || t >= e || ch >= rot / 32) continue;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float cs, sn;
                    rope_cos_sin(t0 + t, A.rope.turns[ch * 16 + j], A.rope.gain, cs, sn);
                    const float x = xk[i][j], y = xk[i + 1][j];
                    xk[i][j] = fmaf(x, cs, -(y * sn));
                    xk[i + 1][j] = fmaf(y, cs, x * sn);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kTasks; ++i)
#pragma unroll
            for (int j = 0; j < 16; ++j) mb = abs_bits(xk[i][j]) > mb ? abs_bits(xk[i][j]) : mb;
    } else {
        uint32_t m2 = 0u;
#pragma unroll
        for (int i = 0; i < MAXT; ++i) {
            const int u = tid + i * kThreads;
            const int g = u / dp * kGran, p = u % dp;
#pragma unroll
            for (int t = 0; t < 16; ++t) {
                xv[i][t] = 0u;
                if (g + t >= a && g + t < e) {
                    const int r = row_of(g + t);
                    xv[i][t] = r < 0 ? 0x7E007E00u : *reinterpret_cast<const uint32_t*>(src + (size_t)r * stride + 2 * p);
                }
                m2 = max_abs2(m2, xv[i][t]);
            }
        }
        const uint32_t top = (m2 & 0xFFFFu) > (m2 >> 16) ? (m2 & 0xFFFFu) : (m2 >> 16);
        mb = abs_bits((float)__builtin_bit_cast(f16, (unsigned short)top));
    }
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
    const bool bad = mb >= 0x7F800000u || !finite(s0);
    const float s = bad ? __builtin_nanf("") : fmaxf(s0, __uint_as_float(mb) / Codes<FMT>::kMax);
    const bool grew = !bad && s > s0 && a > 0;
    const bool zero = bad || s == 0.f;
    const float inv = zero ? 0.f : 1.f / s, r = grew ? s0 / s : 1.f;
    if (tid == 0) *scale = s;

    if (!is_v) {
#pragma unroll
        for (int i = 0; i < kTasks; ++i) {
            int t, ch;
            if (!place(i, t, ch)) continue;
            u32x4* at = reinterpret_cast<u32x4*>(dst + (size_t)(t / 4 * 4 * d + ch * 64 + t % 4 * 16));
            if (t >= a && t < e) {
                u32x4 o = {Codes<FMT>::kZero4, Codes<FMT>::kZero4, Codes<FMT>::kZero4, Codes<FMT>::kZero4};
                if (!zero) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        o[j] = encode4<FMT>(quotient(xk[i][4 * j], s, inv), quotient(xk[i][4 * j + 1], s, inv),
                                            quotient(xk[i][4 * j + 2], s, inv), quotient(xk[i][4 * j + 3], s, inv));
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
    store_v<FMT, kThreads, MAXT>(dst, xv, tid, dp, a, e, s, inv, r, zero, grew);
}

hipError_t launch_kv_append_rope(const KvCache& c, const KvBatch& b, const Rope* rope, const int32_t* rows, int n_src, const h16* k,
                                 long long k_stride, const h16* v, long long v_stride, const h16* q, long long q_stride,
                                 int n_head, h16* q_out, long long out_stride, hipStream_t s) {
    AppendArgs A{c, b, rope ? *rope : Rope{0, 0, 1.f, nullptr}, rows, n_src, k, v, q, k_stride, v_stride, q_stride, out_stride,
                 n_head, 0, 0, q_out};
    const long long items = touched(b, c.page);
    const int e = c.page * c.d;
    const int units = q ? rope_units(A.rope, c.d) : 0;
    // four heads share a thread's angles from kRopeShareFrom units on, where a token's threads still fill a wave
    const bool share = q && (long long)b.n_tok * n_head * units >= kRopeShareFrom && n_head * units >= 4 * kWave;
    A.units = units;
    A.groups = !q ? 0 : share ? (n_head + 3) / 4 : n_head;
#define PI_APPEND(F, W, T, H)                                                                              \
    do {                                                                                                   \
        constexpr int kBlockWaves = kAppThreads(W) / kWave;                                                \
        const long long waves = (long long)b.n_tok * ((A.groups * units + kWave - 1) / kWave);             \
        const long long blocks_q = (waves + kBlockWaves - 1) / kBlockWaves;                                \
        long long gx = (items * (W) + kBlockWaves - 1) / kBlockWaves;                                      \
        if (gx * 32768 < blocks_q) gx = (blocks_q + 32767) / 32768;   /* a grid has at most 65535 rows */  \
        const long long rows_q = (blocks_q + gx - 1) / gx;                                                 \
        hipLaunchKernelGGL((k_kv_append_rope<F, W, T, H>), dim3((unsigned)gx, (unsigned)(2 * c.n_kv + rows_q)), \
                           dim3(kAppThreads(W)), 0, s, A);                                                 \
    } while (0)
#define PI_APPEND_E(F, H)                        \
    if (e <= 2048) PI_APPEND(F, 1, 1, H);        \
    else if (e <= 4096) PI_APPEND(F, 1, 2, H);   \
    else if (e <= 8192) PI_APPEND(F, 4, 1, H);   \
    else if (e <= 16384) PI_APPEND(F, 4, 2, H);  \
    else if (e <= 32768) PI_APPEND(F, 16, 1, H); \
    else PI_APPEND(F, 16, 2, H)
#define PI_APPEND_F(F) \
    if (share) { PI_APPEND_E(F, 4); } else { PI_APPEND_E(F, 1); }
    if (c.fmt == 0) { PI_APPEND_F(0); } else { PI_APPEND_F(1); }
#undef PI_APPEND_F
#undef PI_APPEND_E
#undef PI_APPEND
    return hipGetLastError();
}

}  // namespace pi
