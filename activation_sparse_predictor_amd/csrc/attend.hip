// Attention over the 8-bit paged cache.
//
// For a row (query token, head) and its keys j: x_j = scale log2(e) q . K_j,
// p_j = 2^(x_j - R), l = sum p_j, y = sum p_j V_j / l, in one pass over the
// cache with running references in place of R.
//
// K_j = ks code and V_j = vs code, one ks and vs a page and head.  Codes are
// exact in fp16, so q . code runs on the matrix cores without rounding the
// cache a second time; ks multiplies the fp32 score and vs the weight.  A
// weight p vs can lie anywhere between 2^-31 and 2^9 times p, so the weights
// have a reference of their own: M follows max (x + log2 vs), the weights are
// w = 2^(x + log2 vs - M + 14), and y = (sum w code) 2^(M - R - 14) / l.  Both
// references move only when a new maximum is more than 1 above them, so w
// stays within 2^15 and fp16 holds it, down to 2^-39 of the row's largest; M is
// kept above R - 60, below which nothing of the row can reach fp16.
//
// Operands.  A wave takes 64 keys (four granules of 16) a step, as the rows of
// S^T = K Q^T and the inner axis of O^T = V^T P^T, with 16x16x32 products.
// Row i of score tile t is token 4 t + i % 4 of granule i / 4.  Then lane
// (n, g) = (lane % 16, lane / 16) ends up with the 16 scores of query n against
// the tokens of granule g, in order: they are, as they stand, the second
// operand of the output's products, all share one page, and the V operand is
// 16 contiguous bytes (a dimension's 16 tokens).  So nothing is shuffled or
// staged between the two products, and a lane has one ks and one vs a step.
#include "kv.hpp"

namespace pi {

constexpr int kTile = 64;          // keys a wave takes at a time
constexpr int kAttWaves = 4;
constexpr int kAttThreads = kAttWaves * kWave;
constexpr int kAttRows = 16;       // query rows of a workgroup
constexpr int kAttMinTiles = 4;    // fewest tiles worth a workgroup of their own
// workgroups the work is split into: those that run at once, by the registers
__host__ __device__ constexpr int att_target(int kj) { return kj == 4 ? 256 : kj == 2 ? 512 : 768; }
constexpr int kAttSlots = 2 * 768;   // pieces of split items: ceil(t / C) < 2 t / C where t > C
constexpr int kAttCtrStride = 16;  // words between arrival counters

constexpr float kLift = 14.f, kSlack = 1.f, kFloor = 60.f, kNone = -1e30f, kLn2 = 0.69314718055994531f;

// max over the lanes that hold the same query (lane ^ 16, lane ^ 32)
__device__ __forceinline__ float max_groups(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
    const uint32_t w = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_groups(float v) { return add_swap<32>(add_swap<16>(v)); }

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_fast(float x) { return __builtin_amdgcn_logf(x); }

struct AttArgs {
    KvCache c;
    KvBatch b;
    const h16* q;
    long long q_stride;
    int n_head, group, window, target;
    float scale2;   // scale * log2(e)
    h16* y;
    float* lse;
    uint32_t* ctr;
    float* part;
};

// What a workgroup works on: `rows` query rows of a sequence from row0 on,
// tiles [t0, t1), head h, piece `split` of `splits`.
struct AttUnit {
    Seq q;
    int h, row_tile, t0, t1, split, splits, slot;
};

// First tile of a sequence that any of its rows attends to, and the tiles in all (at least one).
__device__ __forceinline__ int att_first_tile(const Seq& q, int window) {
    const int lo = q.ctx - q.n - window + 1;
    return window > 0 && lo > 0 ? lo / kTile : 0;
}
__device__ __forceinline__ int att_tiles(const Seq& q, int window) {
    const int n = (q.ctx + kTile - 1) / kTile - att_first_tile(q, window);
    return n > 0 ? n : 1;
}

// Splits the whole batch's tiles over about kAttTarget workgroups: C tiles a
// workgroup, the same for every sequence, from the lengths as they are on the
// device.  Each item (sequence, row tile) becomes ceil(tiles / C) pieces of
// nearly equal size, for each head.  Every wave computes it for itself: a
// round of 64 sequences is one round of loads.  Fills in unit `item`, if there
// is one, and returns how many there are (of each head).  With at most 2^24
// rows and 2^10 sequences, whatever the lengths say, the sums stay below 2^31.
__device__ __forceinline__ int att_plan(const AttArgs& A, int item, AttUnit& w) {
    constexpr int ROWS = kAttRows;
    const KvBatch& b = A.b;
    float all = 0.f, items = 0.f;   // C only has to be the same everywhere
    Seq q{-1, 0, 0, 0};
    int rt = 0, tiles = 1;
    for (int s0 = 0; s0 < b.n_seq; s0 += kWave) {
        const int s = s0 + lane_id();
        rt = 0;
        if (s < b.n_seq) {
            q = kv_seq(b, s);
            rt = (q.n * A.group + ROWS - 1) / ROWS;
            tiles = att_tiles(q, A.window);
        }
        all += group_sum<64>((float)rt * (float)tiles);
        items += group_sum<64>((float)rt);
    }
    const float room = (float)A.target / (float)A.c.n_kv;   // workgroups a head has
    const float want = all / room * 1.001f;                 // a little above: the slots rest on it
    int C = want < kAttMinTiles ? kAttMinTiles : (int)want + 1;
    if (b.n_seq <= kWave && items <= room) {
        // All items can run at once: the smallest C (to a sixteenth) whose rounded-up pieces still do.
        for (int i = 0; i < 24; ++i) {
            if (group_sum<64>((float)(rt * ((tiles + C - 1) / C))) <= room) break;
            C += C / 16 + 1;
        }
    }
    int before = 0, slots = 0;
    for (int s0 = 0; s0 < b.n_seq; s0 += kWave) {
        const int s = s0 + lane_id();
        if (b.n_seq > kWave) {   // otherwise the first loop's values are still there
            rt = 0;
            if (s < b.n_seq) {
                q = kv_seq(b, s);
                rt = (q.n * A.group + ROWS - 1) / ROWS;
                tiles = att_tiles(q, A.window);
            }
        }
        const int ns = (tiles + C - 1) / C;
        const int upto = before + wave_scan(rt * ns), held = ns > 1 ? rt * ns : 0;
        const int slots_upto = slots + wave_scan(held);
        const uint64_t hit = __ballot(upto > item);
        if (hit && before <= item) {
            const int l = __builtin_ctzll(hit);
            w.q.s = s0 + l;
            w.q.row0 = __builtin_amdgcn_readlane(q.row0, l);
            w.q.n = __builtin_amdgcn_readlane(q.n, l);
            w.q.ctx = __builtin_amdgcn_readlane(q.ctx, l);
            w.splits = __builtin_amdgcn_readlane(ns, l);
            const int T = __builtin_amdgcn_readlane(tiles, l);
            const int inside = item - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(rt, l) * w.splits);
            w.row_tile = inside / w.splits;
            w.split = inside - w.row_tile * w.splits;
            w.slot = __builtin_amdgcn_readlane(slots_upto, l) - __builtin_amdgcn_readlane(held, l) +
                     w.row_tile * w.splits;   // the item's first slot
            const int each = T / w.splits, more = T - each * w.splits;
            w.t0 = att_first_tile(w.q, A.window) + w.split * each + (w.split < more ? w.split : more);
            w.t1 = w.t0 + each + (w.split < more ? 1 : 0);
        }
        before = __builtin_amdgcn_readlane(upto, kWave - 1);
        slots = __builtin_amdgcn_readlane(slots_upto, kWave - 1);
    }
    return before;
}

// 16 bytes of a piece's results, written and read past the caches that other
// XCDs do not see (as the agent-scope atomics do).
__device__ __forceinline__ void st16_coherent(__amdgpu_buffer_rsrc_t r, uint32_t at, f32x4 v) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, (int)at, 0, 16);
}
__device__ __forceinline__ f32x4 ld16_coherent(__amdgpu_buffer_rsrc_t r, uint32_t at) {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)at, 0, 16));
}

typedef const __attribute__((address_space(4))) int32_t* const_i32;
typedef const __attribute__((address_space(4))) float* const_f32;

// v[i] for a lane's i in 0 .. 3
template <class T>
__device__ __forceinline__ T pick(const T (&v)[4], int i) {
    const T a = i & 1 ? v[1] : v[0], b = i & 1 ? v[3] : v[2];
    return i & 2 ? b : a;
}

// KJ: 64-dimension steps of a head.
template <int FMT, int KJ>
__device__ __forceinline__ void attend_unit(const AttArgs& A, const AttUnit& w) {
    constexpr int ROWS = kAttRows, DP = 64 * KJ, LD = DP + 4;
    extern __shared__ float lds[];   // [waves][ROWS][LD] outputs, [waves][3][ROWS] statistics
    __shared__ int s_last;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int lane = lane_id(), n16 = lane & 15, g = lane >> 4;
    const int d = A.c.d, dc = d / 16, page = A.c.page, group = A.group;
    const int ctx = w.q.ctx, first = ctx - w.q.n, rows_all = w.q.n * group;
    const int shift = __builtin_ctz(page), last_gran = ctx > 0 ? (ctx - 1) / kGran : 0;

    // The pages of a tile's four granules and their scales, through the scalar
    // cache: uniform over the wave, and off the counter that the K and V loads
    // wait on.  Granules past the end: some page of the sequence, masked.
    const const_i32 table = (const_i32)(A.b.table + (size_t)w.q.s * A.b.table_stride);
    const const_f32 k_scale = (const_f32)A.c.k_scale, v_scale = (const_f32)A.c.v_scale;
    auto gran = [&](int tile, int i) {
        const int gi = tile * (kTile / kGran) + i;
        return gi < last_gran ? gi : last_gran;
    };
    auto lookup = [&](int tile, int (&id)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) id[i] = ctx > 0 ? table[gran(tile, i) * kGran >> shift] : -1;
    };
    auto known = [&](int id) { return id >= 0 && id < A.c.n_pages; };
    auto scales = [&](const int (&id)[4], float (&ks)[4], float (&vs)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const size_t at = (size_t)(known(id[i]) ? id[i] : 0) * A.c.n_kv + w.h;
            ks[i] = known(id[i]) ? k_scale[at] : __builtin_nanf("");
            vs[i] = known(id[i]) ? v_scale[at] : __builtin_nanf("");
        }
    };
    auto gran_base = [&](const int (&id)[4], int tile, int i) {   // i: per lane
        int p = pick(id, i);
        p = known(p) ? p : 0;
        return ((size_t)p * A.c.n_kv + w.h) * (size_t)(page * d) + (size_t)((gran(tile, i) * kGran & (page - 1)) * d);
    };

    // byte offsets of this lane's pieces inside a granule
    int ko[KJ];
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
        const int ch = j * 4 + g < dc ? j * 4 + g : dc - 1;   // beyond d: any finite code, its query is 0
        ko[j] = ch * 64 + (n16 & 3) * 16;
    }
    const int gk = n16 >> 2;
    u32x4 kc[4][KJ], vc[4 * KJ];
    auto load_k = [&](const int (&id)[4], int tile) {
        const uint8_t* at = A.c.k + gran_base(id, tile, gk);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < KJ; ++j) kc[t][j] = ld16_stream(at + t * 4 * d + ko[j]);
    };
    auto load_v = [&](const int (&id)[4], int tile) {
        const uint8_t* at = A.c.v + gran_base(id, tile, g) + n16 * 16;
#pragma unroll
        for (int k = 0; k < 4 * KJ; ++k) vc[k] = ld16_stream(at + (k < dc ? k : dc - 1) * 256);
    };

    int tile = w.t0 + wave;
    int id[4];
    float ks[4], vs[4];
    if (tile < w.t1) {
        lookup(tile, id);
        load_k(id, tile);
        load_v(id, tile);
        scales(id, ks, vs);
        lookup(tile + kAttWaves, id);
    }

    // this lane's query: position, and the operand's fragments
    const int my_row = w.row_tile * ROWS + n16;
    const bool live = my_row < rows_all;
    const int my_tok = live ? my_row / group : 0, my_head = w.h * group + (live ? my_row - my_tok * group : 0);
    const int pos = live ? first + my_tok : -1;
    const int lo = A.window > 0 && pos - A.window + 1 > 0 ? pos - A.window + 1 : 0;
    f16x8 qf[2 * KJ];
    {
        const h16* qr = A.q + (size_t)(w.q.row0 + my_tok) * A.q_stride + (size_t)my_head * d;
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
            const int ch = j * 4 + g;
            u32x4 a = {0u, 0u, 0u, 0u}, e = a;
            if (live && ch < dc) {
                a = ld16(qr + ch * 16);
                e = ld16(qr + ch * 16 + 8);
            }
            qf[2 * j] = __builtin_bit_cast(f16x8, a);
            qf[2 * j + 1] = __builtin_bit_cast(f16x8, e);
        }
    }
    // positions that every row of this workgroup attends to need no mask
    const int row_a = w.row_tile * ROWS / group;
    int row_b = (w.row_tile * ROWS + ROWS - 1) / group;
    if (row_b >= w.q.n) row_b = w.q.n - 1;
    const int free_to = first + row_a;                                                   // up to this one
    const int free_from = A.window > 0 ? first + row_b - A.window + 1 : 0;               // from this one on
    // and outside these, none attends
    const int any_to = first + row_b, any_from = A.window > 0 ? first + row_a - A.window + 1 : 0;

    float R = kNone, M = kNone, l = 0.f;
    f32x4 O[4 * KJ];
#pragma unroll
    for (int k = 0; k < 4 * KJ; ++k) O[k] = f32x4{0.f, 0.f, 0.f, 0.f};

    for (; tile < w.t1; tile += kAttWaves) {
        const int next = tile + kAttWaves;
        f32x4 S[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < KJ; ++j) {
                f16x2 c[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) Codes<FMT>::to_f16(kc[t][j][i], c[2 * i], c[2 * i + 1]);
                f16x8 a = {c[0].x, c[0].y, c[1].x, c[1].y, c[2].x, c[2].y, c[3].x, c[3].y};
                f16x8 e = {c[4].x, c[4].y, c[5].x, c[5].y, c[6].x, c[6].y, c[7].x, c[7].y};
                S[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, qf[2 * j], S[t], 0, 0, 0);
                S[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(e, qf[2 * j + 1], S[t], 0, 0, 0);
            }
        }
        if (next < w.t1) load_k(id, next);

        const float kx = pick(ks, g) * A.scale2, vl = pick(vs, g), lv = log2_fast(vl);
        const int key0 = tile * kTile + g * kGran;   // position of this lane's first key
        const bool edge = tile * kTile < free_from || tile * kTile + kTile - 1 > free_to;
        f16x8 ph[2], pl[2];   // the weights' leading and following halves: to 22 bits, at four more products a tile
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = S[i / 4][i % 4] * kx;
        if (edge) {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = key0 + i >= lo && key0 + i <= pos ? x[i] : -__builtin_inff();
        }
        float mx = x[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, x[i]);
        const float mr = max_groups(mx), mw = max_groups(mx + lv);
        if (__ballot(mr > R + kSlack || mw > M + kSlack)) {
            const float r = fmaxf(R, mr), m = fmaxf(fmaxf(M, mw), r - kFloor);
            l *= exp2_fast(R - r);
            const float f = exp2_fast(M - m);
#pragma unroll
            for (int k = 0; k < 4 * KJ; ++k) O[k] *= f;
            R = r;
            M = m;
        }
        const float up = vl * exp2_fast(R - M + kLift);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float p = exp2_fast(x[i] - R);
            sum += p;
            float wt = p * up;
            if (edge) wt = key0 + i >= lo && key0 + i <= pos ? wt : 0.f;
            const f16 hi = (f16)wt;
            ph[i / 8][i % 8] = hi;
            pl[i / 8][i % 8] = (f16)(wt - (float)hi);
        }
        l += sum;
        // fp8 slots that no row here attends to may hold NaN, which a zero weight would not silence
        if (FMT == 1 && (tile * kTile < any_from || tile * kTile + kTile - 1 > any_to)) {
#pragma unroll
            for (int k = 0; k < 4 * KJ; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int k0 = key0 + 4 * i;   // the word's tokens are k0 .. k0 + 3
                    const int have = any_to + 1 - k0, skip = any_from - k0;
                    uint32_t v = vc[k][i];
                    v = have >= 4 ? v : have <= 0 ? 0u : v & ((1u << (8 * have)) - 1u);
                    v = skip <= 0 ? v : skip >= 4 ? 0u : v & ~((1u << (8 * skip)) - 1u);
                    vc[k][i] = v;
                }
        }
#pragma unroll
        for (int k = 0; k < 4 * KJ; ++k) {
            f16x2 c[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) Codes<FMT>::to_f16(vc[k][i], c[2 * i], c[2 * i + 1]);
            f16x8 a = {c[0].x, c[0].y, c[1].x, c[1].y, c[2].x, c[2].y, c[3].x, c[3].y};
            f16x8 e = {c[4].x, c[4].y, c[5].x, c[5].y, c[6].x, c[6].y, c[7].x, c[7].y};
            O[k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, ph[0], O[k], 0, 0, 0);
            O[k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(e, ph[1], O[k], 0, 0, 0);
            O[k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pl[0], O[k], 0, 0, 0);
            O[k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(e, pl[1], O[k], 0, 0, 0);
        }
        if (next < w.t1) {
            load_v(id, next);
            scales(id, ks, vs);
            lookup(next + kAttWaves, id);
        }
    }

    // Join the waves that had tiles: statistics first, then every wave brings
    // its outputs to the common reference and the workgroup adds them up.
    const int parts = w.t1 - w.t0 < kAttWaves ? w.t1 - w.t0 : kAttWaves;
    float* outs = lds;                                   // [parts][ROWS][LD]
    float* stat = lds + kAttWaves * ROWS * LD;           // [parts][3][ROWS]: R, M, l
    float* done = stat + kAttWaves * 3 * ROWS;           // [3][ROWS]: the workgroup's
    const int rows = rows_all - w.row_tile * ROWS < ROWS ? rows_all - w.row_tile * ROWS : ROWS;
    l = sum_groups(l);
    if (g == 0 && wave < parts) {
        stat[(wave * 3 + 0) * ROWS + n16] = R;
        stat[(wave * 3 + 1) * ROWS + n16] = M;
        stat[(wave * 3 + 2) * ROWS + n16] = l;
    }
    __syncthreads();
    if (wave < parts) {
        float Rr = kNone, Mr = kNone, sum = 0.f;
        for (int p = 0; p < parts; ++p) {
            Rr = fmaxf(Rr, stat[(p * 3 + 0) * ROWS + n16]);
            Mr = fmaxf(Mr, stat[(p * 3 + 1) * ROWS + n16]);
        }
        const float f = exp2_fast(M - Mr);
#pragma unroll
        for (int k = 0; k < 4 * KJ; ++k)
            *reinterpret_cast<f32x4*>(&outs[(wave * ROWS + n16) * LD + k * 16 + g * 4]) = O[k] * f;
        if (wave == 0 && g == 0) {
            for (int p = 0; p < parts; ++p)
                sum = fmaf(stat[(p * 3 + 2) * ROWS + n16], exp2_fast(stat[(p * 3 + 0) * ROWS + n16] - Rr), sum);
            done[n16] = Rr;
            done[ROWS + n16] = Mr;
            done[2 * ROWS + n16] = sum;
        }
    }
    __syncthreads();

    // four outputs of a row, from its sum of weights and references in `done`
    auto emit = [&](int r, int i, f32x4 o) {
        const int gr = w.row_tile * ROWS + r, tok = gr / group, head = w.h * group + gr - tok * group;
        const size_t at = (size_t)(w.q.row0 + tok) * A.n_head + head;
        const bool empty = first + tok < 0;
        const float Rr = done[r], sum = done[2 * ROWS + r];
        // no weight at all although there are keys: every score was -infinity
        const float f = sum == 0.f ? __builtin_nanf("") : exp2_fast(done[ROWS + r] - Rr - kLift) / sum;
        typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
        f16x4 v;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = empty ? (f16)0.f : (f16)(o[k] * f);
        *reinterpret_cast<f16x4*>(A.y + at * d + i) = v;
        if (A.lse && i == 0) A.lse[at] = empty ? -__builtin_inff() : (Rr + log2_fast(sum)) * kLn2;
    };
    constexpr int kSlotBytes = ROWS * (DP + 4) * 4;   // outputs [ROWS][DP], then R, M, l and nothing [4][ROWS]
    const size_t step = (size_t)A.c.n_kv * kSlotBytes;
    char* item = reinterpret_cast<char*>(A.part) + ((size_t)w.slot * A.c.n_kv + w.h) * kSlotBytes;
    const __amdgpu_buffer_rsrc_t mine = buf_rsrc(item + w.split * step, kSlotBytes);
    for (int e = threadIdx.x; e < rows * (DP / 4); e += kAttThreads) {
        const int r = e / (DP / 4), i = e % (DP / 4) * 4;
        if (i >= d) continue;
        f32x4 o = *reinterpret_cast<const f32x4*>(&outs[r * LD + i]);
        for (int p = 1; p < parts; ++p) o += *reinterpret_cast<const f32x4*>(&outs[(p * ROWS + r) * LD + i]);
        if (w.splits == 1) emit(r, i, o);
        else st16_coherent(mine, (uint32_t)(r * DP + i) * 4, o);
    }
    if (w.splits == 1) return;
    for (int e = threadIdx.x; e < 3 * ROWS / 4; e += kAttThreads)
        st16_coherent(mine, (uint32_t)(ROWS * DP + e * 4) * 4, *reinterpret_cast<const f32x4*>(&done[e * 4]));

    // the last of the item's pieces to arrive joins them, in their order
    uint32_t* ctr = A.ctr + ((size_t)w.slot * A.c.n_kv + w.h) * kAttCtrStride;
    wait_own_memory();
    __syncthreads();
    if (threadIdx.x == 0) s_last = fetch_add_acq_rel(ctr, 1u) == (uint32_t)(w.splits - 1);
    __syncthreads();
    if (!s_last) return;
    // each row's references and sum over the pieces: a row's lanes take a piece each
    constexpr int kRowLanes = kAttThreads / ROWS;
    {
        const int r = threadIdx.x / kRowLanes, j = threadIdx.x % kRowLanes;
        float Rr = kNone, Mr = kNone, sum = 0.f;
        for (int p = j; p < w.splits; p += kRowLanes) {
            const float* at = reinterpret_cast<const float*>(item + p * step) + ROWS * DP + r;
            const float pr = ld_coherent(at), pm = ld_coherent(at + ROWS), ps = ld_coherent(at + 2 * ROWS);
            const float nr = fmaxf(Rr, pr);
            sum = sum * exp2_fast(Rr - nr) + ps * exp2_fast(pr - nr);
            Rr = nr;
            Mr = fmaxf(Mr, pm);
        }
#pragma unroll
        for (int off = 1; off < kRowLanes; off <<= 1) {
            const float pr = __shfl_xor(Rr, off, kWave), ps = __shfl_xor(sum, off, kWave);
            const float nr = fmaxf(Rr, pr);
            sum = sum * exp2_fast(Rr - nr) + ps * exp2_fast(pr - nr);
            Rr = nr;
            Mr = fmaxf(Mr, __shfl_xor(Mr, off, kWave));
        }
        if (j == 0) {
            done[r] = Rr;
            done[ROWS + r] = Mr;
            done[2 * ROWS + r] = sum;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < rows * (DP / 4); e += kAttThreads) {
        const int r = e / (DP / 4), i = e % (DP / 4) * 4;
        if (i >= d) continue;
        const float Mr = done[ROWS + r];
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
        for (int p = 0; p < w.splits; p += 16) {   // sixteen pieces' loads at a time
            f32x4 v[16];
            float m[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const char* at = item + (p + k < w.splits ? p + k : p) * step;
                v[k] = ld16_coherent(buf_rsrc(at, kSlotBytes), (uint32_t)(r * DP + i) * 4);
                m[k] = ld_coherent(reinterpret_cast<const float*>(at) + ROWS * DP + ROWS + r);
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float f = p + k < w.splits ? exp2_fast(m[k] - Mr) : 0.f;
                if (p + k < w.splits) o += v[k] * f;
            }
        }
        emit(r, i, o);
    }
    if (threadIdx.x == 0) st_flag(ctr, 0u);
}

// A workgroup takes units until there are none: whatever the lengths on the
// device say, every piece of every item runs, and the counters end at zero.
template <int FMT, int KJ>
__global__ __launch_bounds__(kAttThreads, KJ == 4 ? 1 : KJ == 2 ? 2 : 3) void k_attend(AttArgs A) {
    AttUnit w;
    w.h = blockIdx.x;
    const int units = att_plan(A, blockIdx.y, w);
    for (int u = blockIdx.y; u < units;) {
        attend_unit<FMT, KJ>(A, w);
        u += gridDim.y;
        if (u < units) {
            __syncthreads();   // the next unit uses the same shared memory
            att_plan(A, u, w);
        }
    }
}

static int att_kj(int d) { return d <= 64 ? 1 : d <= 128 ? 2 : 4; }

static long long att_row_tiles(const KvBatch& b, int group) {
    const long long each = (long long)b.n_seq * (((long long)b.max_q * group + kAttRows - 1) / kAttRows);
    const long long all = (long long)b.n_tok * group / kAttRows + b.n_seq;
    return each < all ? each : all;
}

size_t kv_attend_zero_bytes() { return (size_t)kAttSlots * kAttCtrStride * 4; }

size_t kv_attend_bytes(int, int, int, int, int, int d) {
    return kv_attend_zero_bytes() + (size_t)kAttSlots * kAttRows * (64 * att_kj(d) + 4) * 4;
}

hipError_t launch_kv_attend(const KvCache& c, const KvBatch& b, const h16* q, long long q_stride, int n_head,
                            float scale, int window, h16* y, float* lse, char* data, hipStream_t s) {
    const int group = n_head / c.n_kv, kj = att_kj(c.d), target = att_target(kj);
    AttArgs A{c, b, q, q_stride, n_head, group, window, target, scale * 1.4426950408889634f, y, lse,
              reinterpret_cast<uint32_t*>(data), reinterpret_cast<float*>(data + kv_attend_zero_bytes())};
    const long long items = att_row_tiles(b, group);
    const long long cap = ((long long)b.table_stride * c.page + kTile - 1) / kTile;
    const long long most = items * ((cap + kAttMinTiles - 1) / kAttMinTiles);
    long long units = items + (target + c.n_kv - 1) / c.n_kv;
    if (units > most) units = most;
    if (units > 65535) units = 65535;
    // heads side by side: the row tiles that read one head's pages run on one
    // XCD where the heads are a multiple of 8, and share its L2
    const dim3 grid(c.n_kv, (unsigned)units);
    const size_t shm = ((size_t)kAttWaves * (64 * kj + 4 + 3) + 3) * kAttRows * 4;
    hipError_t e = hipSuccess;
#define PI_ATT(F, K)                                                                               \
    do {                                                                                           \
        if (shm > 65536)                                                                           \
            e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_attend<F, K>),                \
                                    hipFuncAttributeMaxDynamicSharedMemorySize, (int)shm);         \
        if (e == hipSuccess) hipLaunchKernelGGL((k_attend<F, K>), grid, dim3(kAttThreads), shm, s, A); \
    } while (0)
#define PI_ATT_D(F)                \
    if (kj == 1) PI_ATT(F, 1);      \
    else if (kj == 2) PI_ATT(F, 2); \
    else PI_ATT(F, 4)
    if (c.fmt == 0) { PI_ATT_D(0); } else { PI_ATT_D(1); }
#undef PI_ATT_D
#undef PI_ATT
    if (e != hipSuccess) return e;
    return hipGetLastError();
}

}  // namespace pi
