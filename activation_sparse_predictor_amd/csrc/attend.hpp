// What the two attention kernels share: attend.hip, a wave's keys against 16
// query rows of a sequence (single tokens), and prompt.hip, tiles of keys
// against hundreds of rows.
#pragma once

#include "kv.hpp"

namespace pi {

constexpr int kTile = 64;          // keys a wave takes at a time
constexpr int kAttMaxTarget = 512;   // most workgroups that the work is split into on purpose
// pieces of split items: with C >= tiles / target, ceil(t / C) < 2 t / C where t > C
constexpr int kAttSlots = 2 * kAttMaxTarget;
constexpr int kAttCtrStride = 16;    // words between arrival counters

constexpr float kZeroLog = -64.f, kNone = -1e30f, kLn2 = 0.69314718055994531f;

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
    int n_head, group, window;
    int above, upto;         // this kernel's sequences: those with more rows than `above`, at most `upto`
    int target, min_tiles;   // workgroups the work is split into, and the least tiles of att_plan's C
    float scale2;            // scale * log2(e)
    h16* y;
    float* lse;
    uint32_t* ctr;
    float* part;
};

// What a workgroup works on: a row tile of a sequence, its keys' tiles
// [t0, t1), head h; piece `split` of `splits`, whose first has slot `slot`.
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

// The tiles that rows [row_tile * ROWS, + ROWS) attend to: the first, and how many.
template <int ROWS>
__device__ __forceinline__ int att_row_tiles(const AttArgs& A, const Seq& q, int row_tile, int& first_tile) {
    const int a = row_tile * ROWS / A.group;
    int b = (row_tile * ROWS + ROWS - 1) / A.group;
    b = b < q.n ? b : q.n - 1;
    const int from = A.window > 0 ? q.ctx - q.n + a - A.window + 1 : 0, to = q.ctx - q.n + b;
    first_tile = from > 0 ? from / kTile : 0;
    return to < 0 ? 1 : to / kTile - first_tile + 1;
}

// Tiles of a piece, before items that run at once are fitted: `want`, but at
// least min_tiles, and never above the 2^24 tiles of the longest context (2^30
// tokens), so that the fitting and the divisions stay far below 2^31 (row ranges
// that overlap, or a table that names pages again and again, can ask for more).
__host__ __device__ constexpr int att_piece(float want, int min_tiles) {
    return want < (float)min_tiles ? min_tiles : want < 16777216.f ? (int)want + 1 : 16777216;
}

// Splits the whole batch's tiles over about A.target workgroups: C tiles a
// workgroup, the same for every sequence, from the lengths as they are on the
// device.  Each item (sequence, row tile) becomes ceil(tiles / C) pieces, for
// each head, that share its own tiles evenly (`tiles` is the whole sequence's:
// the early rows of a prompt, and rows under a short window, have fewer, and
// their pieces may have one tile or none); the last rows, which attend to most,
// come first.  Every wave computes it for itself: a
// round of 64 sequences is one round of loads.  Fills in unit `item`, if there
// is one, and returns how many there are (of each head).  With at most 2^24
// rows and 2^10 sequences, whatever the lengths say, the sums stay below 2^31.
template <int ROWS>
__device__ __forceinline__ int att_plan(const AttArgs& A, int item, AttUnit& w) {
    const KvBatch& b = A.b;
    auto row_tiles = [&](const Seq& q) {
        const int rows = q.n * A.group;
        return rows > A.above && rows <= A.upto ? (rows + ROWS - 1) / ROWS : 0;
    };
    float all = 0.f, items = 0.f;   // C only has to be the same everywhere
    Seq q{-1, 0, 0, 0};
    int rt = 0, tiles = 1;
    for (int s0 = 0; s0 < b.n_seq; s0 += kWave) {
        const int s = s0 + lane_id();
        rt = 0;
        if (s < b.n_seq) {
            q = kv_seq(b, s);
            rt = row_tiles(q);
            tiles = att_tiles(q, A.window);
        }
        all += group_sum<64>((float)rt * (float)tiles);
        items += group_sum<64>((float)rt);
    }
    const float room = (float)A.target / (float)A.c.n_kv;   // workgroups a head has
    const float want = all / room * 1.001f;                 // a little above: the slots rest on it
    int C = att_piece(want, A.min_tiles);
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
                rt = row_tiles(q);
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
            const int rts = __builtin_amdgcn_readlane(rt, l);
            const int inside = item - (__builtin_amdgcn_readlane(upto, l) - rts * w.splits);
            const int behind = inside / w.splits;
            w.row_tile = rts - 1 - behind;
            w.split = inside - behind * w.splits;
            w.slot = __builtin_amdgcn_readlane(slots_upto, l) - __builtin_amdgcn_readlane(held, l) +
                     behind * w.splits;   // the item's first slot
            int f;
            const int T = att_row_tiles<ROWS>(A, w.q, w.row_tile, f);
            const int each = T / w.splits, more = T - each * w.splits;
            w.t0 = f + w.split * each + (w.split < more ? w.split : more);
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
__device__ __forceinline__ void st8_coherent(__amdgpu_buffer_rsrc_t r, uint32_t at, float a, float b) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(a), __float_as_uint(b)}, r, (int)at, 0, 16);
}
__device__ __forceinline__ f32x4 ld16_coherent(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t from) {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)at, (int)from, 16));
}
__device__ __forceinline__ float ld4_coherent(__amdgpu_buffer_rsrc_t r, uint32_t at) {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (int)at, 0, 16));
}

// A granule of the sequence: where its bytes start in the pools, and its
// page's scales as the loop uses them.
struct Gran {
    uint32_t lo, hi;   // byte offset
    float kx, lv;      // ks * |scale| * log2(e);  log2 vs
};
constexpr int kSegTiles = 128;   // tiles whose granules are looked up at a time
constexpr int kSegGrans = kSegTiles * (kTile / kGran);

// Looks up granules [first, first + count) of a sequence, `threads` threads an
// entry each.  Past its end: its last granule, masked later.
__device__ __forceinline__ void att_lookup(const AttArgs& A, const AttUnit& w, int d, int first, int count, int tid,
                                           int threads, Gran* out) {
    const int page = A.c.page, shift = __builtin_ctz(page), last = w.q.ctx > 0 ? (w.q.ctx - 1) / kGran : 0;
    const int32_t* table = A.b.table + (size_t)w.q.s * A.b.table_stride;
    const uint32_t page_bytes = (uint32_t)A.c.n_kv * page * d;   // of all heads: at most 2^26
    const float scale2 = fabsf(A.scale2), nan = __builtin_nanf("");
    for (int i = tid; i < count; i += threads) {
        int gi = first + i;
        gi = gi < last ? gi : last;
        int id = w.q.ctx > 0 ? table[gi * kGran >> shift] : -1;
        const bool known = id >= 0 && id < A.c.n_pages;
        id = known ? id : 0;
        const size_t si = (size_t)id * A.c.n_kv + w.h;
        const float ks = A.c.k_scale[si], vs = A.c.v_scale[si];
        const size_t off = (size_t)id * page_bytes + (size_t)(w.h * page * d) + (size_t)((gi * kGran & (page - 1)) * d);
        out[i] = Gran{(uint32_t)off, (uint32_t)(off >> 32), known ? ks * scale2 : nan,
                      !known ? nan : vs < 0x1p-64f ? kZeroLog : log2_fast(vs)};
    }
}
__device__ __forceinline__ const uint8_t* gran_at(const uint8_t* pool, const Gran& e) {
    return pool + (((size_t)e.hi << 32) | e.lo);
}

// A word of four V codes of the tokens from key0 on, those outside [from, to]
// zeroed: fp8 slots that nobody attends to may hold NaN, which a zero weight
// would not silence.
__device__ __forceinline__ uint32_t keep_tokens(uint32_t v, int key0, int from, int to) {
    const int have = to + 1 - key0, skip = from - key0;
    v = have >= 4 ? v : have <= 0 ? 0u : v & ((1u << (8 * have)) - 1u);
    return skip <= 0 ? v : skip >= 4 ? 0u : v & ~((1u << (8 * skip)) - 1u);
}

// Eight codes of two words as fp16.
template <int FMT>
__device__ __forceinline__ f16x8 codes8(uint32_t a, uint32_t b) {
    f16x2 c[4];
    Codes<FMT>::to_f16(a, c[0], c[1]);
    Codes<FMT>::to_f16(b, c[2], c[3]);
    return f16x8{c[0].x, c[0].y, c[1].x, c[1].y, c[2].x, c[2].y, c[3].x, c[3].y};
}

// Row tiles of `rows` rows that the batch can have.
inline long long att_most_row_tiles(const KvBatch& b, int group, int rows) {
    const long long each = (long long)b.n_seq * (((long long)b.max_q * group + rows - 1) / rows);
    const long long all = (long long)b.n_tok * group / rows + b.n_seq;
    return each < all ? each : all;
}
// Units of one head that the plan can come to (more would be taken in turn).
inline unsigned att_grid(const AttArgs& A, int rows) {
    const long long items = att_most_row_tiles(A.b, A.group, rows);
    const long long cap = ((long long)A.b.table_stride * A.c.page + kTile - 1) / kTile;
    const long long most = items * ((cap + A.min_tiles - 1) / A.min_tiles);
    long long units = items + (A.target + A.c.n_kv - 1) / A.c.n_kv;
    if (units > most) units = most;
    return (unsigned)(units < 65535 ? units : 65535);
}

// 64-dimension steps of a head, as the kernels are built for
__host__ __device__ constexpr int att_kj(int d) { return d <= 64 ? 1 : d <= 128 ? 2 : 4; }

// prompt.hip
constexpr int prompt_rows(int kj) { return kj == 4 ? 64 : 128; }
hipError_t launch_attend_prompt(AttArgs A, hipStream_t s);

}  // namespace pi
