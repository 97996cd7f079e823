// What the two attention kernels share: attend.hip, a wave's keys against 16
// query rows of a sequence (single tokens), and prompt.hip, tiles of keys
// against hundreds of rows.
#pragma once

#include <type_traits>

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

// Attention of drafted tokens (pi_kv_attend_tree): every row sees the cached
// tokens, all ctx of them or, under a window, those above its own position less
// the window, and the drafted rows that its mask names.  The drafted rows are
// further tiles of 64 keys, before the cached ones.  In attend.hip their loads are
// under way while the cached granules are looked up; prompt.hip looks up first,
// then loads, stores and multiplies one drafted tile after the other.
struct TreeArgs : AttArgs {
    const h16 *tk, *tv;            // drafted keys and values: n_tok rows
    long long tk_stride, tv_stride;
    const uint64_t* mask;          // n_tok x words
    int words;
    const int32_t* pos;            // n_tok; only read under a window
    int at_once;                   // prompt.hip: workgroups that the chip holds (target: the bound that the slots rest on); attend.hip: 0
};
constexpr int kMaxDrafted = 4;     // tiles of drafted rows (words)
template <class ARGS> constexpr bool is_tree = std::is_same_v<ARGS, TreeArgs>;

// Cached positions below this one are outside a drafted row's window.
__device__ __forceinline__ int tree_from(const TreeArgs& A, int ctx, int row) {
    if (A.window <= 0) return 0;
    const int p = A.pos[row];
    const int from = (p > ctx ? p : ctx) - A.window + 1;
    return from > 0 ? from : 0;
}
// The drafted rows of tile x that row `row` of a sequence of n rows attends to, as bits.
__device__ __forceinline__ uint64_t tree_bits(const TreeArgs& A, int row, int n, int x) {
    if (x >= A.words) return 0ull;
    const uint64_t m = A.mask[(size_t)row * A.words + x];
    const int have = n - x * kTile;
    return have >= kTile ? m : have <= 0 ? 0ull : m & ((1ull << have) - 1);
}
__device__ __forceinline__ uint64_t tree_bits(const AttArgs&, int, int, int) { return 0ull; }   // no drafted rows
// Whether a drafted row attends to anything.
__device__ __forceinline__ bool tree_sees(const TreeArgs& A, const Seq& q, int tok) {
    if (tree_from(A, q.ctx, q.row0 + tok) < q.ctx) return true;
    for (int x = 0; x < A.words; ++x)
        if (tree_bits(A, q.row0 + tok, q.n, x)) return true;
    return false;
}
// A drafted token's value that is not finite would reach, times a weight of 0,
// rows that do not attend to it.  It is taken as 0, and the token's bit goes
// into `bad`, which makes the sums of the rows that do attend to it NaN.
// v: a dimension's 16 tokens.
__device__ __forceinline__ void drop_nonfinite(u32x4 (&v)[2], uint32_t& bad) {
    uint32_t any = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) any |= ((v[i / 4][i % 4] & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
    if (!__ballot(any != 0u)) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t x = v[i / 4][i % 4], top = ((x & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
        bad |= ((top >> 15 & 1u) | (top >> 30 & 2u)) << (2 * i);
        v[i / 4][i % 4] = x & ~((top >> 15) * 0xFFFFu);
    }
}
// Over the 16 lanes of one g: bits that any has, and the largest.
__device__ __forceinline__ uint32_t or_lanes16(uint32_t v) {
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) v |= __shfl_xor(v, m, kWave);
    return v;
}
__device__ __forceinline__ int max_lanes16(int v) {
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) {
        const int o = __shfl_xor(v, m, kWave);
        v = o > v ? o : v;
    }
    return v;
}

// What a workgroup works on: a row tile of a sequence, its keys' tiles
// [t0, t1), head h; piece `split` of `splits`, whose first has slot `slot`.
struct AttUnit {
    Seq q;
    int h, row_tile, t0, t1, split, splits, slot;
};

// First tile of a sequence that any of its rows attends to, and the tiles in all (at least one).
template <bool TREE>
__device__ __forceinline__ int att_first_tile(const Seq& q, int window) {
    const int lo = q.ctx - (TREE ? 0 : q.n) - window + 1;
    return window > 0 && lo > 0 ? lo / kTile : 0;
}
__device__ __forceinline__ int tree_drafted(const TreeArgs& A, const Seq& q) {   // at most the mask's, whatever the lengths say
    const int n = (q.n + kTile - 1) / kTile;
    return n < A.words ? n : A.words;
}
template <class ARGS>
__device__ __forceinline__ int att_tiles(const ARGS& A, const Seq& q) {
    const int n = (q.ctx + kTile - 1) / kTile - att_first_tile<is_tree<ARGS>>(q, A.window);
    if constexpr (is_tree<ARGS>) return n + tree_drafted(A, q);
    return n > 0 ? n : 1;
}

// The tiles that rows [row_tile * ROWS, + ROWS) attend to: the first, and how many.
template <int ROWS, class ARGS>
__device__ __forceinline__ int att_row_tiles(const ARGS& A, const Seq& q, int row_tile, int& first_tile) {
    if constexpr (is_tree<ARGS>) {
        first_tile = 0;   // of its drafted and cached tiles together
        return att_tiles(A, q);
    }
    const int a = row_tile * ROWS / A.group;
    int b = (row_tile * ROWS + ROWS - 1) / A.group;
    b = b < q.n ? b : q.n - 1;
    const int from = A.window > 0 ? q.ctx - q.n + a - A.window + 1 : 0, to = q.ctx - q.n + b;
    first_tile = from > 0 ? from / kTile : 0;
    return to < 0 ? 1 : to / kTile - first_tile + 1;
}

// A unit's tiles as its drafted ones, [w.t0, + drafted), and its cached ones, [from, to).
struct TreeTiles {
    int drafted, from, to;
};
__device__ __forceinline__ TreeTiles tree_tiles(const TreeArgs& A, const AttUnit& w) {
    const int nt = tree_drafted(A, w.q), f = att_first_tile<true>(w.q, A.window) - nt;
    const int a = w.t0 > nt ? w.t0 : nt, b = w.t1 > nt ? w.t1 : nt, d = (w.t1 < nt ? w.t1 : nt) - w.t0;
    return TreeTiles{d > 0 ? d : 0, f + a, f + b};
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
template <int ROWS, class ARGS>
__device__ __forceinline__ int att_plan(const ARGS& A, int item, AttUnit& w) {
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
            tiles = att_tiles(A, q);
        }
        all += group_sum<64>((float)rt * (float)tiles);
        items += group_sum<64>((float)rt);
    }
    const float room = (float)A.target / (float)A.c.n_kv;   // workgroups a head has
    const float want = all / room * 1.001f;                 // a little above: the slots rest on it
    int C = att_piece(want, A.min_tiles);
    // the smallest C from `from` on (to a sixteenth) whose rounded-up pieces are at most `most`
    auto fit = [&](int from, float most) {
        int c = from;
        for (int i = 0; i < 24; ++i) {
            if (group_sum<64>((float)(rt * ((tiles + c - 1) / c))) <= most) break;
            c += c / 16 + 1;
        }
        return c;
    };
    float once = room;
    if constexpr (is_tree<ARGS>) once = A.at_once > 0 ? (float)A.at_once / (float)A.c.n_kv : room;
    if (b.n_seq <= kWave && items <= once) {
        // All items can run at once.
        const float wish = all / once * 1.001f;
        C = fit(att_piece(wish, A.min_tiles), once);
        if constexpr (is_tree<ARGS>) {
            // Items alike in length do not divide into just any number of workgroups:
            // where one turn of pieces would leave many idle, two turns of shorter ones
            // (each with its start and join, about eight tiles' time) may end earlier (9 trees
            // of 64 rows of 64 heads, 8 kv, on 4096 tokens: 137 us against 169).  For
            // single rows' pieces they never did (12 trees of up to 48 rows of 8 kv heads of 256
            // on up to 4096 tokens: 73 us, 68 in one turn).
            const float slots = (float)kAttSlots / (float)A.c.n_kv, twice = 2.f * once < slots ? 2.f * once : slots;
            if (A.at_once > 0 && (float)C > 1.5f * wish && C > 32) {
                const int c = fit(att_piece(0.5f * wish, A.min_tiles), twice);
                if (2 * (c + 8) < C + 8) C = c;
            }
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
                tiles = att_tiles(A, q);
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
            const int T = att_row_tiles<ROWS, ARGS>(A, w.q, w.row_tile, f);
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
inline unsigned att_grid(const AttArgs& A, int rows, int drafted_tiles = 0, int at_once = 0) {
    const long long items = att_most_row_tiles(A.b, A.group, rows);
    const long long cap = ((long long)A.b.table_stride * A.c.page + kTile - 1) / kTile + drafted_tiles;
    const long long most = items * ((cap + A.min_tiles - 1) / A.min_tiles);
    const int most_units = 2 * at_once > A.target ? 2 * at_once : A.target;
    long long units = items + (most_units + A.c.n_kv - 1) / A.c.n_kv;
    if (units > most) units = most;
    return (unsigned)(units < 65535 ? units : 65535);
}

// 64-dimension steps of a head, as the kernels are built for
__host__ __device__ constexpr int att_kj(int d) { return d <= 64 ? 1 : d <= 128 ? 2 : 4; }

// prompt.hip
constexpr int prompt_rows(int kj) { return kj == 4 ? 64 : 128; }
hipError_t launch_attend_prompt(AttArgs A, hipStream_t s);
hipError_t launch_attend_prompt(TreeArgs A, hipStream_t s);

}  // namespace pi
