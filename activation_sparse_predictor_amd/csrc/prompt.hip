// Attention of many rows over the 8-bit paged cache (prompts).
//
// The mathematics, the references and the operands' order are those of
// attend.hip.  Here the matrix cores are the bound, and next to them LDS: a
// workgroup of four waves carries 128 rows (64 for heads above 128 dimensions),
// 32 a wave, and the waves share every tile of 64 keys through LDS, where it is
// kept as fp16 in the order of the operands' fragments (1 KB each, a lane's 16
// bytes in lane order: no bank conflicts).  Each thread turns its 16-byte
// pieces of codes into fp16 once for the workgroup.  Two tiles are held: while
// one is used the next is written, and the one after is on its way in
// registers, so one barrier a tile is all.  A fragment read from LDS serves the
// wave's two 16-row operands.  Two workgroups share a CU, so that one's weights
// (vector work) run beside the other's products.  As in attend.hip the weights
// enter as a leading and a following fp16 half (21 bits), so that which kernel a
// call's sizes choose does not show in a row's precision.  Rounded to fp16 once
// they cost a third fewer products (79-94 us against 97-113 below), but an
// error of 2^-11 a weight, as large as the rounding of the output itself.
//
// Measured: 2048 tokens of 56 heads of 128 (60 GFLOP) in 97-113 us, 530-620
// TFLOP/s, by the card; 509 tokens of 64 heads beside seven short sequences (65
// GFLOP) in 111-124, of which the other kernel's 16.  A large matrix product
// reaches 1.4 PFLOP/s, and the following halves are half as many products again.
// What is between: a tile's 96 products of a wave (1536 cycles, 36 % of the
// kernel's) stand beside 250 vector instructions (weights, codes to fp16; five
// cycles each, more beside another wave's products) and 32 fragments from LDS.
// LDS is a fifth busy, without bank conflicts.
//
// Drafted tokens: 5 trees of 64 rows of 64 heads, 8 kv, on 8192 cached tokens (86 GFLOP)
// 128 us, 670 TFLOP/s; 16 ragged ones of 6 to 16 rows (30 GFLOP, 181 MB) 81 us; 6 of 63
// of 128 heads of 64 under a window (40 GFLOP) 85.  Of those some 20 are a piece's start and
// end: the plan, the granules' look-up, the drafted tile and the join.
#include "attend.hpp"

namespace pi {

// The reference moves when a maximum is more than 2.9 above it, which after a
// row's first tiles hardly happens (a move multiplies all outputs; with 0.25,
// as in attend.hip, moves took a tenth of the time).  fp16 then holds a weight
// down to 2^-37 of the row's largest.
constexpr float kLift = 13.f, kSlack = 2.9f;
constexpr int kProWaves = 4;
constexpr int kProThreads = kProWaves * kWave;
constexpr int pro_target(int kj) { return kj == 4 ? 256 : 512; }   // workgroups that run at once, by LDS
constexpr int kProMinTiles = 8;     // tiles a piece of a whole context has at least
constexpr int kProSeg = 64;         // tiles whose granules are looked up at a time
constexpr int kProRing = 2 * kProSeg;
// Polls before the join gives up on the other pieces, which are done and only
// have their results to write (some microseconds; this is tens of milliseconds).
constexpr int kProWaitLimit = 1 << 16;

// The waves' LDS writes are done and all of them are here.  Unlike
// __syncthreads this does not wait for the loads of the tile after next.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory"); }

// Two numbers as fp16, rounded towards zero.
__device__ __forceinline__ f16x2 cut2(float a, float b) { return __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_pkrtz(a, b)); }

template <int FMT, int KJ, bool FULL, class ARGS>
__device__ __forceinline__ void prompt_unit(const ARGS& A, const AttUnit& w) {
    constexpr bool TREE = is_tree<ARGS>;
    static_assert(kProWaves == 4 && kProWaves % KJ == 0, "a thread's pieces");
    constexpr int NT = KJ == 4 ? 1 : 2, ROWS = kProWaves * 16 * NT, DP = 64 * KJ;
    static_assert(ROWS == prompt_rows(KJ), "rows of a workgroup");
    constexpr int kFrags = 16 * KJ;   // of a tile: 8 KJ of K, 8 KJ of V
    extern __shared__ u32x4 frags[];  // [2][kFrags][64]
    __shared__ Gran grans[kProRing * (kTile / kGran)];
    __shared__ int s_last, s_written;
    __shared__ uint32_t s_bad[TREE ? kMaxDrafted : 1][kTile / kGran];   // drafted tokens whose values are not finite
    // (settled, so that what follows from them is not kept in registers from
    // unit to unit)
    const int lane = settle(lane_id()), wave = __builtin_amdgcn_readfirstlane(settle((int)threadIdx.x) / kWave);
    const int n16 = lane & 15, g = lane >> 4;
    const int d = FULL ? DP : A.c.d, dc = d / 16, group = A.group;
    const int first = w.q.ctx - w.q.n, rows_all = w.q.n * group;
    const int n = w.t1 - w.t0;
    // the unit's first tiles are drafted rows, nd of them; tile x >= nd is the cache's tile c0 + x
    int nd = 0, c0 = w.t0;
    if constexpr (TREE) {
        const TreeTiles t = tree_tiles(A, w);
        nd = t.drafted, c0 = t.from - nd;
    }

    auto fill = [&](int x, int count) {   // tiles [x, x + count) of this unit, into their places of the ring
        att_lookup(A, w, d, (c0 + x) * (kTile / kGran), count * (kTile / kGran), threadIdx.x, kProThreads,
                   &grans[(x & (kProRing - 1)) * (kTile / kGran)]);
    };

    // rows and positions: the workgroup's, this wave's, this lane's
    auto last_tok = [&](int r) {
        const int t = r / group;
        return t < w.q.n ? t : w.q.n - 1;
    };
    const int row_w = w.row_tile * ROWS, row_v = row_w + wave * 16 * (TREE ? 1 : NT);
    // A wave's operand nt has rows [row_of(nt), + 16).  Drafted rows are often fewer
    // than a workgroup's 128: they fill the waves' first operands before any
    // second one, so that no wave has two while another has none.
    auto row_of = [&](int nt) {
        if (!TREE) return row_v + nt * 16;
        return nt == 0 ? row_v : row_w + (kProWaves + wave) * 16;
    };
    const int operands = TREE && NT == 2 && row_of(NT - 1) >= rows_all ? 1 : NT;
    int any_to = first + last_tok(row_w + ROWS - 1);
    int any_from = A.window > 0 ? first + row_w / group - A.window + 1 : 0;
    const bool idle = row_v >= rows_all;
    int v_to = idle ? -1 : first + last_tok(row_v + 16 * NT - 1), v_free_to = first + row_v / group;
    int v_from = A.window > 0 ? first + row_v / group - A.window + 1 : 0;
    int v_free_from = A.window > 0 ? v_to - A.window + 1 : 0;
    if constexpr (TREE) {
        any_to = v_free_to = w.q.ctx - 1;
        v_to = idle ? -1 : w.q.ctx - 1;
        any_from = v_from = A.window > 0 ? w.q.ctx - A.window + 1 : 0;
        v_free_from = 0;
    }
    int pos[NT], lo[NT];
    f16x8 qf[NT][2 * KJ];
    const uint32_t sign = A.scale2 < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = row_of(nt) + n16;
        const bool live = r < rows_all;
        const int tok = live ? r / group : 0, head = w.h * group + (live ? r - tok * group : 0);
        pos[nt] = !live ? -1 : TREE ? w.q.ctx - 1 : first + tok;
        lo[nt] = A.window > 0 && pos[nt] - A.window + 1 > 0 ? pos[nt] - A.window + 1 : 0;
        if constexpr (TREE) {
            lo[nt] = live ? tree_from(A, w.q.ctx, w.q.row0 + tok) : 0;
            const int most = A.window > 0 ? __builtin_amdgcn_readfirstlane(max_lanes16(lo[nt])) : 0;
            v_free_from = most > v_free_from ? most : v_free_from;
        }
        const h16* qr = A.q + (size_t)(w.q.row0 + tok) * A.q_stride + (size_t)head * d;
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
            const int ch = j * 4 + g;
            u32x4 a = {0u, 0u, 0u, 0u}, e = a;
            if (live && ch < dc) {
                a = ld16(qr + ch * 16);
                e = ld16(qr + ch * 16 + 8);
            }
            qf[nt][2 * j] = __builtin_bit_cast(f16x8, a ^ sign);
            qf[nt][2 * j + 1] = __builtin_bit_cast(f16x8, e ^ sign);
        }
    }

    // This thread's 2 KJ pieces of a tile's codes: of the 4 KJ groups of 64
    // pieces of K, then the 4 KJ of V, wave v takes groups v, v + 4, ..., which
    // lie a fixed distance apart.
    u32x4 st[2 * KJ];
    const uint8_t* const k0 = A.c.k + (wave / KJ) * 4 * d + (wave % KJ * 4 + g) * 64 + (n16 & 3) * 16;
    const uint8_t* const v0 = A.c.v + (wave * 16 + n16) * 16;
    auto load = [&](int x) __attribute__((always_inline)) {
        const Gran* gr = &grans[(x & (kProRing - 1)) * (kTile / kGran)];
        const uint8_t* const kp = gran_at(k0, gr[n16 >> 2]);
        const uint8_t* const vp = gran_at(v0, gr[g]);
#pragma unroll
        for (int i = 0; i < KJ; ++i) {
            const u32x4 zero = {Codes<FMT>::kZero4, Codes<FMT>::kZero4, Codes<FMT>::kZero4, Codes<FMT>::kZero4};
            st[i] = st[KJ + i] = zero;
            if (FULL || wave % KJ * 4 + g < dc) st[i] = ld16(kp + i * (kProWaves / KJ) * 4 * d);
            if (FULL || wave + 4 * i < dc) st[KJ + i] = ld16(vp + i * kProWaves * 256);
        }
    };
    auto store = [&](int x, int i) __attribute__((always_inline)) {   // piece i
        const int tile0 = (c0 + x) * kTile, key0 = tile0 + g * kGran;
        u32x4* to = frags + ((x & 1) * kFrags + 2 * wave) * 64 + lane;
        u32x4 v = st[i];
        if (FMT == 1 && i >= KJ && (tile0 < any_from || tile0 + kTile - 1 > any_to)) {   // slots that no row here attends to may hold NaN
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = keep_tokens(v[j], key0 + 4 * j, any_from, any_to);
        }
        // group u of K makes fragments 2 u and 2 u + 1 of the tile, group u of V 8 KJ + 2 u and the next
        to[i * 2 * kProWaves * 64] = __builtin_bit_cast(u32x4, codes8<FMT>(v.x, v.y));
        to[(i * 2 * kProWaves + 1) * 64] = __builtin_bit_cast(u32x4, codes8<FMT>(v.z, v.w));
    };

    // Drafted tile x: fp16 rows as they are, into the fragments' places.  Keys as
    // above; of the values, two neighbouring dimensions of a granule's tokens a thread.
    constexpr int kDraftV = TREE ? (KJ + 1) / 2 : 1;   // (one head dimension in 64: half of the threads)
    u32x4 dk[TREE ? 2 * KJ : 1];
    uint32_t dv[kDraftV][kGran];
    auto load_drafted = [&](int x) __attribute__((always_inline)) {
        if constexpr (TREE) {
            const int tok0 = (w.t0 + x) * kTile, rows = w.q.n;
            auto row = [&](int tok) { return (size_t)(w.q.row0 + (tok < rows ? tok : rows - 1)); };
            const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int i = 0; i < KJ; ++i) {
                const int t = wave / KJ + i * (kProWaves / KJ), ch = wave % KJ * 4 + g;
                const h16* p = A.tk + row(tok0 + (n16 >> 2) * kGran + t * 4 + (n16 & 3)) * A.tk_stride + (size_t)w.h * d + ch * 16;
                dk[2 * i] = dk[2 * i + 1] = zero;
                if (FULL || ch < dc) dk[2 * i] = ld16(p), dk[2 * i + 1] = ld16(p + 8);
            }
#pragma unroll
            for (int t = 0; t < kGran; ++t) {
                const h16* p = A.tv + row(tok0 + g * kGran + t) * A.tv_stride + (size_t)w.h * d;
#pragma unroll
                for (int i = 0; i < kDraftV; ++i) {
                    const int dim = (wave + 4 * i) * 32 + 2 * n16;
                    dv[i][t] = (FULL && KJ > 1) || dim < d ? *reinterpret_cast<const uint32_t*>(p + dim) : 0u;
                }
            }
        }
    };
    auto store_drafted = [&](int x) __attribute__((always_inline)) {
        if constexpr (TREE) {
            u32x4* const tile = frags + (x & 1) * kFrags * 64;
#pragma unroll
            for (int i = 0; i < KJ; ++i) {
                tile[(2 * (wave + 4 * i)) * 64 + lane] = dk[2 * i];
                tile[(2 * (wave + 4 * i) + 1) * 64 + lane] = dk[2 * i + 1];
            }
            uint32_t bad = 0u;
#pragma unroll
            for (int i = 0; i < kDraftV; ++i) {
                if ((wave + 4 * i) * 32 >= DP) continue;
#pragma unroll
                for (int o = 0; o < 2; ++o) {   // dimension (wave + 4 i) 32 + 2 n16 + o: fragment pair, and lane in it
                    u32x4 v[2];
#pragma unroll
                    for (int t = 0; t < 8; ++t)
                        v[t / 4][t % 4] = __builtin_amdgcn_perm(dv[i][2 * t + 1], dv[i][2 * t], o ? 0x07060302u : 0x05040100u);
                    drop_nonfinite(v, bad);
                    u32x4* to = tile + (8 * KJ + 2 * ((wave + 4 * i) * 2 + (n16 >> 3))) * 64 + g * 16 + (2 * n16 + o) % 16;
                    to[0] = v[0];
                    to[64] = v[1];
                }
            }
            if (bad) atomicOr(&s_bad[(w.t0 + x) & (kMaxDrafted - 1)][g], bad);
        }
    };

    const float minus = settle(-1.f);   // (a constant would turn the differences below into a conversion and a subtraction each)
    float M[NT], l[NT];
    f32x4 O[NT][4 * KJ];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        M[nt] = kNone;
        l[nt] = 0.f;
#pragma unroll
        for (int k = 0; k < 4 * KJ; ++k) O[nt][k] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // Tile x against this wave's first LIVE operands, those that have rows.
    auto compute = [&](auto live, auto of_drafted, int x) __attribute__((always_inline)) {
        constexpr int LIVE = decltype(live)::value;
        constexpr bool drafted = decltype(of_drafted)::value;
        const int tile0 = (c0 + x) * kTile;
        if (drafted ? !idle : tile0 <= v_to && tile0 + kTile - 1 >= v_from) {
            const Gran* gr = &grans[(x & (kProRing - 1)) * (kTile / kGran)];
            const float kx = drafted ? fabsf(A.scale2) : gr[g].kx, lv = drafted ? 0.f : gr[g].lv;
            uint32_t mine[LIVE], broken = 0u;   // drafted tokens of granule g: those that the row attends to, and those whose values are not finite
            if constexpr (drafted) {
                broken = s_bad[(w.t0 + x) & (kMaxDrafted - 1)][g];
#pragma unroll
                for (int nt = 0; nt < LIVE; ++nt) {
                    const int r = row_of(nt) + n16;
                    mine[nt] = r < rows_all ? (uint32_t)(tree_bits(A, w.q.row0 + r / group, w.q.n, w.t0 + x) >> (kGran * g)) & 0xFFFFu : 0u;
                }
            }
            const u32x4* kf = frags + (x & 1) * kFrags * 64 + lane;
            // Fragments are read a group of products ahead (the compiler alone reads one and waits for it).
            f32x4 S[LIVE][4];
            f16x8 ka[2][2 * KJ];
#pragma unroll
            for (int k = 0; k < 2 * KJ; ++k) ka[0][k] = __builtin_bit_cast(f16x8, kf[k * 64]);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (t < 3) {
#pragma unroll
                    for (int k = 0; k < 2 * KJ; ++k) ka[(t + 1) % 2][k] = __builtin_bit_cast(f16x8, kf[((t + 1) * 2 * KJ + k) * 64]);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int nt = 0; nt < LIVE; ++nt) S[nt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < 2 * KJ; ++k)
#pragma unroll
                    for (int nt = 0; nt < LIVE; ++nt)
                        S[nt][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ka[t % 2][k], qf[nt][k], S[nt][t], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
            const u32x4* vf = kf + 8 * KJ * 64;
            f16x8 va[2][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) va[0][k] = __builtin_bit_cast(f16x8, vf[k * 64]);
            __builtin_amdgcn_sched_barrier(0);
            const int key0 = tile0 + g * kGran;
            const bool edge = drafted || tile0 < v_free_from || tile0 + kTile - 1 > v_free_to;
            f16x8 ph[LIVE][2], pl[LIVE][2];   // the weights' leading and following halves
#pragma unroll
            for (int nt = 0; nt < LIVE; ++nt) {
                if constexpr (drafted) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float v = S[nt][k / 4][k % 4] * kx;
                        S[nt][k / 4][k % 4] = mine[nt] >> k & 1u ? v : -__builtin_inff();
                    }
                } else if (edge) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float v = S[nt][k / 4][k % 4] * kx;
                        S[nt][k / 4][k % 4] = k >= lo[nt] - key0 && k <= pos[nt] - key0 ? v : -__builtin_inff();
                    }
                }
                float mx = S[nt][0][0];
#pragma unroll
                for (int k = 1; k < 16; ++k) mx = fmaxf(mx, S[nt][k / 4][k % 4]);
                // a lane that attends to none of its keys adds nothing, whatever their page's scale is
                const bool none = edge && mx == -__builtin_inff();
                const float by = edge ? 1.f : kx;
                mx = fmaf(mx, by, lv);
                if (__ballot(mx > M[nt] + kSlack)) {
                    const float m = fmaxf(M[nt], max_groups(mx)), f = exp2_fast(M[nt] - m);
                    l[nt] *= f;
#pragma unroll
                    for (int k = 0; k < 4 * KJ; ++k) O[nt][k] *= f;
                    M[nt] = m;
                }
                const float c = none ? 0.f : lv - M[nt] + kLift, unscale = none ? 0.f : exp2_fast(-lv);
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                    const float a = exp2_fast(fmaf(S[nt][k / 4][k % 4], by, c));
                    const float b = exp2_fast(fmaf(S[nt][k / 4][k % 4 + 1], by, c));
                    sum += a;
                    sum += b;
                    // (towards zero, two a conversion: what the first leaves the second takes up)
                    const f16x2 hi = cut2(a, b), more = cut2(fmaf((float)hi.x, minus, a), fmaf((float)hi.y, minus, b));
                    ph[nt][k / 8][k % 8] = hi.x, ph[nt][k / 8][k % 8 + 1] = hi.y;
                    pl[nt][k / 8][k % 8] = more.x, pl[nt][k / 8][k % 8 + 1] = more.y;
                }
                l[nt] = fmaf(sum, unscale, l[nt]);
                if (drafted && (broken & mine[nt])) l[nt] = __builtin_nanf("");
            }
#pragma unroll
            for (int k = 0; k < 2 * KJ; ++k) {   // two 16-dimension tiles at a time
                if (k + 1 < 2 * KJ) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) va[(k + 1) % 2][i] = __builtin_bit_cast(f16x8, vf[((k + 1) * 4 + i) * 64]);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int nt = 0; nt < LIVE; ++nt) {
                        f32x4& o = O[nt][2 * k + i / 2];
                        o = __builtin_amdgcn_mfma_f32_16x16x32_f16(va[k % 2][i], ph[nt][i % 2], o, 0, 0, 0);
                        o = __builtin_amdgcn_mfma_f32_16x16x32_f16(va[k % 2][i], pl[nt][i % 2], o, 0, 0, 0);
                    }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    auto compute_rows = [&](auto of_drafted, int x) __attribute__((always_inline)) {
        if (TREE && NT == 2 && operands == 1) compute(std::integral_constant<int, 1>{}, of_drafted, x);
        else compute(std::integral_constant<int, NT>{}, of_drafted, x);
    };

    if constexpr (TREE) {
        if (nd > 0) {
            if (threadIdx.x < kMaxDrafted * (kTile / kGran)) (&s_bad[0][0])[threadIdx.x] = 0u;
        }
    }
    if (n > 0) {
        fill(nd, (n < kProSeg ? n : kProSeg) - nd);
        __syncthreads();
        if constexpr (TREE) {
#pragma unroll 1
            for (int x = 0; x < nd; ++x) {
                load_drafted(x);
                store_drafted(x);
                lds_barrier();
                compute_rows(std::true_type{}, x);
            }
        }
        if (n > nd) {
            load(nd);
#pragma unroll
            for (int i = 0; i < 2 * KJ; ++i) store(nd, i);
        }
        if (n > nd + 1) load(nd + 1);
        lds_barrier();
    }
    for (int x = nd; x < n; ++x) {
        // Of the two workgroups of a CU the younger one's waves get what the
        // older one's leave.  A priority that falls every second tile, and starts
        // again, keeps the two abreast, so that they end together.
        switch (x / 2 & 3) {
            case 0: __builtin_amdgcn_s_setprio(3); break;
            case 1: __builtin_amdgcn_s_setprio(2); break;
            case 2: __builtin_amdgcn_s_setprio(1); break;
            default: __builtin_amdgcn_s_setprio(0);
        }
        if (TREE ? x == nd || x % kProSeg == 0 : x % kProSeg == 0) {   // the next segment, in the half of the ring that is done with
            const int next = TREE ? x / kProSeg * kProSeg + kProSeg : x + kProSeg, left = n - next;
            if (left > 0) fill(next, left < kProSeg ? left : kProSeg);
        }
        if (x + 1 < n) {
#pragma unroll
            for (int i = 0; i < 2 * KJ; ++i) store(x + 1, i);
        }
        if (x + 2 < n) load(x + 2);
        compute_rows(std::false_type{}, x);
        lds_barrier();
    }

    // The item's pieces are joined by the one that is done last, which keeps its
    // own results in registers: only the others' travel, as their lanes hold them.
    const int tid = settle((int)threadIdx.x), n16e = settle(lane) & 15, ge = settle(lane) >> 4;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) l[nt] = sum_groups(l[nt]);
    if (w.splits > 1) {
        constexpr int kSlotBytes = ROWS * (DP + 2) * 4;   // [NT][4 KJ][threads] of four outputs, then [ROWS] of M and l
        const uint32_t step = (uint32_t)A.c.n_kv * kSlotBytes, item = ((uint32_t)w.slot * A.c.n_kv + w.h) * kSlotBytes;
        const __amdgpu_buffer_rsrc_t part = buf_rsrc(A.part, (uint32_t)kAttSlots * kSlotBytes);
        const uint32_t at_o = (uint32_t)tid * 16, at_m = (uint32_t)(ROWS * DP + (wave * 16 * NT + n16e) * 2) * 4;
        uint32_t* ctr = A.ctr + ((size_t)w.slot * A.c.n_kv + w.h) * kAttCtrStride;   // pieces done, pieces written
        if (tid == 0) s_last = fetch_add(ctr, 1u) == (uint32_t)(w.splits - 1);
        __syncthreads();
        if (!s_last) {
            const uint32_t mine = item + w.split * step;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int k = 0; k < 4 * KJ; ++k)
                    if (FULL || k < dc) st16_coherent(part, mine + at_o + (nt * 4 * KJ + k) * kProThreads * 16, O[nt][k]);
                if (ge == 0) st8_coherent(part, mine + at_m + nt * 128, M[nt], l[nt]);
            }
            wait_own_memory();
            __syncthreads();
            if (tid == 0) fetch_add(ctr + 1, 1u);
            return;
        }
        // The others are done and running: nothing that they wait for is held
        // here.  Should they not arrive all the same (counters that something
        // else wrote), the rows become NaN and cannot pass as a result.
        if (tid == 0) {
            int polls = 0;
            while ((int)ld_flag(ctr + 1) != w.splits - 1 && polls < kProWaitLimit) {
                __builtin_amdgcn_s_sleep(1);
                ++polls;
            }
            s_written = polls < kProWaitLimit;
            st_flag(ctr, 0u);
            st_flag(ctr + 1, 0u);
        }
        __syncthreads();
        float m[NT], sum[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) m[nt] = M[nt], sum[nt] = s_written ? 0.f : __builtin_nanf("");
        for (int p = 0; p < w.splits; ++p) {
            if (p == w.split) continue;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) m[nt] = fmaxf(m[nt], ld4_coherent(part, item + p * step + at_m + nt * 128));
        }
        f32x4 o[NT][4 * KJ];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4 * KJ; ++k) o[nt][k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int p = 0; p < w.splits; ++p) {   // in their order, whoever joins them
            f32x4 v[NT][4 * KJ];
            float f[NT], pl[NT];
            if (p == w.split) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    f[nt] = M[nt], pl[nt] = l[nt];
#pragma unroll
                    for (int k = 0; k < 4 * KJ; ++k) v[nt][k] = O[nt][k];
                }
            } else {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    f[nt] = ld4_coherent(part, item + p * step + at_m + nt * 128);
                    pl[nt] = ld4_coherent(part, item + p * step + at_m + nt * 128 + 4);
#pragma unroll
                    for (int k = 0; k < 4 * KJ; ++k) {
                        v[nt][k] = f32x4{0.f, 0.f, 0.f, 0.f};
                        if (FULL || k < dc) v[nt][k] = ld16_coherent(part, at_o + (nt * 4 * KJ + k) * kProThreads * 16, item + p * step);
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                f[nt] = exp2_fast(f[nt] - m[nt]);
                sum[nt] = fmaf(pl[nt], f[nt], sum[nt]);
#pragma unroll
                for (int k = 0; k < 4 * KJ; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[nt][k][j] = fmaf(v[nt][k][j], f[nt], o[nt][k][j]);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            M[nt] = m[nt], l[nt] = sum[nt];
#pragma unroll
            for (int k = 0; k < 4 * KJ; ++k) O[nt][k] = o[nt][k];
        }
    }

    // A row's outputs are spread over the four lanes of one n16.
    typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int row = row_of(nt) + n16e;
        if (row >= rows_all) continue;
        const int tok = row / group, head = w.h * group + row - tok * group;
        const size_t to = (size_t)(w.q.row0 + tok) * A.n_head + head;
        bool empty = first + tok < 0;
        if constexpr (TREE) empty = l[nt] == 0.f && !tree_sees(A, w.q, tok);
        // no weight at all although there are keys: every score was -infinity
        const float f = l[nt] == 0.f ? __builtin_nanf("") : 1.f / l[nt];
#pragma unroll
        for (int k = 0; k < 4 * KJ; ++k) {
            if (!FULL && k >= dc) continue;
            f16x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = empty ? (f16)0.f : (f16)(O[nt][k][j] * f);
            *reinterpret_cast<f16x4*>(A.y + to * d + k * 16 + ge * 4) = v;
        }
        if (A.lse && ge == 0) A.lse[to] = empty ? -__builtin_inff() : (M[nt] - kLift + log2_fast(l[nt])) * kLn2;
    }
}

template <int FMT, int KJ, bool FULL, class ARGS>
__global__ __launch_bounds__(kProThreads, is_tree<ARGS> && KJ == 1 ? 3 : 2) void k_attend_prompt(ARGS A) {
    constexpr int ROWS = prompt_rows(KJ);
    AttUnit w;
    w.h = blockIdx.x;
    const int units = att_plan<ROWS, ARGS>(A, blockIdx.y, w);
    for (int u = blockIdx.y; u < units;) {
        prompt_unit<FMT, KJ, FULL, ARGS>(A, w);
        u += gridDim.y;
        if (u < units) {
            __syncthreads();   // the next unit uses the same shared memory
            att_plan<ROWS, ARGS>(A, u, w);
        }
    }
}

template <class ARGS>
static hipError_t launch(ARGS A, hipStream_t s) {
    const int kj = att_kj(A.c.d);
    A.target = pro_target(kj);
    A.min_tiles = kProMinTiles;
    unsigned units;
    if constexpr (is_tree<ARGS>) {
        // Three workgroups of heads of up to 64 dimensions fit a CU; pieces for all of them
        // (6 ragged trees of 63 rows, 128 heads, 8 kv, up to 6000 tokens: 79 us against 97 with
        // pieces for two; 8 of 64 on 4096, which divide well into either: 142 against 140).
        A.at_once = kj == 1 ? 768 : A.target;
        units = att_grid(A, prompt_rows(kj), A.words, A.at_once);
    } else {
        units = att_grid(A, prompt_rows(kj));
    }
    const dim3 grid(A.c.n_kv, units);
    const size_t shm = (size_t)2 * 16 * kj * 1024;
    const bool full = A.c.d == 64 * kj;
    hipError_t e = hipSuccess;
#define PI_PRO(F, K, U)                                                                                   \
    do {                                                                                                  \
        if (shm + 16384 > 65536)                                                                          \
            e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_attend_prompt<F, K, U, ARGS>),       \
                                    hipFuncAttributeMaxDynamicSharedMemorySize, (int)shm);                \
        if (e == hipSuccess) hipLaunchKernelGGL((k_attend_prompt<F, K, U, ARGS>), grid, dim3(kProThreads), shm, s, A); \
    } while (0)
#define PI_PRO_D(F)                                                          \
    if (kj == 1) { if (full) PI_PRO(F, 1, true); else PI_PRO(F, 1, false); }  \
    else if (kj == 2) { if (full) PI_PRO(F, 2, true); else PI_PRO(F, 2, false); } \
    else { if (full) PI_PRO(F, 4, true); else PI_PRO(F, 4, false); }
    if (A.c.fmt == 0) { PI_PRO_D(0); } else { PI_PRO_D(1); }
#undef PI_PRO_D
#undef PI_PRO
    if (e != hipSuccess) return e;
    return hipGetLastError();
}
hipError_t launch_attend_prompt(AttArgs A, hipStream_t s) { return launch(A, s); }
hipError_t launch_attend_prompt(TreeArgs A, hipStream_t s) { return launch(A, s); }

}  // namespace pi
