// Attention over the 8-bit paged cache.
//
// For a row (query token, head) and its keys j, x_j = scale log2(e) q . K_j and
// y = sum 2^x_j V_j / sum 2^x_j, in one pass over the cache.
//
// K_j = ks code and V_j = vs code, one ks and vs a page and head.  Codes are
// exact in fp16, so q . code runs on the matrix cores without rounding the
// cache a second time; ks multiplies the fp32 score and vs the weight.  A vs
// lies anywhere between 2^-33 and 2^9.1, so the running reference M follows the
// largest weight with its scale, max (x + log2 vs):
//   w_j = 2^(x_j + log2 vs_j - M + 15.7),  l = sum w_j / vs_j,  y = sum w_j code_j / l.
// M moves when a maximum is more than 0.25 above it, so w is at most 2^15.95,
// just inside fp16, which holds it down to 2^-40 of the row's largest; l is
// summed in fp32, where its terms 2^(x - M + 15.7) always fit.  A page of zeros (vs = 0) takes part
// as vs = 2^-64: its weights count, and its values stay far below fp16's range.
//
// Operands.  A wave takes 64 keys (four granules of 16) a step, as the rows of
// S^T = K Q^T and the inner axis of O^T = V^T P^T, with 16x16x32 products.
// Row i of score tile t is token 4 t + i % 4 of granule i / 4.  Then lane
// (n, g) = (lane % 16, lane / 16) ends up with the 16 scores of query n against
// the tokens of granule g, in order: they are, as they stand, the second
// operand of the output's products, all share one page, and the V operand is
// 16 contiguous bytes (a dimension's 16 tokens).  So nothing is shuffled or
// staged between the two products, and a lane has one ks and one vs a step.
//
// What bounds it: the cache's bytes, read once, at up to 6.1 TB/s (64 ragged
// sequences of 72 heads, 1.48 GB: 242 us).  Below that a call's fixed chain
// shows: lengths, table, scales, first codes (6 us) and the joins (3-4 us):
// 161 MB in 38 us, 134 MB in 34, 129 MB in 39 with 32 rows a head; 7.5 us for
// one sequence of 128 tokens.  The weights as a leading and a following fp16
// half keep 22 bits where the products are free: the matrix cores are busy a
// tenth of the time.
//
// A chain of 8 drafted tokens behind 128 cached ones, 56 heads: 9.3 us; 4 of 4 rows of 64
// heads, 8 kv, on 16384 tokens (134 MB) 40, as the rows as a chain in the cache do.  Of those
// 10-12 are start and end (13 on 256 tokens); in between each key is read by two items of 16 rows,
// 4.5 TB/s of keys (9 with the second reading, from L2).  With 2 rows, one item: 33 us, 6.7 TB/s.
// 16 of 4 rows of 64 heads of 64 up to 8000 tokens 29.5 (28.5).  The drafted rows' values come
// as pairs of dimensions; with the cached codes read in the pairs' order too, half a
// line an instruction, these took 48 and 34.
#include "attend.hpp"
#include "pi.h"

namespace pi {

constexpr float kLift = 15.7f, kSlack = 0.25f;   // of the references, above
constexpr int kAttRows = 16;   // query rows of a workgroup
constexpr int kHeadRounds = 2;   // of tiles that the waves without drafted ones share among them
constexpr int kMinTiles = 4;   // tiles a piece of a whole context has at least
// workgroups the work is split into: those that run at once, by the registers
constexpr int single_target(int kj, int waves) { return kj == 4 || waves == 8 ? 256 : 512; }

// KJ: 64-dimension steps of a head; FULL: d is all of them; WAVES: of a workgroup.
template <int FMT, int KJ, bool FULL, int WAVES, class ARGS>
__device__ __forceinline__ void attend_unit(const ARGS& A, const AttUnit& w) {
    constexpr bool TREE = is_tree<ARGS>;
    constexpr int kAttWaves = WAVES, kAttThreads = WAVES * kWave, ROWS = kAttRows, DP = 64 * KJ, LD = DP + 4;
    extern __shared__ float lds[];   // while tiles are read: Gran [kSegGrans]; then the joins' arrays
    __shared__ int s_last;
    Gran* grans = reinterpret_cast<Gran*>(lds);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int lane = lane_id(), n16 = lane & 15, g = lane >> 4;
    const int d = FULL ? DP : A.c.d, dc = d / 16, group = A.group;
    const int ctx = w.q.ctx, first = ctx - w.q.n, rows_all = w.q.n * group;
    // byte offsets of this lane's pieces inside a granule
    int ko[KJ];
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
        const int ch = FULL || j * 4 + g < dc ? j * 4 + g : dc - 1;   // beyond d: any finite code, its query is 0
        ko[j] = ch * 64 + (n16 & 3) * 16;
    }
    u32x4 kc[4][KJ], vc[4 * KJ];
    auto load_k = [&](const Gran& e) {
        const uint8_t* p = gran_at(A.c.k, e) + (FULL ? ko[0] : 0);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < KJ; ++j) kc[t][j] = ld16_stream(p + t * 4 * d + (FULL ? j * 256 : ko[j]));
    };
    auto load_v = [&](const Gran& e) {
        const uint8_t* p = gran_at(A.c.v, e) + n16 * 16;
#pragma unroll
        for (int k = 0; k < 4 * KJ; ++k) vc[k] = ld16_stream(p + (FULL || k < dc ? k : dc - 1) * 256);
    };

    // this lane's query: position, and the operand's fragments (negated for a
    // negative scale, so that kx is never below 0)
    const int my_row = w.row_tile * ROWS + n16;
    const bool live = my_row < rows_all;
    const int my_tok = live ? my_row / group : 0, my_head = w.h * group + (live ? my_row - my_tok * group : 0);
    const int pos = !live ? -1 : TREE ? ctx - 1 : first + my_tok;   // the last cached token that the row attends to
    int lo = A.window > 0 && pos - A.window + 1 > 0 ? pos - A.window + 1 : 0;
    if constexpr (TREE) lo = live ? tree_from(A, ctx, w.q.row0 + my_tok) : 0;
    f16x8 qf[2 * KJ];
    {
        const h16* qr = A.q + (size_t)(w.q.row0 + my_tok) * A.q_stride + (size_t)my_head * d;
        const uint32_t sign = A.scale2 < 0.f ? 0x80008000u : 0u;
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
            const int ch = j * 4 + g;
            u32x4 a = {0u, 0u, 0u, 0u}, e = a;
            if (live && ch < dc) {
                a = ld16(qr + ch * 16);
                e = ld16(qr + ch * 16 + 8);
            }
            qf[2 * j] = __builtin_bit_cast(f16x8, a ^ sign);
            qf[2 * j + 1] = __builtin_bit_cast(f16x8, e ^ sign);
        }
    }
    // positions that every row of this workgroup attends to need no mask
    const int row_a = w.row_tile * ROWS / group;
    int row_b = (w.row_tile * ROWS + ROWS - 1) / group;
    if (row_b >= w.q.n) row_b = w.q.n - 1;
    int free_to = first + row_a;                                                         // up to this one
    int free_from = A.window > 0 ? first + row_b - A.window + 1 : 0;                     // from this one on
    // and outside these, none attends
    int any_to = first + row_b, any_from = A.window > 0 ? first + row_a - A.window + 1 : 0;
    if constexpr (TREE) {
        free_to = any_to = ctx - 1;
        if (A.window > 0) free_from = __builtin_amdgcn_readfirstlane(max_lanes16(lo));
        any_from = A.window > 0 ? ctx - A.window + 1 : 0;
    }

    float M = kNone, l = 0.f;
    f32x4 O[4 * KJ];
#pragma unroll
    for (int k = 0; k < 4 * KJ; ++k) O[k] = f32x4{0.f, 0.f, 0.f, 0.f};

    // Weights of a tile's scores S (times kx; -infinity where the row does not attend, which edge says may be) and their sum.
    auto weigh = [&](f32x4 (&S)[4], bool edge, float kx, float lv, f16x8 (&ph)[2], f16x8 (&pl)[2]) __attribute__((always_inline)) {
        float mx = S[0][0];
#pragma unroll
        for (int k = 1; k < 16; ++k) mx = fmaxf(mx, S[k / 4][k % 4]);
        // a lane that attends to none of its keys adds nothing, whatever their page's scale is
        const bool none = edge && mx == -__builtin_inff();
        const float by = edge ? 1.f : kx;
        mx = fmaf(mx, by, lv);
        if (__ballot(mx > M + kSlack)) {
            const float m = fmaxf(M, max_groups(mx)), f = exp2_fast(M - m);
            l *= f;
#pragma unroll
            for (int k = 0; k < 4 * KJ; ++k) O[k] *= f;
            M = m;
        }
        // the weights' leading and following halves: to 22 bits, at twice the output's products
        const float c = none ? 0.f : lv - M + kLift, unscale = none ? 0.f : exp2_fast(-lv);
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float wt = exp2_fast(fmaf(S[k / 4][k % 4], by, c));
            sum += wt;
            const f16 hi = (f16)wt;
            ph[k / 8][k % 8] = hi;
            pl[k / 8][k % 8] = (f16)(wt - (float)hi);
        }
        l = fmaf(sum, unscale, l);
    };

    int c0 = w.t0, c1 = w.t1, nd = 0;   // cached tiles; drafted ones, of waves 0 .. nd - 1
    auto look_up = [&](int seg) __attribute__((always_inline)) {
        const int tiles = c1 - seg < kSegTiles ? c1 - seg : kSegTiles;
        att_lookup(A, w, d, seg * (kTile / kGran), tiles * (kTile / kGran), threadIdx.x, kAttThreads, grans);
        __syncthreads();
    };
    if constexpr (TREE) {
        // The drafted rows: fp16 as they are, K and V of scale 1.  A piece's tiles go
        // round the waves, the drafted ones first, at most one of them a wave; its
        // rows are under way while the first granules are looked up.
        const TreeTiles tt = tree_tiles(A, w);
        c0 = tt.from, c1 = tt.to, nd = tt.drafted;
        const bool has = wave < tt.drafted;
        const int n = w.q.n, tok0 = (w.t0 + wave) * kTile;
        auto row = [&](int tok) { return (size_t)(w.q.row0 + (tok < n ? tok : n - 1)); };
        const u32x4 zero = {0u, 0u, 0u, 0u};
        u32x4 dk[4][2 * KJ];
        uint32_t dv[2 * KJ][kGran], bits = 0u;   // dimensions 2 n16 and the next of 32, of the lane's 16 tokens; those that the row attends to
        auto load_values = [&](int j0, int j1) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < kGran; ++i) {
                const h16* p = A.tv + row(tok0 + g * kGran + i) * A.tv_stride + (size_t)w.h * d + 2 * n16;
#pragma unroll
                for (int j = j0; j < j1; ++j) dv[j][i] = FULL || j * 32 + 2 * n16 < d ? *reinterpret_cast<const uint32_t*>(p + j * 32) : 0u;
            }
        };
        constexpr int kEarly = KJ == 4 ? 0 : 2 * KJ;   // value loads that fit the registers beside the keys'
        if (has) {
            if (live) bits = (uint32_t)(tree_bits(A, w.q.row0 + my_tok, n, w.t0 + wave) >> (kGran * g)) & 0xFFFFu;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const h16* p = A.tk + row(tok0 + (n16 >> 2) * kGran + t * 4 + (n16 & 3)) * A.tk_stride + (size_t)w.h * d + g * 16;
#pragma unroll
                for (int j = 0; j < KJ; ++j) {
                    dk[t][2 * j] = dk[t][2 * j + 1] = zero;
                    if (FULL || j * 4 + g < dc) dk[t][2 * j] = ld16(p + j * 64), dk[t][2 * j + 1] = ld16(p + j * 64 + 8);
                }
            }
            load_values(0, kEarly);
        }
        if (c0 < c1) look_up(c0);
        if (has) {
            const float kx = fabsf(A.scale2);
            f32x4 S[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < 2 * KJ; ++j) S[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, dk[t][j]), qf[j], S[t], 0, 0, 0);
            }
            load_values(kEarly, 2 * KJ);
#pragma unroll
            for (int k = 0; k < 16; ++k) S[k / 4][k % 4] = bits >> k & 1u ? S[k / 4][k % 4] * kx : -__builtin_inff();
            f16x8 ph[2], pl[2];
            weigh(S, true, kx, 0.f, ph, pl);
            uint32_t bad = 0u;
#pragma unroll
            for (int k = 0; k < 4 * KJ; ++k) {
                u32x4 v[2];
#pragma unroll
                for (int i = 0; i < 8; ++i)   // the even or the odd dimension of two tokens
                    v[i / 4][i % 4] = __builtin_amdgcn_perm(dv[k / 2][2 * i + 1], dv[k / 2][2 * i], k % 2 ? 0x07060302u : 0x05040100u);
                drop_nonfinite(v, bad);
                const f16x8 a = __builtin_bit_cast(f16x8, v[0]), b = __builtin_bit_cast(f16x8, v[1]);
                O[k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, ph[0], O[k], 0, 0, 0);
                O[k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, ph[1], O[k], 0, 0, 0);
                O[k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pl[0], O[k], 0, 0, 0);
                O[k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, pl[1], O[k], 0, 0, 0);
            }
            // Tiles k and k + 1 hold the even and the odd dimensions of 32, lane group g
            // those from 8 g on.  They go where the cached tiles' results will: tile k + t has
            // dimensions 16 t + 4 g + r, which group 2 t + g / 2 holds.
#pragma unroll
            for (int k = 0; k < 4 * KJ; k += 2) {
                const f32x4 even = O[k], odd = O[k + 1];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int from = n16 + 16 * (2 * t + (g >> 1));
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float low = __shfl(r % 2 ? odd[r / 2] : even[r / 2], from, kWave);
                        const float high = __shfl(r % 2 ? odd[2 + r / 2] : even[2 + r / 2], from, kWave);
                        O[k + t][r] = g & 1 ? high : low;
                    }
                }
            }
            if (__ballot(bad != 0u)) {
                bad = or_lanes16(bad);
                if (bad & bits) l = __builtin_nanf("");
            }
        }
    }
    // A drafted tile takes a wave some two rounds of cached ones: the others share the tiles of these.
    const int others = kAttWaves - nd, head = TREE ? kHeadRounds * others : 0;
    for (int seg = c0; seg < c1; seg += kSegTiles) {
        const int tiles = c1 - seg < kSegTiles ? c1 - seg : kSegTiles;
        if (seg != c0) __syncthreads();   // the last segment's entries are no longer read
        if (!TREE || seg != c0) look_up(seg);
        int i = TREE && seg == c0 ? wave < nd ? head + wave : wave - nd : wave;   // this wave's tile in the segment
        Gran e;         // of the lane's V granule
        if (i < tiles) {
            load_k(grans[i * 4 + (n16 >> 2)]);
            e = grans[i * 4 + g];
            load_v(e);
        }
        for (int next; i < tiles; i = next) {
            next = i + kAttWaves;
            if (TREE && seg == c0 && i < head) next = i + others < head ? i + others : head + wave;
            const float kx = e.kx, lv = e.lv;
            f32x4 S[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < KJ; ++j) {
                    S[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes8<FMT>(kc[t][j].x, kc[t][j].y), qf[2 * j], S[t], 0, 0, 0);
                    S[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes8<FMT>(kc[t][j].z, kc[t][j].w), qf[2 * j + 1], S[t], 0, 0, 0);
                }
            }
            if (next < tiles) {
                load_k(grans[next * 4 + (n16 >> 2)]);
                e = grans[next * 4 + g];
            }

            const int tile0 = (seg + i) * kTile, key0 = tile0 + g * kGran;   // the tile's first key, and this lane's
            const bool edge = tile0 < free_from || tile0 + kTile - 1 > free_to;
            if (edge) {   // scores of keys that the row does not attend to become -infinity
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float x = S[k / 4][k % 4] * kx;
                    S[k / 4][k % 4] = k >= lo - key0 && k <= pos - key0 ? x : -__builtin_inff();
                }
            }
            f16x8 ph[2], pl[2];
            weigh(S, edge, kx, lv, ph, pl);
            if (FMT == 1 && (tile0 < any_from || tile0 + kTile - 1 > any_to)) {
#pragma unroll
                for (int k = 0; k < 4 * KJ; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) vc[k][j] = keep_tokens(vc[k][j], key0 + 4 * j, any_from, any_to);
            }
#pragma unroll
            for (int k = 0; k < 4 * KJ; ++k) {
                const f16x8 a = codes8<FMT>(vc[k].x, vc[k].y), b = codes8<FMT>(vc[k].z, vc[k].w);
                O[k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, ph[0], O[k], 0, 0, 0);
                O[k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, ph[1], O[k], 0, 0, 0);
                O[k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pl[0], O[k], 0, 0, 0);
                O[k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, pl[1], O[k], 0, 0, 0);
            }
            if (next < tiles) load_v(e);
        }
    }

    // Join the waves that had tiles: references first, then every wave brings
    // its sums to the common one and the workgroup adds them up.
    const int mine_n = w.t1 - w.t0, parts = mine_n < 1 ? 1 : mine_n < kAttWaves ? mine_n : kAttWaves;
    static_assert(kAttWaves * ROWS * LD * 4 >= kSegGrans * (int)sizeof(Gran), "the statistics lie behind the granules");
    float* outs = lds;                                   // [parts][ROWS][LD], over the granules
    float* stat = lds + kAttWaves * ROWS * LD;           // [parts][2][ROWS]: M, l
    float* done = stat + kAttWaves * 2 * ROWS;           // [2][ROWS]: the workgroup's
    const int rows = rows_all - w.row_tile * ROWS < ROWS ? rows_all - w.row_tile * ROWS : ROWS;
    l = sum_groups(l);
    if (g == 0 && wave < parts) {
        stat[(wave * 2 + 0) * ROWS + n16] = M;
        stat[(wave * 2 + 1) * ROWS + n16] = l;
    }
    __syncthreads();
    if (wave < parts) {
        float Mr = kNone;
        for (int p = 0; p < parts; ++p) Mr = fmaxf(Mr, stat[p * 2 * ROWS + n16]);
        const float f = exp2_fast(M - Mr);
#pragma unroll
        for (int k = 0; k < 4 * KJ; ++k) {
            *reinterpret_cast<f32x4*>(&outs[(wave * ROWS + n16) * LD + k * 16 + g * 4]) = O[k] * f;
        }
        if (wave == 0 && g == 0) {
            float sum = 0.f;
            for (int p = 0; p < parts; ++p)
                sum = fmaf(stat[(p * 2 + 1) * ROWS + n16], exp2_fast(stat[p * 2 * ROWS + n16] - Mr), sum);
            done[n16] = Mr;
            done[ROWS + n16] = sum;
        }
    }
    __syncthreads();

    // four outputs of a row, from its sum of weights and reference in `done`
    auto emit = [&](int r, int i, f32x4 o) {
        const int gr = w.row_tile * ROWS + r, tok = gr / group, head = w.h * group + gr - tok * group;
        const size_t to = (size_t)(w.q.row0 + tok) * A.n_head + head;
        const float sum = done[ROWS + r];
        bool empty = first + tok < 0;
        if constexpr (TREE) empty = sum == 0.f && !tree_sees(A, w.q, tok);
        // no weight at all although there are keys: every score was -infinity
        const float f = sum == 0.f ? __builtin_nanf("") : 1.f / sum;
        typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
        f16x4 v;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = empty ? (f16)0.f : (f16)(o[k] * f);
        *reinterpret_cast<f16x4*>(A.y + to * d + i) = v;
        if (A.lse && i == 0) A.lse[to] = empty ? -__builtin_inff() : (done[r] - kLift + log2_fast(sum)) * kLn2;
    };
    constexpr int kSlotBytes = ROWS * (DP + 2) * 4;   // outputs [ROWS][DP], then M and l [2][ROWS]
    // all pieces' results lie in one buffer of at most 2^25 bytes
    const uint32_t step = (uint32_t)A.c.n_kv * kSlotBytes, item = ((uint32_t)w.slot * A.c.n_kv + w.h) * kSlotBytes;
    const uint32_t mine = item + w.split * step;
    const __amdgpu_buffer_rsrc_t part = buf_rsrc(A.part, kAttSlots * kSlotBytes);
    for (int e = threadIdx.x; e < rows * (DP / 4); e += kAttThreads) {
        const int r = e / (DP / 4), i = e % (DP / 4) * 4;
        if (i >= d) continue;
        f32x4 o = *reinterpret_cast<const f32x4*>(&outs[r * LD + i]);
        for (int p = 1; p < parts; ++p) o += *reinterpret_cast<const f32x4*>(&outs[(p * ROWS + r) * LD + i]);
        if (w.splits == 1) emit(r, i, o);
        else st16_coherent(part, mine + (uint32_t)(r * DP + i) * 4, o);
    }
    if (w.splits == 1) return;
    if (threadIdx.x < 2 * ROWS / 4)
        st16_coherent(part, mine + (uint32_t)(ROWS * DP + threadIdx.x * 4) * 4,
                      *reinterpret_cast<const f32x4*>(&done[threadIdx.x * 4]));

    // the last of the item's pieces to arrive joins them, in their order
    uint32_t* ctr = A.ctr + ((size_t)w.slot * A.c.n_kv + w.h) * kAttCtrStride;
    // (the results are written through and waited for, so that the arrival needs
    // no write-back of the whole L2: 32 ragged sequences 38 us against 53)
    wait_own_memory();
    __syncthreads();
    if (threadIdx.x == 0) s_last = fetch_add(ctr, 1u) == (uint32_t)(w.splits - 1);
    __syncthreads();
    if (!s_last) return;
    // Each row's reference and sum over the pieces: kAttThreads / ROWS lanes a
    // row, a piece each.  The first outputs are already on their way meanwhile.
    auto join = [&](auto batch) __attribute__((always_inline)) {
        constexpr int kBatch = decltype(batch)::value;   // pieces loaded at a time
        constexpr int kRowLanes = kAttThreads / ROWS;
        constexpr int kJoin = kAttWaves * LD < 256 ? kAttWaves * LD / 32 * 32 : 256;   // pieces whose factors fit
        float* fac = outs;   // [kJoin][ROWS]: what each piece is multiplied by
        auto load = [&](f32x4 (&v)[kBatch], int p0, int r, int i) __attribute__((always_inline)) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                v[k] = ld16_coherent(part, (uint32_t)(r * DP + i) * 4, item + (p0 + k < w.splits ? p0 + k : w.splits - 1) * step);
        };
        f32x4 v[kBatch];
        const int e0 = threadIdx.x, r0 = e0 / (DP / 4), i0 = e0 % (DP / 4) * 4;
        load(v, 0, r0 < ROWS ? r0 : 0, i0);
        const int sr = threadIdx.x / kRowLanes, sj = threadIdx.x % kRowLanes;
        float Mr = kNone, sum = 0.f;
        for (int p = sj; p < w.splits; p += kRowLanes) {
            const uint32_t st = item + p * step + (ROWS * DP + sr) * 4;
            const float pm = ld4_coherent(part, st), ps = ld4_coherent(part, st + ROWS * 4);
            const float m = fmaxf(Mr, pm);
            sum = sum * exp2_fast(Mr - m) + ps * exp2_fast(pm - m);
            Mr = m;
        }
#pragma unroll
        for (int off = 1; off < kRowLanes; off <<= 1) {
            const float pm = __shfl_xor(Mr, off, kWave), ps = __shfl_xor(sum, off, kWave);
            const float m = fmaxf(Mr, pm);
            sum = sum * exp2_fast(Mr - m) + ps * exp2_fast(pm - m);
            Mr = m;
        }
        if (sj == 0) {
            done[sr] = Mr;
            done[ROWS + sr] = sum;
        }
        __syncthreads();
        // (every thread takes every round: there are barriers in them)
        for (int e = e0; e - e0 < ROWS * (DP / 4); e += kAttThreads) {
            const int r = e / (DP / 4), i = e % (DP / 4) * 4;
            const bool has = r < rows && i < d;
            f32x4 o = {0.f, 0.f, 0.f, 0.f};
            for (int p0 = 0; p0 < w.splits; p0 += kJoin) {
                const int np = w.splits - p0 < kJoin ? w.splits - p0 : kJoin;
                if (e == e0 || w.splits > kJoin) {   // otherwise the factors are still there
                    __syncthreads();
                    for (int p = sj; p < np; p += kRowLanes)
                        fac[p * ROWS + sr] = exp2_fast(ld4_coherent(part, item + (p0 + p) * step + (ROWS * DP + sr) * 4) - done[sr]);
                    __syncthreads();
                }
                if (!has) continue;
                for (int p = 0; p < np; p += kBatch) {
                    if (e != e0 || p0 + p > 0) load(v, p0 + p, r, i);
#pragma unroll
                    for (int k = 0; k < kBatch; ++k)
                        if (p + k < np) o += v[k] * fac[(p + k) * ROWS + r];
                }
            }
            if (has) emit(r, i, o);
        }
    };
    if (w.splits <= 8) join(std::integral_constant<int, 8>{});
    else join(std::integral_constant<int, 32>{});
    if (threadIdx.x == 0) st_flag(ctr, 0u);
}

// A workgroup takes units until there are none: whatever the lengths on the
// device say, every piece of every item runs, and the counters end at zero.
template <int FMT, int KJ, bool FULL, int WAVES, class ARGS>
__global__ __launch_bounds__(WAVES * kWave, KJ == 4 ? 1 : 2) void k_attend(ARGS A) {
    AttUnit w;
    w.h = blockIdx.x;
    const int units = att_plan<kAttRows, ARGS>(A, blockIdx.y, w);
    for (int u = blockIdx.y; u < units;) {
        attend_unit<FMT, KJ, FULL, WAVES, ARGS>(A, w);
        u += gridDim.y;
        if (u < units) {
            __syncthreads();   // the next unit uses the same shared memory
            att_plan<kAttRows, ARGS>(A, u, w);
        }
    }
}

size_t kv_attend_zero_bytes() { return (size_t)kAttSlots * kAttCtrStride * 4; }
static_assert(kSyncBytes + (size_t)kAttSlots * kAttCtrStride * 4 == PI_KV_WS_ZERO_BYTES, "header and counters");

// Whether sequences of more rows than one item holds go to the prompt kernel.
// Where the 16-row items of all heads are few, this kernel's split over the
// context serves them better (one sequence, 64 rows of each of 8 kv heads on
// 30000 tokens, 32 items: 35 us against 83; 4 sequences of 160 rows of 8 kv heads
// on 2000 tokens, 320 items: 25 against 29; 512 tokens of 12 heads of 64, 384
// items: 9.6 against 17).  With more, every item reads its keys again, and the
// prompt kernel is faster (77 sequences of 71 rows of one kv head up to 8000
// tokens, 385 items: 43 us against 60; 1024 rows of 8 kv heads on 8192 tokens, 512
// items: 68 against 87; 8 sequences of 128 rows of 56 heads on 2000 tokens, 3584
// items: 84 against 165).  The count does not see how few keys an item may have:
// there it chooses wrongly (256 rows of 32 heads on as many tokens, 512 items:
// 15.7 us against this kernel's 10.9; 8 sequences of 20 rows of 56 heads on 2000,
// 896 items: 61 against 54).
constexpr int kSingleItems = 384;
static bool uses_prompt(const KvBatch& b, int group, int n_kv) {
    return (long long)b.max_q * group > kAttRows && att_most_row_tiles(b, group, kAttRows) * n_kv > kSingleItems;
}

size_t kv_attend_bytes(int n_seq, int n_tok, int max_q, int n_head, int n_kv, int d) {
    const int kj = att_kj(d);
    const KvBatch b{n_seq, n_tok, max_q, 0, 0, nullptr, nullptr, nullptr};
    const size_t rows = (size_t)kAttSlots * (uses_prompt(b, n_head / n_kv, n_kv) ? prompt_rows(kj) : kAttRows);
    return kv_attend_zero_bytes() + rows * (64 * kj + 2) * 4;
}

template <int FMT, int KJ, bool FULL, int WAVES, class ARGS>
static hipError_t launch_single(const ARGS& A, hipStream_t s) {
    constexpr size_t joins = ((size_t)WAVES * (64 * KJ + 4 + 2) + 2) * kAttRows * 4, looks = kSegGrans * sizeof(Gran);
    constexpr size_t shm = joins > looks ? joins : looks;
    if (shm > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_attend<FMT, KJ, FULL, WAVES, ARGS>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)shm);
        if (e != hipSuccess) return e;
    }
    // heads side by side: the row tiles that read one head's pages run on one
    // XCD where the heads are a multiple of 8, and share its L2
    unsigned units;
    if constexpr (is_tree<ARGS>) units = att_grid(A, kAttRows, A.words);
    else units = att_grid(A, kAttRows);
    hipLaunchKernelGGL((k_attend<FMT, KJ, FULL, WAVES, ARGS>), dim3(A.c.n_kv, units), dim3(WAVES * kWave), shm, s, A);
    return hipGetLastError();
}

template <int FMT, class ARGS>
static hipError_t launch_singles(ARGS A, hipStream_t s) {
    const int kj = att_kj(A.c.d);
    const bool full = A.c.d == 64 * kj;
    // Where all items run at once, one eight-wave workgroup a CU each: half as
    // many pieces to join (16 sequences of 4 x 8 rows, window 4097: 39.7 us
    // against 43.6 with four waves; 131072 tokens: 33 against 35; 8 sequences of
    // 8 kv heads: 17.5 against 18.7; 32 of 4096 tokens each: 51 against 53).
    // Where there are more, two four-wave workgroups a CU, one's start and end
    // beside the other's loads (33 ragged sequences of 8 kv heads: 38 us against
    // 48 with eight; 64: 68 against 71; 64 of 72 heads: 242 against 295).  With
    // 16 to 32 ragged sequences of 8 kv heads eight waves lose 2 us (32: 39.6
    // against 37.5): the pieces are then as long as the longest sequence.
    const int waves = kj < 4 && att_most_row_tiles(A.b, A.group, kAttRows) * A.c.n_kv <= 256 ? 8 : 4;
    A.target = single_target(kj, waves);
    A.min_tiles = kMinTiles;
    if (kj == 4) return full ? launch_single<FMT, 4, true, 4, ARGS>(A, s) : launch_single<FMT, 4, false, 4, ARGS>(A, s);
    if (kj == 2 && waves == 8) return full ? launch_single<FMT, 2, true, 8, ARGS>(A, s) : launch_single<FMT, 2, false, 8, ARGS>(A, s);
    if (kj == 2) return full ? launch_single<FMT, 2, true, 4, ARGS>(A, s) : launch_single<FMT, 2, false, 4, ARGS>(A, s);
    if (waves == 8) return full ? launch_single<FMT, 1, true, 8, ARGS>(A, s) : launch_single<FMT, 1, false, 8, ARGS>(A, s);
    return full ? launch_single<FMT, 1, true, 4, ARGS>(A, s) : launch_single<FMT, 1, false, 4, ARGS>(A, s);
}

template <class ARGS>
static hipError_t launch_attend(ARGS A, hipStream_t s) {
    const KvBatch& b = A.b;
    // Drafted rows, up to two items of 16 a sequence: the second reading of the keys comes from
    // L2 and costs less than the other kernel's idle waves, however many items there are (64 heads, 8
    // kv: 32 ragged sequences of 4 rows on up to 8192 tokens 87 us against 112, 64 on 4096 82
    // against 114, 128 on 1024 60 against 75; 8 kv heads of 256 104 against 182; with three
    // items, 32 of 6 rows on 8192, 121 against 110).
    const bool few = is_tree<ARGS> && (long long)b.max_q * A.group <= 2 * kAttRows;
    if (!few && uses_prompt(b, A.group, A.c.n_kv)) {
        // Drafted rows: where most sequences have about as many as the largest, a
        // workgroup's waves without rows cost less than a second launch that finds
        // little or nothing to do (16 ragged trees of 6 to 16: 79 us against 88).  One tree of
        // 64 beside 31 single rows: 60 us in two launches, 78 in one; 8 beside 56: 72 and 76.
        if (is_tree<ARGS> && 2LL * b.n_tok >= (long long)b.n_seq * b.max_q) return launch_attend_prompt(A, s);
        // rows of long and short sequences: each kernel takes its own (they
        // share the workspace, one after the other)
        A.upto = kAttRows;
        ARGS P = A;
        P.above = kAttRows;
        P.upto = 0x7FFFFFFF;
        const hipError_t e = launch_attend_prompt(P, s);
        if (e != hipSuccess || b.n_tok == (long long)b.n_seq * b.max_q) return e;   // no short ones
    }
    return A.c.fmt == 0 ? launch_singles<0>(A, s) : launch_singles<1>(A, s);
}

hipError_t launch_kv_attend(const KvCache& c, const KvBatch& b, const h16* q, long long q_stride, int n_head,
                            float scale, int window, h16* y, float* lse, char* data, const KvDraft* draft, hipStream_t s) {
    const int group = n_head / c.n_kv;
    if (!draft && window > 0x3FFFFFFF) window = 0;   // above any length (and positions less it would pass 32 bits)
    const AttArgs A{c, b, q, q_stride, n_head, group, window, 0, 0x7FFFFFFF, 0, 0, scale * 1.4426950408889634f, y, lse,
                    reinterpret_cast<uint32_t*>(data), reinterpret_cast<float*>(data + kv_attend_zero_bytes())};
    if (!draft) return launch_attend(A, s);
    return launch_attend(TreeArgs{A, draft->k, draft->v, draft->k_stride, draft->v_stride, draft->mask, draft->words, draft->pos, 0}, s);
}

}  // namespace pi
