// pi_verify: which drafted tokens stay, and the token after them.
//
// At a row with distribution p, the children rejected so far, r of them, leave
// p_r ~ max(p_{r-1} - q, 0) of it.  Unrolled, p_r = max(p - s_r q, 0) / W_r with
//   s_0 = 0, W_0 = 1;  s_{r+1} = s_r + W_r,  W_{r+1} = sum max(p - s_{r+1} q, 0)
// (where p < s q, it stays below), so two numbers are all that a rejection
// leaves behind, and nothing of the distribution's size is written.  A child's
// own test u q(x) W < max(p(x) - s q(x), 0) needs single elements, which are loaded for
// 64 rows at a time before the walk; only a sibling after a rejected one needs
// the sum W.  Drafts without probabilities: the rejected tokens are taken out of
// p, and W_{r+1} = W_r - p(x).
//
// All in 64 bits: the next token is the first whose running sum passes u times
// the whole, where sums of 10^5 terms in 32 bits would decide for a neighbour
// about once in a few hundred times.
//
// Two launches: the walk, a workgroup a sequence; then the sums of what is left at
// its end, a wave a slice of the vocabulary; a sequence's workgroup that is done
// last finds the slice and the element in it.
//
// What bounds it: latency, and how the work is divided.  The second launch is a chain
// (where the walk ended, the row, the sums written through, the arrival, the sums back,
// the slice's elements) of 10 us for one sequence of 32000 tokens and 11.7 for 48 of
// 50257 (9.6 MB of p, and of q where a child was rejected).  For fixed proposals (16 sequences, 128000
// tokens: 13.3 us) its sums add to that single loads with a bit looked up for each, none
// under way ahead, and three barriers for every four slices.  The walk takes 1.9 us
// where no sum is asked for, 25 us where the longest of 48 trees asks for several one
// after the other, each one pass of the sequence's one workgroup over both rows (400 KB,
// some 4 us with eight loads of each a thread under way) while most of the chip is idle:
// one workgroup a sequence is this kernel's choice, not the card's bound.  A third
// launch of one workgroup for the search took 2-5 us more.
#include "common.hpp"
#include "internal.hpp"
#include "pi.h"

namespace pi {

constexpr int kWalkThreads = 1024, kVerThreads = 256, kVerWaves = kVerThreads / kWave;
// Elements that one sum is kept of: as many as the search takes in one step, more for
// a vocabulary that had more than kVerMaxSlices of them.
constexpr int kVerStep = 4 * kVerThreads, kVerMaxSlices = 1024, kVerMaxSlice = PI_VERIFY_MAX_VOCAB / kVerMaxSlices;
// Workgroups of the second launch.  Each is one more arrival on its sequence's
// counter, and arrivals on one cache line wait for each other: with a workgroup
// a slice and the counters side by side 48 sequences of 50257 tokens (2400
// workgroups) took 31 us, so (336) they took 12.5, q read for all.
constexpr int kVerBlocks = 512, kVerCtrStride = 32;

struct VerifyWs {   // kept between the two kernels
    int32_t *path, *cur, *count;   // [n_tok] accepted rows of a sequence, from its first row's place on; [n_seq] the last one; [n_seq]
    uint32_t* arrived;             // [n_seq][kVerCtrStride] workgroups of the second that are done, cleared by the first
    double *s, *part;              // [n_seq] s_r there; [n_seq][slices] sums
};

struct f32x4u { float v[4]; } __attribute__((packed, aligned(4)));   // rows start at any element
__device__ __forceinline__ f32x4u ld4u(const float* p) { return *reinterpret_cast<const f32x4u*>(p); }

// First row and rows of a sequence, clamped to the arrays.
__device__ __forceinline__ void ver_seq(const VerifyArgs& A, int s, int& row0, int& n) {
    const int a = A.q_start[s], e = A.q_start[s + 1];
    row0 = a < 0 ? 0 : a > A.n_tok ? A.n_tok : a;
    const int end = e > A.n_tok ? A.n_tok : e;
    n = end > row0 ? end - row0 : 0;
}

// What is left of an element, 0 at least; `nan` notes a NaN, which the maximum would drop.
__device__ __forceinline__ double left_of(float p, float q, double s, bool& nan) {
    nan |= __builtin_isunordered(p, q);
    return __builtin_fmax(fma(-s, (double)q, (double)p), 0.0);
}

// v of the lane that the DPP control names, 0 where there is none, or where ROWS leaves a row out.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_d(double v) {
    const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, ROWS, 0xF, ROWS == 0xF);
    const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, ROWS, 0xF, ROWS == 0xF);
    return __hiloint2double(hi, lo);
}
// Inclusive sums over the lanes, as wave_scan, and the whole.
__device__ __forceinline__ double wave_scan_d(double v) {
    v += dpp_d<0x111, 0xF>(v);
    v += dpp_d<0x112, 0xF>(v);
    v += dpp_d<0x114, 0xF>(v);
    v += dpp_d<0x118, 0xF>(v);
    v += dpp_d<0x142, 0xA>(v);
    v += dpp_d<0x143, 0xC>(v);
    return v;
}
__device__ __forceinline__ double lane_d(double v, int lane) {   // lane: wave-uniform
    return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), lane), __builtin_amdgcn_readlane(__double2loint(v), lane));
}
__device__ __forceinline__ double wave_sum_d(double v) { return lane_d(wave_scan_d(v), kWave - 1); }

// This thread's share of sum max(p - s q, 0) over [from, to), `threads` threads
// four elements each, kAhead loads of each row under way; NaN if there is one.
template <bool DRAWN, int kAhead>
__device__ __forceinline__ double sum_left(const float* p, const float* q, double s, int from, int to, int tid, int threads) {
    double a[4] = {0.0, 0.0, 0.0, 0.0};
    bool nan = false;
    const int step = threads * 4;
    for (int i0 = from; i0 < to; i0 += kAhead * step) {
        f32x4u x[kAhead], y[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (i0 + k * step >= to) continue;   // (the same for all threads)
            const int at = i0 + k * step + tid * 4;
            x[k] = y[k] = f32x4u{{0.f, 0.f, 0.f, 0.f}};
            if (at + 4 <= to) {
                x[k] = ld4u(p + at);
                if (DRAWN) y[k] = ld4u(q + at);
            } else {
#pragma unroll
                for (int j = 0; j < 3; ++j)
                    if (at + j < to) {
                        x[k].v[j] = p[at + j];
                        if (DRAWN) y[k].v[j] = q[at + j];
                    }
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (i0 + k * step >= to) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] += left_of(x[k].v[j], y[k].v[j], s, nan);
        }
    }
    const double sum = (a[0] + a[1]) + (a[2] + a[3]);
    return nan ? __builtin_nan("") : sum;
}

// Wave 0 walks; the others wait for a sum to be asked for.
template <bool DRAWN>
__global__ __launch_bounds__(kWalkThreads) void k_verify_walk(VerifyArgs A, VerifyWs w) {
    __shared__ double s_sum[kWalkThreads / kWave], s_s;
    __shared__ int s_row;   // whose sum; -1: the walk is over
    const int seq = blockIdx.x, tid = threadIdx.x, lane = lane_id();
    int row0, n;
    ver_seq(A, seq, row0, n);
    auto part = [&](int row, double s) {
        const double v = wave_sum_d(sum_left<DRAWN, 8>(A.p + row * A.p_stride, DRAWN ? A.q + row * A.q_stride : nullptr, s, 0, A.vocab,
                                                       tid, kWalkThreads));
        if (lane == 0) s_sum[tid / kWave] = v;
    };
    if (tid >= kWave) {
        if (!DRAWN) return;
        for (;;) {   // ends with the walk, which takes at most n steps
            __syncthreads();
            const int row = s_row;
            if (row < 0) return;
            part(row, s_s);
            __syncthreads();
        }
    }
    int cur = 0, count = n > 0 ? 1 : 0;
    double s = 0.0, W = 1.0;
    bool stale = false;   // W is the one before the last rejection
    if (lane == 0 && n > 0) w.path[row0] = row0;
    for (int c0 = 0; c0 < n; c0 += kWave) {
        const int j = c0 + lane, row = row0 + j;
        int parent = -1, token = -1;
        float u = 0.f, pj = 0.f, qj = 0.f;
        if (j > 0 && j < n) {
            parent = A.parent[row];
            token = A.tokens[row];
            u = A.u[row];
            parent = parent < j ? parent : -1;
        }
        if (parent >= 0 && token >= 0 && token < A.vocab) {
            pj = A.p[(row0 + parent) * A.p_stride + token];
            if (DRAWN) qj = A.q[(row0 + parent) * A.q_stride + token];
        }
        uint64_t after = ~0ull;
        for (;;) {
            const uint64_t m = __ballot(parent == cur) & after;   // (row 0 has no parent, so cur >= 0 finds none but children)
            if (!m) break;
            const int l = __builtin_ctzll(m);
            after = l == 63 ? 0ull : ~0ull << (l + 1);
            const double P = __shfl(pj, l, kWave), Q = __shfl(qj, l, kWave), U = __shfl(u, l, kWave);
            const int T = __shfl(token, l, kWave);
            bool good;
            if (DRAWN) {
                if (stale) {
                    if (lane == 0) s_row = row0 + cur, s_s = s;
                    __syncthreads();
                    part(row0 + cur, s);
                    __syncthreads();
                    W = 0.0;
                    for (int k = 0; k < kWalkThreads / kWave; ++k) W += s_sum[k];
                    stale = false;
                }
                const double d = P - s * Q;
                good = U * Q * W < (!(d <= 0.0) ? d : 0.0);
                if (!good) s += W, stale = true;
            } else {
                // a token that a rejected sibling had is no longer there
                bool gone = (__ballot(parent == cur && token == T) & ((1ull << l) - 1)) != 0;
                for (int b = cur + 1; b < c0 && !gone; b += kWave)
                    gone = __ballot(b + lane < c0 && A.parent[row0 + b + lane] == cur && A.tokens[row0 + b + lane] == T) != 0;
                const double of = gone ? 0.0 : P;
                good = U * W < of;
                if (!good) W -= of;
            }
            if (good) {
                cur = c0 + l;
                if (lane == 0) w.path[row0 + count] = row0 + cur;
                ++count;
                s = 0.0, W = 1.0, stale = false;
            }
        }
    }
    if (lane == 0) {
        w.cur[seq] = cur;
        w.count[seq] = count;
        w.s[seq] = s;
        w.arrived[seq * kVerCtrStride] = 0u;
        if (DRAWN) s_row = -1;
    }
    if (DRAWN) __syncthreads();
}

// The tokens of row cur's children among the `count` from `from` on, as bits: they were all rejected.
__device__ __forceinline__ void mark_children(const VerifyArgs& A, int row0, int n, int cur, int from, int count, uint32_t* gone, int tid) {
    const int to = from + count;
    __syncthreads();   // the last bits are no longer read
    for (int i = tid; i < count / 32; i += kVerThreads) gone[i] = 0u;
    __syncthreads();
    for (int j = cur + 1 + tid; j < n; j += kVerThreads) {
        const int t = A.tokens[row0 + j];
        if (A.parent[row0 + j] == cur && t >= from && t < to) atomicOr(&gone[(t - from) / 32], 1u << ((t - from) % 32));
    }
    __syncthreads();
}

template <bool DRAWN>
__global__ __launch_bounds__(kVerThreads) void k_verify_next(VerifyArgs A, VerifyWs w) {
    __shared__ double s_part[kVerMaxSlices], s_wave[kVerWaves], s_base, s_total;
    __shared__ uint32_t gone[DRAWN ? 1 : kVerWaves * kVerMaxSlice / 32];
    __shared__ int s_before[kVerWaves], s_all[kVerWaves], s_slice, s_found, s_last;
    const int seq = blockIdx.y, tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
    int row0, n;
    ver_seq(A, seq, row0, n);
    const int cur = w.cur[seq], count = w.count[seq], row = row0 + (n > 0 ? cur : 0);
    const float *p = A.p + row * A.p_stride, *q = DRAWN ? A.q + row * A.q_stride : nullptr;
    double s = DRAWN ? w.s[seq] : 0.0;
    bool whole = false;   // the row's own distribution, nothing taken from it
    auto bounds = [&](int slice, int& from, int& to) {
        from = slice * A.slice;
        to = from + A.slice < A.vocab ? from + A.slice : A.vocab;
    };
    auto taken = [&](int i, int from) { return !DRAWN && (gone[(i - from) / 32] >> ((i - from) % 32) & 1u) != 0u; };
    auto block_sum = [&](double v) {
        v = wave_sum_d(v);
        if (lane == 0) s_wave[wave] = v;
        __syncthreads();
        return (s_wave[0] + s_wave[1]) + (s_wave[2] + s_wave[3]);
    };

    int before = 0, all = 0;   // accepted rows of the sequences before, and of all (loaded here, for the last workgroup)
    for (int i = tid; i < A.n_seq; i += kVerThreads) {
        const int c = w.count[i];
        all += c;
        before += i < seq ? c : 0;
    }
    const double u_next = (double)A.u_next[seq];

    // a wave's slices: their sums
    if (n > 0) {
        const int first = blockIdx.x * A.each, end = first + A.each < A.slices ? first + A.each : A.slices;
        for (int i0 = first; i0 < end; i0 += kVerWaves) {
            const int i = i0 + wave;
            int from, to;
            bounds(i, from, to);
            double v = 0.0;
            if (DRAWN) {
                // (no child rejected: q has no part in it, and may hold anything in a row that nothing hangs below)
                if (i < end) v = s != 0.0 ? sum_left<true, 4>(p, q, s, from, to, lane, kWave) : sum_left<false, 4>(p, nullptr, 0.0, from, to, lane, kWave);
            } else {
                mark_children(A, row0, n, cur, i0 * A.slice, kVerWaves * A.slice, gone, tid);
                bool nan = false;
                if (i < end)
                    for (int at = from + lane * 4; at < to; at += kWave * 4)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (at + j < to) {
                                const double x = left_of(p[at + j], 0.f, 0.0, nan);
                                v += taken(at + j, i0 * A.slice) ? 0.0 : x;
                            }
                if (nan) v = __builtin_nan("");
            }
            v = wave_sum_d(v);
            if (lane == 0 && i < end)
                __hip_atomic_store(&w.part[(size_t)seq * A.slices + i], v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    wait_own_memory();   // written through before the arrival is seen
    __syncthreads();
    if (tid == 0) s_found = fetch_add(&w.arrived[seq * kVerCtrStride], 1u) == gridDim.x - 1;
    __syncthreads();
    if (!s_found) return;

    // The last one: where the sequence's accepted rows start, and the rows.
    for (int i = tid; i < A.slices; i += kVerThreads)
        s_part[i] = n > 0 ? __hip_atomic_load(&w.part[(size_t)seq * A.slices + i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
    before = (int)group_sum_u32<kWave>((uint32_t)before);
    all = (int)group_sum_u32<kWave>((uint32_t)all);
    if (lane == 0) s_before[wave] = before, s_all[wave] = all;
    __syncthreads();
    before = all = 0;
    for (int i = 0; i < kVerWaves; ++i) before += s_before[i], all += s_all[i];
    for (int i = tid; i < count; i += kVerThreads)
        if (before + i < A.n_tok) A.rows[before + i] = w.path[row0 + i];
    for (long long i = all + (long long)seq * kVerThreads + tid; i < A.n_tok; i += (long long)A.n_seq * kVerThreads) A.rows[i] = -1;
    if (tid == 0) {
        A.start[seq] = before;
        A.new_ctx[seq] = A.ctx[seq] + count;
        if (seq == A.n_seq - 1) A.start[A.n_seq] = all;
        if (n == 0) A.next[seq] = -1;
    }
    if (n == 0) return;

    for (;;) {
        // wave 0: the whole, and the first slice whose running sum passes the mark
        if (wave == 0) {
            double total = 0.0;
            for (int i = 0; i < A.slices; i += kWave) total += wave_sum_d(i + lane < A.slices ? s_part[i + lane] : 0.0);
            const double mark = u_next * total;
            double base = 0.0, base_found = 0.0;
            int found = -1, last = 0;
            for (int i = 0; i < A.slices && found < 0; i += kWave) {
                const double v = i + lane < A.slices ? s_part[i + lane] : 0.0, upto = base + wave_scan_d(v);
                const uint64_t hit = __ballot(i + lane < A.slices && upto > mark), some = __ballot(v > 0.0);
                const double until = lane_d(upto - v, hit ? __builtin_ctzll(hit) : 0);
                if (hit) found = i + __builtin_ctzll(hit), base_found = until;
                if (some) last = i + 63 - __builtin_clzll(some);
                base = lane_d(upto, kWave - 1);
            }
            if (lane == 0) {
                s_total = total;
                s_slice = found >= 0 ? found : last;   // (u so near 1 that the sums' rounding decides: the last element with any weight)
                s_base = found >= 0 ? base_found : __builtin_inf();
                s_found = 0x7FFFFFFF, s_last = -1;
            }
        }
        __syncthreads();
        if (s_total != 0.0 || whole) break;
        // nothing is left: the row as it is
        whole = true;
        s = 0.0;
        for (int i = 0; i < A.slices; ++i) {
            int from, to;
            bounds(i, from, to);
            __syncthreads();
            const double v = block_sum(sum_left<false, 4>(p, nullptr, 0.0, from, to, tid, kVerThreads));
            if (tid == 0) s_part[i] = v;
        }
        __syncthreads();
    }
    const double total = s_total;
    if (!(total > 0.0 && total < __builtin_inf())) {   // NaN or infinity among the probabilities, or nothing at all
        if (tid == 0) A.next[seq] = -1;
        return;
    }

    // the element inside the slice: four neighbours a thread
    int from, to;
    bounds(s_slice, from, to);
    if (!DRAWN && !whole) mark_children(A, row0, n, cur, from, A.slice, gone, tid);
    const double mark = u_next * total;
    double base = s_base;
    int found = 0x7FFFFFFF, last = -1;
    for (int i0 = from; i0 < to; i0 += kVerStep) {
        double v[4], mine = 0.0;
        bool nan = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + tid * 4 + j;
            v[j] = 0.0;
            if (i < to) v[j] = left_of(p[i], DRAWN && s != 0.0 ? q[i] : 0.f, s, nan);
            if (i < to && !whole && taken(i, from)) v[j] = 0.0;
            mine += v[j];
        }
        const double scan = wave_scan_d(mine);
        __syncthreads();   // the last step's sums are no longer read
        if (lane == kWave - 1) s_wave[wave] = scan;
        __syncthreads();
        double at = base + (scan - mine);
        for (int i = 0; i < wave; ++i) at += s_wave[i];
        base += (s_wave[0] + s_wave[1]) + (s_wave[2] + s_wave[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + tid * 4 + j;
            at += v[j];
            if (v[j] > 0.0) {
                last = i;
                if (at > mark && at < __builtin_inf() && found > i) found = i;
            }
        }
    }
    if (found != 0x7FFFFFFF) atomicMin(&s_found, found);
    if (last >= 0) atomicMax(&s_last, last);
    __syncthreads();
    if (tid == 0) A.next[seq] = s_found != 0x7FFFFFFF ? s_found : s_last;
}

static int ver_slice(int vocab) {
    const int least = (vocab + kVerMaxSlices - 1) / kVerMaxSlices;
    return (least + kVerStep - 1) / kVerStep * kVerStep;
}

size_t verify_bytes(int n_seq, int n_tok, int vocab) {
    const int slice = ver_slice(vocab), slices = (vocab + slice - 1) / slice;
    return (size_t)n_seq * (1 + slices) * 8 + ((size_t)n_seq * (2 + kVerCtrStride) + n_tok) * 4;
}

hipError_t launch_verify(VerifyArgs A, char* ws, hipStream_t st) {
    A.slice = ver_slice(A.vocab);
    A.slices = (A.vocab + A.slice - 1) / A.slice;
    const long long all = (long long)A.slices * A.n_seq, each = (all + kVerBlocks - 1) / kVerBlocks;
    A.each = (int)((each + kVerWaves - 1) / kVerWaves * kVerWaves);
    const dim3 grid((A.slices + A.each - 1) / A.each, A.n_seq);
    VerifyWs w;
    w.s = reinterpret_cast<double*>(ws);
    w.part = w.s + A.n_seq;
    w.cur = reinterpret_cast<int32_t*>(w.part + (size_t)A.n_seq * A.slices);
    w.count = w.cur + A.n_seq;
    w.arrived = reinterpret_cast<uint32_t*>(w.count + A.n_seq);
    w.path = w.count + (size_t)A.n_seq * (1 + kVerCtrStride);
    if (A.q) {
        hipLaunchKernelGGL((k_verify_walk<true>), dim3(A.n_seq), dim3(kWalkThreads), 0, st, A, w);
        hipLaunchKernelGGL((k_verify_next<true>), grid, dim3(kVerThreads), 0, st, A, w);
    } else {
        hipLaunchKernelGGL((k_verify_walk<false>), dim3(A.n_seq), dim3(kWalkThreads), 0, st, A, w);
        hipLaunchKernelGGL((k_verify_next<false>), grid, dim3(kVerThreads), 0, st, A, w);
    }
    return hipGetLastError();
}

}  // namespace pi
