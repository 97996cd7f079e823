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
// Three launches: the walk, a workgroup a sequence; the sums of what is left at
// its end, a workgroup a slice of the vocabulary; the search in one slice.
#include "common.hpp"
#include "internal.hpp"
#include "pi.h"

namespace pi {

constexpr int kVerMinSlice = 1024, kVerMaxSlice = 16384;   // elements of the vocabulary a workgroup sums
constexpr int kVerMaxSlices = PI_VERIFY_MAX_VOCAB / kVerMaxSlice;
constexpr int kWalkThreads = 1024, kVerThreads = 256, kVerWaves = kVerThreads / kWave;

struct VerifyWs {   // kept between the three kernels
    int32_t *path, *cur, *count;   // [n_tok] accepted rows of a sequence, from its first row's place on; [n_seq] the last one; [n_seq]
    double *s, *part;              // [n_seq] s_r there; [n_seq][slices] sums
};

struct f32x4u { float v[4]; } __attribute__((packed, aligned(4)));
__device__ __forceinline__ f32x4u ld4u(const float* p) { return *reinterpret_cast<const f32x4u*>(p); }

// First row and rows of a sequence, clamped to the arrays.
__device__ __forceinline__ void ver_seq(const VerifyArgs& A, int s, int& row0, int& n) {
    const int a = A.q_start[s], e = A.q_start[s + 1];
    row0 = a < 0 ? 0 : a > A.n_tok ? A.n_tok : a;
    const int end = e > A.n_tok ? A.n_tok : e;
    n = end > row0 ? end - row0 : 0;
}

// What is left of an element; NaN stays.
__device__ __forceinline__ double left_of(float p, float q, double s) {
    const double d = (double)p - s * (double)q;
    return !(d <= 0.0) ? d : 0.0;
}

__device__ __forceinline__ double shfl_xor_d(double v, int m) { return __shfl_xor(v, m, kWave); }
__device__ __forceinline__ double wave_sum_d(double v) {
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) v += shfl_xor_d(v, m);
    return v;
}
__device__ __forceinline__ double wave_scan_d(double v) {   // inclusive
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) {
        const double o = __shfl_up(v, m, kWave);
        if (lane_id() >= m) v += o;
    }
    return v;
}

// This thread's share of sum max(p - s q, 0) over [from, to), `threads` threads four elements each.
template <bool DRAWN>
__device__ __forceinline__ double sum_left(const float* p, const float* q, double s, int from, int to, int tid, int threads) {
    double a[4] = {0.0, 0.0, 0.0, 0.0};
    int i = from + tid * 4;
    const int step = threads * 4;
    for (; i + 3 * step + 4 <= to; i += 4 * step) {   // four loads of each row under way
        f32x4u x[4], y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[k] = ld4u(p + i + k * step);
            if (DRAWN) y[k] = ld4u(q + i + k * step);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) a[j] += left_of(x[k].v[j], DRAWN ? y[k].v[j] : 0.f, s);
    }
    for (; i < to; i += step)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < to) a[j] += left_of(p[i + j], DRAWN ? q[i + j] : 0.f, s);
    return (a[0] + a[1]) + (a[2] + a[3]);
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
        const double v = wave_sum_d(sum_left<DRAWN>(A.p + row * A.p_stride, DRAWN ? A.q + row * A.q_stride : nullptr, s, 0, A.vocab, tid,
                                                    kWalkThreads));
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
        if (DRAWN) s_row = -1;
    }
    if (DRAWN) __syncthreads();
}

// The tokens of `row`'s children inside [from, to), as bits: they were all rejected.
__device__ __forceinline__ void mark_children(const VerifyArgs& A, int row0, int n, int cur, int from, int to, uint32_t* gone, int tid) {
    for (int i = tid; i < (to - from + 31) / 32; i += kVerThreads) gone[i] = 0u;
    __syncthreads();
    for (int j = cur + 1 + tid; j < n; j += kVerThreads) {
        const int t = A.tokens[row0 + j];
        if (A.parent[row0 + j] == cur && t >= from && t < to) atomicOr(&gone[(t - from) / 32], 1u << ((t - from) % 32));
    }
    __syncthreads();
}

template <bool DRAWN>
__global__ __launch_bounds__(kVerThreads) void k_verify_sum(VerifyArgs A, VerifyWs w) {
    __shared__ double s_sum[kVerWaves];
    __shared__ uint32_t gone[DRAWN ? 1 : kVerMaxSlice / 32];
    const int seq = blockIdx.y, tid = threadIdx.x;
    int row0, n;
    ver_seq(A, seq, row0, n);
    if (n == 0) return;
    const int from = blockIdx.x * A.slice, to = from + A.slice < A.vocab ? from + A.slice : A.vocab;
    const int cur = w.cur[seq], row = row0 + cur;
    const float* p = A.p + row * A.p_stride;
    double v = 0.0;
    if (DRAWN) {
        v = sum_left<true>(p, A.q + row * A.q_stride, w.s[seq], from, to, tid, kVerThreads);
    } else {
        mark_children(A, row0, n, cur, from, to, gone, tid);
        for (int i = from + tid * 4; i < to; i += kVerThreads * 4) {
            const uint32_t out = gone[(i - from) / 32] >> ((i - from) % 32);
            if (i + 4 <= to) {
                const f32x4u x = ld4u(p + i);
#pragma unroll
                for (int j = 0; j < 4; ++j) v += out >> j & 1u ? 0.0 : left_of(x.v[j], 0.f, 0.0);
            } else {
                for (int j = 0; i + j < to; ++j) v += out >> j & 1u ? 0.0 : left_of(p[i + j], 0.f, 0.0);
            }
        }
    }
    v = wave_sum_d(v);
    if (lane_id() == 0) s_sum[tid / kWave] = v;
    __syncthreads();
    if (tid == 0) w.part[(size_t)seq * A.slices + blockIdx.x] = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
}

template <bool DRAWN>
__global__ __launch_bounds__(kVerThreads) void k_verify_next(VerifyArgs A, VerifyWs w) {
    __shared__ double s_part[kVerMaxSlices], s_wave[kVerWaves];
    __shared__ uint32_t gone[DRAWN ? 1 : kVerMaxSlice / 32];
    __shared__ int s_before[kVerWaves], s_all[kVerWaves], s_slice, s_found, s_last;
    __shared__ double s_base, s_total;
    const int seq = blockIdx.x, tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
    int row0, n;
    ver_seq(A, seq, row0, n);

    // where this sequence's accepted rows start
    int before = 0, all = 0;
    for (int i = tid; i < A.n_seq; i += kVerThreads) {
        const int c = w.count[i];
        all += c;
        before += i < seq ? c : 0;
    }
    before = (int)group_sum_u32<kWave>((uint32_t)before);
    all = (int)group_sum_u32<kWave>((uint32_t)all);
    if (lane == 0) s_before[wave] = before, s_all[wave] = all;
    __syncthreads();
    before = all = 0;
    for (int i = 0; i < kVerWaves; ++i) before += s_before[i], all += s_all[i];
    const int count = w.count[seq];
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

    const int cur = w.cur[seq], row = row0 + cur;
    const float *p = A.p + row * A.p_stride, *q = DRAWN ? A.q + row * A.q_stride : nullptr;
    double s = DRAWN ? w.s[seq] : 0.0;
    bool whole = false;   // the row's own distribution, nothing taken from it
    for (int i = tid; i < A.slices; i += kVerThreads) s_part[i] = w.part[(size_t)seq * A.slices + i];
    __syncthreads();
    for (;;) {
        // wave 0: the whole, and the first slice whose running sum passes the mark
        if (wave == 0) {
            double total = 0.0;
            for (int i = 0; i < A.slices; i += kWave) total += wave_sum_d(i + lane < A.slices ? s_part[i + lane] : 0.0);
            const double mark = (double)A.u_next[seq] * total;
            double base = 0.0, base_found = 0.0;
            int found = -1, last = 0;
            for (int i = 0; i < A.slices && found < 0; i += kWave) {
                const double v = i + lane < A.slices ? s_part[i + lane] : 0.0, upto = base + wave_scan_d(v);
                const uint64_t hit = __ballot(i + lane < A.slices && upto > mark), some = __ballot(v > 0.0);
                const double until = __shfl(upto - v, hit ? __builtin_ctzll(hit) : 0, kWave);
                if (hit) found = i + __builtin_ctzll(hit), base_found = until;
                if (some) last = i + 63 - __builtin_clzll(some);
                base = __shfl(upto, kWave - 1, kWave);
            }
            if (lane == 0) {
                s_total = total;
                s_slice = found >= 0 ? found : last;   // (u so near 1 that the sums' rounding decides: the last element with any weight)
                s_base = found >= 0 ? base_found : __builtin_inf();
            }
        }
        __syncthreads();
        if (s_total != 0.0 || whole) break;
        // nothing is left: the row as it is
        whole = true;
        s = 0.0;
        __syncthreads();
        for (int i = 0; i < A.slices; ++i) {
            const int from = i * A.slice, to = from + A.slice < A.vocab ? from + A.slice : A.vocab;
            const double v = wave_sum_d(sum_left<false>(p, nullptr, 0.0, from, to, tid, kVerThreads));
            if (lane == 0) s_wave[wave] = v;
            __syncthreads();
            if (tid == 0) s_part[i] = (s_wave[0] + s_wave[1]) + (s_wave[2] + s_wave[3]);
            __syncthreads();
        }
    }
    const double total = s_total;
    if (!(total > 0.0 && total < __builtin_inf())) {   // NaN or infinity among the probabilities, or nothing at all
        if (tid == 0) A.next[seq] = -1;
        return;
    }

    // the element inside the slice: a run of neighbours a thread
    const int from = s_slice * A.slice, to = from + A.slice < A.vocab ? from + A.slice : A.vocab;
    if (!DRAWN && !whole) mark_children(A, row0, n, cur, from, to, gone, tid);
    const int each = (A.slice + kVerThreads - 1) / kVerThreads, a = from + tid * each, e = a + each < to ? a + each : to;
    auto weight = [&](int i) {
        if (!DRAWN && !whole && (gone[(i - from) / 32] >> ((i - from) % 32) & 1u)) return 0.0;
        return left_of(p[i], DRAWN ? q[i] : 0.f, s);
    };
    double mine = 0.0;
    for (int i = a; i < e; ++i) mine += weight(i);
    const double scan = wave_scan_d(mine);
    if (lane == kWave - 1) s_wave[wave] = scan;
    if (tid == 0) s_found = 0x7FFFFFFF, s_last = -1;
    __syncthreads();
    double base = s_base;
    for (int i = 0; i < wave; ++i) base += s_wave[i];
    const double mark = (double)A.u_next[seq] * total;
    base += scan - mine;
    int found = 0x7FFFFFFF, last = -1;
    for (int i = a; i < e; ++i) {
        const double v = weight(i);
        base += v;
        if (v > 0.0) {
            last = i;
            if (base > mark && base < __builtin_inf() && found > i) found = i;
        }
    }
    if (found != 0x7FFFFFFF) atomicMin(&s_found, found);
    if (last >= 0) atomicMax(&s_last, last);
    __syncthreads();
    if (tid == 0) A.next[seq] = s_found != 0x7FFFFFFF ? s_found : s_last;
}

// A slice of the vocabulary for each workgroup: about 512 workgroups.
static int ver_slice(int n_seq, int vocab) {
    long long each = (long long)vocab * n_seq / 512 + 1;
    each = (each + kVerMinSlice - 1) / kVerMinSlice * kVerMinSlice;
    return (int)(each < kVerMaxSlice ? each : kVerMaxSlice);
}

size_t verify_bytes(int n_seq, int n_tok, int vocab) {
    const int slice = ver_slice(n_seq, vocab), slices = (vocab + slice - 1) / slice;
    return ((size_t)n_seq * (1 + slices)) * 8 + ((size_t)n_tok + 2 * (size_t)n_seq) * 4;
}

hipError_t launch_verify(VerifyArgs A, char* ws, hipStream_t st) {
    A.slice = ver_slice(A.n_seq, A.vocab);
    A.slices = (A.vocab + A.slice - 1) / A.slice;
    VerifyWs w;
    w.s = reinterpret_cast<double*>(ws);
    w.part = w.s + A.n_seq;
    w.cur = reinterpret_cast<int32_t*>(w.part + (size_t)A.n_seq * A.slices);
    w.count = w.cur + A.n_seq;
    w.path = w.count + A.n_seq;
    if (A.q) {
        hipLaunchKernelGGL((k_verify_walk<true>), dim3(A.n_seq), dim3(kWalkThreads), 0, st, A, w);
        hipLaunchKernelGGL((k_verify_sum<true>), dim3(A.slices, A.n_seq), dim3(kVerThreads), 0, st, A, w);
        hipLaunchKernelGGL((k_verify_next<true>), dim3(A.n_seq), dim3(kVerThreads), 0, st, A, w);
    } else {
        hipLaunchKernelGGL((k_verify_walk<false>), dim3(A.n_seq), dim3(kWalkThreads), 0, st, A, w);
        hipLaunchKernelGGL((k_verify_sum<false>), dim3(A.slices, A.n_seq), dim3(kVerThreads), 0, st, A, w);
        hipLaunchKernelGGL((k_verify_next<false>), dim3(A.n_seq), dim3(kVerThreads), 0, st, A, w);
    }
    return hipGetLastError();
}

}  // namespace pi
