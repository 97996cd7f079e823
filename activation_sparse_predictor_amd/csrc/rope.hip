// pi_rotate: rotary positions of rows that the caller keeps.
//
// Bytes bound it: two in and two out an element, no more than once.  2048 tokens of 72
// heads of 128, 75 MB: 13.1 us over the same buffers again, which the last-level cache
// serves in part (a copy of as many bytes: 11.4), 17.4 through 3 GB of buffers in turn
// (copy: 16.2).  8192 tokens: 49.5 and 54.8 us (copy 57).  The angles cost some 30
// operations a pair, which is why four heads share them.  The pairs layout, whose
// thread has 16 neighbouring dimensions, takes 14.8 and 19.6 us for 2048 tokens, 53.8 and
// 56.9 for 8192 (with eight, half the angles a thread reads together: 17.3 and 63 over
// the same buffers).  One token of 56 heads: 2.7 us, a launch.
#include "rope.hpp"

namespace pi {

constexpr int kRotThreads = 256;

// Threads of a block take the units of one token, or of several where a token
// has fewer than 256.
template <int HPT>
__global__ __launch_bounds__(kRotThreads) void k_rotate(Rope R, const int32_t* __restrict__ pos, int n_tok, const h16* x,
                                                        long long x_stride, int n_head, int d, h16* y, long long y_stride,
                                                        int groups, int units, int tokens) {
    const int slots = groups * units, tid = threadIdx.x;
    const int in = tokens > 1 ? tid / slots : 0;
    const int slot = tokens > 1 ? tid - in * slots : (int)blockIdx.y * kRotThreads + tid;
    const long long tok = (long long)blockIdx.x * tokens + in;
    if (slot >= slots || in >= tokens || tok >= n_tok) return;
    rotate_heads<HPT>(R, d, n_head, groups, units, pos[tok], x + tok * x_stride, y + tok * y_stride, slot);
}

template <int HPT>
static hipError_t launch(const Rope& R, const int32_t* pos, int n_tok, const h16* x, long long x_stride, int n_head, int d,
                         h16* y, long long y_stride, int units, hipStream_t s) {
    const int groups = (n_head + HPT - 1) / HPT, slots = groups * units;
    const int tokens = slots >= kRotThreads ? 1 : kRotThreads / slots;
    const dim3 grid((n_tok + tokens - 1) / tokens, tokens > 1 ? 1 : (slots + kRotThreads - 1) / kRotThreads);
    hipLaunchKernelGGL((k_rotate<HPT>), grid, dim3(kRotThreads), 0, s, R, pos, n_tok, x, x_stride, n_head, d, y, y_stride, groups,
                       units, tokens);
    return hipGetLastError();
}

hipError_t launch_rotate(const Rope& R, const int32_t* pos, int n_tok, const h16* x, long long x_stride, int n_head, int d,
                         h16* y, long long y_stride, hipStream_t s) {
    const int units = rope_units(R, d);
    if ((long long)n_tok * n_head * units >= kRopeShareFrom) return launch<4>(R, pos, n_tok, x, x_stride, n_head, d, y, y_stride, units, s);
    return launch<1>(R, pos, n_tok, x, x_stride, n_head, d, y, y_stride, units, s);
}

}  // namespace pi
