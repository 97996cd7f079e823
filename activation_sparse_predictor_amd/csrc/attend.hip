// Attention over the 8-bit paged cache.
//
// One wave a (row, query head): 64 keys a step, a key a lane for the scores, a
// running maximum and sum, and d / 64 dimensions a lane for the output.
#include "kv.hpp"

namespace pi {

template <int FMT>
__global__ __launch_bounds__(256) void k_attend(KvCache c, KvBatch b, const h16* __restrict__ q, long long q_stride,
                                                int n_head, float scale, int window, h16* __restrict__ y,
                                                float* __restrict__ lse) {
    const int lane = lane_id();
    const long long unit = (long long)blockIdx.x * 4 + threadIdx.x / kWave;
    const int row = (int)(unit / n_head), head = (int)(unit % n_head);
    if (row >= b.n_tok) return;
    int inside;
    const Seq sq = find_seq(b, row, inside, [](const Seq& x) { return x.n; });
    if (sq.s < 0) return;
    const int h = head / (n_head / c.n_kv), d = c.d;
    const int pos = sq.ctx - sq.n + inside;
    const int lo = window > 0 && pos - window + 1 > 0 ? pos - window + 1 : 0;
    const h16* qr = q + (size_t)row * q_stride + (size_t)head * d;
    float m = -__builtin_inff(), l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = lo & ~63; j0 <= pos; j0 += kWave) {
        const int j = j0 + lane;
        const bool in = j >= lo && j <= pos;
        float x = -__builtin_inff(), vs = 0.f;
        size_t at = 0;
        if (in) {
            int id = b.table[(size_t)sq.s * b.table_stride + j / c.page];
            const bool known = id >= 0 && id < c.n_pages;
            id = known ? id : 0;
            const size_t si = (size_t)id * c.n_kv + h;
            const float ks = known ? c.k_scale[si] : __builtin_nanf("");
            vs = known ? c.v_scale[si] : __builtin_nanf("");
            at = page_base(c, id, h);
            const int t = j & (c.page - 1);
            float dot = 0.f;
            for (int i = 0; i < d; ++i) dot = fmaf((float)qr[i], Codes<FMT>::value(c.k[at + k_byte(t, i, d)]), dot);
            x = dot * ks * scale;
        }
        float mx = x;
        for (int off = 1; off < kWave; off <<= 1) mx = fmaxf(mx, __shfl_xor(mx, off, kWave));
        const float mn = fmaxf(m, mx);
        const float f = m == mn ? 1.f : expf(m - mn);
        const float p = in ? expf(x - mn) : 0.f;
        l = fmaf(l, f, group_sum<64>(p));
        m = mn;
        for (int i = 0; i < 4; ++i) acc[i] *= f;
        const float w = in ? p * vs : 0.f;
        for (int k = 0; k < kWave; ++k) {
            if (j0 + k < lo || j0 + k > pos) continue;
            const float wk = __shfl(w, k, kWave);
            const size_t ak = ((size_t)(uint32_t)__shfl((int)(at >> 32), k, kWave) << 32) | (uint32_t)__shfl((int)at, k, kWave);
            const int t = (j0 + k) & (c.page - 1);
            for (int i = 0; i < 4; ++i)
                if (lane + 64 * i < d)
                    acc[i] = fmaf(wk, Codes<FMT>::value(c.v[ak + v_byte(t, lane + 64 * i, d)]), acc[i]);
        }
    }
    h16* yr = y + ((size_t)row * n_head + head) * d;
    for (int i = 0; i < 4; ++i)
        if (lane + 64 * i < d) yr[lane + 64 * i] = (h16)(pos < 0 ? 0.f : acc[i] / l);
    if (lse && lane == 0) lse[(size_t)row * n_head + head] = pos < 0 ? -__builtin_inff() : m + logf(l);
}

size_t kv_attend_bytes(int, int, int, int, int, int) { return 256; }
size_t kv_attend_zero_bytes() { return 256; }

hipError_t launch_kv_attend(const KvCache& c, const KvBatch& b, const h16* q, long long q_stride, int n_head,
                            float scale, int window, h16* y, float* lse, char*, hipStream_t s) {
    const long long units = (long long)b.n_tok * n_head;
    const dim3 grid((unsigned)((units + 3) / 4));
    if (c.fmt == 0)
        hipLaunchKernelGGL(k_attend<0>, grid, dim3(256), 0, s, c, b, q, q_stride, n_head, scale, window, y, lse);
    else
        hipLaunchKernelGGL(k_attend<1>, grid, dim3(256), 0, s, c, b, q, q_stride, n_head, scale, window, y, lse);
    return hipGetLastError();
}

}  // namespace pi
