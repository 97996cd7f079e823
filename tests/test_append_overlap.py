"""pi_kv_append_rope's turned queries lie outside the keys' and values' rows: the host's
check against sets of bytes, and its refusals, before any HIP call."""

import os

import pytest

from activation_sparse_predictor_amd import binding as B
from tests.test_draft_host import A, FAR, write
from tests.test_kv_plan import host_program

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libpi.so not built")


def test_rows_that_meet(tmp_path):
    """rows_meet against byte by byte, for all small places, strides, widths and counts."""
    out = host_program(tmp_path, r"""
    long long wrong = 0, met = 0, all = 0;
    for (int stride = 1; stride <= 5; ++stride) for (int row = 1; row <= stride; ++row) for (int n = 1; n <= 3; ++n)
    for (int step = 1; step <= 5; ++step) for (int other = 1; other <= step; ++other) for (int m = 1; m <= 3; ++m)
    for (int a = 0; a <= 16; ++a) {
        const int b = 16;   // a before and at b; b before a by the roles exchanged
        bool hit = false;
        for (int i = 0; i < n; ++i) for (int j = 0; j < m; ++j)
            hit |= a + i * stride < b + j * step + other && b + j * step < a + i * stride + row;
        wrong += rows_meet(a, stride, row, n, b, step, other, m) != hit;
        wrong += rows_meet(b, step, other, m, a, stride, row, n) != hit;
        met += hit, ++all;
    }
    printf("%lld %lld %lld\n", wrong, met, all);
    return 0;""")
    wrong, met, count = (int(x) for x in out)
    assert wrong == 0 and 0 < met < count


# 3 tokens; k and v: 2 heads of 64, 256 bytes a row; queries: 8 heads, 1024 bytes
@pytest.mark.parametrize("kw", [
    dict(k=FAR), dict(v=FAR), dict(k=FAR + 1008), dict(k=FAR - 240), dict(v=FAR + 2 * 1024 + 1008), dict(v=FAR - 2 * 256 - 240),
    dict(k=FAR + 1008, k_stride=512), dict(v=FAR - 512 + 768 + 16, v_stride=512),
    dict(q_out=A, q_stride=640, k_stride=640, out_stride=640),   # the queries' own place, which the keys share
    dict(q=A, q_out=A, q_stride=640, out_stride=640, k=A + 1008, k_stride=640, v=FAR, v_stride=640),   # one projection, the keys a vector too early
    dict(q=A, q_out=A, q_stride=640, out_stride=640, k=A + 1024, k_stride=640, v=A + 1264, v_stride=640)])   # the values' end in the next token's queries
def test_refused(kw):
    assert write(**kw) == B.PI_ERR_INVALID_ARG and "q_out overlaps" in B.last_error()
