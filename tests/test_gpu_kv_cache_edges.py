"""The paged cache at the ends of what a call may hold, against 64 bits (bounds derived in kv_util)."""
import math

import pytest
import torch

import kv_util
from test_gpu_kv_cache import BF16, FP16, Setup, tf  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("rope", ["interleaved", "neox", None])
def test_rows_whose_squares_overflow_beside_ordinary_ones(tf, rope, page, D):  # noqa: F811
    """Rows share a warp: NaN, infinities and sums of squares beyond fp32 in some do not touch the others."""
    s = Setup(tf, [150, 33], [140, 33], D=D, page=page, H=4, Hkv=2, seed=21)
    plain = [t.clone() for t in s.q]
    want = s.append(tf, rope=rope)
    special = [3, 4, 21, 50, 77, 139, 150]
    for t in (s.k[0], s.q[0]):
        t[3, 0, 5] = math.nan
        t[4, 1] = math.nan
        t[21, 0, D - 1] = math.inf
        t[50, 1, 0] = -math.inf
        t[77] = (t[77].sign() * 1e19).to(BF16)   # the sum of the squares overflows, their mean does not
        t[139] *= 3e18
        t[150, 1, 2] = 2.0 ** 66
    s.append(tf, rope=rope, q=False)
    got = tf.kv_append(*s.args, s.k, s.v, s.q, rope=rope, q_weight=s.weights[0], k_weight=s.weights[1])
    same = torch.ones(s.T, dtype=torch.bool, device="cuda")
    same[special] = False
    assert torch.equal(got[0][same], want[0][same]) and bool(plain[0][same].isfinite().all())
    at = torch.cat([torch.arange(10, 150), torch.arange(33)]).cuda()
    ref, size = kv_util.rotated(s.q[0], s.weights[0], rope, kv_util.table(s.most * s.page, D), at)
    assert torch.equal(got[0].isnan(), ref.isnan())
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -20 * size + 2.0 ** -25
    assert bool((((got[0].double() - ref).abs() <= tol) | ref.isnan()).all())


@pytest.mark.parametrize("starts", [[1000, 1000, 1000], [1000, 1001, 1005], [2 ** 31 - 3] * 3, [24, 24, 40], [0, 1000, 1000], [-7, -7, -7],
                                    [23, 1, 0]])
def test_starts_that_do_not_ascend_within_the_rows(tf, starts):  # noqa: F811
    """Both calls say so, also where no sequence has new tokens or all of them lie behind the rows."""
    s = Setup(tf, [70, 33], [20, 3], page=16, seed=22)
    assert s.T == 23
    s.starts.copy_(torch.tensor(starts, dtype=torch.int32))
    before, out = s.copy(), [torch.full_like(t, 7.0) for t in s.q]
    tf.kv_append(*s.args, s.k, s.v, s.q, [t.clone() for t in out])
    assert tf.device_status(clear=True) == 8
    tf.kv_attend(*s.args, s.q, out)
    assert tf.device_status(clear=True) == 8
    if starts[0] > s.T or starts[-1] < 0:
        assert bool((out[0] == 7).all())
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, s.copy()))
