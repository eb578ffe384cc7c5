"""The residual norm over the whole of its accepted range: eps of zero, rows
side by side with rows past the end.  Oracle and tolerances as in
``test_gpu_resnorm.py``, whose derivation does not depend on eps or on the rows' size."""
import numpy as np
import pytest
import torch

from tests.test_gpu_resnorm import _check, _np, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import qlora_fine_tuning_nf4_amd as pkg
    pkg.lib()
    return pkg


@pytest.mark.parametrize("d", [40, 64, 1000, 1500, 2048, 4096, 8192, 9000])
@pytest.mark.parametrize("m", [1, 3, 5, 9])
def test_without_eps(q, m, d):
    """eps = 0: rows of numbers are as good as with one, whatever stands beside the last row."""
    g = np.random.default_rng(m + d)
    for act, res in (("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")):
        _check(q, g, m, d, act, res, kind="channel", eps=0.0)
    _check(q, g, m, d, "bf16", "f32", kind="full", eps=0.0)
    _check(q, g, m, d, "f16", "f16", kind="token", pre=False, eps=0.0)
    _check(q, g, m, d, "bf16", "bf16", kind="none", eps=0.0)


@pytest.mark.parametrize("kind", ["none", "channel", "token", "full"])
def test_earlier_rows_beside_the_last(q, kind):
    """An infinite gradient reaches its column's sum once: the places beside the last row, where it
    may still stand, add nothing (infinity times zero is no number)."""
    g = np.random.default_rng(21)
    m, d, row, col = 8 * 256 + 1, 64, 3, 5
    for act, res in (("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")):
        y, h = _rows(g.standard_normal((m, d)), act), _rows(g.standard_normal((m, d)), res)
        dh = _rows(g.standard_normal((m, d)), res)
        dh[row, col] = float("inf")
        gate = {"none": None, "channel": torch.ones(d, device="cuda"), "token": torch.ones(m, device="cuda"),
                "full": torch.ones_like(y)}[kind]
        dx, _, _, dw, _ = q.qlora_resnorm_bwd(None, dh, h, y, gate, pre=False)
        assert torch.equal(dx, dh)
        want = np.sign(_np(y)[row, col]) * np.inf
        assert dw[col].item() == want and torch.isfinite(dw).sum() == d - 1
