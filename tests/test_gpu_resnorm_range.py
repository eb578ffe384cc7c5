"""The residual norm over the whole of its accepted range: eps of zero, rows
side by side with rows past the end, rows of large and small numbers.  Oracle and tolerances as in
``test_gpu_resnorm.py``, whose derivation does not depend on eps or on the rows' size."""
import numpy as np
import pytest
import torch

from oracle import train_ops as T
from tests.test_gpu_resnorm import DT, _case, _check, _close, _gate_np, _np, _rows

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


def _even(g, shape):
    """Normal numbers, none smaller than a half in magnitude, so that no row is much smaller than 1."""
    v = g.standard_normal(shape)
    return np.sign(v) * np.maximum(np.abs(v), 0.5)


def _sized(q, g, m, d, act, res, kind, sh, sy, eps, offset=0.25, extra=0.0):
    """Both directions with residual rows of the size `sh`, block outputs of the size `sy`, and gradients that keep both
    terms of dx of one size."""
    a = _case(g, m, d, act, res, "f32", kind, True, True)
    a["x"], a["y"] = (_rows(_even(g, (m, d)) * s, t) for s, t in ((sh, res), (sy, act)))
    eps = float(np.float32(eps))
    kw = dict(scale=0.75, eps=eps, w_offset=offset)
    args = (_gate_np(a, kind), kind, _np(a["w_post"]), _np(a["w_pre"]), True, True, 0.75, eps, offset)
    h, z = q.qlora_resnorm_fwd(a["x"], a["y"], a["gate"], a["w_post"], a["w_pre"], **kw)
    hw, zw = T.resnorm_fwd(_np(a["x"]), _np(a["y"]), *args)
    mag = np.abs(_np(a["x"])) + np.abs(hw - _np(a["x"]))
    _close(h, hw, mag, res, extra, name="h")
    r = 1 / np.sqrt((hw * hw).mean(1, keepdims=True) + eps)
    w = np.abs(offset + _np(a["w_pre"]))
    _close(z, zw, r * w * (mag + np.abs(hw) * (r * r * (np.abs(hw) * mag).mean(1, keepdims=True))), act, extra, name="z")
    h, dz, dh = (_rows(_even(g, (m, d)) * s, t) for s, t in ((sh, res), (1.0, act), (1 / sh, res)))
    for given in (None, dh):
        got = q.qlora_resnorm_bwd(dz, given, h, a["y"], a["gate"], a["w_post"], a["w_pre"], **kw)
        want, mg = T.resnorm_bwd(_np(dz), _np(given), _np(h), _np(a["y"]), *args)
        for k, t in zip(("dx", "dy", "dgate", "dw_post", "dw_pre"), got):
            if k not in want:
                continue
            dt = res if k == "dx" else act if k == "dy" or (k == "dgate" and kind == "full") else "f32"
            col = k in ("dw_post", "dw_pre") or (k == "dgate" and kind == "channel")
            _close(t if t.dim() == want[k].ndim else t[:, 0], want[k], mg[k], dt, extra + (m * 2.0 ** -24 if col else 0.0), k)


@pytest.mark.parametrize("size,eps", [(1e13, 1e-5), (1e15, 1e-5), (1e17, 1e-5), (1e-14, 0.0), (1e-14, 1e-30),
                                      (1e-17, 0.0)])
@pytest.mark.parametrize("d", [64, 1001, 4096, 9000])
def test_large_and_small_rows(q, size, eps, d):
    """Rows whose squares binary32 holds, though the cube of their root is out of its range."""
    g = np.random.default_rng(d)
    for act, res in (("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")):
        for sh, sy in ((size, size), (size, 1.0), (1.0, size)):
            _sized(q, g, 3, d, act, res, "channel", sh, sy, eps)
    for kind in ("none", "token", "full"):
        _sized(q, g, 3, d, "f32", "f32", kind, size, size, eps)


@pytest.mark.parametrize("eps", [0.0, 1e-42])
@pytest.mark.parametrize("d", [5, 64, 1001, 4096, 9000])
def test_subnormal_mean_squares(q, eps, d):
    """Rows of 2^-65, whose squares and their mean are subnormal.  Each square is off by half of the
    spacing 2^-149 and so is the mean: 2^-149 in all, of a mean of 2^-130 and at least a quarter of that
    in these rows, 2^-17 relative; its root is off by half of that, and the outputs hold at most three roots:
    2^-14 covers them."""
    g = np.random.default_rng(d)
    size = 2.0 ** -65
    for act, res in (("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")):
        for sh, sy in ((size, 1.0), (1.0, size)):
            _sized(q, g, 3, d, act, res, "channel", sh, sy, eps, extra=2.0 ** -14)
        x, dz = _rows(_even(g, (3, d)) * size, res), _rows(g.standard_normal((3, d)), act)
        w = torch.from_numpy(g.standard_normal(d).astype(np.float32)).cuda()
        e = float(np.float32(eps))
        _, z = q.qlora_resnorm_fwd(x, w_pre=w, eps=eps, act_dtype=DT[act])
        _, zw = T.resnorm_fwd(_np(x), None, None, "none", None, _np(w), False, True, 1.0, e, 0.0)
        _close(z, zw, np.abs(zw), act, 2.0 ** -14)
        dx, _, _, _, dw = q.qlora_resnorm_bwd(dz, None, x, w_pre=w, eps=eps)
        want, mg = T.resnorm_bwd(_np(dz), None, _np(x), None, None, "none", None, _np(w), False, True, 1.0, e, 0.0)
        _close(dx, want["dx"], mg["dx"], res, 2.0 ** -14)
        _close(dw, want["dw_pre"], mg["dw_pre"], "f32", 2.0 ** -14)


def _alike(got, want):
    """Finite, infinite (with its sign) and no number in the same places."""
    got = _np(got)
    return (np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), np.isinf(want))
            and np.array_equal(np.sign(got[np.isinf(got)]), np.sign(want[np.isinf(want)])))


@pytest.mark.filterwarnings("ignore::RuntimeWarning")
@pytest.mark.parametrize("d", [5, 9, 64, 1001, 1500, 4097, 8191, 9001])
def test_infinite_weight_near_the_end_of_a_row(q, d):
    """An infinite weight acts on its own column and on what the formulas sum over, also where the row's last
    vector lies over columns of the thread before."""
    g = np.random.default_rng(d)
    m = 3
    for act, res in (("f32", "f32"), ("bf16", "f32"), ("f16", "f16")):
        for col in sorted({max(0, d - 8), max(0, d // 8 * 8 - 1), d - 1}):
            x, y, dz, dh = (_rows(_even(g, (m, d)), t) for t in (res, act, act, res))
            w, bad = (torch.from_numpy(_even(g, d).astype(np.float32)).cuda() for _ in range(2))
            bad[col] = float("inf")
            for w_post, w_pre in ((bad, w), (w, bad)):
                a = (None, "none", _np(w_post), _np(w_pre), True, True, 1.0, float(np.float32(1e-5)), 0.0)
                h, z = q.qlora_resnorm_fwd(x, y, None, w_post, w_pre, eps=1e-5)
                hw, zw = T.resnorm_fwd(_np(x), _np(y), *a)
                assert _alike(h, hw) and _alike(z, zw)
                # any residual for the backward: the ordinary x
                got = q.qlora_resnorm_bwd(dz, dh, x, y, None, w_post, w_pre, eps=1e-5)
                want, mg = T.resnorm_bwd(_np(dz), _np(dh), _np(x), _np(y), *a)
                for k, t in zip(("dx", "dy", "dgate", "dw_post", "dw_pre"), got):
                    assert t is None or _alike(t, want[k]), k
                _close(got[4], want["dw_pre"], mg["dw_pre"], "f32", m * 2.0 ** -24)
                if w_post is bad:
                    _close(got[0], want["dx"], mg["dx"], res)
                    _close(got[3], want["dw_post"], mg["dw_post"], "f32", m * 2.0 ** -24)
