"""The AdamW step over the whole of its accepted range: eps of zero with subnormal second moments.
Oracle and tolerances as in ``test_gpu_adamw.py``; a subnormal second moment
is off by half the spacing 2^-149 at each of its three roundings besides."""
import numpy as np
import pytest
import torch

from oracle import train_ops as T
from tests.test_gpu_adamw import U, _np, _sections, _tensors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import qlora_fine_tuning_nf4_amd as pkg
    pkg.lib()
    return pkg


@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-30, 1e-20, 1e-12, 1e-8])
@pytest.mark.parametrize("bits", [32, 8])
def test_subnormal_second_moments(q, bits, eps):
    """Gradients near 1e-20: their squares are subnormal, the steps are as large as with any other."""
    g = np.random.default_rng(bits)
    sizes = [3000, 5]
    b1, b2, lr, step = 0.9, 0.99, 0.01, 4
    p, gr = _tensors(g, sizes, "f32"), _tensors(g, sizes, "f32")
    for t in gr:
        t.copy_(torch.from_numpy((np.sign(g.standard_normal(t.numel())) * g.uniform(1e-19, 3e-19, t.numel())).astype(np.float32)))
    plan = q.qlora_adamw_init(p, gr, state_bits=bits)
    st = plan.new_state()
    if bits == 32:
        for a, b in zip(_sections(st.m, sizes), _sections(st.v, sizes)):
            a.copy_(torch.from_numpy((g.standard_normal(len(a)) * 1e-20).astype(np.float32)))
            b.copy_(torch.from_numpy(g.uniform(1e-40, 1e-39, len(b)).astype(np.float32)))
    m, v = (x.double().cpu().numpy() for x in st.moments())
    p0 = [_np(t) for t in p]
    q.qlora_adamw_step(plan, st, step, lr, betas=(b1, b2), eps=eps)
    for i, x0 in enumerate(p0):
        m0, v0 = _sections(m, sizes)[i], _sections(v, sizes)[i]
        m1, v1 = T.adamw_moments(_np(gr[i]), m0, v0, b1, b2)
        want = T.adamw_param(x0, m1, v1, step, lr, b1, b2, eps, 0.0)
        size = lr / (1 - b1 ** step) * (b1 * np.abs(m0) + (1 - b1) * np.abs(_np(gr[i]))) / (
            np.sqrt(v1 / (1 - b2 ** step)) + eps)
        assert (np.abs(_np(p[i]) - want) <= (32 * U + 3 * 2.0 ** -150 / v1) * size + 4 * U * np.abs(x0)).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_subnormal_eps_beside_zero_moments(q, bits):
    """Parameters that never had a gradient stay as they are for any eps above zero."""
    g = np.random.default_rng(1)
    p = _tensors(g, [700], "f32")
    plan = q.qlora_adamw_init(p, [torch.zeros_like(p[0])], state_bits=bits)
    before = p[0].clone()
    for eps in (1e-44, 1e-40, 1e-20, 1e-8):
        q.qlora_adamw_step(plan, plan.new_state(), 1, 0.1, eps=eps)
        assert torch.equal(p[0], before)


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan"), 1e25])
def test_one_bad_gradient_leaves_its_block(q, bad):
    """8-bit moments: a value whose moments are not finite changes nothing of its block's other values, in
    this step and the next, against a run where its gradient is 0."""
    g = np.random.default_rng(9)
    n, at = 600, 300
    grads = [torch.from_numpy(g.standard_normal(n).astype(np.float32)).cuda() for _ in range(3)]
    start = torch.from_numpy(g.standard_normal(n).astype(np.float32)).cuda()
    runs = []
    for value in (0.0, bad):
        p, gr = start.clone(), grads[0].clone()
        plan = q.qlora_adamw_init([p], [gr], state_bits=8)
        st = plan.new_state()
        steps = []
        for t in range(3):
            gr.copy_(grads[t])
            if t < 2:
                gr[at] = value if t else 0.0
            q.qlora_adamw_step(plan, st, t + 1, 0.01, seed=5)
            steps.append([x.clone() for x in (p, st.m.view(torch.uint8), st.v.view(torch.uint8), st.m_scale, st.v_scale)])
        runs.append(steps)
    other = torch.arange(n, device="cuda") != at
    code = (torch.arange(768, device="cuda") != at).view(3, 256)
    good, got = (r[1] for r in runs)
    assert torch.equal(got[2][code], good[2][code]) and torch.equal(got[4], good[4])
    assert got[2].view(-1)[at] == 0x7B                                 # 57344 in e5m2
    if abs(bad) != 1e25:                                               # 1e25: a finite first moment, and the block's largest
        assert torch.equal(got[1][code], good[1][code]) and torch.equal(got[3], good[3])
        assert got[1].view(-1)[at] & 0x7F == 0x7E                      # 448 in e4m3
        if bad == bad:
            assert (got[1].view(-1)[at] >= 0x80) == (bad < 0)
    good, got = (r[2] for r in runs)
    assert torch.isfinite(got[0][other]).all()
    if abs(bad) != 1e25:
        assert torch.equal(got[0][other], good[0][other])
        assert torch.isnan(got[0][at])
        # the third step's own gradient at the place is an ordinary one: the scales may hold it
        assert torch.isfinite(got[3]).all() and torch.isfinite(got[4]).all()


def test_norm_after_calls_that_overlapped(q):
    """Two calls on one plan at a time are against the rule and may return anything, but the next call is right."""
    p = torch.zeros(1 << 28, device="cuda")      # long enough for the calls to run side by side
    gr = torch.ones_like(p)
    plan = q.qlora_adamw_init([p], [gr])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                q.qlora_grad_norm(plan, 1.0)
    torch.cuda.synchronize()
    for value in (1.0, 0.5):
        gr.fill_(value)
        assert q.qlora_grad_norm(plan)[0].item() == 16384 * value
    assert not plan.table[:4].any()
