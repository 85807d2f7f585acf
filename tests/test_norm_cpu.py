"""The norms around a block: the oracle's pins (autograd, library norms,
differences) and the refusals of the entry points.  No GPU."""
import numpy as np
import pytest
import torch

import chunked_kl_loss_tcgen05_b200 as fk
import oracle
from chunked_kl_loss_tcgen05_b200 import FcklNormProblem
from chunked_kl_loss_tcgen05_b200 import torch_api as ta
from chunked_kl_loss_tcgen05_b200.build import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()


def _case(N=5, H=12, seed=0):
    r = np.random.default_rng(seed)
    return (r.standard_normal((N, H)), r.standard_normal((N, H)), r.standard_normal(H),
            r.standard_normal(H), r.standard_normal(H), r.standard_normal((N, H)),
            r.standard_normal((N, H)))


@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False)])
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_oracle_matches_autograd(post, pre, offset):
    x, b, w1, g, w2, dy, dv = _case()
    t = {k: torch.tensor(a, requires_grad=True)
         for k, a in dict(x=x, b=b, w1=w1, g=g, w2=w2).items()}
    F = torch.nn.functional
    u = F.rms_norm(t["b"], (12,), t["w1"] + offset, eps=1e-5) if post else t["b"]
    v = t["x"] + 0.3 * t["g"] * u
    total = (v * torch.tensor(dv)).sum()
    if pre:
        y = F.rms_norm(v, (12,), t["w2"] + offset, eps=1e-5)
        total = total + (y * torch.tensor(dy)).sum()
    kw = dict(w1=w1 if post else None, g=g, w2=w2 if pre else None, scale=0.3, post=post, pre=pre,
              eps=1e-5, offset=offset)
    ov, oy = oracle.block_norm(x, b, **kw)
    np.testing.assert_allclose(ov, v.detach().numpy(), atol=1e-13)
    if pre:
        np.testing.assert_allclose(oy, y.detach().numpy(), atol=1e-13)
    o = oracle.block_norm_grads(x, b, dy if pre else None, dv, **kw)
    names = [("x", "dx"), ("b", "dblock"), ("g", "dg")]
    names += [("w1", "dw1")] * post + [("w2", "dw2")] * pre
    for (k, name), grad in zip(names, torch.autograd.grad(total, [t[k] for k, _ in names])):
        np.testing.assert_allclose(o[name], grad.numpy(), atol=1e-12)


def test_oracle_plain_norm_and_differences():
    x, b, w1, g, w2, dy, dv = _case(3, 7, 1)
    v, y = oracle.block_norm(x, w2=w2)
    assert v is not None and np.allclose(y, x / np.sqrt((x * x).mean(1, keepdims=True) + 1e-6) * w2)
    kw = dict(w1=w1, g=g, w2=w2, scale=0.7)
    o = oracle.block_norm_grads(x, b, dy, None, **kw)
    for i in np.ndindex(b.shape):
        keep = b[i]
        lo_hi = []
        for d in (1e-6, -1e-6):
            b[i] = keep + d
            lo_hi.append((oracle.block_norm(x, b, **kw)[1] * dy).sum())
        b[i] = keep
        assert abs((lo_hi[0] - lo_hi[1]) / 2e-6 - o["dblock"][i]) < 1e-6


F = 1 << 20


@pytest.mark.parametrize("bad", [
    dict(N=0), dict(H=0), dict(N=2**31), dict(eps=-1e-6), dict(eps=float("nan")),
    dict(scale=float("inf")), dict(weight_offset=float("nan")), dict(flags=4), dict(flags=-1),
    dict(x_type=2), dict(weight_type=-1), dict(dy_type=9)])
def test_invalid_problem_rejected(bad):
    p = FcklNormProblem(**{**dict(N=8, H=64), **bad})
    assert fk.fckl_block_norm_workspace_bytes(p) == 0
    assert fk.fckl_block_norm_fwd(p, F, F, F, F, F, F, F, None) == fk.FCKL_ERR_INVALID_ARG


@pytest.mark.parametrize("H", [12, 8200, 60])
def test_unsupported_width_rejected(H):
    p = FcklNormProblem(8, H)
    assert fk.fckl_block_norm_workspace_bytes(p) == 0
    assert fk.fckl_block_norm_fwd(p, F, F, F, F, F, F, F, None) == fk.FCKL_ERR_UNSUPPORTED
    assert fk.fckl_block_norm_bwd(p, F, F, F, F, F, F, F, F, F, F, F, F, F, 1 << 40,
                                  None) == fk.FCKL_ERR_UNSUPPORTED


def test_inconsistent_arguments_rejected():
    both = FcklNormProblem(8, 64)
    pre = FcklNormProblem(8, 64, flags=fk.FCKL_NORM_PRE)
    post = FcklNormProblem(8, 64, flags=fk.FCKL_NORM_POST)

    def fwd(p, *a):
        return fk.fckl_block_norm_fwd(p, *a, None)

    bad = fk.FCKL_ERR_INVALID_ARG
    assert fwd(both, None, F, F, F, F, F, F) == bad        # no x
    assert fwd(both, F, None, None, None, F, None, F) == bad   # post-norm of nothing
    assert fwd(pre, F, None, None, F, F, None, F) == bad   # gate of nothing
    assert fwd(pre, F, None, None, None, F, F, F) == bad   # v is x itself
    assert fwd(pre, F, F, F, None, F, F, F) == bad         # weight of a norm that is not there
    assert fwd(post, F, F, F, None, F, F, None) == bad
    assert fwd(both, F, F, F, F, F, F, None) == bad        # pre-norm without y
    assert fwd(post, F, F, F, F, None, F, F) == bad        # y without pre-norm
    assert fwd(post, F, F, F, F, None, None, None) == bad  # no output
    for i in range(7):
        a = [F] * 7
        a[i] = F + 8
        assert fwd(both, *a) == bad, i

    def bwd(p, *a, ws=F, n=1 << 40):
        return fk.fckl_block_norm_bwd(p, *a, ws, n, None)

    good = [F] * 12
    for i in (0, 5):
        a = list(good)
        a[i] = None
        assert bwd(both, *a) == bad, i
    for i in range(12):
        a = list(good)
        a[i] = F + 4
        assert bwd(both, *a) == bad, i
    assert bwd(both, F, F, None, F, F, F, F, F, F, F, F, F) == bad   # gradient of an absent weight
    assert bwd(both, F, F, F, F, F, F, F, None, None, None, None, None) == bad
    assert bwd(post, F, F, F, F, None, None, None, F, F, F, F, None) == bad   # no upstream
    assert bwd(both, *good, ws=None) == fk.FCKL_ERR_WORKSPACE
    need = fk.fckl_block_norm_workspace_bytes(both)
    assert need > 0 and bwd(both, *good, n=need - 1) == fk.FCKL_ERR_WORKSPACE


def _t(N=4, H=16, **over):
    bf = torch.bfloat16
    t = dict(x=torch.zeros(N, H, dtype=bf), block=torch.zeros(N, H, dtype=bf),
             post_weight=torch.ones(H, dtype=bf), pre_weight=torch.ones(H, dtype=bf))
    t.update(over)
    return t


@pytest.mark.parametrize("over,exc", [
    (dict(x=torch.zeros(16)), ValueError),
    (dict(x=torch.zeros(4, 16, dtype=torch.float16)), TypeError),
    (dict(block=torch.zeros(4, 16)), TypeError),
    (dict(block=torch.zeros(3, 16, dtype=torch.bfloat16)), ValueError),
    (dict(post_weight=torch.ones(8, dtype=torch.bfloat16)), ValueError),
    (dict(gate=torch.ones(16)), TypeError),                       # mixed weight types
    (dict(gate=torch.ones(4, 16, dtype=torch.bfloat16)), ValueError),
    ({}, ValueError),                                             # host tensors
])
def test_tensor_checks(over, exc):
    with pytest.raises(exc):
        ta.block_norm_fwd(**_t(**over))
    with pytest.raises(exc):
        ta.block_norm_bwd(**_t(**over), dy=torch.zeros(4, 16))


def test_backward_and_wrapper_checks():
    with pytest.raises(ValueError, match="dy"):
        ta.block_norm_bwd(**_t())
    t = _t()
    t.pop("pre_weight")
    with pytest.raises(ValueError, match="dv"):
        ta.block_norm_bwd(**t, pre=False)
    with pytest.raises(TypeError, match="dv"):
        ta.block_norm_bwd(**_t(), dy=torch.zeros(4, 16), dv=torch.zeros(4, 16))
    with pytest.raises(TypeError, match="dy"):
        ta.block_norm_bwd(**_t(), dy=torch.zeros(4, 16, dtype=torch.float64))
    with pytest.raises(ValueError, match="pre-norm"):
        ta.block_norm(torch.zeros(4, 16), pre=False)
