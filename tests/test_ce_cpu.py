"""Cross entropy against labels: the oracle's pins (library cross entropy,
autograd, finite differences) and every refusal of the entry points that the
host can decide.  No GPU."""
import numpy as np
import pytest
import torch

import chunked_kl_loss_tcgen05_b200 as fk
import oracle
from chunked_kl_loss_tcgen05_b200 import FcklCeProblem
from chunked_kl_loss_tcgen05_b200 import torch_api as ta
from chunked_kl_loss_tcgen05_b200.build import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()


def _case(N=7, H=12, V=19, seed=0):
    rng = np.random.default_rng(seed)
    h, W = rng.standard_normal((N, H)), rng.standard_normal((V, H)) * 0.4
    y = rng.integers(0, V, N)
    y[1] = -100
    return h, W, y, rng.random(N) + 0.5


@pytest.mark.parametrize("smooth", [0.0, 0.1, 1.0])
@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_oracle_matches_library_cross_entropy_and_autograd(smooth, reduction):
    h, W, y, _ = _case()
    T = 1.7
    o = oracle.cross_entropy(h, W, y, T=T, label_smoothing=smooth, reduction=reduction)
    ht, Wt = (torch.tensor(a, requires_grad=True) for a in (h, W))
    a = ht @ Wt.T / T
    loss = torch.nn.functional.cross_entropy(a, torch.tensor(y), label_smoothing=smooth,
                                             reduction=reduction)
    gh, gW = torch.autograd.grad(loss, (ht, Wt))
    assert abs(o["loss"] - loss.item()) < 1e-12
    np.testing.assert_allclose(o["dH"], gh.numpy(), atol=1e-13)
    np.testing.assert_allclose(o["dW"], gW.numpy(), atol=1e-13)
    keep = y != -100
    np.testing.assert_allclose(o["lse"][keep], torch.logsumexp(a, 1).detach().numpy()[keep])
    assert o["row_loss"][1] == 0 and (o["dH"][1] == 0).all()


def test_oracle_gradients_by_differences():
    h, W, y, w = _case(N=4, H=5, V=9, seed=3)
    kw = dict(row_weight=w[:4], T=0.8, label_smoothing=0.2, z_loss=0.05)
    o = oracle.cross_entropy(h, W, y, **kw)
    d = 1e-5
    for X, g in ((h, o["dH"]), (W, o["dW"])):
        for i in np.ndindex(X.shape):
            keep = X[i]
            X[i] = keep + d
            up = oracle.cross_entropy(h, W, y, **kw)["loss"]
            X[i] = keep - d
            down = oracle.cross_entropy(h, W, y, **kw)["loss"]
            X[i] = keep
            assert abs((up - down) / (2 * d) - g[i]) < 1e-8
    # the row gradient form: sum_r k_r l_r
    k = np.array([0.3, 1.0, -2.0, 0.7])
    kw.pop("row_weight")
    r = oracle.cross_entropy(h, W, y, row_grad=k, **kw)
    s = oracle.cross_entropy(h, W, y, row_weight=k, reduction="sum", **kw)
    np.testing.assert_allclose(r["dW"], s["dW"])


def test_no_kept_row_gives_zero():
    h, W, y, _ = _case()
    o = oracle.cross_entropy(h, W, np.full_like(y, -100))
    assert o["loss"] == 0 and not o["dH"].any() and not o["dW"].any()


@pytest.mark.parametrize("bad", [
    dict(N=0), dict(H=0), dict(V=0), dict(T=0.0), dict(T=float("nan")), dict(T=float("inf")),
    dict(label_smoothing=-0.1), dict(label_smoothing=1.5), dict(label_smoothing=float("nan")),
    dict(z_loss=-1.0), dict(z_loss=float("inf")), dict(reduction=2), dict(label_type=7),
    dict(grad_type=3), dict(chunk=-1), dict(n_valid_total=-1), dict(N=2**31), dict(V=2**31)])
def test_invalid_problem_rejected(bad):
    p = FcklCeProblem(**{**dict(N=64, H=64, V=512), **bad})
    assert fk.fckl_ce_workspace_bytes(p, True) == 0
    f = 1 << 20
    args = [f] * 3
    assert fk.fckl_ce_fwd(p, *args, None, f, None, None, f, 1 << 40, None) == fk.FCKL_ERR_INVALID_ARG
    assert fk.fckl_ce_bwd(p, *args, f, f, f, f, f, 1 << 40, None) == fk.FCKL_ERR_INVALID_ARG


def test_null_misaligned_and_unsupported_arguments_rejected():
    p = FcklCeProblem(64, 64, 512)
    ws = fk.fckl_ce_workspace_bytes(p, True)
    assert ws > fk.fckl_ce_workspace_bytes(p, False) > 0
    f = 1 << 20

    def train(*a, nbytes=ws):
        return fk.fckl_ce_fwd_bwd(p, *a, nbytes, None)

    good = [f, f, f, f, f, f, f, f, f, f]
    for i in (0, 1, 2, 4):
        a = list(good)
        a[i] = None
        assert train(*a) == fk.FCKL_ERR_INVALID_ARG, i
    for i, off in ((0, 8), (1, 2), (2, 4), (3, 2), (4, 2), (5, 1), (6, 2), (7, 8), (8, 4)):
        a = list(good)
        a[i] = f + off
        assert train(*a) == fk.FCKL_ERR_INVALID_ARG, i
    a = list(good)
    a[7] = a[8] = None          # no gradient asked for
    assert train(*a) == fk.FCKL_ERR_INVALID_ARG
    assert train(*good, nbytes=ws - 1) == fk.FCKL_ERR_WORKSPACE
    a = list(good)
    a[9] = f + 16
    assert train(*a) == fk.FCKL_ERR_WORKSPACE
    odd = FcklCeProblem(64, 60, 512)
    assert fk.fckl_ce_workspace_bytes(odd, True) == 0
    assert fk.fckl_ce_fwd(odd, f, f, f, None, f, None, None, f, 1 << 40, None) == fk.FCKL_ERR_UNSUPPORTED
    # int32 labels need 4-byte alignment only
    p32 = FcklCeProblem(64, 64, 512, label_type=fk.FCKL_LABELS_INT)
    st = fk.fckl_ce_fwd(p32, f, f, f + 4, None, f, None, None, None, 0, None)
    assert st == fk.FCKL_ERR_WORKSPACE
    # backward needs the log-sum-exps and the row gradient
    for lse, g in ((None, f), (f, None)):
        assert fk.fckl_ce_bwd(p, f, f, f, lse, g, f, f, f, ws, None) == fk.FCKL_ERR_INVALID_ARG
    for a in ((None, 4, 0, f), (f, 0, 0, f), (f, 4, 2, f), (f, 4, 0, None), (f + 4, 4, 0, f)):
        assert fk.fckl_scale_gradient(*a, None) == fk.FCKL_ERR_INVALID_ARG


def test_workspace_rules():
    """One chunk of 16-bit dlogits; the fp32 sum of dW only for bf16 gradients of
    several chunks."""
    one = dict(N=4096, H=1024, V=128256)
    a = fk.fckl_ce_workspace_bytes(FcklCeProblem(**one, grad_type=fk.FCKL_GRAD_BFLOAT), True)
    b = fk.fckl_ce_workspace_bytes(FcklCeProblem(**one), True)
    assert a == b and a >= 4096 * 128256 * 2
    many = dict(one, N=40960)
    fp32 = fk.fckl_ce_workspace_bytes(FcklCeProblem(**many), True)
    bf16 = fk.fckl_ce_workspace_bytes(FcklCeProblem(**many, grad_type=fk.FCKL_GRAD_BFLOAT), True)
    # ten chunks of 4096 rows: the row list and the rows' loss shares grow
    assert fp32 - b == 36864 * 8
    assert bf16 - fp32 == 128256 * 1024 * 4
    small = fk.fckl_ce_workspace_bytes(FcklCeProblem(**many, chunk=256), True)
    assert small < fp32 - 3800 * 128256 * 2


def _t(N=6, H=16, V=64, **over):
    t = dict(hidden=torch.zeros(N, H, dtype=torch.bfloat16),
             W=torch.zeros(V, H, dtype=torch.bfloat16), labels=torch.zeros(N, dtype=torch.int64))
    t.update(over)
    return t


@pytest.mark.parametrize("over,kw,exc", [
    (dict(labels=torch.zeros(5, dtype=torch.int64)), {}, ValueError),
    (dict(labels=torch.zeros(6, 1, dtype=torch.int64)), {}, ValueError),
    (dict(labels=torch.zeros(6)), {}, TypeError),
    (dict(hidden=torch.zeros(6, 16)), {}, TypeError),
    (dict(W=torch.zeros(64, 8, dtype=torch.bfloat16)), {}, ValueError),
    ({}, dict(row_weight=torch.ones(5)), TypeError),
    ({}, dict(row_weight=torch.ones(6, dtype=torch.float64)), TypeError),
    ({}, dict(reduction="none"), ValueError),
    ({}, {}, ValueError),                                       # host tensors
])
@pytest.mark.parametrize("fn", [ta.fused_ce_fwd, ta.fused_ce_fwd_bwd])
def test_tensor_checks(fn, over, kw, exc):
    with pytest.raises(exc):
        fn(**_t(**over), **kw)


def test_backward_and_autograd_checks():
    t, row = _t(), torch.zeros(6)
    with pytest.raises(TypeError, match="lse"):
        ta.fused_ce_bwd(**t, lse=torch.zeros(5), row_grad=row)
    with pytest.raises(TypeError, match="row_grad"):
        ta.fused_ce_bwd(**t, lse=row, row_grad=torch.zeros(6, dtype=torch.float64))
    with pytest.raises(TypeError):
        ta.fused_ce_bwd(**t, lse=None, row_grad=row)
    with pytest.raises(ValueError, match="both"):
        ta.fused_ce_bwd(**t, lse=row, row_grad=row, want=(False, False))
    with pytest.raises(TypeError, match="grad_dtype"):
        ta.fused_ce_bwd(**t, lse=row, row_grad=row, grad_dtype=torch.float16)
    with pytest.raises(ValueError, match="reduction"):
        ta.fused_cross_entropy_loss(**t, reduction="average")
    with pytest.raises(ValueError, match="row_weight"):
        ta.fused_cross_entropy_loss(**t, row_weight=torch.ones(6, requires_grad=True))
    with pytest.raises(ValueError, match="row_weight"):
        ta.fused_cross_entropy_loss(**t, row_weight=torch.ones(6), reduction="none")
