"""Options of the cross entropy and norm calls given as tensors: every call sees
the value of that moment.  The library calls are recorded, not made.  No GPU."""
import numpy as np
import pytest
import torch

from chunked_kl_loss_tcgen05_b200 import torch_api as ta
from chunked_kl_loss_tcgen05_b200.build import build

bf = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()


@pytest.fixture
def calls(monkeypatch):
    """The problems the library would be called with; host tensors stand in for
    device ones."""
    seen = []

    def record(index, call, *args):
        if len(args) > 1:
            seen.append(args[0])
        return 0

    monkeypatch.setattr(ta, "_on_device", record)
    monkeypatch.setattr(ta, "_placed", lambda index, tensors: True)
    monkeypatch.setattr(ta, "_check_placement", lambda cuda, tensors: None)
    return seen


def _ce_args():
    return (torch.zeros(6, 16, dtype=bf), torch.zeros(64, 16, dtype=bf),
            torch.zeros(6, dtype=torch.int64))


def _ce_calls(**kw):
    h, W, y = _ce_args()
    z = torch.zeros(6)
    ta.fused_ce_fwd(h, W, y, check=False, **kw)
    ta.fused_ce_fwd_bwd(h, W, y, check=False, **kw)
    kw.pop("n_valid_total", None)
    ta.fused_ce_bwd(h, W, y, z, z, check=False, **kw)


@pytest.mark.parametrize("name,first,second", [
    ("T", 1.0, 2.0), ("label_smoothing", 0.0, 0.25), ("z_loss", 0.5, 0.125),
    ("ignore_index", -100, 7), ("chunk", 3, 2), ("n_valid_total", 5, 9)])
@pytest.mark.parametrize("make", [torch.tensor, np.array])
def test_cross_entropy_option_changed_in_place(calls, name, first, second, make):
    option = make(first)
    _ce_calls(**{name: option})
    option[...] = second
    _ce_calls(**{name: option})
    if name == "n_valid_total":        # the backward for row gradients has no mean
        calls = calls[:2] + calls[3:5]
    half = len(calls) // 2
    assert [getattr(p, name) for p in calls] == [first] * half + [second] * half


@pytest.mark.parametrize("name,first,second", [
    ("scale", 0.5, 3.0), ("eps", 0.25, 0.125), ("weight_offset", 0.0, 1.0)])
def test_norm_option_changed_in_place(calls, name, first, second):
    x, w = torch.zeros(4, 16, dtype=bf), torch.ones(16)
    option = torch.nn.Parameter(torch.tensor(first))
    for value in (first, second):
        option.data.fill_(value)
        ta.block_norm_fwd(x, x, w, pre_weight=w, **{name: option})
        ta.block_norm_bwd(x, x, dy=x, post_weight=w, pre_weight=w, **{name: option})
    assert [getattr(p, name) for p in calls] == [first] * 2 + [second] * 2


def test_backward_uses_the_options_of_its_forward(calls):
    h, W, y = _ce_args()
    T = torch.tensor(2.0)
    rows = ta.fused_cross_entropy_loss(h.requires_grad_(), W, y, T=T, reduction="none")
    T.fill_(4.0)
    rows.backward(torch.ones(6))
    x, s = torch.zeros(4, 16, dtype=bf, requires_grad=True), torch.tensor(0.5)
    v, _ = ta.block_norm(x, torch.zeros(4, 16, dtype=bf), scale=s)
    s.fill_(3.0)
    v.backward(torch.ones(4, 16, dtype=bf))
    assert [p.T for p in calls[:2]] == [2.0, 2.0]
    assert [p.scale for p in calls[2:]] == [0.5, 0.5]


def test_options_that_would_need_a_gradient_are_refused(calls):
    h, W, y = _ce_args()
    learned = torch.nn.Parameter(torch.tensor(0.5))
    for name in ("T", "label_smoothing", "z_loss"):
        with pytest.raises(ValueError, match=name):
            ta.fused_cross_entropy_loss(h.requires_grad_(), W, y, **{name: learned})
    x = torch.zeros(4, 16, dtype=bf)
    for name in ("scale", "eps", "weight_offset"):
        with pytest.raises(ValueError, match=name):
            ta.block_norm(x, x, **{name: learned})
    with torch.no_grad():
        ta.block_norm(x, x, scale=learned)
    assert [p.scale for p in calls] == [0.5]


def test_whole_number_options_refuse_fractions(calls):
    h, W, y = _ce_args()
    for name in ("ignore_index", "chunk", "n_valid_total"):
        with pytest.raises(TypeError):
            ta.fused_ce_fwd(h, W, y, check=False, **{name: 1.5})
    assert not calls


def test_held_gradients_are_float32_or_bfloat16(calls):
    h, W, y = _ce_args()
    with pytest.raises(TypeError, match="grad_dtype"):
        ta.fused_cross_entropy_loss(h.requires_grad_(), W, y, grad_dtype=torch.float16)
    for dtype in (torch.float32, torch.bfloat16):
        ta.fused_cross_entropy_loss(h.requires_grad_(), W, y, grad_dtype=dtype, check=False)
    assert [p.grad_type for p in calls] == [0, 1]


def test_mean_over_more_rows_than_the_call_s(calls):
    h, W, y = _ce_args()
    loss = ta.fused_cross_entropy_loss(h.requires_grad_(), W, y, n_valid_total=40, check=False)
    with torch.no_grad():
        ta.fused_cross_entropy_loss(h, W, y, n_valid_total=40, check=False)
    assert [p.n_valid_total for p in calls] == [40, 40]
