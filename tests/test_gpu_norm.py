"""The norms around a block on the GPU, against the fp64 oracle.

Tolerances: a bf16 output is rounded once (2^-8 of it), an fp32 one 2^-24.  The
fp32 arithmetic before that is a few dozen roundings of 2^-24 of the terms'
magnitudes (row sums over up to 8192 values in a tree of threads, 16-value
chains in each: at most ~32 additions deep; rsqrt 2^-22): 2^-17 of the summed
magnitudes covers it, with cancellation counted by taking magnitudes.  Column
sums over N rows add at most N 2^-24 of the summed magnitudes.
"""
import numpy as np
import pytest
import torch

import oracle
from chunked_kl_loss_tcgen05_b200.torch_api import (TailNorm, arrays_to_device, block_norm,
                                                    block_norm_bwd, block_norm_fwd,
                                                    fused_ce_fwd_bwd, fused_chunked_kl_loss,
                                                    fused_cross_entropy_loss, fused_kl_fwd_bwd)

pytestmark = pytest.mark.gpu
BF16, FP32 = 2.0 ** -8, 2.0 ** -24
EPS32 = 2.0 ** -17
bf, f32 = torch.bfloat16, torch.float32


def own(t):
    return BF16 if t.dtype == bf else FP32


def np64(t):
    return None if t is None else t.double().cpu().numpy()


class Case:
    def __init__(self, N, H, xt=bf, wt=bf, dyt=bf, post=True, gate=True, pre=True, dv=True,
                 offset=0.0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed * 1000 + N + H)

        def rnd(*s):
            return torch.randn(*s, generator=g, device="cuda")

        self.x = (rnd(N, H) * 1.5).to(xt)
        self.block = rnd(N, H).to(bf)
        self.w1 = (1 - offset + 0.2 * rnd(H)).to(wt) if post else None
        self.g = rnd(H).to(wt) if gate else None
        self.w2 = (1 - offset + 0.2 * rnd(H)).to(wt) if pre else None
        self.dy = rnd(N, H).to(dyt) if pre else None
        self.dv = rnd(N, H).to(xt) if dv or not pre else None
        self.kw = dict(post_weight=self.w1, gate=self.g, pre_weight=self.w2, scale=0.4, post=post,
                       pre=pre, eps=1e-5, weight_offset=offset)
        self.okw = dict(w1=np64(self.w1), g=np64(self.g), w2=np64(self.w2), scale=0.4, post=post,
                        pre=pre, eps=1e-5, offset=offset)

    def magnitudes(self):
        """Oracle values and the magnitudes of the terms they are summed from."""
        x, b = np64(self.x), np64(self.block)
        k = self.okw
        post, pre, off = k["post"], k["pre"], k["offset"]
        one = np.ones(x.shape[1])
        a1 = np.abs(one if k["w1"] is None else k["w1"] + off)
        a2 = np.abs(one if k["w2"] is None else k["w2"] + off)
        ag = np.abs(one if k["g"] is None else k["g"])
        rb = 1 / np.sqrt((b * b).mean(1, keepdims=True) + 1e-5) if post else 1.0
        bn = np.abs(b) * rb
        u = bn * a1 if post else np.abs(b)
        v, y = oracle.block_norm(x, b, **k)
        vm = np.abs(x) + 0.4 * ag * u
        m = dict(v=vm)
        dvm = np.zeros_like(x) if self.dv is None else np.abs(np64(self.dv))
        if pre:
            rv = 1 / np.sqrt((v * v).mean(1, keepdims=True) + 1e-5)
            # an error of v moves rho too, by the rows' mean
            ill = 1 + (vm * vm).mean(1, keepdims=True) * rv ** 2
            m["y"] = vm * rv * a2 * ill
            if self.dy is not None:
                dy = np.abs(np64(self.dy))
                t = dy * a2
                dvm = dvm + ill * (rv * t + vm * rv ** 3 * (vm * t).mean(1, keepdims=True))
                m["dw2"] = (dy * vm * rv * ill).sum(0)
        m["dx"] = dvm
        m["dg"] = (0.4 * dvm * u).sum(0)
        du = 0.4 * ag * dvm
        if post:
            m["dw1"] = (du * bn).sum(0)
            t = du * a1
            m["dblock"] = rb * (t + bn * (bn * t).mean(1, keepdims=True))
        else:
            m["dblock"] = du
        return v, y, m

    def check(self, grads=True):
        v, y = block_norm_fwd(self.x, self.block, **self.kw)
        ov, oy, m = self.magnitudes()
        assert v.dtype == self.x.dtype
        self.near("v", v, ov, m["v"])
        if self.w2 is not None:
            assert y.dtype == bf
            self.near("y", y, oy, m["y"])
        else:
            assert y is None
        if not grads:
            return
        got = block_norm_bwd(self.x, self.block, dy=self.dy, dv=self.dv, **self.kw)
        o = oracle.block_norm_grads(np64(self.x), np64(self.block), np64(self.dy), np64(self.dv),
                                    **self.okw)
        N = self.x.shape[0]
        for name, t in zip(("dx", "dblock", "dw1", "dg", "dw2"), got):
            if t is None:
                continue
            extra = N * FP32 if name in ("dw1", "dg", "dw2") else 0.0
            self.near(name, t, o[name], m[name], extra)
        assert got[0].dtype == self.x.dtype and got[1].dtype == bf
        assert (got[2] is None) == (self.w1 is None) and (got[3] is None) == (self.g is None)
        assert all(t.dtype == f32 for t in got[2:] if t is not None)

    @staticmethod
    def near(name, got, want, mag, extra=0.0):
        e = np.abs(np64(got) - want)
        bound = own(got) * np.abs(want) + (EPS32 + extra) * (1 + own(got)) * mag + 1e-30
        assert (e <= bound).all(), (name, (e / bound).max())


@pytest.mark.parametrize("N,H", [(1, 8), (1, 4096), (2, 248), (3, 264), (7, 1000), (33, 2048),
                                 (5, 2056), (40, 2880), (17, 8192), (700, 256), (1500, 1024),
                                 (3, 64), (31, 64), (33, 24), (10007, 40), (5, 72), (17, 128),
                                 (10001, 128), (9, 136), (6001, 512), (3, 520), (2, 4104)])
def test_sizes(N, H):
    Case(N, H).check()


@pytest.mark.parametrize("xt", [bf, f32])
@pytest.mark.parametrize("wt", [bf, f32])
@pytest.mark.parametrize("dyt", [bf, f32])
@pytest.mark.parametrize("H", [264, 4096])
def test_types(xt, wt, dyt, H):
    Case(50, H, xt, wt, dyt).check()


@pytest.mark.parametrize("post,gate,pre,dv", [
    (True, False, True, True), (False, True, True, False), (False, False, True, True),
    (True, True, False, True), (False, True, False, True), (True, True, True, False)])
@pytest.mark.parametrize("H", [520, 2320])
def test_parts(post, gate, pre, dv, H):
    Case(61, H, post=post, gate=gate, pre=pre, dv=dv, offset=1.0).check()


def test_more_rows_than_blocks():
    Case(5000, 72).check()


@pytest.mark.parametrize("H", [64, 4096])
def test_plain_norm_and_weightless_norms(H):
    c = Case(30, H)
    _, y = block_norm_fwd(c.x, pre_weight=c.w2, eps=1e-5)
    v, _ = block_norm_fwd(c.x, pre_weight=c.w2)
    assert v is c.x
    _, oy = oracle.block_norm(np64(c.x), w2=np64(c.w2), eps=1e-5)
    Case.near("y", y, oy, 2 * np.abs(oy))
    dx, db, d1, dg, d2 = block_norm_bwd(c.x, dy=c.dy, pre_weight=c.w2, eps=1e-5)
    o = oracle.block_norm_grads(np64(c.x), None, np64(c.dy), None, w2=np64(c.w2), eps=1e-5)
    xs = np.abs(np64(c.x))
    r = 1 / np.sqrt((xs * xs).mean(1, keepdims=True) + 1e-5)
    t = np.abs(np64(c.dy) * np64(c.w2))
    Case.near("dx", dx, o["dx"], 2 * (r * t + xs * r ** 3 * (xs * t).mean(1, keepdims=True)))
    Case.near("dw2", d2, o["dw2"], 2 * np.abs(np64(c.dy) * xs * r).sum(0), 30 * FP32)
    assert db is None and d1 is None and dg is None
    # both norms without weights
    v, y = block_norm_fwd(c.x, c.block, post=True, eps=1e-5)
    ov, oy = oracle.block_norm(np64(c.x), np64(c.block), post=True, eps=1e-5)
    Case.near("v", v, ov, np.abs(np64(c.x)) + 4 * np.abs(np64(c.block)))
    assert (np.abs(np64(y) - oy) <= BF16 * np.abs(oy) + EPS32 * 20).all()


def test_rows_of_zeros_and_far_values():
    """A zero row stays zero (eps > 0); rows near the ends of the bf16 range that
    still square in fp32; a row with NaN or inf spoils itself alone."""
    c = Case(12, 512)
    c.x[0] = 0; c.block[0] = 0
    c.x[1] *= 1e15; c.block[1] *= 1e15
    c.x[2] *= 1e-18; c.block[2] *= 1e-15
    c.x[3, 5] = float("nan")
    c.block[4, 7] = float("inf")
    good = [0, 1, 2] + list(range(5, 12))
    v, y = block_norm_fwd(c.x, c.block, **c.kw)
    ov, oy, m = c.magnitudes()
    Case.near("v", v[good], ov[good], m["v"][good])
    Case.near("y", y[good], oy[good], m["y"][good])
    assert not y[0].any() and not v[0].any()
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).any()
    dx, db, *_ = block_norm_bwd(c.x, c.block, dy=c.dy, dv=c.dv, **c.kw)
    assert torch.isfinite(dx[good].float()).all()
    assert torch.isnan(dx[3]).all()


def test_gradients_by_differences():
    """<dy, y> + <dv, v> differenced along one direction of x, block and each
    weight, everything in fp32 but the bf16 block and y: the step is large
    enough for y's rounding (2^-9 sqrt(N H) in the sum) to be small against it."""
    c = Case(64, 256, xt=f32, wt=f32, dyt=f32)

    def value(x, w1, g, w2):
        kw = dict(c.kw, post_weight=w1, gate=g, pre_weight=w2)
        v, y = block_norm_fwd(x, c.block, **kw)
        return ((y.double() * c.dy.double()).sum() + (v.double() * c.dv.double()).sum()).item()

    got = block_norm_bwd(c.x, c.block, dy=c.dy, dv=c.dv, **c.kw)
    base = [c.x, c.w1, c.g, c.w2]
    noise = 2 * BF16 * (c.dy.double().abs() * 4).norm().item()
    for i, k in ((0, 0), (1, 2), (2, 3), (3, 4)):
        d = torch.sign(got[k])                      # the direction of steepest change
        h = 2.0 ** -6
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + h * d, base[i] - h * d
        lu, l0, ld = value(*up), value(*base), value(*down)
        want = (got[k].double() * d.double()).sum().item() * h
        curve = abs(lu - 2 * l0 + ld)
        assert abs((lu - ld) / 2 - want) <= noise + 0.5 * curve, (k, lu - ld, want)
        assert abs(want) > 2 * noise


def test_repeated_calls_give_the_same_bits_and_want_selects():
    c = Case(3000, 520)
    runs = [block_norm_bwd(c.x, c.block, dy=c.dy, dv=c.dv, **c.kw) for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))
    for i in range(5):
        want = tuple(j == i for j in range(5))
        r = block_norm_bwd(c.x, c.block, dy=c.dy, dv=c.dv, want=want, **c.kw)
        assert [t is not None for t in r] == list(want)
        assert torch.equal(r[i], runs[0][i])
    v, y = block_norm_fwd(c.x, c.block, want_residual=False, **c.kw)
    assert v is None and torch.equal(y, block_norm_fwd(c.x, c.block, **c.kw)[1])


def test_autograd_matches_the_direct_call():
    c = Case(64, 512, wt=f32)
    leaves = [t.clone().requires_grad_() for t in (c.x, c.block, c.w1, c.g, c.w2)]
    kw = dict(scale=0.4, eps=1e-5)
    v, y = block_norm(*leaves[:2], post_weight=leaves[2], gate=leaves[3], pre_weight=leaves[4], **kw)
    full = dict(c.kw, dy=c.dy, dv=c.dv)
    direct = block_norm_bwd(c.x, c.block, **full)
    got = torch.autograd.grad((v, y), leaves, (c.dv, c.dy), retain_graph=True)
    for g, d, leaf in zip(got, direct, leaves):
        assert g.dtype == leaf.dtype and torch.equal(g, d.to(g.dtype))
    # y alone, v alone
    got = torch.autograd.grad(y, leaves, c.dy, retain_graph=True)
    direct = block_norm_bwd(c.x, c.block, **dict(full, dv=None))
    assert all(torch.equal(g, d.to(g.dtype)) for g, d in zip(got, direct))
    got = torch.autograd.grad(v, leaves[:4], c.dv)
    direct = block_norm_bwd(c.x, c.block, **dict(full, dy=None, pre_weight=None, pre=False))
    assert all(torch.equal(g, d.to(g.dtype)) for g, d in zip(got, direct))
    x = c.x.clone().requires_grad_()
    same, y = block_norm(x, pre_weight=c.w2)
    assert same is x
    (g,) = torch.autograd.grad(y, x, c.dy)
    assert torch.equal(g, block_norm_bwd(c.x, dy=c.dy, pre_weight=c.w2)[0])


def test_captured_and_on_another_stream():
    a, b = Case(200, 1024, seed=1), Case(200, 1024, seed=2)
    bufs = [t.clone() for t in (a.x, a.block, a.dy, a.dv)]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kw = dict(a.kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        block_norm_fwd(bufs[0], bufs[1], **kw)
        block_norm_bwd(bufs[0], bufs[1], dy=bufs[2], dv=bufs[3], workspace=ws, **kw)
    side.synchronize()
    with torch.cuda.graph(graph):
        v, y = block_norm_fwd(bufs[0], bufs[1], **kw)
        grads = block_norm_bwd(bufs[0], bufs[1], dy=bufs[2], dv=bufs[3], workspace=ws, **kw)
    for c in (b, a):
        for t, s in zip(bufs, (c.x, c.block, c.dy, c.dv)):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        ev, ey = block_norm_fwd(c.x, c.block, **kw)
        eg = block_norm_bwd(c.x, c.block, dy=c.dy, dv=c.dv, **kw)
        assert torch.equal(v, ev) and torch.equal(y, ey)
        assert all(torch.equal(p, q) for p, q in zip(grads, eg))


def test_offsets_past_31_bits():
    """More than 2^31 values: the last rows are normed as alone."""
    N, H = 270000, 8192
    x = torch.empty(N, H, dtype=bf, device="cuda")
    x[:1000].normal_(); x[-1000:].normal_()
    x[1000:-1000] = 1.0
    w = torch.rand(H, device="cuda") + 0.5
    _, y = block_norm_fwd(x, pre_weight=w)
    _, tail = block_norm_fwd(x[-1000:].contiguous(), pre_weight=w)
    assert torch.equal(y[-1000:], tail)
    dx, _, _, _, dw = block_norm_bwd(x, dy=y, pre_weight=w)
    dt = block_norm_bwd(x[-1000:].contiguous(), dy=tail, pre_weight=w)[0]
    assert torch.equal(dx[-1000:], dt)
    assert torch.isfinite(dw).all()


@pytest.mark.parametrize("loss", ["ce", "kl"])
@pytest.mark.parametrize("xt", [bf, f32])
def test_tail_norm_then_loss(loss, xt):
    """The student's tail as it is used: block output joins the residual stream,
    final norm, fused projection and loss, gradients back to all of them --
    against the same chain put together from the direct calls."""
    c = Case(300, 256, xt=xt, wt=f32, dv=False)
    W = (torch.randn(1000, 256, device="cuda") * 0.1).bfloat16()
    if loss == "ce":
        target = (torch.randint(0, 1000, (300,), device="cuda"),)
        target[0][::7] = -100
        direct, fused = fused_ce_fwd_bwd, fused_cross_entropy_loss
    else:
        ids = torch.stack([torch.randperm(1000, device="cuda")[:16] for _ in range(300)])
        target = (ids.int(), torch.randn(300, 16, device="cuda"))
        direct, fused = fused_kl_fwd_bwd, fused_chunked_kl_loss
    leaves = [t.clone().requires_grad_() for t in (c.x, c.block, c.w1, c.g, c.w2, W)]
    norm = TailNorm(pre_weight=leaves[4], block=leaves[1], post_weight=leaves[2], gate=leaves[3],
                    scale=0.4, eps=1e-5)
    value = fused(leaves[0], leaves[5], *target, norm=norm)
    got = torch.autograd.grad(value, leaves)
    _, y = block_norm_fwd(c.x, c.block, **c.kw)
    ref, _, dH, dW = direct(y, W, *target)
    assert value.item() == pytest.approx(ref.item(), rel=1e-6)
    grads = block_norm_bwd(c.x, c.block, dy=dH.bfloat16(), **c.kw)
    for g, d, leaf in zip(got, grads + (dW,), leaves):
        assert g.dtype == leaf.dtype
        # the KL loss sums its split-K partials in any order: one bf16 step of dH
        assert ((g.double() - d.double()).norm() <= 2 * BF16 * d.double().norm()).item()
    # the fp32 dH of a direct call can go straight into the norm's backward
    exact = block_norm_bwd(c.x, c.block, dy=dH.float(), **c.kw)
    for a, b in zip(exact, grads):
        assert ((a.double() - b.double()).norm() <= 2 * BF16 * b.double().norm()).item()
