"""Cross entropy rows whose label lies far below the other columns, or at minus
infinity, against the fp64 oracle; and the sizes at which calls change their way.

Far labels: logits are exact here (one nonzero hidden value a row, or sums of few terms), so a
log-sum-exp is off only by its own arithmetic: the exponent of each column
(relative 2^-24 of at most 2^5), ex2 (2^-22) and a few fp32 roundings of values up
to |LSE| + 1: 8 2^-22 (1 + |LSE|).  A row loss adds five roundings of
2^-24 of itself (log2 e and its product, the difference, ln 2 and its product): 2^-21.
"""
import numpy as np
import pytest
import torch

import oracle
import synth
from chunked_kl_loss_tcgen05_b200 import fckl_profile_begin, fckl_profile_end
from chunked_kl_loss_tcgen05_b200.torch_api import (fused_ce_bwd, fused_ce_fwd, fused_ce_fwd_bwd,
                                                    fused_cross_entropy_loss, TailNorm)

pytestmark = pytest.mark.gpu
BF16, FP16 = 2.0 ** -8, 2.0 ** -11


def device(bits):
    return torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)


@pytest.mark.parametrize("N,V", [(1, 300), (2, 300), (40, 300), (40, 5000)])
def test_label_far_below_the_others(N, V):
    """z = h_0 W_v0 exactly: other columns between -4 and 4, the labels between
    -100 and -3400."""
    rng = np.random.default_rng(N + V)
    H = 8
    h, W = np.zeros((N, H), np.float32), np.zeros((V, H), np.float32)
    h[:, 0] = 1
    W[:, 0] = rng.integers(-16, 17, V) / 4
    y = rng.permutation(V)[:N]
    h[:, 1] = rng.integers(100, 256, N) / 8       # hits only the labels' rows of W
    W[y, 1] = -rng.integers(8, 108, N).astype(np.float32)
    hb, Wb = synth.f32_to_bf16_bits(h), synth.f32_to_bf16_bits(W)
    o = oracle.cross_entropy(hb, Wb, y)
    labels = torch.from_numpy(y).cuda()
    runs = [fused_ce_fwd(device(hb), device(Wb), labels)[1:]]
    runs.append((fused_ce_fwd_bwd(device(hb), device(Wb), labels)[1], None))
    tol = 8 * 2.0 ** -22 * (1 + np.abs(o["lse"]))
    for rows, lse in runs:
        err = np.abs(rows.cpu().numpy() - o["row_loss"])
        assert (err <= tol + 2.0 ** -21 * o["row_loss"]).all(), err.max()
        if lse is not None:
            err = np.abs(lse.cpu().numpy() - o["lse"])
            assert (err <= tol).all(), (err.max(), tol.max())


@pytest.mark.parametrize("kw", [dict(), dict(label_smoothing=0.1, z_loss=1e-3)])
@pytest.mark.parametrize("N,H,V,at", [
    (1, 64, 300, 0), (2, 64, 300, 1), (50, 64, 300, 7), (1300, 64, 700, 1200),
    (1400, 64, 48000, 7)])                       # streamed, in a block, a warp a row, recomputed
def test_label_at_minus_infinity(N, H, V, at, kw):
    """h . W_y overflows to -inf for one row: its loss is infinite, its log-sum-exp
    and all gradients are what they are without that column."""
    rng = np.random.default_rng(N + V)
    h = rng.standard_normal((N, H)).astype(np.float32)
    W = (rng.standard_normal((V, H)) * 0.1).astype(np.float32)
    A = float((np.abs(h[:64]) @ np.abs(W[:4096]).T).max()) * 1.5
    y = rng.integers(0, V, N)
    h[:, 0], W[:, 0] = 0, 0
    h[at, 0], W[y[at], 0] = 2.0 ** 100, -2.0 ** 100
    hb, Wb = synth.f32_to_bf16_bits(h), synth.f32_to_bf16_bits(W)
    o = oracle.cross_entropy(hb, Wb, y, **kw)
    g = rng.standard_normal(N).astype(np.float32)
    og = oracle.cross_entropy(hb, Wb, y, row_grad=g, **kw)
    hd, Wd, labels = device(hb), device(Wb), torch.from_numpy(y).cuda()
    dz = H * 2.0 ** -23 * A
    tol = (2 * dz + 8 * 2.0 ** -22 * (1 + np.abs(o["lse"]).max())) * 1.1
    rest = np.arange(N) != at
    loss, rows, lse = fused_ce_fwd(hd, Wd, labels, **kw)
    both = fused_ce_fwd_bwd(hd, Wd, labels, **kw)
    assert np.abs(lse.cpu().numpy() - o["lse"]).max() <= tol
    for r in (rows, both[1]):
        r = r.cpu().numpy()
        assert r[at] == np.inf
        assert (np.abs(r - o["row_loss"])[rest] <= tol).all()
    assert loss.item() == np.inf and both[0].item() == np.inf
    grads = fused_ce_bwd(hd, Wd, labels, lse, torch.from_numpy(g).cuda(), **kw)
    for ref, pair in ((o, both[2:]), (og, grads)):
        for name, t in zip(("dH", "dW"), pair):
            # dlogits' rounding; and of q = G + e / V, to which a smoothed G can be
            # small (q near e / V), the 16-bit exponential's, the logits' error and
            # the fp32 exponent's (z/T - LSE) few 2^-20
            err = np.abs(t.double().cpu().numpy() - ref[name])
            bound = (1.05 * (BF16 + 2 * dz + 2.0 ** -20) * ref[name + "_abs"]
                     + 2.0 ** -22 * np.abs(ref[name]) + 1e-30
                     + 1.05 * (FP16 + 2 * dz + 2.0 ** -18) * ref[name + "_q"])
            assert (err <= bound).all(), (name, (err / bound).max())


@pytest.mark.parametrize("N,H,V,dtype,side_by_side", [
    (8, 256, 65000, torch.bfloat16, True), (8, 256, 70000, torch.bfloat16, False),
    (256, 256, 70000, torch.bfloat16, True), (257, 64, 1000, torch.bfloat16, False),
    (256, 64, 1000, torch.float32, True), (8, 256, 262144, torch.float32, True),
    (8, 256, 262145, torch.float32, False), (256, 4096, 128256, torch.bfloat16, False)])
def test_gradient_products_side_by_side(N, H, V, dtype, side_by_side):
    """Which calls run dH and dW in one launch, and that both ways give the gradients
    that the dW of one-row-tile chunks, in launches of their own, adds up to."""
    g = torch.Generator(device="cuda").manual_seed(N + V)
    h = torch.randn(N, H, generator=g, device="cuda").bfloat16()
    W = torch.empty(V, H, dtype=torch.bfloat16, device="cuda").normal_(0, 0.05, generator=g)
    y = torch.randint(0, V, (N,), generator=g, device="cuda")
    fckl_profile_begin()
    _, _, dH, dW = fused_ce_fwd_bwd(h, W, y, grad_dtype=dtype, check=False)
    kinds = {k["name"] for k in fckl_profile_end()}
    assert ("dH_dW_gemm" in kinds) == side_by_side
    assert bool(kinds & {"dH_gemm", "dW_gemm"}) != side_by_side
    _, _, rH, rW = fused_ce_fwd_bwd(h, W, y, chunk=N // 2 + 1, check=False)
    for t, r in ((dH, rH), (dW, rW)):
        # the same bf16 dlogits; fp32 sums in another order (the tensor cores cut a
        # segment's sum at most 2100 times here, 0.18 2^-23 of it each on average)
        # and, in bf16, one rounding
        own = BF16 if dtype == torch.bfloat16 else 0.0
        e = (t.float() - r).abs()
        assert (e <= own * r.abs() + 2.0 ** -10 * r.abs().max()).all()
        assert (e.double().norm() <= (own / 2 + 2.0 ** -14) * r.double().norm()).item()


@pytest.mark.parametrize("N", [49_151, 200_000])
def test_long_sums_of_one_sign(N):
    """dW of classes that no row is labelled with, for positive hidden values: sums of
    one sign over all rows.  With chunks of at most 49152 rows the tensor cores cut
    49152 / 16 partial sums, less than 2^-23 of the whole each on average; the bf16
    rounding of each row's share is random and averages out."""
    H, V = 64, 64
    g = torch.Generator(device="cuda").manual_seed(N)
    h = torch.randn(N, H, generator=g, device="cuda").abs().bfloat16()
    W = (torch.randn(V, H, generator=g, device="cuda") * 0.02).bfloat16()
    y = torch.zeros(N, dtype=torch.int64, device="cuda")
    dW = fused_ce_fwd_bwd(h, W, y)[3].double()
    q = torch.softmax(h.double() @ W.double().t(), 1)
    off = (dW / (q.t() @ h.double() / N) - 1)[1:]
    assert off.mean().abs().item() <= 49152 / 16 * 2.0 ** -23
    assert off.abs().max().item() <= 49152 / 16 * 2.0 ** -23 + 8 * BF16 / N ** 0.5


@pytest.mark.parametrize("kw", [dict(), dict(reduction="sum"), dict(chunk=64)])
def test_gradients_kept_in_float32_are_rounded_once(kw):
    """The gradients of 0.3 loss are those of the float32 call, times 0.3 in float32,
    rounded once; the same again from a retained graph; frozen operands get none."""
    N, H, V = 200, 128, 900
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(N, H, generator=g, device="cuda").bfloat16()
    W = (torch.randn(V, H, generator=g, device="cuda") * 0.1).bfloat16()
    y = torch.randint(0, V, (N,), generator=g, device="cuda")
    weight = torch.rand(N, generator=g, device="cuda")
    kw = dict(kw, row_weight=weight)
    direct = fused_ce_fwd_bwd(h, W, y, **kw)
    factor = torch.tensor(0.3, device="cuda")
    for frozen in (None, 0, 1):
        leaves = [t.clone().requires_grad_(i != frozen) for i, t in enumerate((h, W))]
        loss = fused_cross_entropy_loss(*leaves, y, grad_dtype=torch.float32, **kw)
        assert torch.equal(loss, direct[0][0])
        wanted = [i for i in (0, 1) if i != frozen]
        for scale in (factor, factor * 7):
            got = torch.autograd.grad(loss * scale, [leaves[i] for i in wanted], retain_graph=True)
            for i, t in zip(wanted, got):
                assert torch.equal(t, (direct[2 + i] * scale).bfloat16())
    rows = fused_cross_entropy_loss(leaves[0], leaves[1], y, reduction="none",
                                    grad_dtype=torch.float32)
    rows.sum().backward()
    assert leaves[0].grad.dtype == torch.bfloat16


@pytest.mark.parametrize("grad_dtype", [torch.bfloat16, torch.float32])
def test_mean_over_the_rows_of_all_shards(grad_dtype):
    """Two shards of a batch, each dividing by the kept rows of both: their losses and
    gradients are those of the direct calls, from a retained graph too, and sum to the
    whole batch's."""
    N, H, V, cut = 150, 64, 400, 61
    g = torch.Generator(device="cuda").manual_seed(2)
    h = torch.randn(N, H, generator=g, device="cuda").bfloat16()
    W = (torch.randn(V, H, generator=g, device="cuda") * 0.1).bfloat16()
    y = torch.randint(0, V, (N,), generator=g, device="cuda")
    y[::5] = -100
    total = int((y >= 0).sum())
    losses, sums = [], torch.zeros(V, H, device="cuda")
    for rows in (slice(0, cut), slice(cut, N)):
        leaves = [h[rows].clone().requires_grad_(), W.clone().requires_grad_()]
        loss = fused_cross_entropy_loss(*leaves, y[rows], n_valid_total=total,
                                        grad_dtype=grad_dtype)
        direct = fused_ce_fwd_bwd(h[rows], W, y[rows], n_valid_total=total)
        for _ in range(2):
            got = torch.autograd.grad(loss, leaves, retain_graph=True)
            for t, d in zip(got, direct[2:]):
                # bf16 of the same sums; computed again, the dlogits may fall on the
                # other side of a rounding
                e = (t.float() - d).norm() / d.norm()
                assert e.item() <= BF16
        with torch.no_grad():
            alone = fused_cross_entropy_loss(*leaves, y[rows], n_valid_total=total)
        assert alone.item() == pytest.approx(loss.item(), rel=1e-6)
        losses.append(loss.item())
        sums += direct[3]
    whole = fused_ce_fwd_bwd(h, W, y)
    assert sum(losses) == pytest.approx(whole[0].item(), rel=1e-6)
    assert ((sums - whole[3]).norm() / whole[3].norm()).item() <= 2.0 ** -12


@pytest.mark.parametrize("grad_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("reduction", ["mean", "none"])
def test_captured_step_through_the_tail(reduction, grad_dtype):
    """Loss and gradients of a student's tail captured as one graph; replays on new
    inputs give the eager step's results.  (No eager graph of the leaves lives during the
    capture: torch's engine would synchronise with the stream it was made on, which
    invalidates any capture of a backward pass.)"""
    N, H, V = 300, 128, 700
    g = torch.Generator(device="cuda").manual_seed(3)

    def inputs():
        return (torch.randn(N, H, generator=g, device="cuda").bfloat16(),
                torch.randint(0, V, (N,), generator=g, device="cuda"))

    x, y = inputs()
    x.requires_grad_()
    W = (torch.randn(V, H, generator=g, device="cuda") * 0.1).bfloat16().requires_grad_()
    w2 = torch.rand(H, generator=g, device="cuda").requires_grad_()
    leaves, up = (x, W, w2), torch.rand(N, generator=g, device="cuda")

    def step():
        loss = fused_cross_entropy_loss(x, W, y, reduction=reduction, check=False,
                                        norm=TailNorm(pre_weight=w2), grad_dtype=grad_dtype)
        return (loss, *torch.autograd.grad(loss, leaves, up if reduction == "none" else up[0]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(3):
        nx, ny = inputs()
        with torch.no_grad():
            x.copy_(nx), y.copy_(ny), up.mul_(0.7)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, step()))
