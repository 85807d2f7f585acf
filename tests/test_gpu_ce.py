"""Cross entropy against labels on the GPU, against the fp64 oracle.

Tolerances, counted in roundings (eps/2: bf16 2^-8, fp16 2^-11, fp32 2^-24):
* a logit z is an fp32 sum of H exact products, each addition off by at most
  2^-23 of what it holds (the tensor cores may cut instead of round), so
  |dz| <= H 2^-23 A with A = max_v sum_j |h_j W_vj|; log, exp and merging add a
  few 2^-22 of values near |LSE| + 1.  A row loss is a difference of two such.
* G's entries are rounded once to bf16 and may carry the rounding of a 16-bit
  exponential before (2^-11); they also inherit the logits' error (relative,
  through exp).  |ddH| <= (2^-8 + 2^-11 + dz + ...) |G| |W| elementwise, plus
  fp32 sums (far smaller), plus 2^-8 |dH| when dH is bf16.  SLACK covers the
  fp32 sums.
* exp's relative error is one of q, not of G = q - 1 at the label: with one
  class, q = 1 and G = 0, and the fp32 exponent z/T - LSE (values up to ~16 in
  base 2, so each of its few roundings is up to 2^-20 in the exponent) leaves
  q - 1 up to a few 2^-20 from 0.  So (2 dz + 2^-18) of the magnitudes with q in
  G's place (dH_q, dW_q) is added.
"""
import numpy as np
import pytest
import torch

import oracle
import synth
from chunked_kl_loss_tcgen05_b200 import (FCKL_ERR_BAD_INDEX, FCKL_OK, FcklCeProblem, FcklError,
                                          fckl_ce_workspace_bytes, fckl_profile_begin,
                                          fckl_profile_end, fckl_scale_gradient)
from chunked_kl_loss_tcgen05_b200.torch_api import (fused_ce_bwd, fused_ce_fwd, fused_ce_fwd_bwd,
                                                    fused_cross_entropy_loss)

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24
SLACK = 1.05


class Case:
    def __init__(self, N, H, V, seed=0, ignored=0.15, std=0.1, labels=torch.int64, lift=0.0):
        rng = np.random.default_rng(seed + N + 7 * H + 13 * V)
        W = (rng.standard_normal((V, H)) * std).astype(np.float32)
        y = rng.integers(0, V, N)
        h = rng.standard_normal((N, H)).astype(np.float32) + lift * W[y]
        y[rng.random(N) < ignored] = -100
        self.h_bits, self.W_bits = synth.f32_to_bf16_bits(h), synth.f32_to_bf16_bits(W)
        self.y = y
        self.w = (rng.random(N) + 0.5).astype(np.float32)
        self.g = rng.standard_normal(N).astype(np.float32)
        self.N, self.H, self.V = N, H, V
        self.hidden = torch.from_numpy(self.h_bits.view(np.int16)).cuda().view(torch.bfloat16)
        self.W = torch.from_numpy(self.W_bits.view(np.int16)).cuda().view(torch.bfloat16)
        self.labels = torch.from_numpy(y).to(labels).cuda()
        self.weight = torch.from_numpy(self.w).cuda()
        self.row_grad = torch.from_numpy(self.g).cuda()
        hv, Wv = synth.bf16_bits_to_f32(self.h_bits), synth.bf16_bits_to_f32(self.W_bits)
        self.A = float((np.abs(hv[:64]) @ np.abs(Wv[:4096]).T).max()) * 1.5

    def dz(self, T):
        return self.H * 2.0 ** -23 * self.A / T

    def oracle(self, **kw):
        return oracle.cross_entropy(self.h_bits, self.W_bits, self.y, **kw)


def check_losses(c, o, loss, row_loss, lse=None, T=1.0, z_loss=0.0):
    tol = 2 * c.dz(T) + 8 * 2.0 ** -22 * (1 + np.abs(o["lse"]).max())
    tol *= 1 + 2 * z_loss * np.abs(o["lse"]).max()
    rl = row_loss.detach().cpu().numpy()
    assert np.abs(rl - o["row_loss"]).max() <= tol, (np.abs(rl - o["row_loss"]).max(), tol)
    assert (rl[c.y == -100] == 0).all()
    if lse is not None:
        assert np.abs(lse.cpu().numpy() - o["lse"]).max() <= tol
        assert (lse.cpu().numpy()[c.y == -100] == 0).all()
    if loss is not None:
        kept = max(1, int((c.y != -100).sum()))
        scale = abs(o["loss"]) / max(np.abs(o["row_loss"]).mean() * c.N / kept, 1e-30)
        assert abs(loss.item() - o["loss"]) <= 2 * tol * max(1.0, scale) + 4 * FP32 * abs(o["loss"])


def check_grads(c, o, dH, dW, T=1.0):
    rel = SLACK * (BF16 + FP16 + 2 * c.dz(T) + 2.0 ** -20)
    for got, name in ((dH, "dH"), (dW, "dW")):
        if got is None:
            continue
        own = BF16 if got.dtype == torch.bfloat16 else 4 * FP32
        err = np.abs(got.double().cpu().numpy() - o[name])
        bound = (rel * (1 + own) * o[name + "_abs"] + own * np.abs(o[name]) + 1e-38
                 + (2 * c.dz(T) + 2.0 ** -18) * o[name + "_q"])
        assert (err <= bound).all(), (name, (err / bound).max())
        # rounding errors are independent: over the matrix they average like
        # 2^-8 / sqrt(3) per rounding (dlogits, and the result when bf16)
        n = np.linalg.norm(o[name])
        if c.V > 1:
            assert np.linalg.norm(err) <= 6e-3 * n, (name, np.linalg.norm(err) / n)
    if dH is not None:
        assert (dH.cpu().float().numpy()[c.y == -100] == 0).all()


SHAPES = [
    # N, H, V, chunk
    (1, 8, 1, 0),            # one row, one class: loss 0, zero gradients
    (1, 128, 700, 0),
    (3, 8, 255, 0),
    (64, 64, 256, 0),
    (65, 72, 257, 0),        # one row and one column past a tile
    (130, 200, 513, 0),
    (257, 320, 1000, 0),     # H % 256 <= 128: half-width last tile
    (300, 520, 1003, 100),   # three chunks
    (300, 136, 4099, 37),
    (511, 384, 2048, 256),
    (1000, 264, 333, 0),
]


@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,H,V,chunk", SHAPES)
def test_train_matches_oracle(N, H, V, chunk, grad_dtype):
    c = Case(N, H, V, ignored=0.15 if N > 3 else 0.0)
    loss, row_loss, dH, dW = fused_ce_fwd_bwd(c.hidden, c.W, c.labels, chunk=chunk,
                                              grad_dtype=grad_dtype)
    o = c.oracle()
    check_losses(c, o, loss, row_loss)
    check_grads(c, o, dH, dW)
    assert dH.dtype == dW.dtype == grad_dtype


@pytest.mark.parametrize("N,H,V,chunk", SHAPES)
def test_score_and_row_backward_match_oracle(N, H, V, chunk):
    c = Case(N, H, V, seed=5, ignored=0.3 if N > 3 else 0.0, lift=2.0)
    loss, row_loss, lse = fused_ce_fwd(c.hidden, c.W, c.labels, chunk=chunk, reduction="sum")
    o = c.oracle(reduction="sum", row_grad=c.g)
    check_losses(c, o, loss, row_loss, lse)
    dH, dW = fused_ce_bwd(c.hidden, c.W, c.labels, lse, c.row_grad, chunk=chunk)
    check_grads(c, o, dH, dW)


@pytest.mark.parametrize("kw", [
    dict(label_smoothing=0.1), dict(label_smoothing=1.0), dict(z_loss=1e-3), dict(T=0.5),
    dict(T=3.0, label_smoothing=0.2, z_loss=1e-2), dict(reduction="sum")])
@pytest.mark.parametrize("chunk", [0, 128])
def test_options_match_oracle(kw, chunk):
    c = Case(333, 200, 1111, seed=2)
    loss, row_loss, dH, dW = fused_ce_fwd_bwd(c.hidden, c.W, c.labels, row_weight=c.weight,
                                              chunk=chunk, **kw)
    o = c.oracle(row_weight=c.w, **kw)
    check_losses(c, o, loss, row_loss, T=kw.get("T", 1.0), z_loss=kw.get("z_loss", 0.0))
    check_grads(c, o, dH, dW, T=kw.get("T", 1.0))
    kw.pop("reduction", None)
    _, _, lse = fused_ce_fwd(c.hidden, c.W, c.labels, chunk=chunk, **kw)
    dH, dW = fused_ce_bwd(c.hidden, c.W, c.labels, lse, c.row_grad, chunk=chunk,
                          grad_dtype=torch.bfloat16, **kw)
    check_grads(c, c.oracle(row_grad=c.g, **kw), dH, dW, T=kw.get("T", 1.0))


def test_confident_rows():
    """Rows whose label holds almost all the mass: q_y - 1 is formed in fp32."""
    c = Case(200, 256, 3000, seed=9, std=0.3, lift=1.2)
    loss, row_loss, dH, dW = fused_ce_fwd_bwd(c.hidden, c.W, c.labels)
    o = c.oracle()
    assert np.median(o["row_loss"][c.y != -100]) < 1e-2
    check_losses(c, o, loss, row_loss)
    # elementwise as everywhere, plus the logits' error on the label's q, which
    # is large against 1 - q_y but not against 1
    q_err = 2 * c.dz(1.0) + 2.0 ** -22
    kept = (c.y != -100).sum()
    for got, name in ((dH, "dH"), (dW, "dW")):
        big = np.abs(synth.bf16_bits_to_f32(c.W_bits if name == "dH" else c.h_bits)).max()
        err = np.abs(got.cpu().numpy() - o[name])
        rows = 1 if name == "dH" else kept
        bound = (SLACK * (BF16 + FP16 + 2 * c.dz(1.0)) * o[name + "_abs"]
                 + (2 * q_err + 2.0 ** -24) * big * rows / kept)
        assert (err <= bound).all(), (name, (err / bound).max())


@pytest.mark.parametrize("labels", [torch.int32, torch.int64])
@pytest.mark.parametrize("n_kept", [0, 1, 63, 64, 65, 299, 300])
def test_kept_counts(n_kept, labels):
    """From no kept row to all of them, with chunks that end up empty or partly
    filled; left-out rows hold NaN and inf, which must not show anywhere."""
    c = Case(300, 128, 600, seed=n_kept, ignored=0.0, labels=labels)
    drop = np.random.default_rng(n_kept).permutation(300)[n_kept:]
    c.y[drop] = -100
    c.labels[torch.from_numpy(drop).cuda()] = -100
    hidden, weight, row_grad = c.hidden.clone(), c.weight.clone(), c.row_grad.clone()
    d = torch.from_numpy(drop).cuda()
    hidden[d] = float("nan")
    hidden[d[::2]] = float("inf")
    weight[d] = float("nan")
    row_grad[d] = float("nan")
    o, og = c.oracle(row_weight=c.w), c.oracle(row_grad=c.g)
    for chunk in (0, 100):
        for gd in (torch.float32, torch.bfloat16):
            prob = FcklCeProblem(300, 128, 600, chunk=chunk, grad_type=int(gd == torch.bfloat16))
            ws = torch.full((fckl_ce_workspace_bytes(prob, True),), 255, dtype=torch.uint8,
                            device="cuda")       # NaN wherever nothing was written
            loss, row_loss, dH, dW = fused_ce_fwd_bwd(hidden, c.W, c.labels, row_weight=weight,
                                                      chunk=chunk, grad_dtype=gd, workspace=ws)
            check_losses(c, o, loss, row_loss)
            check_grads(c, o, dH, dW)
            ws.fill_(255)
            _, _, lse = fused_ce_fwd(hidden, c.W, c.labels, chunk=chunk, workspace=ws)
            lse[d] = float("nan")
            dH, dW = fused_ce_bwd(hidden, c.W, c.labels, lse, row_grad, chunk=chunk, workspace=ws,
                                  grad_dtype=gd)
            check_grads(c, og, dH, dW)
    if n_kept == 0:
        assert loss.item() == 0 and not dW.any() and not dH.any()


def test_many_rows_select_over_several_blocks():
    """More rows than one block selects: 30000 rows, 40% left out."""
    c = Case(30000, 64, 500, ignored=0.4)
    loss, row_loss, dH, dW = fused_ce_fwd_bwd(c.hidden, c.W, c.labels, chunk=7000)
    o = c.oracle()
    check_losses(c, o, loss, row_loss)
    check_grads(c, o, dH, dW)


@pytest.mark.parametrize("bad", [-1, 600, 2 ** 31, -(2 ** 40)])
def test_bad_labels_are_reported_and_left_out(bad):
    c = Case(100, 64, 600, ignored=0.1)
    c.labels[17] = bad
    with pytest.raises(FcklError) as e:
        fused_ce_fwd_bwd(c.hidden, c.W, c.labels)
    assert e.value.status == FCKL_ERR_BAD_INDEX
    loss, row_loss, dH, dW = fused_ce_fwd_bwd(c.hidden, c.W, c.labels, check=False)
    c.y[17] = -100
    o = c.oracle()
    check_losses(c, o, loss, row_loss)
    check_grads(c, o, dH, dW)


@pytest.mark.parametrize("N", [1, 300, 1024, 1025])
def test_row_count_of_an_earlier_call_is_never_used(N):
    """Calls with different counts in turn on one workspace, whose control block
    then holds the other call's count (or, poisoned, nothing sensible) while the
    next call's kernels start early."""
    a, b = Case(N, 64, 700, ignored=0.0), Case(N, 64, 700, seed=1, ignored=0.5)
    prob = FcklCeProblem(N, 64, 700)
    ws = torch.full((fckl_ce_workspace_bytes(prob, True),), 127, dtype=torch.uint8, device="cuda")
    refs = [(c, c.oracle(row_grad=c.g), c.oracle()) for c in (a, b)]
    for turn in range(6):
        c, og, o = refs[turn % 2]
        _, rows, lse = fused_ce_fwd(c.hidden, c.W, c.labels, workspace=ws)
        check_losses(c, o, None, rows, lse)
        if turn >= 4:
            ws.fill_(127)
        check_grads(c, og, *fused_ce_bwd(c.hidden, c.W, c.labels, lse, c.row_grad, workspace=ws))
        loss, rows, dH, dW = fused_ce_fwd_bwd(c.hidden, c.W, c.labels, workspace=ws)
        check_losses(c, o, loss, rows)
        check_grads(c, o, dH, dW)


def test_ignore_index_inside_the_vocabulary():
    c = Case(200, 64, 300, ignored=0.0)
    c.labels[::3] = 7
    loss, row_loss, dH, dW = fused_ce_fwd_bwd(c.hidden, c.W, c.labels, ignore_index=7)
    c.y[::3] = 7
    c.y[c.y == 7] = -100
    o = c.oracle()
    check_losses(c, o, loss, row_loss)
    check_grads(c, o, dH, dW)


def test_global_row_count_and_output_buffers():
    c = Case(150, 64, 400)
    out = (torch.empty(1, device="cuda"), torch.empty(150, 64, device="cuda"),
           torch.empty(400, 64, device="cuda"))
    loss, _, dH, dW = fused_ce_fwd_bwd(c.hidden, c.W, c.labels, n_valid_total=1000, out=out)
    assert dH.data_ptr() == out[1].data_ptr()
    o = c.oracle(row_weight=np.full(150, (c.y != -100).sum() / 1000.0))
    assert abs(loss.item() - o["loss"]) <= 1e-5 * o["loss"]
    check_grads(c, o, dH, dW)


def test_repeated_calls_give_the_same_bits():
    c = Case(700, 520, 3001)
    for chunk in (0, 256):
        runs = [fused_ce_fwd_bwd(c.hidden, c.W, c.labels, chunk=chunk) for _ in range(3)]
        for r in runs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_autograd_mean_scaled_and_twice():
    c = Case(200, 128, 900)
    o = c.oracle(row_weight=c.w)
    h, W = c.hidden.clone().requires_grad_(), c.W.clone().requires_grad_()
    loss = fused_cross_entropy_loss(h, W, c.labels, row_weight=c.weight)
    for scale in (1.0, 4.0):     # the second pass computes the gradients again
        gh, gW = torch.autograd.grad(loss * scale, (h, W), retain_graph=True)
        assert gh.dtype == gW.dtype == torch.bfloat16
        check_grads(c, o, gh / scale, gW / scale)
    loss = fused_cross_entropy_loss(h, W, c.labels, row_weight=c.weight)
    (loss * 4.0).backward()      # a power of two: exact
    check_grads(c, o, h.grad / 4.0, W.grad / 4.0)


def test_autograd_row_losses_and_frozen_operands():
    c = Case(200, 128, 900)
    o = c.oracle(row_grad=c.g)
    h, W = c.hidden.clone().requires_grad_(), c.W.clone().requires_grad_()
    rows = fused_cross_entropy_loss(h, W, c.labels, reduction="none")
    check_losses(c, o, None, rows)
    gh, gW = torch.autograd.grad(rows, (h, W), c.row_grad)
    check_grads(c, o, gh, gW)
    om = c.oracle()
    for frozen_W in (True, False):
        h, W = c.hidden.clone(), c.W.clone()
        leaf = (h if frozen_W else W).requires_grad_()
        for red, ref, up in (("mean", om, None), ("none", o, c.row_grad)):
            for chunk in (0, 64):
                out = fused_cross_entropy_loss(h, W, c.labels, reduction=red, chunk=chunk)
                (g,) = torch.autograd.grad(out, leaf, up)
                check_grads(c, ref, g if frozen_W else None, None if frozen_W else g)
    empty = torch.full_like(c.labels, -100)
    h, W = c.hidden.clone(), c.W.clone().requires_grad_()
    (g,) = torch.autograd.grad(fused_cross_entropy_loss(h, W, empty), W)
    assert not g.any()


def test_upstream_factor_not_a_power_of_two():
    c = Case(90, 64, 333)
    o = c.oracle()
    h, W = c.hidden.clone().requires_grad_(), c.W.clone().requires_grad_()
    gh, gW = torch.autograd.grad(fused_cross_entropy_loss(h, W, c.labels) * 0.3, (h, W))
    # one more bf16 rounding of the result
    for got, name in ((gh, "dH"), (gW, "dW")):
        err = np.abs(got.double().cpu().numpy() - 0.3 * o[name])
        rel = SLACK * (BF16 + FP16 + 2 * c.dz(1.0) + 2.0 ** -20)
        assert (err <= 0.3 * (rel * (1 + BF16) ** 2 * o[name + "_abs"]
                              + (2 * c.dz(1.0) + 2.0 ** -18) * o[name + "_q"]
                              + 2.1 * BF16 * np.abs(o[name])) + 1e-38).all()


def test_captured_call_replays_with_new_inputs():
    a, b = Case(300, 128, 700, seed=1), Case(300, 128, 700, seed=2)
    h, W, y = a.hidden.clone(), a.W.clone(), a.labels.clone()
    prob = FcklCeProblem(300, 128, 700, chunk=128)
    ws = torch.empty(fckl_ce_workspace_bytes(prob, True), dtype=torch.uint8, device="cuda")
    out = (torch.empty(1, device="cuda"), torch.empty(300, 128, device="cuda"),
           torch.empty(700, 128, device="cuda"))

    def step():
        return fused_ce_fwd_bwd(h, W, y, chunk=128, workspace=ws, out=out, check=False)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, rows, _, _ = step()
    for c in (a, b, a):
        h.copy_(c.hidden); W.copy_(c.W); y.copy_(c.labels)
        graph.replay()
        torch.cuda.synchronize()
        o = c.oracle()
        check_losses(c, o, out[0], rows)
        check_grads(c, o, out[1], out[2])


def test_two_streams_at_once_match_solo_calls():
    cases = [Case(400, 256, 2000, seed=s) for s in range(2)]
    solo = [fused_ce_fwd_bwd(c.hidden, c.W, c.labels) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[] for _ in cases]
    for _ in range(5):
        for i, (c, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                got[i].append(fused_ce_fwd_bwd(c.hidden, c.W, c.labels, check=False))
    torch.cuda.synchronize()
    for g, ref in zip(got, solo):
        for r in g:
            assert all(torch.equal(x, y) for x, y in zip(r, ref))


def test_gradients_by_differences():
    """The loss itself, differenced along a direction, against dH . direction.
    Steps of 2^-4 on entries of size ~1 keep the perturbed bf16 rows exact for
    most entries; the difference quotient's own error (second order, fp32 loss)
    is bounded by the spread of one-sided quotients."""
    c = Case(64, 128, 500, seed=4)
    _, _, dH, _ = fused_ce_fwd_bwd(c.hidden, c.W, c.labels, reduction="sum")
    d = torch.randn(64, 128, device="cuda")
    up, down = (c.hidden.float() + s * d * 2.0 ** -4 for s in (1, -1))
    up, down = up.bfloat16(), down.bfloat16()
    lu, l0, ld = (fused_ce_fwd(h, c.W, c.labels, reduction="sum")[0].item()
                  for h in (up, c.hidden, down))
    step = (up.double() - down.double()) / 2
    want = (dH.double() * step).sum().item()
    # central difference: third-order remainder, well below the second-order spread
    spread = abs((lu - l0) - (l0 - ld)) / 2
    shift = (up.double() + down.double() - 2 * c.hidden.double()) / 2   # rounding asymmetry
    assert abs((lu - ld) / 2 - want) <= 0.2 * spread + BF16 * abs(want) + \
        (dH.double().abs() * shift.abs()).sum().item() + 1e-3


def test_offsets_past_31_bits():
    """W of more than 2^31 elements: rows at its end are scored and their
    gradients land there."""
    N, H, V = 40, 16384, 140000
    g = torch.Generator(device="cuda").manual_seed(3)
    W = (torch.randn(V, H, generator=g, device="cuda", dtype=torch.bfloat16) * 0.01)
    h = torch.randn(N, H, generator=g, device="cuda").bfloat16()
    y = torch.randint(V - 2000, V, (N,), generator=g, device="cuda")
    loss, row_loss, dH, dW = fused_ce_fwd_bwd(h, W, y, grad_dtype=torch.bfloat16)
    z = torch.cat([h.double() @ W[i:i + 20000].double().t() for i in range(0, V, 20000)], 1)
    lse = torch.logsumexp(z, 1)
    want = lse - z[torch.arange(N, device="cuda"), y]
    A = (h[:4].float().abs() @ W[:4096].float().abs().t()).max().item() * 1.5
    assert (row_loss.double() - want).abs().max().item() <= 2 * H * 2.0 ** -23 * A + 1e-4
    G = torch.exp(z - lse[:, None])
    G[torch.arange(N, device="cuda"), y] -= 1
    G /= N
    for v0 in (0, V - 2000):
        ref = G[:, v0:v0 + 2000].t() @ h.double()
        err = (dW[v0:v0 + 2000].double() - ref).norm() / ref.norm()
        assert err.item() <= 6e-3, (v0, err.item())
    ref = sum(G[:, i:i + 20000] @ W[i:i + 20000].double() for i in range(0, V, 20000))
    assert ((dH.double() - ref).norm() / ref.norm()).item() <= 6e-3


@pytest.mark.parametrize("chunk", [1, 2, 5, 64, 1000])
def test_chunks_of_any_size(chunk):
    c = Case(70, 72, 300, ignored=0.3)
    o, og = c.oracle(), c.oracle(row_grad=c.g)
    for gd in (torch.float32, torch.bfloat16):
        loss, rows, dH, dW = fused_ce_fwd_bwd(c.hidden, c.W, c.labels, chunk=chunk, grad_dtype=gd)
        check_losses(c, o, loss, rows)
        check_grads(c, o, dH, dW)
        _, _, lse = fused_ce_fwd(c.hidden, c.W, c.labels, chunk=chunk)
        check_grads(c, og, *fused_ce_bwd(c.hidden, c.W, c.labels, lse, c.row_grad, chunk=chunk,
                                         grad_dtype=gd))


@pytest.mark.parametrize("V", [1, 2, 7, 9, 64, 127, 128, 129])
def test_small_vocabularies(V):
    c = Case(40, 40, V, ignored=0.2)
    o = c.oracle(label_smoothing=0.3)
    loss, rows, dH, dW = fused_ce_fwd_bwd(c.hidden, c.W, c.labels, label_smoothing=0.3)
    check_losses(c, o, loss, rows)
    check_grads(c, o, dH, dW)


def test_very_many_rows():
    """Rows selected over many blocks, more row tiles than SMs."""
    c = Case(300_000, 16, 60, ignored=0.5)
    o = c.oracle(row_weight=c.w, reduction="sum")
    loss, rows, dH, dW = fused_ce_fwd_bwd(c.hidden, c.W, c.labels, row_weight=c.weight,
                                          reduction="sum")
    check_losses(c, o, loss, rows)
    # 150000 rows add up in dW in fp32: at most 2^-24 of the magnitudes per 16-row step
    c.dz = lambda T, d=c.dz(1.0): d + 150_000 / 16 * 2.0 ** -24
    check_grads(c, o, dH, dW)


def test_without_gradients_only_the_forward_runs():
    c = Case(100, 64, 500)
    h, W = c.hidden.clone().requires_grad_(), c.W.clone().requires_grad_()
    fckl_profile_begin()
    with torch.no_grad():
        loss = fused_cross_entropy_loss(h, W, c.labels)
    kinds = {k["name"] for k in fckl_profile_end()}
    assert not loss.requires_grad and "merge_loss" in kinds
    assert not kinds & {"ce_scale", "dH_gemm", "dW_gemm", "dH_dW_gemm"}
    check_losses(c, c.oracle(), loss, fused_ce_fwd(c.hidden, c.W, c.labels)[1])


def test_negative_and_zero_weights():
    c = Case(120, 64, 400)
    c.w[:] = np.random.default_rng(0).standard_normal(120).astype(np.float32)
    c.w[::5] = 0
    weight = torch.from_numpy(c.w).cuda()
    o = c.oracle(row_weight=c.w, reduction="sum", z_loss=1e-2)
    loss, rows, dH, dW = fused_ce_fwd_bwd(c.hidden, c.W, c.labels, row_weight=weight,
                                          reduction="sum", z_loss=1e-2)
    check_grads(c, o, dH, dW)
    assert abs(loss.item() - o["loss"]) <= 1e-4 * np.abs(c.w * o["row_loss"]).sum()


@pytest.mark.parametrize("n", [1, 3, 4, 13, 1027])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("factor", [1.0, 0.3])
def test_scale_gradient_any_length(n, dtype, factor):
    t = torch.randn(n + 8, device="cuda").to(dtype)
    before, f = t.clone(), torch.tensor([factor], device="cuda")
    st = fckl_scale_gradient(t.data_ptr(), n, int(dtype == torch.bfloat16), f.data_ptr(),
                             torch.cuda.current_stream().cuda_stream)
    assert st == FCKL_OK
    assert torch.equal(t[:n], (before[:n].float() * f).to(dtype))
    assert torch.equal(t[n:], before[n:])


def test_labels_decide_over_infinities():
    """An overflowed logit of a kept row shows in that row's loss, not elsewhere."""
    c = Case(50, 64, 300, ignored=0.0)
    hidden = c.hidden.clone()
    hidden[7, 3] = float("inf")
    loss, rows, lse = fused_ce_fwd(hidden, c.W, c.labels)
    o = c.oracle()
    keep = np.arange(50) != 7
    tol = 2 * c.dz(1.0) + 8 * 2.0 ** -22 * (1 + np.abs(o["lse"]).max())
    assert np.abs(rows.cpu().numpy() - o["row_loss"])[keep].max() <= tol
    assert not torch.isfinite(rows[7]) and not torch.isfinite(loss).any()


def test_host_threads_on_their_own_streams():
    import threading
    cases = [Case(256 + 10 * i, 128, 900, seed=i) for i in range(4)]
    solo = [fused_ce_fwd_bwd(c.hidden, c.W, c.labels) for c in cases]
    got, torch_err = [None] * 4, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    r = fused_ce_fwd_bwd(cases[i].hidden, cases[i].W, cases[i].labels)
                torch.cuda.current_stream().synchronize()
                got[i] = r
        except Exception as e:  # noqa: BLE001
            torch_err.append(e)

    torch.cuda.synchronize()
    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not torch_err
    for g, ref in zip(got, solo):
        assert all(torch.equal(a, b) for a, b in zip(g, ref))


@pytest.mark.parametrize("N,H,V,kw", [
    (1400, 64, 48000, {}),                                  # logits computed twice
    (1400, 64, 48000, dict(label_smoothing=0.1, z_loss=1e-3)),
    (2900, 40, 48001, dict(chunk=1450)),                    # the same in chunks
    (1000, 40, 70000, {}),                                  # and selected in one launch
    (1300, 72, 700, {}), (1300, 72, 8192, {}),              # a warp a row of dlogits
    (1184, 72, 700, {}), (1300, 72, 8200, {})])             # just past those
def test_both_sides_of_every_rule(N, H, V, kw):
    c = Case(N, H, V, ignored=0.2, std=0.2)
    w = {k: v for k, v in kw.items() if k != "chunk"}
    o = c.oracle(row_weight=c.w, **w)
    loss, rows, dH, dW = fused_ce_fwd_bwd(c.hidden, c.W, c.labels, row_weight=c.weight, **kw)
    check_losses(c, o, loss, rows, z_loss=w.get("z_loss", 0.0))
    check_grads(c, o, dH, dW)
    again = fused_ce_fwd_bwd(c.hidden, c.W, c.labels, row_weight=c.weight, **kw)
    assert torch.equal(dH, again[2]) and torch.equal(dW, again[3])


@pytest.mark.parametrize("kw", [dict(), dict(T=0.7, label_smoothing=0.2, z_loss=1e-3)])
@pytest.mark.parametrize("N,H,V,chunk", [
    (1, 8, 1, 0), (1, 8, 31, 0), (2, 40, 33, 0),
    (1, 256, 1003, 0), (1, 264, 64, 0), (2, 1024, 777, 0), (2, 1032, 97, 0),
    (1, 4104, 2050, 0), (2, 4104, 2050, 0),
    (5, 136, 300, 1), (5, 136, 300, 2),
])
def test_few_rows_are_streamed(N, H, V, chunk, kw):
    c = Case(N, H, V, seed=11, ignored=0.0, lift=1.0)
    loss, row_loss, lse = fused_ce_fwd(c.hidden, c.W, c.labels, chunk=chunk, **kw)
    check_losses(c, c.oracle(**kw), loss, row_loss, lse, T=kw.get("T", 1.0),
                 z_loss=kw.get("z_loss", 0.0))


@pytest.mark.parametrize("left_out", [(0,), (1,), (0, 1)])
def test_few_rows_with_some_left_out(left_out):
    c = Case(2, 72, 130, seed=3, ignored=0.0)
    hidden = c.hidden.clone()
    for r in left_out:
        c.y[r] = -100
        hidden[r] = float("nan")
    labels = torch.from_numpy(c.y).cuda()
    loss, row_loss, lse = fused_ce_fwd(hidden, c.W, labels)
    check_losses(c, c.oracle(), loss, row_loss, lse)


def test_few_rows_with_infinities():
    # an infinite logit apart from the label's: the row's loss is no number, or
    # infinite; minus infinity: the column has no share
    c = Case(2, 64, 100, seed=4, ignored=0.0)
    W = c.W.clone()
    hidden = c.hidden.clone()
    hidden[:, 0] = torch.tensor([-1.0, 1.0])
    W[:, 0] = 0
    at = next(v for v in range(c.V) if v not in c.y)
    W[at, 0] = float("inf")
    _, row_loss, _ = fused_ce_fwd(hidden, W, c.labels)
    z = hidden[0].double() @ torch.where(W.isinf(), 0, W).double().T
    z[at] = -float("inf")
    want = (torch.logsumexp(z, 0) - z[c.y[0]]).item()
    assert abs(row_loss[0].item() - want) <= 2 * c.dz(1.0) + 8 * 2.0 ** -22 * (1 + abs(want))
    assert not np.isfinite(row_loss[1].item())
