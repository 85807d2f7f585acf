"""How near the cross entropy comes, at the widths that it is made for: row losses,
log-sum-exps and dH against 64 bits on the same bf16 inputs.

The tensor cores cut every partial sum of a logit instead of rounding it, H / 16
times; UNIT(H) = (H / 16) 2^-23 is one last bit of the sum for each.  A sum that is
random noise around its value loses 0.13 to 0.18 UNIT of it, one of a single sign up
to 0.7, a short or exact one nothing; every logit is scaled up by 0.14 UNIT.  So a
logit is left off by -0.6 to +0.15 UNIT of itself, and within 0.05 where the scale fits.
The label's logit and the streamed rows are fp32 sums, rounded.
"""
import pytest
import torch

from chunked_kl_loss_tcgen05_b200.torch_api import fused_ce_fwd, fused_ce_fwd_bwd

pytestmark = pytest.mark.gpu
BF16 = 2.0 ** -8


def unit(H):
    return H / 16 * 2.0 ** -23


def arithmetic(lse):
    """exp, log, merging: a few 2^-22 of values up to |LSE| + 1."""
    return 4 * 2.0 ** -22 * (1 + lse.abs())


def rng(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


def logits(h, W):
    return h.double() @ W.double().t()


@pytest.mark.parametrize("H", [4096, 16384])
@pytest.mark.parametrize("kind,low,high", [
    ("noise", -0.05, 0.05), ("one sign", -0.6, 0.0), ("one hot", 0.13, 0.15)])
def test_log_sum_exp_of_one_large_logit(kind, low, high, H):
    """A column that is not the label's carries the row: its logit, 30, is the
    log-sum-exp up to the others near 0."""
    R, N, V, top = rng(H), 64, 512, 30.0
    h, W = R(N, H), R(V, H) * 1e-4
    if kind == "noise":
        W[:N] = R(N, H) * 0.02
        h += W[:N] * (top / W[:N].square().sum(1, keepdim=True))
    elif kind == "one sign":
        W[:N] = h * (top / h.square().sum(1, keepdim=True))
    else:
        h.zero_(), W.zero_()
        h[:, 3], W[:N, 3] = top, 1.0
    h, W = h.bfloat16(), W.bfloat16()
    a = logits(h, W)
    ref = torch.logsumexp(a, 1)
    _, _, lse = fused_ce_fwd(h, W, torch.full((N,), V - 1, device="cuda"))
    e = lse.double() - ref
    share = e / (a.amax(1) * unit(H))
    slack = arithmetic(ref) / (a.amax(1) * unit(H))
    assert (share >= low - slack).all() and (share <= high + slack).all(), (share.min(), share.max())
    assert low - 0.01 <= share.mean().item() <= high + 0.01


@pytest.mark.parametrize("N", [1, 2, 64, 300])
@pytest.mark.parametrize("smooth", [0.0, 0.1])
def test_row_losses_of_spread_logits(N, smooth):
    """Logits of spread 1 and labels among them: every column counts.  Streamed rows
    (N <= 2) sum 64 products a lane and 6 levels; rounding errors are random, sqrt(70)
    2^-25 of partial sums up to 4, ten times that is 1e-5; the tiles' logits are off by
    0.05 UNIT of values up to 4, 6e-6, and average in the log-sum-exp."""
    R, H, V = rng(N), 4096, 2050
    h, W = R(N, H).bfloat16(), (R(V, H) / 64).bfloat16()
    y = torch.arange(N, device="cuda") * 7 % V
    a = logits(h, W)
    ref = torch.logsumexp(a, 1)
    want = ref - (1 - smooth) * a.gather(1, y[:, None])[:, 0] - smooth * a.mean(1)
    loss, rows, lse = fused_ce_fwd(h, W, y, label_smoothing=smooth)
    assert (lse.double() - ref).abs().max().item() <= 1e-5
    assert (rows.double() - want).abs().max().item() <= 1e-5
    assert abs(loss.item() - want.mean().item()) <= 1e-5
    rows = fused_ce_fwd_bwd(h, W, y, label_smoothing=smooth)[1]
    assert (rows.double() - want).abs().max().item() <= 1e-5


@pytest.mark.parametrize("N", [1, 2, 64])
def test_small_losses_keep_their_relative_accuracy(N):
    """The label's logit stands out by 20: its row loss is about 1e-5, and the error
    of R = sum exp(a_v - a_y) is that of the exponents -- the label's own (fp32: 16
    vectors of 8 a thread in two chains, then 8 levels, 72 roundings of 2^-24 of the
    sum of magnitudes, 20), the others' (UNIT of values near 1.3) and 2^-18 of
    arithmetic.  As a tensor-core sum of one sign the label's would be off by 0.3 UNIT
    of 20 and more, 1.8e-4."""
    R, H, V = rng(N), 4096, 2050
    h = R(N, H).bfloat16()
    W = R(V, H) * 0.02
    W[:N] = h.float() * (20 / h.float().square().sum(1, keepdim=True))
    W = W.bfloat16()
    y = torch.arange(N, device="cuda")
    a = logits(h, W)
    others = a.scatter(1, y[:, None], -float("inf"))
    want = torch.log1p(torch.exp(torch.logsumexp(others, 1) - a.gather(1, y[:, None])[:, 0]))
    assert want.max().item() < 1e-4     # 2050 e^(-20 + 1.28^2 / 2) = 1e-5, give or take
    bound = 72 / 4 * 2.0 ** -24 * 20 + 1.3 * unit(H) + 2.0 ** -18   # (a quarter: random)
    for rows in (fused_ce_fwd(h, W, y)[1], fused_ce_fwd_bwd(h, W, y)[1]):
        assert ((rows.double() - want) / want).abs().max().item() <= bound


@pytest.mark.parametrize("grad_chunk", [0, 32])
def test_the_label_s_entry_reaches_dH_in_full(grad_chunk):
    """dH = q_y - 1 times the label's row of W, mostly: bf16 would round that entry by
    up to 2^-9.  The other columns' entries are small and their roundings average, so
    what is left is far less than the label's would be."""
    R, N, H, V = rng(5), 64, 1024, 2000
    W = (R(V, H) * 0.05).bfloat16()
    y = torch.arange(N, device="cuda")
    lift = torch.linspace(3, 7, N, device="cuda")[:, None]
    h = (R(N, H) * 0.2 + W[:N].float() * lift / W[:N].float().square().sum(1, keepdim=True)).bfloat16()
    q = torch.softmax(logits(h, W), 1)
    G = q.clone()
    G[torch.arange(N), y] -= 1
    dH = fused_ce_fwd_bwd(h, W, y, reduction="sum", chunk=grad_chunk)[2].double()
    err = (dH - G @ W.double()).norm(dim=1)
    wn = W.double().norm(dim=1)
    q.scatter_(1, y[:, None], 0.0)
    # each other entry: its bf16 rounding and the 16-bit exponential's, independent;
    # and the logits' error, UNIT of a few, common to the row
    left = (BF16 + 2.0 ** -11) * (q.square() @ wn.square()).sqrt() + 8 * unit(H) * G.norm(dim=1) * wn.max()
    label = 2.0 ** -9 / 3 ** 0.5 * G[torch.arange(N), y].abs() * wn[y]
    assert (err <= left).all(), (err / left).max()
    assert err.square().sum() <= label.square().sum() / 16
