"""Workspace of the cross entropy calls: what a size can need, and no more.  No GPU."""
import pytest

from chunked_kl_loss_tcgen05_b200 import (FCKL_GRAD_BFLOAT, FCKL_GRAD_FLOAT, FcklCeProblem,
                                          fckl_ce_workspace_bytes)
from chunked_kl_loss_tcgen05_b200.build import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()


def _sizes(N, H, V, **kw):
    p = FcklCeProblem(N, H, V, **kw)
    return fckl_ce_workspace_bytes(p, False), fckl_ce_workspace_bytes(p, True)


@pytest.mark.parametrize("N,H,V", [(1, 8, 1), (1, 64, 64), (16, 512, 1000), (256, 256, 4096),
                                   (100, 1000, 257), (2000, 512, 3000), (4000, 4096, 300)])
def test_slabs_follow_the_vocabulary(N, H, V):
    """The dH product's segments: at most one per 64 columns of the vocabulary, 128
    in all, 256 x H fp32 values each per 256 rows."""
    score, train = _sizes(N, H, V)
    rows = -(-N // 256) * 256
    segments = min(-(-V // 64), 128)
    dlogits = N * -(-V // 64) * 64 * 2
    assert train - score <= segments * rows * H * 4 + dlogits + 512


def test_small_steps_take_little():
    assert _sizes(16, 512, 1000)[1] < 9 << 20
    assert _sizes(256, 256, 4096)[1] < 20 << 20
    for gt in (FCKL_GRAD_FLOAT, FCKL_GRAD_BFLOAT):
        assert _sizes(64, 64, 256, grad_type=gt)[1] < 1 << 20


@pytest.mark.parametrize("N,V,chunk", [
    # 1 GiB of rows at this vocabulary is fewer than 4096
    (1, 201088, 1), (4096, 201088, 4096), (6143, 201088, 6143), (6145, 201088, 3200),
    (10239, 201088, 5120), (10240, 201088, 3456), (16384, 201088, 4096),
    (6143, 10 ** 6, 6143), (6145, 10 ** 6, 3200),
    # and this many at these
    (8000, 64000, 8000), (100_000, 32000, 16768), (40_000, 16384, 40_000),
    # small vocabularies stop at 32768 rows (times 3/4 to 3/2)
    (49_151, 1000, 49_151), (49_153, 1000, 24_704), (262_144, 1000, 32768),
    (1_000_000, 60, 32384)])
@pytest.mark.parametrize("gt", [FCKL_GRAD_FLOAT, FCKL_GRAD_BFLOAT])
def test_automatic_chunk(N, V, chunk, gt):
    """The workspace of an automatic chunk is that of the rows the rule gives."""
    assert _sizes(N, 64, V, grad_type=gt) == _sizes(N, 64, V, grad_type=gt, chunk=chunk)
    if chunk < N:
        assert _sizes(N, 64, V, grad_type=gt) != _sizes(N, 64, V, grad_type=gt, chunk=chunk + 128)
