"""The widest rows of the norms in the types that fill shared memory, and calls on two
streams at once; tolerances as in test_gpu_norm."""
import pytest
import torch

from test_gpu_norm import Case, bf, f32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [1, 3, 400])
@pytest.mark.parametrize("H", [8192, 8184, 4104])
@pytest.mark.parametrize("xt,wt,dyt", [(f32, f32, f32), (f32, bf, bf), (bf, f32, f32)])
def test_widest_rows(N, H, xt, wt, dyt):
    """H = 8192 with x, dv and dy in float32: two stages of 114688 bytes."""
    Case(N, H, xt, wt, dyt).check()


@pytest.mark.parametrize("H", [256, 512, 4096, 8192])
def test_full_types_without_parts(H):
    Case(30, H, f32, f32, f32, post=False, gate=False).check()
    Case(30, H, f32, f32, f32, pre=False).check()


def test_two_streams_at_once_match_solo_calls():
    from chunked_kl_loss_tcgen05_b200.torch_api import block_norm_bwd, block_norm_fwd
    cases = [Case(900, 2880, f32, f32, f32, seed=s) for s in range(2)]

    def both(c):
        return (block_norm_fwd(c.x, c.block, **c.kw),
                block_norm_bwd(c.x, c.block, dy=c.dy, dv=c.dv, **c.kw))

    solo = [both(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for c, s, ref in zip(cases, streams, solo):
            with torch.cuda.stream(s):
                got.append((both(c), ref))
    torch.cuda.synchronize()
    for (fwd, bwd), (rf, rb) in got:
        assert all(torch.equal(a, b) for a, b in zip(fwd + bwd, rf + rb))
