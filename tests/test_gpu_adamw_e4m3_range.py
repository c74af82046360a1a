"""8-bit moments over blocks whose elements span many powers of two, and past fp32's range.

Constant gradients, one element of each block S and the others far smaller.  The block's scales are S's,
whose stored moments are exact, so that AdamW moves every element by lr (1 at most, eps lowers it).  Let a
small element be worth x codes of 2^-9.  Its first moment is at every step a mean of the stored code and x,
so the code stays at most ceil(x); the root is a root mean square of the stored code and x, so the code stays at
least max(1, floor(x)) where no positive root is stored as zero.  In units of lr, with w = b2 c2(t) / c2(t + 1) >= 1/2 the
stored code's weight:  x >= 1: ceil(x) / floor(x) <= 2;  x < 1: 1 / sqrt(w + (1 - w) x^2) <= sqrt(2).
Where the gradient of x < 1 is zero at some steps the same holds with x = 0.  Once in 65536 roundings the
largest code, a rounding below 448, falls to 416: 448 / 416 = 1.08 on top."""
import numpy as np
import pytest
import torch

from sparse_moe_layer_03_b200 import optim

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("S", [100.0, 1.0, 0.1])
@pytest.mark.parametrize("gap", [False, True])
def test_small_elements_of_a_block_move_by_the_rate(S, gap):
    lr, ratios = 1e-4, (1e-6, 3e-7, 1e-8) if gap else (1e-3, 1e-4, 1e-5, 3e-6, 1e-6, 1e-7)
    n = 256 * 32 * len(ratios)
    g = torch.cat([torch.full((256 * 32,), S * r, device=DEV) for r in ratios])
    g[1::2] *= -1.0
    small = torch.arange(n, device=DEV) % 256 != 77
    g[~small] = S
    off = torch.where(small, 0.0, g)
    p = torch.zeros(n, device=DEV)
    opt = optim.AdamW([p], lr=lr, state="e4m3", seed=5)
    worst = torch.zeros((), device=DEV)
    for t in range(300):
        had = p.clone()
        opt.step([off if gap and t % 2 else g])
        worst = torch.maximum(worst, (p - had).abs().max())
    assert float(worst) / lr <= 2.0 * 1.08 * 1.001, float(worst) / lr
    codes = opt.buffers["v"].view(torch.uint8)
    assert int(codes.min()) >= 1                          # every element has had a gradient


def test_a_root_of_zero_stays_zero():
    p = torch.zeros(300, device=DEV)
    opt = optim.AdamW([p], lr=1e-3, state="e4m3")
    g = torch.zeros(300, device=DEV)
    g[0], g[299] = 1.0, 2.0
    opt.step([g])
    codes = opt.buffers["v"].view(torch.uint8)
    assert torch.equal(torch.nonzero(codes).flatten().cpu(), torch.tensor([0, 299]))
    assert int(torch.count_nonzero(p)) == 2


def test_a_second_moment_past_fp32_takes_the_first_with_it():
    # 1e25 squared is infinite in fp32: its block's second moments start again from zero, and a first moment
    # that stayed would then be divided by the next step's gradient alone
    lr = 1e-3
    gen = torch.Generator().manual_seed(3)
    p = torch.zeros(1024, device=DEV)
    opt = optim.AdamW([p], lr=lr, state="e4m3", seed=1)
    g = (torch.rand(1024, generator=gen) + 0.5).to(DEV)
    opt.step([g])
    big = g.clone()
    big[300] = 1e25
    opt.step([big])
    assert torch.isfinite(p).all()
    assert float(opt.part("v_scale", 0)[1]) == 0.0 and float(opt.part("m_scale", 0)[1]) == 0.0
    for _ in range(4):
        had = p.clone()
        opt.step([g])
        # a first step's own ratio at step t: (1 - b1) g / c1 over sqrt(1 - b2) g / sqrt(c2), largest 0.1 / 0.2
        # over sqrt(0.001 / 0.003) = 0.9 at t = 3, rising to 3.2 as t grows; below 4 with the codes' eighths
        assert float((p - had).abs().max()) <= 4 * lr
    assert torch.isfinite(opt.buffers["m_scale"]).all() and torch.isfinite(opt.buffers["v_scale"]).all()
