"""AdamW with eps = 0 over gradients whose squares fall out of fp32's range."""
import pytest
import torch

from sparse_moe_layer_03_b200 import optim

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_gradients_of_any_size_move_by_the_rate(state):
    # constant gradient g: m / c1 = g.  Where 0.001 g^2 is a normal number the ratio to sqrt(v / c2) is 1.  It is
    # rounded to zero below 8.4e-22, where g is at most the least denominator, 2^-70 = 8.5e-22; between, v's
    # unit is 2^-149 and 0.001 g^2 at least half of one, rounded up to it at most: root within sqrt(1/2) and
    # sqrt(2), and in 8 bits one code of the block's largest, itself.
    lr = 1e-3
    sizes = [1e-37, 1e-30, 1e-25, 1e-23, 4e-22, 8.3e-22, 9e-22, 1.3e-21, 3e-21, 1e-20, 1e-15, 1.0]
    g = torch.cat([torch.full((256,), s, device=DEV) for s in sizes])
    g[::2] *= -1.0
    p = torch.zeros_like(g)
    opt = optim.AdamW([p], lr=lr, eps=0.0, state=state, seed=2)
    worst = torch.zeros(len(sizes), device=DEV)
    for _ in range(40):
        had = p.clone()
        opt.step([g])
        worst = torch.maximum(worst, (p - had).abs().view(len(sizes), 256).max(1).values)
    assert float(worst.max()) <= 1.5 * lr, (worst / lr).tolist()
    assert 0.99 * lr <= float(worst[-1]) <= 1.01 * lr


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_no_gradient_leaves_a_parameter_as_it_is(state):
    p = torch.ones(300, device=DEV)
    opt = optim.AdamW([p], lr=1e-2, eps=0.0, state=state)
    for _ in range(3):
        opt.step([torch.zeros(300, device=DEV)])
    assert torch.equal(p, torch.ones_like(p))
