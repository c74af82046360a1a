"""An optimizer's state taken and restored while other streams step it, and tensors that the vectors do not fit."""
import pytest
import torch

from sparse_moe_layer_03_b200 import inputs as I
from sparse_moe_layer_03_b200 import optim

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LATE = 20_000_000          # clock cycles, some 10 ms


def _layer_optimizer():
    from sparse_moe_layer_03_b200.layer import LayerShape, MoELayer
    w = I.small_workload(64, 64, 128, 4, 2, 1, "bf16", "topk", seed=3)
    layer = MoELayer(LayerShape(w.T, w.D, w.H, w.E, w.K, w.n_shared, w.dtype, w.routing, w.alpha), I.make_inputs(w))
    opt = layer.optimizer(lr=1e-2, ema_decay=0.9)
    gen = torch.Generator().manual_seed(1)
    return opt, {n: torch.randn(p.numel(), generator=gen).to(DEV) for n, p in zip(opt.grad_names, opt.params)}


def _plain_optimizer():
    gen = torch.Generator().manual_seed(2)
    opt = optim.AdamW([torch.randn(5000, generator=gen).to(DEV)], lr=1e-2, ema_decay=0.9)
    return opt, [torch.randn(5000, generator=gen).to(DEV)]


def _all(opt):
    return [b.clone() for b in opt.buffers.values()] + [p.clone() for p in opt.params]


def _late(opt, name):
    """The optimizer's method, with the current stream held up before (``_init``) or behind it."""
    call = getattr(opt, name)

    def wrapped(*args):
        if name == "_init":
            torch.cuda._sleep(LATE)
        out = call(*args)
        if name != "_init":
            torch.cuda._sleep(LATE)
        return out
    setattr(opt, name, wrapped)


@pytest.mark.parametrize("make", [_plain_optimizer, _layer_optimizer])
def test_a_step_right_behind_state_dict_is_not_in_it(make):
    opt, grads = make()
    opt.step(grads)
    torch.cuda.synchronize()
    want, side = _all(opt), torch.cuda.Stream()
    torch.cuda.synchronize()
    _late(opt, "steps_taken")                             # the copies wait on the current stream
    saved = opt.state_dict()
    with torch.cuda.stream(side):
        opt.step(grads)
    torch.cuda.synchronize()
    got = [saved[k] for k in opt.buffers] + list(saved.get("params", opt.params[:0]))
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert saved["step"] == 1


@pytest.mark.parametrize("make", [_plain_optimizer, _layer_optimizer])
def test_a_step_ahead_of_load_state_dict_does_not_mix_with_it(make):
    opt, grads = make()
    opt.step(grads)
    saved, side = opt.state_dict(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LATE)
        opt.step(grads)
    opt.load_state_dict(saved)
    torch.cuda.synchronize()
    for k in opt.buffers:
        assert torch.equal(opt.buffers[k], saved[k]), k
    for p, q in zip(opt.params, saved.get("params", ())):
        assert torch.equal(p, q)
    assert opt.steps_taken() == 1


@pytest.mark.parametrize("make", [_plain_optimizer, _layer_optimizer])
def test_a_step_right_behind_load_state_dict_starts_from_it(make):
    opt, grads = make()
    held = [p.clone() for p in opt.params]
    opt.step(grads)
    saved = opt.state_dict()
    start = [p.clone() for p in opt.params]
    opt.step(grads)
    want, side = _all(opt), torch.cuda.Stream()
    for p, q in zip(opt.params, start if "params" not in saved else held):
        p.copy_(q)                                        # the layer's come from its own state
    torch.cuda.synchronize()
    _late(opt, "_init")
    opt.load_state_dict(saved)
    with torch.cuda.stream(side):
        opt.step(grads)
    torch.cuda.synchronize()
    for a, b in zip(want, _all(opt)):
        assert torch.equal(a, b)
    assert opt.steps_taken() == 2


@pytest.mark.parametrize("what", ["params", "weights", "grads", "norm"])
def test_tensors_off_the_vectors_are_refused_by_name(what):
    p, odd = torch.zeros(64, device=DEV), torch.zeros(65, device=DEV)[1:]
    with pytest.raises(ValueError, match="16-byte aligned"):
        if what == "params":
            optim.AdamW([p, odd], lr=1e-3)
        elif what == "weights":
            optim.AdamW([p], [torch.zeros(65, dtype=torch.half, device=DEV)[1:]], lr=1e-3)
        elif what == "grads":
            optim.AdamW([p], lr=1e-3).step([odd])
        else:
            optim.GradNorm(DEV)([p, odd])
    # nothing there, nothing to align
    optim.AdamW([p, odd[:0]], lr=1e-3).step([p, odd[:0]], max_norm=1.0)
    torch.cuda.synchronize()
