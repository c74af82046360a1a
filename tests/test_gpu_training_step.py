"""A layer's whole training step -- forward, backward with the loss per image, clipped AdamW -- eagerly, replayed
from a graph, and of two layers at once on two streams: the same bits."""
import numpy as np
import pytest
import torch

from sparse_moe_layer_03_b200 import inputs as I

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
STEPS = 3


def _make(dt, routing, state, seed=0, D=128):
    from sparse_moe_layer_03_b200.layer import LayerShape, MoELayer
    w = I.small_workload(384, D, 256, 8, 2, 1, dt, routing, seed=31 + seed)
    inp = I.make_inputs(w, bias_std=0.1)
    layer = MoELayer(LayerShape(w.T, w.D, w.H, w.E, w.K, w.n_shared, w.dtype, w.routing, w.alpha), inp)
    opt = layer.optimizer(lr=1e-3, weight_decay=0.05, state=state, ema_decay=0.99, seed=7)
    rng = np.random.default_rng(seed)
    on = lambda a: torch.as_tensor(I._store(a, dt)).to(DEV, layer.act_dtype)  # noqa: E731
    data = [(on(rng.standard_normal((w.T, D))), on(rng.standard_normal((w.T, D)))) for _ in range(STEPS)]
    offsets = [torch.tensor(o, dtype=torch.int32, device=DEV) for o in ([0, 100, 384], [10, 11, 200, 200], [5, 90, 300])]
    return layer, opt, data, offsets


def _step(layer, opt, x, dout, offsets):
    layer.forward(x)
    g = layer.backward(x, dout, aux_scale=10.0, seq_offsets=offsets)
    opt.step(g, max_norm=1.0)
    return g


def _bits(layer, opt):
    torch.cuda.synchronize()
    layer.check()
    assert opt.steps_taken() == STEPS
    return [t.clone().view(torch.uint8) for t in opt.params + [w for w in opt.weights if w is not None] + list(opt.buffers.values())]


def _eager(*args):
    layer, opt, data, offsets = _make(*args)
    for (x, dout), off in zip(data, offsets):
        _step(layer, opt, x, dout, torch.cat([off, off[-1:].expand(4 - off.numel())]))   # the graph's count of sequences
    return _bits(layer, opt)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("routing,state,D", [("topk", "f32", 128), ("race", "e4m3", 128), ("topk", "e4m3", 704)])
def test_a_captured_step_replays_as_the_next(dt, routing, state, D):
    want = _eager(dt, routing, state, 0, D)
    layer, opt, data, offsets = _make(dt, routing, state, 0, D)
    x, dout = (torch.zeros_like(t) for t in data[0])
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    # buffers and modules before the capture; then the state from the beginning
    start = opt.state_dict()
    _step(layer, opt, x, dout, off)
    opt.load_state_dict(start)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        g = _step(layer, opt, x, dout, off)
    for (a, b), o in zip(data, offsets):
        x.copy_(a)
        dout.copy_(b)
        off.copy_(torch.cat([o, o[-1:].expand(4 - o.numel())]))
        graph.replay()
    got = _bits(layer, opt)
    assert all(torch.isfinite(v).all() for v in g.values() if v is not None and v.is_floating_point())
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_two_layers_step_at_once():
    shapes = [("bf16", "topk", "e4m3", 1, 704), ("f16", "race", "f32", 2, 128)]
    want = [_eager(*s) for s in shapes]
    made = [_make(*s) for s in shapes]
    streams = [torch.cuda.Stream() for _ in made]
    torch.cuda.synchronize()
    for i in range(STEPS):
        for (layer, opt, data, offsets), s in zip(made, streams):
            with torch.cuda.stream(s):
                o = offsets[i]
                _step(layer, opt, *data[i], torch.cat([o, o[-1:].expand(4 - o.numel())]))
    for w, (layer, opt, _, _) in zip(want, made):
        for a, b in zip(w, _bits(layer, opt)):
            assert torch.equal(a, b)
