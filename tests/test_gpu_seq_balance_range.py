"""moe_seq_balance where one call's values or shapes are at the ends of their range: experts that are hardly
ever chosen, every shape of the one-kernel form, no tokens."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from sparse_moe_layer_03_b200 import binding as B
from sparse_moe_layer_03_b200 import inputs as I
from tests import parity as PA
from tests.test_gpu_seq_balance import ALPHA, TYPES, U, Case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("T,D,E", [(4096, 256, 8), (8192, 768, 8), (4096, 512, 16), (2048, 128, 16), (2048, 192, 20)])
@pytest.mark.parametrize("low", [-12.0, -25.0])
@pytest.mark.parametrize("dt", list(TYPES))
def test_the_gate_row_of_a_rare_expert(T, D, E, low, dt):
    # fp16 keeps dl in two parts under one scale for each expert and 16 tokens: 2^-21 of the largest of that
    # expert's own dl among them, whatever the others' are
    c = Case(T, D, E, 2, dt, offsets=[0, T // 2, T])
    rare = E - 3
    c.bias[rare] = low
    c.P = O.softmax_scores(O.gate_logits(c.x, c.wg, c.bias))
    c.idx = np.asarray(O.topk_route(c.P, 2)[0]).reshape(T, -1)
    c.inp["router_bias"] = c.bias
    c.gate = (np.random.default_rng(4).standard_normal(c.idx.shape) * 0.05).astype(np.float32)
    o = c.run()
    c.check(o)
    P = c.P
    dP = O.balance_packed(c.idx, P, 2, ALPHA, c.offsets)[3]
    adP = np.abs(dP)
    for k in range(2):
        np.add.at(dP, (np.arange(T), c.idx[:, k]), c.gate[:, k])
        np.add.at(adP, (np.arange(T), c.idx[:, k]), np.abs(c.gate[:, k]))
    pc = (P * dP).sum(1, keepdims=True)
    dl = P * (dP - pc)
    eP = PA.score_error_bound(c.inp)
    e = eP * np.abs(dP - pc) + P * (eP * np.abs(dP)).sum(1, keepdims=True) + (E + 16) * U * P * (adP + (P * adP).sum(1, keepdims=True))
    a = np.abs(dl) + e
    if dt == "f16":
        e = e + 2.0 ** -21 * np.maximum.reduceat(a, np.arange(0, T, 16), 0).repeat(16, 0)[:T]
    elif dt == "bf16":
        e = e + 2.0 ** -17 * a
    x = O.as_f64(c.x)
    gam = (T + 8) * U / (1 - (T + 8) * U)
    tol = (e.T @ np.abs(x) + gam * (a.T @ np.abs(x)))[rare]
    off = np.abs(o["dwg"].double().cpu().numpy() - dl.T @ x)[rare]
    assert np.all(off <= 1.01 * tol), (float((off / tol).max()), float(off.max()), float(np.abs(dl.T @ x)[rare].max()))


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("T,D,E,routing,off", [
    (6001, 1152, 16, "race", [5, 700, 700, 3000, 5987]),   # one block of dx held; first and last rows inside a token block
    (9000, 576, 9, "topk", [19, 4000, 8990]),
    (8000, 1088, 12, "topk", [3, 4, 8000]),
    (14300, 768, 8, "topk", [9, 7000, 14291]),             # the ring of x and both blocks of dx go round
    (333, 1152, 16, "race", [17, 333]),
    (14300, 512, 13, "race", [1, 14299]),
    (7200, 1152, 1, "topk", [40, 41, 7199]),
])
def test_every_shape_of_the_one_kernel_form(T, D, E, routing, off, dt):
    if dt == "f32" and E * D > 51200:
        D = 64 * (51200 // E // 64)
    c = Case(T, D, E, min(2, E), dt, routing, off, dead=np.nan)
    c.check(c.run(aux=3.0), aux=3.0)
    c.check(c.run(accumulate=False), accumulate=False)
    o = c.run(dx=False)
    c.check(o)


@pytest.mark.parametrize("how", ["seq_balance", "router_backward"])
def test_no_tokens_with_a_dx_to_add_to(how):
    # an empty tensor's pointer is null
    cfg = B.make_config(0, 128, 64, 4, 2, 0)
    z = lambda *s: torch.full(s, 5.0, device=DEV)  # noqa: E731
    dx, dwg, db = torch.empty((0, 128), dtype=torch.bfloat16, device=DEV), z(4, 128), z(4)
    st = torch.cuda.current_stream().cuda_stream
    if how == "seq_balance":
        nb = B.moe_seq_balance_workspace_size(cfg, 2)
        bws, ws = torch.zeros(nb, dtype=torch.uint8, device=DEV), torch.zeros(256, dtype=torch.uint8, device=DEV)
        counts, loss = torch.full((2, 4), 5, dtype=torch.int32, device=DEV), z(1)
        B.moe_seq_balance(cfg, dx, z(4, 128).bfloat16(), None, torch.zeros(3, dtype=torch.int32, device=DEV), 2, None, None,
                          None, 1.0, counts, z(2), loss, dwg, db, dx, 1, bws, nb, ws, st)
        torch.cuda.synchronize()
        assert torch.count_nonzero(counts) == 0 and float(loss) == 0.0
    else:
        nb = B.moe_backward_workspace_size(cfg)
        bws = torch.zeros(max(nb, 1), dtype=torch.uint8, device=DEV)
        B.moe_router_backward(cfg, dx, z(4, 128).bfloat16(), None, torch.zeros(4, dtype=torch.int32, device=DEV), None, None,
                              None, 1.0, dwg, db, dx, 1, bws, nb, st)
        torch.cuda.synchronize()
    assert torch.count_nonzero(dwg) == 0 and torch.count_nonzero(db) == 0


@pytest.mark.parametrize("seq_len", [0, 64])
@pytest.mark.parametrize("offsets", [False, True])
@pytest.mark.parametrize("routing", ["topk", "race"])
def test_a_layer_without_tokens(seq_len, offsets, routing):
    from sparse_moe_layer_03_b200.layer import LayerShape, MoELayer
    w = I.small_workload(64, 64, 128, 4, 2, 1, "bf16", routing, seed=3)
    layer = MoELayer(LayerShape(0, w.D, w.H, w.E, w.K, w.n_shared, w.dtype, w.routing, w.alpha, seq_len=seq_len), I.make_inputs(w))
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    layer.forward(x)
    off = torch.zeros(3, dtype=torch.int32, device=DEV) if offsets else None
    g = layer.backward(x, torch.empty_like(x), seq_offsets=off)
    torch.cuda.synchronize()
    layer.check()
    for n in ("dw1", "dw2", "dws1", "dws2", "dwg", "dbias", "db1", "db2"):
        assert torch.count_nonzero(g[n]) == 0, n
    assert g["dx"].shape == (0, 64)
    if seq_len or offsets:
        assert float(g["balance_loss"]) == 0.0
