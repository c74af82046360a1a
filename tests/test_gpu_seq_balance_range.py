"""moe_seq_balance where one call's values or shapes are at the ends of their range: experts that are hardly
ever chosen, every shape of the one-kernel form, no tokens, rows of no sequence that carry their gates' gradient."""
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
    (8100, 640, 9, "topk", [19, 4000, 8090]),              # its narrowest rows
    (7300, 640, 8, "race", [2, 7300]),
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


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("T,D,E,routing,off", [
    (700, 256, 8, "topk", [0, 300, 612]), (333, 128, 16, "race", [17, 40, 333]), (400, 192, 24, "topk", [399, 400]),
    (5001, 768, 8, "topk", [9, 2000, 4991]), (2500, 1152, 16, "race", [5, 2000]), (5001, 128, 20, "topk", [33, 4000]),
    (6000, 64, 4, "topk", [0, 3001]), (90, 64, 4, "topk", [7, 7]), (300, 512, 2, "topk", [300, 300]), (100, 640, 4, "topk", [50])])
def test_gates_of_every_row(T, D, E, routing, off, dt):
    c = Case(T, D, E, 2, dt, routing, off)
    held = []
    for acc in (True, False):
        o = c.run(aux=3.0, accumulate=acc, hold=held)
        o["dx"].copy_(torch.as_tensor(c.old).to(DEV, TYPES[dt]))
        args = held[-1]
        st = torch.cuda.current_stream().cuda_stream
        B.moe_seq_balance(*args, st, all_gates=1)
        B.moe_check_status(args[-1], st)
        live = c.live.copy()
        c.live[:] = True
        c.check(o, aux=3.0, accumulate=acc)
        c.live = live
    # an expert out of range is reported in any row
    if not c.live.all():
        idx = args[6].clone()
        idx[int(np.nonzero(~c.live & (c.n_sel > 0))[0][0]), 0] = E
        args = args[:6] + (idx,) + args[7:]
        B.moe_seq_balance(*args, st, all_gates=1)
        with pytest.raises(B.MoeError, match="bad index"):
            B.moe_check_status(args[-1], st)


def test_gates_of_every_row_where_all_belong_to_sequences():
    # the flag changes nothing: the same bits
    c = Case(1000, 768, 8, 2, "bf16", offsets=[0, 400, 1000])
    held = []
    o = c.run(hold=held)
    want = {k: v.clone() for k, v in o.items()}
    o["dx"].copy_(torch.as_tensor(c.old).to(DEV, torch.bfloat16))
    B.moe_seq_balance(*held[0], torch.cuda.current_stream().cuda_stream, all_gates=1)
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(want[k], o[k]), k


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("routing", ["topk", "race"])
def test_a_layers_rows_of_no_sequence_keep_their_gates_gradient(dt, routing):
    # J = <dout, MoE(x)> + aux L with L over some of the rows: the first term is every row's
    from sparse_moe_layer_03_b200.layer import LayerShape, MoELayer
    T = 512
    w = I.small_workload(T, 256, 512, 8, 2, 1, dt, routing, seed=23)
    inp = I.make_inputs(w, bias_std=0.1)
    layer = MoELayer(LayerShape(w.T, w.D, w.H, w.E, w.K, w.n_shared, w.dtype, w.routing, w.alpha), inp)
    x = torch.as_tensor(inp["x"]).to(DEV, layer.act_dtype)
    off = [101, 200, 200, 390]
    off_d = torch.tensor(off, dtype=torch.int32, device=DEV)
    # the rows outside matter most, so that leaving them out is far beyond the bound
    d = np.random.default_rng(2).standard_normal((T, w.D))
    d[off[0]:off[-1]] *= 0.1
    dout = I._store(d, dt)
    layer.forward(x)
    g = layer.backward(x, torch.as_tensor(dout).to(DEV, layer.act_dtype), aux_scale=50.0, seq_offsets=off_d)
    torch.cuda.synchronize()
    layer.check()
    idx = PA.gpu_selection(PA.fetch(layer))
    P = O.softmax_scores(O.gate_logits(inp["x"], inp["wg"], inp.get("router_bias")))
    loss, per, counts, dP = O.balance_packed(idx, P, w.K, w.alpha, off)
    assert np.array_equal(g["seq_counts"].cpu().numpy(), counts)
    assert abs(float(g["balance_loss"]) - loss) <= 1e-4 * loss
    ref = O.layer_backward(inp, idx, dout, w.K, w.alpha, aux_scale=0.0)
    add = O.router_backward(inp["x"], inp["wg"], 50.0 * O.softmax_backward(P, dP))
    ref["dwg"], ref["dbias"], ref["dx"] = ref["dwg"] + add[0], ref["dbias"] + add[1], ref["dx"] + add[2]
    for n in ("dwg", "dbias", "dx", "dw1", "dw2"):
        assert PA.rel_err(g[n].float().cpu().numpy(), ref[n]) <= PA.out_tol(w), n
    rows = np.r_[0:off[0], off[-1]:T]
    assert PA.rel_err(g["dx"].float().cpu().numpy()[rows], ref["dx"][rows]) <= PA.out_tol(w)
