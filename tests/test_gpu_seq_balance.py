"""GPU parity of moe_seq_balance against the fp64 oracle: counts, losses and gradients.

Bounds, element by element, from the arithmetic.  With u = 2^-23 (a unit in the last place, which
covers truncating accumulators) and dP_err the scores' own bound (parity.score_error_bound):
    dP       aux C: the factor, its products and the sum with dgate, 8 roundings
    dl       P (dP - pc): the scores' error in either factor, and E + 8 roundings of P (|dP| + sum P |dP|)
    parts    dl as hi + lo of 16-bit values: bf16 2^-17 of the value; fp16 2^-21 of the largest of its row
             (dx) or of its 16 tokens (dWg); fp32 none
    dWg, db  sums over T tokens in any order, gamma_T with T u, of |dl| |x|
    dx       sums over 2 E products, then the sum with the old value and one rounding to the type
"""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from sparse_moe_layer_03_b200 import binding as B
from sparse_moe_layer_03_b200 import inputs as I
from tests import parity as PA

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -23
ALPHA = 0.01
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}


class Case:
    def __init__(self, T, D, E, K, dt, routing="topk", offsets=None, seq_len=0, seed=0, gate=True, bias=True, dead=None):
        rng = np.random.default_rng(seed + T + 7 * D + 13 * E)
        self.T, self.D, self.E, self.K, self.dt, self.routing = T, D, E, K, dt, routing
        st = lambda a: I._store(a, dt)  # noqa: E731
        self.x = st(rng.standard_normal((T, D)))
        self.wg = st(rng.standard_normal((E, D)) / np.sqrt(D))
        self.bias = (rng.standard_normal(E) * 0.7).astype(np.float32) if bias else None
        self.inp = {"x": self.x, "wg": self.wg, "router_bias": self.bias}
        self.P = O.softmax_scores(O.gate_logits(self.x, self.wg, self.bias))
        if routing == "race":
            got = O.race_route(self.P, K * T)
        else:
            got = O.topk_route(self.P, K)
        self.idx = np.asarray(got[0]).reshape(T, -1)
        self.n_sel = (self.idx >= 0).sum(1).astype(np.int32)
        self.gate = (rng.standard_normal(self.idx.shape) * 0.05 * (self.idx >= 0)).astype(np.float32) if gate else None
        self.old = st(rng.standard_normal((T, D)) * 0.02)
        self.seq_len = seq_len
        if offsets is None:
            step = seq_len or T
            self.offsets, self.given = list(range(0, T + 1, step)), False
        else:
            self.offsets, self.given = list(offsets), True
        self.n = len(self.offsets) - 1
        live = np.zeros(T, bool)
        live[self.offsets[0]:self.offsets[-1]] = True
        self.live = live
        self.x_dev = self.x.copy()
        if dead is not None:                          # what rows of no sequence hold
            self.x_dev[~live] = dead
            if self.gate is not None:
                self.gate[~live] = dead

    def run(self, aux=1.0, grads=True, accumulate=True, dx=True, dbias=True, stream=None, hold=None):
        t = lambda a, d: None if a is None else torch.as_tensor(a).to(DEV, d)  # noqa: E731
        dt = TYPES[self.dt]
        cfg = B.make_config(self.T, self.D, 64, self.E, self.K, 0, self.dt, self.routing, ALPHA, seq_len=self.seq_len)
        nb = B.moe_seq_balance_workspace_size(cfg, self.n)
        bws = torch.full((nb + 256,), 0xA5, dtype=torch.uint8, device=DEV)
        status = torch.zeros(256, dtype=torch.uint8, device=DEV)
        junk = lambda *s: torch.full(s, 7.5, device=DEV)  # noqa: E731
        o = {"counts": torch.full((self.n, self.E), -9, dtype=torch.int32, device=DEV), "seq_loss": junk(self.n),
             "loss": junk(1), "dwg": junk(self.E, self.D) if grads else None,
             "dbias": junk(self.E) if grads and dbias else None, "dx": t(self.old, dt) if grads and dx else None}
        args = (cfg, t(self.x_dev, dt), t(self.wg, dt), t(self.bias, torch.float32),
                t(np.array(self.offsets, np.int32), torch.int32) if self.given else None, self.n,
                t(self.idx.astype(np.int32), torch.int32), t(self.n_sel, torch.int32),
                t(self.gate, torch.float32) if grads else None, aux, o["counts"], o["seq_loss"], o["loss"], o["dwg"],
                o["dbias"], o["dx"], int(accumulate and grads and dx), bws, nb, status)
        torch.cuda.synchronize()
        if hold is not None:
            hold.append(args)                          # the tensors of a captured call live as long as its graph
        s = torch.cuda.current_stream() if stream is None else stream
        self.again = lambda st: B.moe_seq_balance(*args, st.cuda_stream)
        self.again(s)
        if hold is None:
            s.synchronize()
            B.moe_check_status(status, s.cuda_stream)
            assert bool((bws[nb:] == 0xA5).all())
        return o

    def check(self, o, aux=1.0, accumulate=True):
        T, E, K = self.T, self.E, self.K
        loss, per, counts, dP = O.balance_packed(self.idx, self.P, K, ALPHA, self.offsets)
        assert np.array_equal(o["counts"].cpu().numpy(), counts)
        eP = PA.score_error_bound(self.inp)
        full = max(1, sum(b > a for a, b in zip(self.offsets, self.offsets[1:])))
        C = dP * full
        share = (self.P * C + eP * C).sum(1)
        got = o["seq_loss"].double().cpu().numpy()
        tol_all = 0.0
        for b, (lo, hi) in enumerate(zip(self.offsets, self.offsets[1:])):
            tol = (eP * C)[lo:hi].sum() + (E + 8) * U * share[lo:hi].sum()
            tol_all += tol
            assert abs(got[b] - per[b]) <= 1.01 * tol, (b, got[b], per[b], tol)
        assert abs(float(o["loss"]) - loss) <= 1.01 * (tol_all / full + U * loss)
        if o.get("dwg") is None:
            return
        dP = aux * dP
        adP = np.abs(dP)
        if self.gate is not None:
            for k in range(self.idx.shape[1]):
                r = np.nonzero((k < self.n_sel) & self.live)[0]
                dP[r, self.idx[r, k]] += self.gate[r, k]
                adP[r, self.idx[r, k]] += np.abs(self.gate[r, k])
        P = self.P
        pc = (P * dP).sum(1, keepdims=True)
        dl = P * (dP - pc) * self.live[:, None]
        e_dl = eP * np.abs(dP - pc) + P * (eP * np.abs(dP)).sum(1, keepdims=True) \
            + (E + 16) * U * P * (adP + (P * adP).sum(1, keepdims=True))
        e_dl *= self.live[:, None]
        a = np.abs(dl) + e_dl
        if self.dt == "f32":
            e_x = e_w = e_dl
        elif self.dt == "bf16":
            e_x = e_w = e_dl + 2.0 ** -17 * a
        else:
            e_x = e_dl + 2.0 ** -21 * a.max(1, keepdims=True)
            blk = np.maximum.reduceat(a.max(1), np.arange(0, T, 16)).repeat(16)[:T]
            e_w = e_dl + 2.0 ** -21 * blk[:, None]
        x, wg = O.as_f64(self.x), O.as_f64(self.wg)
        dwg, db, dx = O.router_backward(x * self.live[:, None], wg, dl)
        gam = (T + 8) * U / (1 - (T + 8) * U)
        ax = np.abs(x) * self.live[:, None]
        self._near(o["dwg"], dwg, e_w.T @ ax + gam * (a.T @ ax), "dwg")
        if o["dbias"] is not None:
            self._near(o["dbias"], db, e_dl.sum(0) + gam * a.sum(0), "dbias")
        if o["dx"] is not None:
            old = O.as_f64(self.old) if accumulate else 0.0
            want = dx + old
            tol = e_x @ np.abs(wg) + (2 * E + 4) * U * (a @ np.abs(wg) + np.abs(old))
            tol = tol + HALF[self.dt] * (np.abs(want) + tol) + TINY[self.dt]
            got = o["dx"].double().cpu().numpy()
            assert np.array_equal(got[~self.live], O.as_f64(self.old)[~self.live])
            off = np.abs(got - want)[self.live]
            assert np.all(off <= 1.01 * tol[self.live]), ("dx", float((off / tol[self.live]).max()))

    @staticmethod
    def _near(got, want, tol, what):
        off = np.abs(got.double().cpu().numpy() - want)
        bad = ~(off <= 1.01 * tol + 2.0 ** -140)
        assert not bad.any(), (what, int(bad.sum()), float(off.max()), float(np.abs(want).max()))


SHAPES = [  # T, D, E, K, routing, offsets
    (1, 64, 1, 1, "topk", [0, 1]),
    (15, 64, 3, 2, "topk", [0, 0, 15]),
    (16, 128, 8, 1, "topk", [0, 16]),
    (17, 192, 8, 8, "topk", [0, 1, 2, 17]),
    (100, 384, 9, 2, "topk", [3, 50, 50, 51, 90]),
    (333, 256, 16, 4, "race", [0, 100, 333]),
    (513, 1152, 8, 2, "topk", [16, 32, 400, 500]),
    (1000, 320, 17, 3, "topk", [0, 999]),
    (700, 640, 32, 2, "race", [1, 300, 640, 700]),
    (257, 1600, 5, 2, "topk", [0, 257]),
    (64, 2304, 20, 6, "topk", [10, 54]),
    (2100, 64, 4, 2, "topk", list(range(0, 2101))),       # one row each: more offsets than shared memory keeps
    (200, 128, 6, 2, "topk", [7, 7, 7]),                    # no row at all
]


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "T%d_D%d_E%d_K%d_%s_n%d" % (*s[:5], len(s[5]) - 1))
def test_against_the_oracle(shape, dt):
    T, D, E, K, routing, off = shape
    if dt == "f32" and E * D > 51200:
        D = 64 * (51200 // E // 64)                       # the gate weight's limit of the router
    c = Case(T, D, E, K, dt, routing, off, dead=np.nan)
    c.check(c.run(aux=3.0), aux=3.0)
    c.check(c.run(aux=1.0, accumulate=False), accumulate=False)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("seq_len", [0, 60, 300])
def test_images_of_one_length(dt, seq_len):
    c = Case(600, 384, 8, 2, dt, seq_len=seq_len, seed=3)
    o = c.run()
    c.check(o)
    # and as offsets: the same bits
    d = Case(600, 384, 8, 2, dt, offsets=list(range(0, 601, seq_len or 600)), seed=3)
    p = d.run()
    for k in o:
        assert torch.equal(o[k], p[k]), k


@pytest.mark.parametrize("dt", list(TYPES))
def test_optional_outputs(dt):
    c = Case(345, 192, 8, 2, dt, offsets=[0, 100, 345])
    whole = c.run()
    c.check(whole)
    loss = c.run(grads=False)                           # the loss alone: another kernel, within the same bounds
    c.check(loss)
    assert torch.equal(whole["counts"], loss["counts"])
    part = c.run(dx=False, dbias=False)
    for k in ("counts", "seq_loss", "loss", "dwg"):
        assert torch.equal(part[k], whole[k])
    d = Case(345, 192, 8, 2, dt, offsets=[0, 100, 345], gate=False, bias=False)
    d.check(d.run(aux=-2.0), aux=-2.0)
    d.check(d.run(aux=0.0), aux=0.0)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_gates_of_very_different_sizes(dt):
    # the fp16 parts are scaled by row and by block: tokens a million times apart share a block
    c = Case(160, 256, 8, 2, dt, offsets=[0, 160])
    c.gate *= np.where(np.arange(160) % 3 == 0, 1e-6, np.where(np.arange(160) % 3 == 1, 1.0, 1e3))[:, None].astype(np.float32)
    c.old[:] = 0
    c.check(c.run())


@pytest.mark.parametrize("dt", list(TYPES))
def test_full_size_with_many_sequences(dt):
    T, D, E = (32768, 1152, 8) if dt != "f32" else (8192, 384, 8)
    rng = np.random.default_rng(5)
    off = np.sort(np.concatenate([[0, T - 77], rng.integers(0, T - 77, 60)])).tolist()
    c = Case(T, D, E, 2, dt, offsets=off)
    c.check(c.run())


@pytest.mark.parametrize("dt,T,D,E", [("f32", 1000, 384, 8), ("bf16", 1000, 384, 8), ("f16", 1000, 384, 8),
                                      ("bf16", 3000, 768, 8), ("f16", 5000, 512, 16), ("f32", 6000, 128, 20),
                                      ("bf16", 3000, 320, 24)])
def test_equal_bits_again_captured_and_on_another_stream(dt, T, D, E):
    c = Case(T, D, E, 2, dt, offsets=[0, 400, T - 10])
    want = c.run(accumulate=False)
    want = {k: v.clone() for k, v in want.items()}
    side = torch.cuda.Stream()
    got = c.run(accumulate=False, stream=side)
    for k in want:
        assert torch.equal(want[k], got[k]), k
    graph, hold = torch.cuda.CUDAGraph(), []
    with torch.cuda.stream(side):
        o = c.run(accumulate=False, stream=side, hold=hold)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            c.again(side)
    for _ in range(2):
        for v in o.values():
            v.fill_(3)
        if o["dx"] is not None:
            o["dx"].copy_(torch.as_tensor(c.old).to(DEV, o["dx"].dtype))
        graph.replay()
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(want[k], o[k]), k


@pytest.mark.parametrize("T,D", [(900, 256), (4000, 768)])
def test_two_calls_at_once_on_two_streams(T, D):
    cases = [Case(T, D, 8, 2, "bf16", offsets=[0, T], seed=s) for s in (1, 2)]
    want = [c.run() for c in cases]
    want = [{k: v.clone() for k, v in w.items()} for w in want]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [c.run(stream=s, hold=[]) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        for k in w:
            assert torch.equal(w[k], o[k])


def test_bad_offsets_and_experts_are_reported():
    # every index is checked in the kernel before it is used: rows outside a sequence take no part
    for off in ([0, 60, 30, 100], [0, 50, 140], [-5, 50, 100]):
        c = Case(100, 64, 4, 2, "bf16", offsets=[0, 100])
        c.offsets, c.n = off, len(off) - 1
        with pytest.raises(B.MoeError, match="bad index"):
            c.run()
    c = Case(100, 64, 4, 2, "bf16", offsets=[0, 100])
    c.idx[50, 1] = 9
    with pytest.raises(B.MoeError, match="bad index"):
        c.run()


@pytest.mark.parametrize("dt", list(TYPES))
def test_no_sequences(dt):
    c = Case(40, 64, 4, 2, dt, offsets=[0, 40])
    c.offsets, c.n = [0], 0
    c.live[:] = False
    o = c.run()
    assert float(o["loss"]) == 0.0 and torch.count_nonzero(o["dwg"]) == 0 and torch.count_nonzero(o["dbias"]) == 0
    assert np.array_equal(o["dx"].double().cpu().numpy(), O.as_f64(c.old))


@pytest.mark.parametrize("E,dt", [(8, "bf16"), (32, "bf16"), (16, "f16"), (8, "f32")])
def test_the_most_tokens_a_call_takes(E, dt):
    # 262144 tokens of one sequence, and of 4096: against fp64 on the device (the CPU oracle's sums take
    # minutes).  Normwise: dl is good to 1e-5 of its largest (logits of 64 products), sums of 2^18 rounded
    # terms in fp32 to 2^18 u / 100 at the very worst order, u = 2^-24
    T, D, K = 262144, 64, 2
    g = torch.Generator(device=DEV).manual_seed(E)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    x, wg = rn(T, D).to(TYPES[dt]), (rn(E, D) / 8).to(TYPES[dt])
    P = torch.softmax(x.double() @ wg.double().t(), 1)
    idx = P.topk(K, 1).indices.to(torch.int32)
    for n in (1, 4096):
        off = torch.arange(n + 1, dtype=torch.int32, device=DEV) * (T // n)
        cfg = B.make_config(T, D, 64, E, K, 0, dt, alpha=ALPHA)
        nb = B.moe_seq_balance_workspace_size(cfg, n)
        bws, st = torch.empty(nb, dtype=torch.uint8, device=DEV), torch.zeros(256, dtype=torch.uint8, device=DEV)
        counts = torch.empty((n, E), dtype=torch.int32, device=DEV)
        f = lambda *s: torch.empty(s, device=DEV)  # noqa: E731
        per, loss, dwg, db, dx = f(n), f(1), f(E, D), f(E), torch.empty_like(x)
        B.moe_seq_balance(cfg, x, wg, None, off, n, idx, None, None, 1e6, counts, per, loss, dwg, db, dx, 0, bws, nb, st,
                          torch.cuda.current_stream().cuda_stream)
        B.moe_check_status(st, torch.cuda.current_stream().cuda_stream)
        sel = torch.zeros((T, E), dtype=torch.float64, device=DEV).scatter_(1, idx.long(), 1.0).view(n, T // n, E)
        want = sel.sum(1)
        assert torch.equal(counts, want.to(torch.int32))
        C = (ALPHA * E / (K * (T // n) ** 2) * want)[:, None].expand(n, T // n, E).reshape(T, E)
        assert torch.allclose(per.double(), (P * C).sum(1).view(n, -1).sum(1), rtol=2e-5)
        assert abs(float(loss) - float((P * C).sum() / n)) <= 2e-5 * float(loss)
        dP = 1e6 * C / n
        dl = P * (dP - (P * dP).sum(1, keepdim=True))
        for got, ref in ((dwg, dl.t() @ x.double()), (db, dl.sum(0))):
            scale = float((dl.abs().t() @ x.double().abs()).max()) if ref.dim() == 2 else float(dl.abs().sum(0).max())
            assert float((got.double() - ref).abs().max()) <= 2e-4 * scale
        ref = dl @ wg.double()
        assert float((dx.double() - ref).abs().max()) <= (HALF[dt] + 3e-5) * float(ref.abs().max()) + TINY[dt]


def test_no_tokens():
    cfg = B.make_config(0, 128, 64, 4, 2, 0)
    nb = B.moe_seq_balance_workspace_size(cfg, 2)
    z = lambda *s: torch.full(s, 5.0, device=DEV)  # noqa: E731
    counts = torch.full((2, 4), 5, dtype=torch.int32, device=DEV)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    bws, st = torch.zeros(nb, dtype=torch.uint8, device=DEV), torch.zeros(256, dtype=torch.uint8, device=DEV)
    o = [counts, z(2), z(1), z(4, 128), z(4)]
    B.moe_seq_balance(cfg, None, None, None, off, 2, None, None, None, 1.0, *o, None, 0, bws, nb, st,
                      torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    for t in o:
        assert torch.count_nonzero(t) == 0


@pytest.mark.parametrize("routing", ["topk", "race"])
@pytest.mark.parametrize("how", ["seq_len", "offsets"])
def test_a_layer_trained_on_the_loss_per_image(how, routing):
    # the layer's own backward, then its optimizer: gradients against the oracle's, normwise at the
    # storage type's bound as the layer's other gradients
    T, L = 512, 128
    w = I.small_workload(T, 256, 512, 8, 2, 1, "bf16", routing, seed=17)
    inp = I.make_inputs(w, bias_std=0.1)
    from sparse_moe_layer_03_b200.layer import LayerShape, MoELayer
    layer = MoELayer(LayerShape(w.T, w.D, w.H, w.E, w.K, w.n_shared, w.dtype, w.routing, w.alpha,
                                seq_len=L if how == "seq_len" else 0), inp)
    x = torch.as_tensor(inp["x"]).to(DEV, layer.act_dtype)
    off = [0, 128, 256, 384, 512] if how == "seq_len" else [0, 100, 100, 400, 512]
    off_d = None if how == "seq_len" else torch.tensor(off, dtype=torch.int32, device=DEV)
    opt = layer.optimizer(lr=1e-3, state="e4m3", ema_decay=0.99, seed=4)
    dout = I._store(np.random.default_rng(2).standard_normal((T, w.D)), "bf16")
    dout_d = torch.as_tensor(dout).to(DEV, layer.act_dtype)
    layer.forward(x)
    ev = layer.seq_balance(x, off_d)
    g = layer.backward(x, dout_d, aux_scale=50.0, seq_offsets=off_d)
    torch.cuda.synchronize()
    layer.check()
    idx = PA.gpu_selection(PA.fetch(layer))
    P = O.softmax_scores(O.gate_logits(inp["x"], inp["wg"], inp.get("router_bias")))
    loss, per, counts, dP = O.balance_packed(idx, P, w.K, w.alpha, off)
    assert np.array_equal(g["seq_counts"].cpu().numpy(), counts)
    assert torch.equal(ev["seq_counts"], g["seq_counts"])
    for got in (ev, g):
        assert abs(float(got["balance_loss"]) - loss) <= 1e-4 * loss
        np.testing.assert_allclose(got["seq_loss"].cpu().numpy(), per, rtol=1e-4)
    if how == "seq_len":
        assert abs(float(layer.aux) - loss) <= 1e-4 * loss      # the forward's own per-image loss
    ref = O.layer_backward(inp, idx, dout, w.K, w.alpha, aux_scale=0.0)
    add = O.router_backward(inp["x"], inp["wg"], 50.0 * O.softmax_backward(P, dP))
    ref["dwg"], ref["dbias"], ref["dx"] = ref["dwg"] + add[0], ref["dbias"] + add[1], ref["dx"] + add[2]
    for n in ("dwg", "dbias", "dx", "dw1", "dw2"):
        assert PA.rel_err(g[n].float().cpu().numpy(), ref[n]) <= PA.out_tol(w), n
    before = [p.clone() for p in opt.params]
    opt.step(g, max_norm=1.0)
    assert all(not torch.equal(a, b) for a, b in zip(before, opt.params))
    out = layer.forward(x)                                       # and on the new weights
    layer.check()
    assert torch.isfinite(out).all()


def test_a_layer_refuses_tensors_that_do_not_fit():
    w = I.small_workload(64, 64, 128, 4, 2, 0, "bf16", "topk", seed=3)
    inp = I.make_inputs(w)
    from sparse_moe_layer_03_b200.layer import LayerShape, MoELayer
    layer = MoELayer(LayerShape(w.T, w.D, w.H, w.E, w.K, w.n_shared, w.dtype, w.routing, w.alpha), inp)
    x = torch.as_tensor(inp["x"]).to(DEV, layer.act_dtype)
    layer.forward(x)
    g = dict(dwg=torch.zeros(4, 64, device=DEV))
    off = torch.tensor([0, 64], dtype=torch.int32, device=DEV)
    bad = [dict(x=x[:63]), dict(x=x.float()), dict(x=x.cpu()), dict(x=x.t().contiguous().t()),
           dict(dgate=torch.zeros(64, 3, device=DEV), grads=g), dict(dgate=torch.zeros(64, 2, device=DEV).half(), grads=g),
           dict(grads=dict(dwg=torch.zeros(4, 63, device=DEV))), dict(grads=dict(g, dbias=torch.zeros(5, device=DEV))),
           dict(grads=dict(g, dx=torch.zeros(64, 64, device=DEV))), dict(seq_offsets=off.long()), dict(seq_offsets=off.cpu()),
           dict(seq_offsets=off[:0])]
    for kw in bad:
        with pytest.raises(ValueError):
            layer.seq_balance(kw.pop("x", x), **kw)
    out = layer.seq_balance(x, off, grads=dict(g, dbias=None, dx=None))
    torch.cuda.synchronize()
    layer.check()
    assert int(out["seq_counts"].sum()) == 64 * 2
