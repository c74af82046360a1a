"""GPU parity of the gradient norm and of AdamW (fp32 and 8-bit moments) against the fp64 oracle.

Bounds, with u = 2^-24 (half a step of fp32, relative).  Each is the sum of the roundings on the
way, every constant (beta, 1 - beta, lr / c1, ...) itself rounded once:
    m   u (4 |(1 - b1) g s| + 2 |b1 m| + |m'|)         s the clip factor, rounded once
    v   u (6 (1 - b2) g^2 s^2 + 2 b2 v + v')           (g s enters twice); at the smallest values, fp32's
        least step 2^-149 a few times
    p   2 u |p keep| + u |p'| + the update's: its quotient m / (root rs2 + eps) by the errors of m, of
        root (half that of v, relative, and u), of rs2, eps and the two sums (4 u), of the division
        (2 units: 4 u), of lr / c1 and the product (2 u)
A second of margin, 1%, is for the products of these.
"""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from sparse_moe_layer_03_b200 import optim
from sparse_moe_layer_03_b200 import inputs as I
from tests import parity as PA

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
SIZES = [1, 2, 3, 4, 5, 127, 255, 256, 257, 1000, 2047, 2048, 2049, 5001, 12345, 70000]


def _rand(n, gen, scale=1.0, dtype=torch.float32):
    return (torch.randn(n, generator=gen) * scale).to(dtype).to(DEV)


def _np(t):
    return t.detach().double().cpu().numpy()


def _expect(p, g, m, v, t, scale, h, wd):
    """The oracle's step and the bounds of the module's docstring."""
    lr, (b1, b2), eps = h
    gs = scale * g
    q, m1, v1 = O.adamw(p, gs, m, v, t, lr, (b1, b2), eps, wd)
    dm = U * (4 * np.abs((1 - b1) * gs) + 2 * np.abs(b1 * m) + np.abs(m1)) + 4 * 2.0 ** -149
    dv = U * (6 * (1 - b2) * gs ** 2 + 2 * b2 * v + v1) + 4 * 2.0 ** -149
    root, rs2 = np.sqrt(v1), 1 / np.sqrt(1 - b2 ** t)
    den = root * rs2 + eps
    droot = np.minimum(dv / np.maximum(root, 1e-300), np.sqrt(dv)) + U * root
    dquot = dm / den + np.abs(m1) / den * ((droot * rs2 + 4 * U * den) / den + 6 * U)
    dp = 2 * U * np.abs(p * (1 - lr * wd)) + U * np.abs(q) + lr / (1 - b1 ** t) * dquot
    return (q, m1, v1), (1.01 * dp + 2.0 ** -149, 1.01 * dm, 1.01 * dv)


def _near(got, want, bound, what):
    off = np.abs(got - want)
    bad = ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(off[bad].max()), float(bound[bad].min()))


GRADS = [torch.float32, torch.bfloat16, torch.float16]


@pytest.mark.parametrize("gdt", GRADS, ids=str)
@pytest.mark.parametrize("wdt", [None, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("ema,max_norm", [(None, None), (0.99, 1.5), (0.99, 0.0)])
def test_adamw_follows_the_formula(gdt, wdt, ema, max_norm):
    gen = torch.Generator().manual_seed(11)
    params = [_rand(n, gen, 0.1) for n in SIZES]
    weights = None if wdt is None else [torch.zeros(n, dtype=wdt, device=DEV) for n in SIZES]
    decay = [0.1 if i % 2 else 0.0 for i in range(len(SIZES))]
    h = (2e-3, (0.9, 0.99), 1e-8)
    opt = optim.AdamW(params, weights, lr=h[0], betas=h[1], eps=h[2], weight_decay=decay, ema_decay=ema)
    for t in range(1, 4):
        grads = [_rand(n, gen, 10.0 ** (i % 5 - 3), gdt) for i, n in enumerate(SIZES)]
        had = [(_np(p), _np(g), _np(opt.part("m", i)), _np(opt.part("v", i)),
                _np(opt.part("ema", i)) if ema else None) for i, (p, g) in enumerate(zip(params, grads))]
        opt.step(grads, max_norm=max_norm, grad_mult=0.25)
        scale = 0.25
        if max_norm is not None:
            norm, scale = O.grad_norm([x[1] for x in had], 0.25, max_norm)
            # squares and sums in fp64 leave the one rounding to fp32
            assert abs(float(opt.grad_norm) - norm) <= 1.01 * U * norm
            assert abs(float(opt.grad_scale) - scale) <= 1.01 * U * scale
        for i, (p, g, m, v, e) in enumerate(had):
            want, bound = _expect(p, g, m, v, t, scale, h, decay[i])
            got = [_np(params[i]), _np(opt.part("m", i)), _np(opt.part("v", i))]
            for name, a, b, c in zip("pmv", got, want, bound):
                _near(a, b, c, (name, i, t))
            if weights:                                  # the copy is the master's own rounding
                assert torch.equal(weights[i], params[i].to(wdt))
            if ema:
                w = ema * e + (1 - ema) * got[0]
                _near(_np(opt.part("ema", i)), w, 1.01 * U * (2 * np.abs(ema * e) + 2 * np.abs((1 - ema) * got[0]) + np.abs(w)),
                      ("ema", i, t))
    assert opt.steps_taken() == 3
    for k, b in opt.buffers.items():                     # nothing behind a tensor's end
        gap = torch.ones(b.numel(), dtype=torch.bool, device=DEV)
        for i, at in enumerate(opt.starts):
            gap[at:at + SIZES[i]] = False
        assert torch.count_nonzero(b[gap]) == 0, k


@pytest.mark.parametrize("gdt", GRADS, ids=str)
@pytest.mark.parametrize("wdt,ema,max_norm", [(None, None, None), (torch.bfloat16, 0.99, 1.5), (torch.float16, None, 0.0)])
def test_adamw_with_8_bit_moments(gdt, wdt, ema, max_norm):
    # The codes are compared with the oracle's rounding of the fp64 moments by the same bits; where
    # value and bits come within 1e-3 of a whole number of gaps (the fp32 moments are off by about
    # 1e-6 of the value, at most 16 gaps) either neighbour may be taken.
    gen = torch.Generator().manual_seed(12)
    params = [_rand(n, gen, 0.1) for n in SIZES]
    weights = None if wdt is None else [torch.zeros(n, dtype=wdt, device=DEV) for n in SIZES]
    h = (2e-3, (0.9, 0.99), 1e-8)
    opt = optim.AdamW(params, weights, lr=h[0], betas=h[1], eps=h[2], weight_decay=0.05, state="e4m3", ema_decay=ema,
                      seed=99)
    close = total = 0
    for t in range(1, 4):
        grads = [_rand(n, gen, 10.0 ** (i % 5 - 3), gdt) for i, n in enumerate(SIZES)]
        spread = lambda k, i: _np(opt.part(k, i)) * np.repeat(_np(opt.part(k + "_scale", i)), 256)[:SIZES[i]]  # noqa: E731
        had = [(_np(p), _np(g), spread("m", i), spread("v", i) ** 2) for i, (p, g) in enumerate(zip(params, grads))]
        opt.step(grads, max_norm=max_norm, grad_mult=0.25)
        scale = 0.25 if max_norm is None else O.grad_norm([x[1] for x in had], 0.25, max_norm)[1]
        for i, (p, g, m, v) in enumerate(had):
            want, bound = _expect(p, g, m, v, t, scale, h, 0.05)
            # decoding adds one rounding to m and three to v (the product, twice in the square)
            bound = (bound[0] * 4, bound[1] + U * np.abs(m), bound[2] + 3 * U * v)
            _near(_np(params[i]), want[0], bound[0], ("p", i, t))
            if weights:
                assert torch.equal(weights[i], params[i].to(wdt))
            r = O.rounding_bits(99, t, i, SIZES[i])
            for name, val, bits in (("m", want[1], r & 0xFFFF), ("v", np.sqrt(want[2]), r >> 16)):
                n = SIZES[i]
                top = np.abs(np.pad(val, (0, -n % 256))).reshape(-1, 256).max(1)
                sc = _np(opt.part(name + "_scale", i))
                np.testing.assert_allclose(sc, top / 448, rtol=1e-5)
                a = np.abs(val) / np.repeat(sc, 256)[:n]
                want_code, room = O.e4m3_round(np.minimum(a, 448.0), bits)
                got = _np(opt.part(name, i))
                sure = room > 1e-3
                close += int((~sure).sum())
                total += n
                assert np.array_equal(np.abs(got)[sure], want_code[sure]), (name, i, t)
                gap = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
                assert np.all(np.abs(np.abs(got) - a) <= gap * 1.01), (name, i, t)
                assert np.all((np.sign(got) == np.sign(val)) | (got == 0))
    assert close < 0.01 * total
    for k in ("m", "v"):
        gap = torch.ones(opt.buffers[k].numel(), dtype=torch.bool, device=DEV)
        for i, at in enumerate(opt.starts):
            gap[at:at + SIZES[i]] = False
        assert torch.count_nonzero(opt.buffers[k].view(torch.uint8)[gap]) == 0


def test_8_bit_moments_follow_a_slow_average():
    # constant gradient: after n steps v is (1 - b2^n) g^2; a moment that stood still would be far off.
    # The mean over 65536 elements of the stored root's rounding has a standard deviation of at most a
    # gap (1/8 of the value) / sqrt(65536) per step; the sum of 300 such steps, each decaying, is below
    # 300^0.5 * 2^-3 / 256 = 0.85% (v: twice), and five of those is the bound.
    n, steps, b2 = 65536, 300, 0.999
    p = torch.zeros(n, device=DEV)
    opt = optim.AdamW([p], lr=0.0, betas=(0.9, b2), state="e4m3", seed=5)
    g = torch.full((n,), 0.01, device=DEV)
    g[::256] = 0.05                                      # the scale is another element's
    for _ in range(steps):
        opt.step([g])
    r = _np(opt.buffers["v"]) * np.repeat(_np(opt.buffers["v_scale"]), 256)
    small = np.arange(n) % 256 != 0
    want = (1 - b2 ** steps) * 0.01 ** 2
    assert abs(np.mean(r[small] ** 2) / want - 1) < 0.0085 * 2 * 5
    m = _np(opt.buffers["m"]) * np.repeat(_np(opt.buffers["m_scale"]), 256)
    assert abs(np.mean(m[small]) / 0.01 - 1) < 0.05


@pytest.mark.parametrize("count,state", [(41, "f32"), (340, "e4m3"), (341, "f32"), (700, "e4m3")])
def test_many_tensors(count, state):
    # over 40 and over 340 tensors the launches' parameters change shape and number
    gen = torch.Generator().manual_seed(count)
    sizes = [int(x) for x in torch.randint(0, 700, (count,), generator=gen)]
    params = [_rand(n, gen) for n in sizes]
    grads = [_rand(n, gen) for n in sizes]
    had = [p.clone() for p in params]
    opt = optim.AdamW(params, lr=1e-2, state=state, seed=3)
    opt.step(grads, max_norm=0.0)
    norm, _ = O.grad_norm([_np(g) for g in grads])
    assert abs(float(opt.grad_norm) - norm) <= 1.01 * U * norm
    assert opt.steps_taken() == 1
    for p, q, g in zip(params, had, grads):
        z = np.zeros(p.numel())
        want, bound = _expect(_np(q), _np(g), z, z, 1, 1.0, (1e-2, (0.9, 0.999), 1e-8), 0.0)
        _near(_np(p), want[0], bound[0], "p")


def test_norm_over_more_tensors_than_one_launch_holds():
    gen = torch.Generator().manual_seed(8)
    flat = _rand(2400 * 8, gen)
    grads = [flat[8 * i:8 * i + 5] for i in range(2400)]
    norm, scale = optim.GradNorm(DEV)(grads, max_norm=2.0)
    want, f = O.grad_norm([_np(g) for g in grads], 1.0, 2.0)
    assert abs(float(norm) - want) <= 1.01 * U * want and abs(float(scale) - f) <= 1.01 * U * f


@pytest.mark.parametrize("dt", GRADS, ids=str)
@pytest.mark.parametrize("sizes", [[1], [4095, 4096, 4097], [3, 0, 100001, 8], [2 ** 22 + 5]], ids=str)
def test_norm(dt, sizes):
    gen = torch.Generator().manual_seed(len(sizes))
    grads = [_rand(n, gen, 3.0, dt) for n in sizes]
    run = optim.GradNorm(DEV)
    for most, mult in ((0.0, 1.0), (0.5, 1.0), (1e9, 2.0 ** -10)):
        norm, scale = run(grads, max_norm=most, grad_mult=mult)
        want, f = O.grad_norm([_np(g) for g in grads], mult, most)
        assert abs(float(norm) - want) <= 1.01 * U * want
        assert abs(float(scale) - f) <= 1.01 * U * f
        assert int(run.nonfinite) == 0


def test_norm_of_nothing_and_of_extremes():
    run = optim.GradNorm(DEV)
    for grads in ([], [torch.zeros(0, device=DEV)], [torch.zeros(77, device=DEV)], [None]):
        norm, scale = run(grads, max_norm=1.0)
        assert float(norm) == 0.0 and float(scale) == 1.0 and int(run.nonfinite) == 0
    for v in (1e-30, 1e30, 3e38):                         # squares leave fp32's range, the norm does not
        norm, _ = run([torch.full((1,), v, device=DEV)])
        assert abs(float(norm) - v) <= 2 * U * v
    for v in (float("nan"), float("inf"), -float("inf")):
        for n, at in ((1, 0), (5000, 4999), (20000, 777)):
            g = torch.ones(n, device=DEV)
            g[at] = v
            _, scale = run([torch.ones(3, device=DEV), g], max_norm=1.0)
            assert int(run.nonfinite) == 1 and float(scale) == 0.0
    norm, scale = run([torch.ones(4, device=DEV)], max_norm=1.0)      # and the next call is clean
    assert float(norm) == 2.0 and int(run.nonfinite) == 0


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_a_gradient_that_is_not_finite_leaves_everything(state):
    gen = torch.Generator().manual_seed(21)
    params = [_rand(n, gen) for n in (300, 5000)]
    weights = [p.bfloat16() for p in params]
    opt = optim.AdamW(params, weights, lr=1e-2, state=state, ema_decay=0.9, seed=1)
    good = [_rand(n, gen) for n in (300, 5000)]
    opt.step(good, max_norm=1.0)
    before = [t.clone() for t in params + weights] + [b.clone() for b in opt.buffers.values()]
    bad = [g.clone() for g in good]
    bad[1][4321] = float("inf")
    opt.step(bad, max_norm=1.0)
    after = params + weights + list(opt.buffers.values())
    for a, b in zip(before, after):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert opt.steps_taken() == 1 and int(opt.skipped) == 1
    opt.step(good, max_norm=1.0)
    assert opt.steps_taken() == 2 and int(opt.skipped) == 1
    # without the norm a NaN reaches its own element; its block's 8-bit moments become zero, others stay whole
    bad[1][4321] = float("nan")
    opt.step(bad)
    assert int(torch.isnan(params[1]).sum()) == 1 and int(torch.isnan(params[0]).sum()) == 0
    if state == "e4m3":
        assert float(opt.part("m_scale", 1)[4321 // 256]) == 0.0
        assert torch.isfinite(opt.buffers["m_scale"]).all() and torch.isfinite(opt.buffers["v_scale"]).all()


def test_zero_moments_and_tiny_ones():
    p = torch.ones(600, device=DEV)
    opt = optim.AdamW([p], lr=1e-2, eps=1e-8, state="e4m3")
    opt.step([torch.zeros(600, device=DEV)])
    assert torch.equal(p, torch.ones_like(p)) and torch.count_nonzero(opt.buffers["m_scale"]) == 0
    g = torch.full((600,), 1e-32, device=DEV)            # its moments are below 2^-100: stored as zero
    opt.step([g])
    assert torch.isfinite(p).all() and torch.count_nonzero(opt.buffers["m"].view(torch.uint8)) == 0


def test_missing_gradients_and_empty_tensors():
    gen = torch.Generator().manual_seed(2)
    params = [_rand(500, gen), torch.zeros(0, device=DEV), _rand(70, gen)]
    had = [p.clone() for p in params]
    opt = optim.AdamW(params, lr=1e-2)
    opt.step([None, torch.zeros(0, device=DEV), torch.ones(70, device=DEV)], max_norm=1.0)
    assert torch.equal(params[0], had[0]) and not torch.equal(params[2], had[2])
    opt.step([torch.ones(500, device=DEV), None, None])
    assert not torch.equal(params[0], had[0]) and opt.steps_taken() == 2
    opt.step([None] * 3)                                  # nothing to update is still a step
    assert opt.steps_taken() == 3


def _clone_run(state, seed, steps=3):
    gen = torch.Generator().manual_seed(31)
    params = [_rand(n, gen) for n in (3000, 257, 100000)]
    opt = optim.AdamW(params, [p.half() for p in params], lr=1e-2, state=state, ema_decay=0.9, seed=seed)
    grads = [[_rand(p.numel(), gen) for p in params] for _ in range(steps)]
    return opt, params, grads


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_equal_calls_give_equal_bits_eagerly_and_captured(state):
    outs = []
    for how in ("eager", "eager", "graph", "stream"):
        opt, params, grads = _clone_run(state, 7)
        if how == "graph":
            buf = [torch.zeros_like(p) for p in params]
            opt.step([None] * 3, max_norm=1.0)            # scratch and modules before the capture
            opt._init(0, opt.betas)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                opt.step(buf, max_norm=1.0)
            for gs in grads:
                for b, g in zip(buf, gs):
                    b.copy_(g)
                graph.replay()
        elif how == "stream":
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                for gs in grads:
                    opt.step(gs, max_norm=1.0)
            side.synchronize()
        else:
            for gs in grads:
                opt.step(gs, max_norm=1.0)
        torch.cuda.synchronize()
        assert opt.steps_taken() == 3
        outs.append([t.clone().view(torch.uint8) for t in params + opt.weights + list(opt.buffers.values())])
    for other in outs[1:]:
        for a, b in zip(outs[0], other):
            assert torch.equal(a, b)
    if state == "e4m3":                                   # another seed rounds otherwise
        opt, params, grads = _clone_run(state, 8)
        for gs in grads:
            opt.step(gs, max_norm=1.0)
        assert not torch.equal(opt.buffers["m"].view(torch.uint8).cpu(),
                               outs[0][len(params) * 2].cpu())


@pytest.mark.parametrize("gdt", GRADS, ids=str)
def test_tensors_aligned_to_16_bytes_only(gdt):
    # 32-byte vectors need more than the 16 bytes that the call asks for: the same bits either way
    n, outs = 5003, []
    for shift in (0, 4):
        gen = torch.Generator().manual_seed(6)
        hold = torch.full((n + 16,), 9.0, device=DEV)
        p = hold[shift:shift + n]
        p.copy_(_rand(n, gen))
        gh = torch.full((n + 16,), 9.0, device=DEV, dtype=gdt)
        s = shift if gdt == torch.float32 else 2 * shift
        g = gh[s:s + n]
        g.copy_(_rand(n, gen, 1.0, gdt))
        opt = optim.AdamW([p], lr=1e-2, ema_decay=0.5)
        for _ in range(2):
            opt.step([g], max_norm=1.0)
        outs.append([p.clone(), opt.part("m", 0).clone(), opt.part("v", 0).clone(), opt.part("ema", 0).clone(), opt.grad_norm.clone()])
        assert bool((hold[shift + n:] == 9).all()) and bool((hold[:shift] == 9).all())
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_rate_factor_on_the_device():
    p = torch.ones(10, device=DEV)
    opt = optim.AdamW([p], lr=1.0, betas=(0.0, 0.0), eps=0.0)
    opt.lr_scale.fill_(0.125)
    opt.step([torch.full((10,), 3.0, device=DEV)])        # m / sqrt(v) = 1: the step is lr * 0.125
    assert float((p - 0.875).abs().max()) <= 8 * U
    opt.lr = 2.0
    opt.step([torch.full((10,), 3.0, device=DEV)])
    assert float((p - 0.625).abs().max()) <= 16 * U


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_state_dict_resumes(state):
    opt, params, grads = _clone_run(state, 3)
    opt.step(grads[0])
    saved, held = opt.state_dict(), [p.clone() for p in params]
    opt.step(grads[1])
    want = [p.clone() for p in params]
    other = optim.AdamW(held, lr=1e-2, state=state, ema_decay=0.9, seed=3)
    other.load_state_dict(saved)
    other.step(grads[1])
    # beta^1 by a product and by a power are the same numbers
    for a, b in zip(want, held):
        assert torch.equal(a, b)
    with pytest.raises(ValueError):
        other.load_state_dict({"step": 1})
    with pytest.raises(ValueError):
        other.load_state_dict(dict(saved, m=saved["m"][:-1]))


def test_python_refusals():
    p = torch.zeros(64, device=DEV)
    bad = [dict(params=[p.half()]), dict(params=[p[::2]]), dict(params=[p, p]), dict(params=[p[:40], p[32:]]),
           dict(params=[p], weights=[torch.zeros(63, dtype=torch.half, device=DEV)]), dict(params=[p], weights=[p.clone()]),
           dict(params=[p], state="int8"), dict(params=[p], betas=(1.0, 0.9)), dict(params=[p], weight_decay=[0.1, 0.2]),
           dict(params=[p], weights=[])]
    for kw in bad:
        with pytest.raises(ValueError):
            optim.AdamW(**kw, lr=1e-3)
    opt = optim.AdamW([p], lr=1e-3)
    for grads in ([], [p.double()], [torch.zeros(63, device=DEV)], [torch.zeros(64)], [torch.zeros(128, device=DEV)[::2]]):
        with pytest.raises(ValueError):
            opt.step(grads)
    with pytest.raises(Exception, match="aligned"):
        optim.AdamW([torch.zeros(65, device=DEV)[1:]], lr=1e-3).step([p])
    with pytest.raises(Exception, match="max_norm"):
        opt.step([p], max_norm=-1.0)
    assert opt.steps_taken() == 0


@pytest.mark.parametrize("n", [1184 * 2048, 1184 * 2048 + 1, 5_000_000])
def test_steps_are_counted_once_whatever_the_blocks(n):
    # up to 1184 blocks count the step themselves, more leave it to a kernel of its own
    p = torch.zeros(n, device=DEV)
    g = torch.ones(n, device=DEV)
    opt = optim.AdamW([p], lr=1.0, betas=(0.5, 0.5), eps=0.0)
    for t in range(1, 4):
        opt.step([g])                                     # m / c1 = sqrt(v / c2) = 1: every step moves by 1
        assert opt.steps_taken() == t
        assert float((p + t).abs().max()) <= t * 16 * U
    g[n - 1] = float("inf")
    opt.step([g], max_norm=1.0)
    assert opt.steps_taken() == 3 and int(opt.skipped) == 1 and float((p + 3).abs().max()) <= 48 * U


def test_offsets_beyond_32_bits():
    # 2^31 + 300 elements: byte offsets pass 2^33 in the master, element offsets 2^31
    n = 2 ** 31 + 300
    p = torch.zeros(n, device=DEV)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    at = torch.tensor([0, 2 ** 31 - 1, 2 ** 31, 2 ** 31 + 255, 2 ** 31 + 256, n - 1], device=DEV)
    g[at] = 2.0
    opt = optim.AdamW([p], lr=1.0, betas=(0.5, 0.5), eps=0.0625, state="e4m3")
    opt.step([g], max_norm=0.0)
    assert abs(float(opt.grad_norm) - 2 * 6 ** 0.5) <= 2 * U * 5
    # m / c1 = 2 and sqrt(v / c2) = 2: every touched parameter moves by 2 / 2.0625
    assert float((p[at] + 2 / 2.0625).abs().max()) <= 16 * U
    assert int(torch.count_nonzero(p)) == 6
    assert torch.count_nonzero(opt.buffers["m_scale"]) == 4


def test_a_layer_is_trained_by_its_own_step():
    # forward, backward, step: the layer's weights become the oracle's step of the gradients it returned
    w = I.small_workload(512, 128, 256, 4, 2, 1, "bf16", "topk", seed=5)
    inp = dict(I.make_inputs(w, bias_std=0.1), router_bias=np.linspace(-0.2, 0.2, 4).astype(np.float32))
    L, x = PA.run_layer(w, inp)
    opt = L.optimizer(lr=1e-3, weight_decay=0.1, state="f32")
    dout = torch.randn((w.T, w.D), generator=torch.Generator().manual_seed(1)).to(DEV, L.act_dtype)
    had = {n: _np(p).ravel() for n, p in zip(opt.grad_names, opt.params)}
    g = L.backward(x, dout)
    opt.step(g, max_norm=1.0)
    _, scale = O.grad_norm([_np(g[n]) for n in opt.grad_names], 1.0, 1.0)
    assert opt.grad_names[:5] == ["dwg", "dw1", "dw2", "dws1", "dws2"] and len(opt.grad_names) == 10
    for i, (n, p, wt) in enumerate(zip(opt.grad_names, opt.params, opt.weights)):
        z = np.zeros(p.numel())
        want, bound = _expect(had[n], _np(g[n]).ravel(), z, z, 1, scale, (1e-3, (0.9, 0.999), 1e-8), 0.1 if i < 5 else 0.0)
        _near(_np(p).ravel(), want[0], bound[0], n)
        assert wt is None or torch.equal(wt, p.to(wt.dtype))
    assert opt.params[5].data_ptr() == L.router_bias.data_ptr()      # fp32: its own master
    L.forward(x)                                                    # and the next forward runs on them
    L.check()


def test_a_captured_norm_keeps_its_scratch():
    # more tensors than one launch takes need more scratch; the graph's own must outlive that
    norm = optim.GradNorm(DEV)
    g = [torch.full((100,), 2.0, device=DEV)]
    norm(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm(g)
    held = list(norm._ws)
    many = [torch.ones(1, device=DEV) for _ in range(1200)]
    assert abs(float(norm(many)[0]) - 1200 ** 0.5) <= 1200 ** 0.5 * U
    assert len(norm._ws) == 2 and norm._ws[0] is held[0]
    graph.replay()
    torch.cuda.synchronize()
    assert float(norm.grad_norm) == 20.0


def test_the_step_count_waits_for_other_streams():
    p = torch.ones(1000, device=DEV)
    opt = optim.AdamW([p], lr=1e-3)
    g = torch.ones(1000, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)                     # some 10 ms
        opt.step([g])
    assert opt.steps_taken() == 1
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        opt.step([g])
    assert opt.state_dict()["step"] == 2


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_layers_optimizer_resumes_with_its_masters(dt):
    from sparse_moe_layer_03_b200.layer import LayerShape, MoELayer
    w = I.small_workload(64, 64, 128, 4, 2, 1, dt, "topk", seed=3)
    inp = I.make_inputs(w)
    make = lambda: MoELayer(LayerShape(w.T, w.D, w.H, w.E, w.K, w.n_shared, w.dtype, w.routing, w.alpha), inp)  # noqa: E731
    layer, gen = make(), torch.Generator().manual_seed(9)
    settings = dict(lr=1e-4, weight_decay=0.1, state="e4m3", ema_decay=0.9, seed=2)
    opt = layer.optimizer(**settings)
    grads = [{n: _rand(p.numel(), gen) for n, p in zip(opt.grad_names, opt.params)} for _ in range(2)]
    opt.step(grads[0])
    saved = opt.state_dict()
    opt.step(grads[1])
    again = make()
    other = again.optimizer(**settings)
    other.load_state_dict(saved)
    for p, wt in zip(other.params, other.weights):
        assert wt is None or torch.equal(p.to(wt.dtype), wt)
    other.step(grads[1])
    for a, b in zip(opt.params + [t for t in opt.weights if t is not None],
                    other.params + [t for t in other.weights if t is not None]):
        assert torch.equal(a, b)
    assert torch.equal(layer.w1, again.w1) and other.steps_taken() == 2
    for bad in (dict(saved, params=saved["params"][:-1]), {k: v for k, v in saved.items() if k != "params"},
                dict(saved, step=-1)):
        with pytest.raises(ValueError):
            other.load_state_dict(bad)
