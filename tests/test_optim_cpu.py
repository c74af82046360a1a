"""The optimizer without a GPU: the oracle's AdamW against torch's, the rounding's random bits,
and the calls that the library refuses before it launches anything."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from sparse_moe_layer_03_b200 import binding as B

FAKE = 1 << 40          # never dereferenced: validation fails first


def test_oracle_adamw_matches_torch():
    g = torch.Generator().manual_seed(3)
    p0 = torch.randn(37, 5, generator=g, dtype=torch.float64)
    p = torch.nn.Parameter(p0.clone())
    opt = torch.optim.AdamW([p], lr=3e-3, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    q, m, v = p0.numpy(), np.zeros((37, 5)), np.zeros((37, 5))
    for t in range(1, 6):
        grad = torch.randn(37, 5, generator=g, dtype=torch.float64)
        p.grad = grad
        opt.step()
        q, m, v = O.adamw(q, grad.numpy(), m, v, t, 3e-3, (0.8, 0.95), 1e-6, 0.1)
        np.testing.assert_allclose(q, p.detach().numpy(), rtol=1e-12, atol=1e-14)


def test_oracle_norm_matches_torch():
    g = torch.Generator().manual_seed(4)
    ts = [torch.randn(n, generator=g, dtype=torch.float64) for n in (1, 50, 333)]
    ps = [torch.nn.Parameter(torch.zeros_like(t)) for t in ts]
    for p, t in zip(ps, ts):
        p.grad = t.clone()
    norm, f = O.grad_norm([t.numpy() for t in ts], 1.0, 2.5)
    got = torch.nn.utils.clip_grad_norm_(ps, 2.5)
    assert abs(norm - float(got)) <= 1e-12 * norm
    np.testing.assert_allclose(ps[2].grad.numpy(), f * ts[2].numpy(), rtol=1e-12)
    assert O.grad_norm([np.ones(4)], 1.0, 100.0)[1] == 1.0 and O.grad_norm([np.ones(4)], 0.5, 0.0) == (1.0, 0.5)


@pytest.mark.parametrize("seed,step,tensor", [(0, 1, 0), (1, 1, 0), (0, 2, 0), (0, 1, 1), (2 ** 63 + 5, 10 ** 6, 300)])
def test_rounding_bits_are_uniform_and_uncorrelated(seed, step, tensor):
    n = 1 << 18
    r = O.rounding_bits(seed, step, tensor, n)
    # each of the 32 bits, and each half's mean: five standard deviations
    bits = (r[:, None] >> np.arange(32, dtype=np.uint32)) & 1
    assert np.all(np.abs(bits.mean(0) - 0.5) < 5 * 0.5 / np.sqrt(n))
    lo, hi = (r & 0xFFFF) / 65536.0, (r >> 16) / 65536.0
    sd = np.sqrt(1 / 12.0)
    for u in (lo, hi):
        assert abs(u.mean() - 0.5 + 0.5 / 65536) < 5 * sd / np.sqrt(n)
        for lag in (1, 2, 4, 128, 256):              # neighbours in a lane, a warp, a block
            c = np.mean((u[:-lag] - 0.5) * (u[lag:] - 0.5)) * 12
            assert abs(c) < 5 / np.sqrt(n - lag)
    assert abs(np.mean((lo - 0.5) * (hi - 0.5)) * 12) < 5 / np.sqrt(n)
    other = O.rounding_bits(seed, step + 1, tensor, n)  # the next step's are others
    assert np.mean(other == r) < 1e-3
    assert abs(np.mean(((other & 0xFFFF) / 65536.0 - 0.5) * (lo - 0.5)) * 12) < 5 / np.sqrt(n)


def test_random_rounding_is_right_on_average():
    # values between two codes, over the normal and the subnormal codes
    for a in (0.0, 1e-4, 2.0 ** -9 * 0.3, 2.0 ** -9 * 5.75, 2.0 ** -6 * 0.999, 0.0501, 1.0, 1.03, 17.2, 447.0, 448.0):
        r = O.rounding_bits(7, 3, 1, 1 << 16) & 0xFFFF
        val, _ = O.e4m3_round(np.full(1 << 16, a), r)
        codes = torch.tensor(val).to(torch.float8_e4m3fn).double().numpy()
        assert np.array_equal(codes, val)                # every result is an e4m3 value
        gap = max(2.0 ** -9, 2.0 ** (np.floor(np.log2(max(a, 2.0 ** -6))) - 3))
        assert np.all(np.abs(val - a) < gap + 1e-12)
        assert abs(val.mean() - a) < gap * (5 * 0.5 / 256 + 1 / 65536)


def _tensor(**kw):
    t = B.MoeAdamwTensor(FAKE, FAKE, None, FAKE, FAKE, None, None, None, 100, 0.0, B.MOE_F32, 0, 0)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def _step(t, n=1, ctl=FAKE, **kw):
    h = B.MoeAdamw(1e-3, 0.9, 0.999, 1e-8, 0.5, 1.0, 0, B.MOE_MOMENTS_F32, 0)
    for k, v in kw.items():
        setattr(h, k, v)
    return B.lib.moe_adamw_step(ctypes.byref(h), ctypes.byref(t) if t is not None else None, n, ctl, None)


@pytest.mark.parametrize("kw,word", [
    (dict(param=None), b"param"), (dict(param=FAKE + 4), b"aligned"), (dict(grad=None), b"grad"),
    (dict(grad=FAKE + 2), b"aligned"), (dict(m=None), b"m or v"), (dict(v=FAKE + 8), b"aligned"),
    (dict(weight=FAKE, weight_dtype=B.MOE_F32), b"weight_dtype"), (dict(weight=FAKE + 2, weight_dtype=1), b"aligned"),
    (dict(ema=FAKE + 4), b"aligned"), (dict(n=-1), b"n=-1"), (dict(grad_dtype=3), b"grad_dtype"),
    (dict(weight_decay=float("nan")), b"weight_decay"),
])
def test_adamw_refuses_bad_tensors(kw, word):
    assert _step(_tensor(**kw)) == B.MOE_ERR_INVALID_ARG
    assert word in B.lib.moe_last_error()


@pytest.mark.parametrize("kw,word", [
    (dict(beta1=1.0), b"beta1"), (dict(beta2=-0.1), b"beta2"), (dict(eps=-1.0), b"eps"), (dict(lr=float("inf")), b"lr"),
    (dict(state=2), b"state"), (dict(grad_mult=float("nan")), b"grad_mult"), (dict(state=1), b"m_scale"),
])
def test_adamw_refuses_bad_settings(kw, word):
    assert _step(_tensor(), **kw) == B.MOE_ERR_INVALID_ARG
    assert word in B.lib.moe_last_error()


def test_adamw_refuses_the_rest():
    assert _step(None) == B.MOE_ERR_INVALID_ARG and b"tensors" in B.lib.moe_last_error()
    assert _step(_tensor(), n=-1) == B.MOE_ERR_INVALID_ARG
    assert _step(_tensor(), ctl=None) == B.MOE_ERR_INVALID_ARG and b"ctl" in B.lib.moe_last_error()
    assert _step(_tensor(), ctl=FAKE + 16) == B.MOE_ERR_INVALID_ARG and b"256-byte" in B.lib.moe_last_error()
    assert _step(_tensor(ema=FAKE), ema_decay=1.5) == B.MOE_ERR_INVALID_ARG and b"ema_decay" in B.lib.moe_last_error()
    assert _step(_tensor(n=(1 << 40) + 1)) == B.MOE_ERR_UNSUPPORTED
    t = _tensor()
    assert B.lib.moe_adamw_step(None, ctypes.byref(t), 1, FAKE, None) == B.MOE_ERR_INVALID_ARG


def test_grad_norm_refusals():
    n = B.moe_grad_norm_workspace_size(1)
    assert n > 0 and B.moe_grad_norm_workspace_size(5000) > n
    with pytest.raises(B.MoeError):
        B.moe_grad_norm_workspace_size(-1)
    t = _tensor()

    def call(t=t, k=1, mult=1.0, most=1.0, ctl=FAKE, ws=FAKE, nb=n):
        return B.lib.moe_grad_norm(ctypes.byref(t), k, mult, most, ctl, ws, nb, None)
    assert call(nb=n - 1) == B.MOE_ERR_WORKSPACE
    for kw, word in [(dict(mult=0.0), b"grad_mult"), (dict(mult=float("inf")), b"grad_mult"), (dict(most=-1.0), b"max_norm"),
                     (dict(most=float("nan")), b"max_norm"), (dict(ws=None), b"ws"), (dict(ws=FAKE + 8), b"ws"),
                     (dict(ctl=None), b"ctl"), (dict(k=-1), b"n_tensors"), (dict(t=_tensor(grad=None)), b"grad"),
                     (dict(t=_tensor(grad_dtype=9)), b"grad_dtype")]:
        assert call(**kw) == B.MOE_ERR_INVALID_ARG, kw
        assert word in B.lib.moe_last_error(), kw


def test_optim_init_refusals():
    for args, word in [((None, 0, 0.9, 0.9), b"ctl"), ((FAKE, -1, 0.9, 0.9), b"step"), ((FAKE, 0, 1.0, 0.9), b"beta1"),
                       ((FAKE, 0, 0.9, float("nan")), b"beta2")]:
        assert B.lib.moe_optim_init(*args, None) == B.MOE_ERR_INVALID_ARG
        assert word in B.lib.moe_last_error()


def test_python_checks_without_a_gpu():
    from sparse_moe_layer_03_b200 import optim
    with pytest.raises(ValueError, match="CUDA"):
        optim.AdamW([torch.zeros(4)], lr=1e-3)
    with pytest.raises(ValueError, match="CUDA"):
        optim.AdamW([], lr=1e-3)
