"""What the training step's operators are measured on: cases, inputs, plain forms and 64-bit values.

The operators are the ones a DiT-MoE layer needs to be trained beyond its expert and router
gradients:

* ``balance``: the expert-level balance loss over packed sequences (images of one or of many
  lengths), with its per-sequence expert counts and its gradient, joined with the gates'
  gradient, through the softmax to the gate weight, the router bias and the tokens;
* ``norm``: the gradient norm over many tensors and the clip factor;
* ``adamw``: one AdamW step over many tensors (with clipping, 16-bit weight copies and the
  weights' moving average where the case asks for them), moments in 32 bits;
* ``adamw`` with ``state = "e4m3"``: the same with both moments in 8 bits.

``run`` with ``own`` false is the plain form: elementary torch operations in 32 bits (64 for the
long sums).  With ``own`` true it makes the framework's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
DEV = "cuda"
BLOCK = 256          # elements that share one scale of an 8-bit moment; tensors start on such blocks
E4M3_MAX = 448.0
MASK = 0xFFFFFFFF


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the smallest configured layer (fp32, two images of 256 tokens): latency
        dict(name="balance_s2_f32", kind="balance", T=512, D=384, E=8, K=2, dtype="f32", routing="topk", seqs=2,
             ragged=False, pad=0, dgate=True, grads=True, accumulate=True),
        # evaluation: loss and counts only, 16 experts, 64 images of 256 tokens
        dict(name="balance_s2_16e_loss", kind="balance", T=16384, D=384, E=16, K=2, dtype="bf16", routing="topk",
             seqs=64, ragged=False, pad=0, dgate=False, grads=False, accumulate=False),
        # the flagship layer's router gradient: 32 images of 1024 tokens, added to the experts' dx
        dict(name="balance_xl_bf16", kind="balance", T=32768, D=1152, E=8, K=2, dtype="bf16", routing="topk",
             seqs=32, ragged=False, pad=0, dgate=True, grads=True, accumulate=True),
        # images of many sizes packed into one call, some empty, padding behind the last
        dict(name="balance_b_f16_packed", kind="balance", T=10007, D=768, E=8, K=3, dtype="f16", routing="topk",
             seqs=53, ragged=True, pad=519, dgate=True, grads=True, accumulate=False),
        # Expert-Race routing: up to 16 experts for a token
        dict(name="balance_xl_race", kind="balance", T=32768, D=1152, E=16, K=2, dtype="bf16", routing="race",
             seqs=32, ragged=False, pad=0, dgate=True, grads=True, accumulate=True),
        # gradient norm of a small layer, and of the flagship layer
        dict(name="norm_s2", kind="norm", D=384, H=1536, E=8, shared=2, grad="f32", max_norm=1.0),
        dict(name="norm_xl", kind="norm", D=1152, H=4608, E=8, shared=2, grad="f32", max_norm=1.0),
        # a narrow test layer's tensors: little work, latency counts
        dict(name="adamw_small", kind="adamw", D=256, H=512, E=4, shared=1, grad="f32", weight="bf16", state="f32",
             ema=False, max_norm=0.0),
        # fp32 layer (the weights are the masters), bf16 gradients as an all-reduce in 16 bits leaves them
        dict(name="adamw_s2_f32", kind="adamw", D=384, H=1536, E=8, shared=2, grad="bf16", weight="none",
             state="f32", ema=False, max_norm=1.0),
        # the flagship layer's whole step: clip, update, bf16 copy, moving average
        dict(name="adamw_xl_ema", kind="adamw", D=1152, H=4608, E=8, shared=2, grad="f32", weight="bf16", state="f32",
             ema=True, max_norm=1.0),
        # 8-bit moments: a small 16-expert layer in fp16, and the flagship layer
        dict(name="adamw8_s2_16e", kind="adamw", D=384, H=1536, E=16, shared=2, grad="f32", weight="f16",
             state="e4m3", ema=False, max_norm=1.0),
        dict(name="adamw8_xl", kind="adamw", D=1152, H=4608, E=8, shared=2, grad="f32", weight="bf16", state="e4m3",
             ema=False, max_norm=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["balance", "balance", "balance", "norm", "adamw", "adamw", "adamw"])
    if kind == "balance":
        dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
        D = 64 * _log(rng, 1, 32)
        E = rng.randint(1, min(32, 51200 // D) if dtype == "f32" else 32)
        K = rng.randint(1, min(E, 6))
        T = min(_log(rng, 1, 32768), 32768 * 1152 // D)
        grads = rng.random() < 0.8
        pad = rng.choice([0, 0, rng.randint(0, T)])
        return dict(kind="balance", T=T, D=D, E=E, K=K, dtype=dtype, routing=rng.choice(["topk", "topk", "race"]),
                    seqs=_log(rng, 1, 400), ragged=True, pad=pad, dgate=grads and rng.random() < 0.8, grads=grads,
                    accumulate=grads and rng.random() < 0.5)
    D = rng.randint(3, 1152)
    E = rng.randint(1, 16)
    shared = rng.randint(0, 2)
    H = max(1, min(_log(rng, 16, 4608), 52_000_000 // (D * (E + shared))))
    case = dict(kind=kind, D=D, H=H, E=E, shared=shared, grad=rng.choice(["f32", "f32", "bf16", "f16"]),
                max_norm=rng.choice([1.0, 0.05, 30.0]))
    if kind == "adamw":
        state = rng.choice(["f32", "e4m3"])
        case.update(weight=rng.choice(["none", "bf16", "f16"]), state=state, ema=rng.random() < 0.4,
                    max_norm=rng.choice([0.0, 1.0, 0.05]))
    return case


# ---------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _offsets(case, seed):
    """[seqs + 1] borders of the packed sequences; the last `pad` rows belong to none."""
    T, B = case["T"], case["seqs"]
    if not case["ragged"]:
        return torch.arange(B + 1, dtype=torch.int32, device=DEV) * (T // B)
    end = T - case["pad"]
    cuts = torch.randint(0, end + 1, (B - 1,), generator=torch.Generator().manual_seed(int(seed) + 1))
    return torch.cat([torch.zeros(1, dtype=torch.int64), cuts.sort().values,
                      torch.tensor([end])]).to(torch.int32).to(DEV)


def _balance_inputs(case, seed):
    g = _gen(seed)
    T, D, E, K = case["T"], case["D"], case["E"], case["K"]
    dt = DTYPES[case["dtype"]]
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    x = rn(T, D).to(dt)
    wg = (rn(E, D) / math.sqrt(D)).to(dt)
    bias = rn(E) * math.sqrt(0.5)
    logits = x.float() @ wg.float().t() + bias
    if case["routing"] == "race":
        # the K * T largest scores of the whole matrix; each token's winners first, then -1
        P = torch.softmax(logits, 1)
        won = torch.zeros(T * E, dtype=torch.bool, device=DEV)
        won[P.reshape(-1).topk(K * T).indices] = True
        won = won.view(T, E)
        order = torch.where(won, P, -1.0).argsort(dim=1, descending=True)
        n_sel = won.sum(1).to(torch.int32)
        idx = torch.where(torch.arange(E, device=DEV)[None] < n_sel[:, None], order, -1).to(torch.int32)
    else:
        idx = logits.topk(K, dim=1).indices.to(torch.int32)
        n_sel = torch.full((T,), K, dtype=torch.int32, device=DEV)
    kmax = idx.shape[1]
    # gates' gradients <dout, e_i(x)>: zero mean, and 0 on unused slots, as the expert backward writes them
    dgate = rn(T, kmax) * 0.05 * (idx >= 0) if case["dgate"] else None
    dx = (rn(T, D) * 0.02).to(dt) if case["accumulate"] else torch.zeros((T, D), dtype=dt, device=DEV)
    s = dict(case=case, x=x, wg=wg, bias=bias, idx=idx.contiguous(), n_sel=n_sel, dgate=dgate, dx=dx,
             offsets=_offsets(case, seed))
    return s


def _sizes(case):
    """Elements of the layer's parameter tensors: gate, experts and shared experts, then the biases."""
    D, H, E, n = case["D"], case["H"], case["E"], case["shared"]
    mats = [E * H * D, E * D * H, E * D] + ([n * H * D, n * D * H] if n else [])
    vecs = [E * H, E * D, E] + ([n * H, n * D] if n else [])
    return mats, vecs


def _layout(case):
    mats, vecs = _sizes(case)
    at, spans = 0, []
    for n in mats + vecs:
        spans.append((at, n))
        at += -(-n // BLOCK) * BLOCK
    return spans, at, spans[len(mats)][0]


def _quantised(v):
    """Codes and scales of 8-bit moments: the nearest e4m3 values of v / scale, 256 elements to a scale."""
    b = v.view(-1, BLOCK)
    scale = b.abs().amax(1) / E4M3_MAX
    codes = (b / torch.where(scale > 0, scale, 1.0)[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes.view(-1), scale


def _flat_inputs(case, seed):
    g = _gen(seed)
    spans, total, vec_at = _layout(case)
    real = torch.zeros(total, device=DEV)
    for at, n in spans:
        real[at:at + n] = 1.0
    rn = lambda: torch.randn(total, generator=g, device=DEV)  # noqa: E731
    # gradients of a layer in training: zero mean, a scale that differs from row to row
    rows = torch.exp(torch.randn(total // BLOCK, generator=g, device=DEV)).repeat_interleave(BLOCK)
    grad = (rn() * rows * 1e-3 * real).to(DTYPES[case["grad"]])
    s = dict(case=case, grad=grad, spans=spans, total=total, vec_at=vec_at)
    if case["kind"] == "norm":
        return s
    s["master"] = rn() * 0.03 * real
    m = (0.4 * grad.float() + 0.3e-3 * rows * rn()) * real
    v = torch.square(rows * 1e-3) * (0.5 + torch.rand(total, generator=g, device=DEV)) * real
    if case["state"] == "f32":
        s.update(m=m, v=v)
    else:
        s["m"], s["m_scale"] = _quantised(m)
        s["v"], s["v_scale"] = _quantised(torch.sqrt(v))      # the root of the second moment is what is kept
    if case["weight"] != "none":
        s["weight"] = s["master"].to(DTYPES[case["weight"]])
    if case["ema"]:
        s["ema"] = s["master"] + 1e-4 * rn() * real
    s.update(step=1000, seed=int(seed) * 2654435761 % (1 << 63))
    return s


HYPER = dict(lr=1e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, ema_decay=0.9999)


def prepare(case, seed):
    if case["kind"] == "balance":
        s = _balance_inputs(case, seed)
        if own:
            _own_balance(s)
        return s
    s = _flat_inputs(case, seed)
    if own:
        _own_optimizer(s)
    return s


# ---------------------------------------------------------------------------------------- one pass
def run(state):
    kind = state["case"]["kind"]
    if own:
        return _run_own(state)
    if kind == "balance":
        return _plain_balance(state)
    if kind == "norm":
        return _plain_norm(state["grad"], state["case"]["max_norm"])
    return _plain_adamw(state)


def _plain_balance(s):
    c = s["case"]
    T, E, K, alpha, B = c["T"], c["E"], c["K"], 0.01, c["seqs"]
    x, wg, off = s["x"].float(), s["wg"].float(), s["offsets"].long()
    logits = x @ wg.t() + s["bias"]
    z = torch.exp(logits - logits.amax(1, keepdim=True))
    P = z / z.sum(1, keepdim=True)
    t = torch.arange(T, device=DEV)
    live = (t >= off[0]) & (t < off[-1])
    sid = (torch.searchsorted(off, t, right=True) - 1).clamp(0, B - 1)
    used = (torch.arange(s["idx"].shape[1], device=DEV)[None] < s["n_sel"][:, None]) & live[:, None]
    slot = s["idx"].long().clamp(min=0)
    taken = torch.zeros((T, E), device=DEV).scatter_add_(1, slot, used.float())
    counts = torch.zeros((B, E), device=DEV).index_add_(0, sid, taken)
    length = (off[1:] - off[:-1]).float()
    full = length > 0
    nb = full.sum().clamp(min=1).float()
    coef = torch.where(full, alpha * E / (K * torch.square(length.clamp(min=1))), 0.0)
    C = (counts * coef[:, None])[sid] * live[:, None]
    seq_loss = torch.zeros(B, dtype=torch.float64, device=DEV).index_add_(0, sid, (P * C).double().sum(1))
    out = dict(counts=counts.to(torch.int32), seq_loss=seq_loss.float(), loss=(seq_loss.sum() / nb).float().view(1))
    if not c["grads"]:
        return out
    dP = C / nb
    if s["dgate"] is not None:
        dP = dP + torch.zeros((T, E), device=DEV).scatter_add_(1, slot, torch.where(used, s["dgate"], 0.0))
    dl = P * (dP - (P * dP).sum(1, keepdim=True)) * live[:, None]
    dx = dl @ wg
    if c["accumulate"]:
        dx = s["dx"].float() + dx
    s["dx"] = torch.where(live[:, None], dx.to(s["dx"].dtype), s["dx"])
    out.update(dwg=dl.t() @ x, dbias=dl.double().sum(0).float(), dx=s["dx"])
    return out


def _plain_norm(grad, max_norm):
    norm = torch.sqrt(torch.square(grad.double()).sum())
    return dict(norm=norm.float().view(1), scale=(max_norm / (norm + 1e-6)).clamp(max=1.0).float().view(1))


# Odd multipliers: the fractions of the golden ratio's inverse and of the square roots of 2 and 3.
PHI32, RT2_32 = 0x9E3779B9, 0x6A09E667
PHI64, RT2_64, RT3_64 = 0x9E3779B97F4A7C15, 0x6A09E667F3BCC909, 0xBB67AE8584CAA73B


def _key(seed, step, k):
    """The key of a step's k-th tensor: below 2^63."""
    h = (seed + step * PHI64 + k * RT3_64) % (1 << 64)
    h = ((h ^ (h >> 29)) * RT2_64) % (1 << 64)
    return (h ^ (h >> 32)) >> 1


def _random_bits(s):
    """32 random bits for each element from its tensor's key and its place in the tensor: twice a
    32 x 32 -> 64 bit product, folded.  As 64-bit integers."""
    n = len(s["spans"])
    starts = torch.tensor([at for at, _ in s["spans"]], device=DEV)
    spans = torch.diff(starts, append=torch.tensor([s["total"]], device=DEV))
    keys = torch.tensor([_key(s["seed"], s["step"], k) for k in range(n)], device=DEV).repeat_interleave(spans)
    i = torch.arange(s["total"], device=DEV) - starts.repeat_interleave(spans)
    z = ((i + keys) & MASK) * PHI32
    z = ((z ^ (z >> 32) ^ (keys >> 32)) & MASK) * RT2_32
    return (z ^ (z >> 32)) & MASK


def _to_e4m3(x, r16):
    """|x| <= 448 rounded up or down to a neighbouring e4m3 value, up where 16 random bits fall below the rest."""
    a = x.abs()
    low = a < 2.0 ** -6
    bits = torch.where(low, a + 2.0 ** -6, a).view(torch.int32) + (r16 << 4)
    code = ((bits >> 20) - 960 - 8 * low.int()).clamp(max=126)
    return (code | torch.where(x < 0, 128, 0)).to(torch.uint8).view(torch.float8_e4m3fn)


def _store8(v, r16):
    b = v.view(-1, BLOCK)
    big = b.abs().amax(1)
    ok = big >= 2.0 ** -100
    inv = torch.where(ok, E4M3_MAX / big, 0.0)
    return _to_e4m3((b * inv[:, None]).view(-1), r16), torch.where(ok, big / E4M3_MAX, 0.0)


def _plain_adamw(s):
    c, h = s["case"], HYPER
    b1, b2 = h["betas"]
    s["step"] += 1
    out = {}
    g = s["grad"].float()
    if c["max_norm"] > 0:
        out = _plain_norm(s["grad"], c["max_norm"])
        g = g * out["scale"]
    q8 = c["state"] == "e4m3"
    if q8:
        spread = lambda codes, scale: (codes.float().view(-1, BLOCK) * scale[:, None]).view(-1)  # noqa: E731
        m, v = spread(s["m"], s["m_scale"]), torch.square(spread(s["v"], s["v_scale"]))
    else:
        m, v = s["m"], s["v"]
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * torch.square(g)
    root = torch.sqrt(v)
    p = s["master"]
    kept = torch.cat([p[:s["vec_at"]] * (1 - h["lr"] * h["weight_decay"]), p[s["vec_at"]:]])   # no decay on biases
    c1, c2 = 1 - b1 ** s["step"], 1 - b2 ** s["step"]
    p = kept - (h["lr"] / c1) * (m / (root * (1 / math.sqrt(c2)) + h["eps"]))
    if q8:
        r = _random_bits(s)
        s["m"], s["m_scale"] = _store8(m, (r & 0xFFFF).int())
        s["v"], s["v_scale"] = _store8(root, (r >> 16).int())
    else:
        s["m"], s["v"] = m, v
    s["master"] = p
    if "weight" in s:
        s["weight"] = p.to(s["weight"].dtype)
    if c["ema"]:
        s["ema"] = h["ema_decay"] * s["ema"] + (1 - h["ema_decay"]) * p
    out.update({k: s[k] for k in ("master", "weight", "m", "v", "m_scale", "v_scale", "ema") if k in s})
    return out


# ---------------------------------------------------------------------------------------- the framework's calls
def _own_balance(s):
    from sparse_moe_layer_03_b200 import binding as B
    c = s["case"]
    T, D, E, n = c["T"], c["D"], c["E"], c["seqs"]
    cfg = B.make_config(T, D, 64, E, c["K"], 0, c["dtype"], c["routing"], 0.01)
    nb = B.moe_seq_balance_workspace_size(cfg, n)
    f = lambda *z: torch.empty(z, device=DEV)  # noqa: E731
    s.update(B=B, cfg=cfg, bws=torch.empty(nb, dtype=torch.uint8, device=DEV), bws_bytes=nb,
             counts=torch.empty((n, E), dtype=torch.int32, device=DEV), seq_loss=f(n), loss=f(1),
             dwg=f(E, D) if c["grads"] else None, dbias=f(E) if c["grads"] else None,
             status=torch.zeros(256, dtype=torch.uint8, device=DEV))


def _own_optimizer(s):
    from sparse_moe_layer_03_b200 import optim
    c = s["case"]
    cut = lambda flat: [flat[at:at + n] for at, n in s["spans"]]  # noqa: E731
    s["grads"] = cut(s["grad"])
    if c["kind"] == "norm":
        s["norm"] = optim.GradNorm(DEV)
        return
    mats = sum(1 for at, _ in s["spans"] if at < s["vec_at"])
    decay = [HYPER["weight_decay"]] * mats + [0.0] * (len(s["spans"]) - mats)
    opt = optim.AdamW(cut(s["master"]), weights=cut(s["weight"]) if "weight" in s else None, lr=HYPER["lr"],
                      betas=HYPER["betas"], eps=HYPER["eps"], weight_decay=decay, state=c["state"],
                      ema_decay=HYPER["ema_decay"] if c["ema"] else None, seed=s["seed"])
    had = {k: s.pop(k) for k in ("m", "v", "m_scale", "v_scale", "ema") if k in s}
    opt.load_state_dict(dict(had, step=s["step"]))
    s["opt"] = opt


def _run_own(s):
    c = s["case"]
    if c["kind"] == "balance":
        s["B"].moe_seq_balance(s["cfg"], s["x"], s["wg"], s["bias"], s["offsets"], c["seqs"], s["idx"], s["n_sel"],
                               s["dgate"], 1.0, s["counts"], s["seq_loss"], s["loss"], s["dwg"], s["dbias"],
                               s["dx"] if c["grads"] else None, int(c["accumulate"]), s["bws"], s["bws_bytes"],
                               s["status"], torch.cuda.current_stream().cuda_stream)
        out = dict(counts=s["counts"], seq_loss=s["seq_loss"], loss=s["loss"])
        if c["grads"]:
            out.update(dwg=s["dwg"], dbias=s["dbias"], dx=s["dx"])
        return out
    if c["kind"] == "norm":
        norm, scale = s["norm"](s["grads"], max_norm=c["max_norm"])
        return dict(norm=norm, scale=scale)
    opt = s["opt"]
    opt.step(s["grads"], max_norm=c["max_norm"] if c["max_norm"] > 0 else None)
    out = dict(master=s["master"], **opt.buffers)
    if "weight" in s:
        out["weight"] = s["weight"]
    if c["max_norm"] > 0:
        out.update(norm=opt.grad_norm, scale=opt.grad_scale)
    return out


# ---------------------------------------------------------------------------------------- work
def work(case):
    if case["kind"] == "balance":
        T, D, E = case["T"], case["D"], case["E"]
        eb = 4 if case["dtype"] == "f32" else 2
        kmax = E if case["routing"] == "race" else case["K"]
        slots = case["K"] * T                       # selected pairs; unused slots of a race are not needed
        nbytes = T * D * eb + E * D * eb + slots * 4 + (T * 4 if kmax != case["K"] else 0) + case["seqs"] * (E + 2) * 4
        products = 1
        if case["grads"]:
            nbytes += T * D * eb * (2 if case["accumulate"] else 1) + E * D * 4
            nbytes += slots * 4 if case["dgate"] else 0
            products = 3                            # logits, dx and dWg
        return {"bytes": nbytes, "flops": 2 * products * T * D * E}
    mats, vecs = _sizes(case)
    n = sum(mats) + sum(vecs)
    gb = 4 if case["grad"] == "f32" else 2
    if case["kind"] == "norm":
        return {"bytes": n * gb, "flops": 2 * n}
    per = gb + 8 + (16 if case["state"] == "f32" else 4 + 16 / BLOCK) + (8 if case["ema"] else 0)
    per += 2 if case["weight"] != "none" else 0
    return {"bytes": int(n * per), "flops": n * (16 if case["state"] == "f32" else 40)}


# ---------------------------------------------------------------------------------------- 64-bit values
def exact(case, seed):
    if case["kind"] == "balance":
        return _exact_balance(_balance_inputs(case, seed))
    s = _flat_inputs(case, seed)
    g = s["grad"].to(torch.float64)
    norm = g.pow(2).sum().sqrt()
    scale = min(1.0, case["max_norm"] / (float(norm) + 1e-6)) if case["max_norm"] > 0 else 1.0
    clip = dict(norm=norm.view(1), scale=torch.full((1,), scale, dtype=torch.float64))
    if case["kind"] == "norm":
        return clip
    lr, (b1, b2), eps = HYPER["lr"], HYPER["betas"], HYPER["eps"]
    t = s["step"] + 1
    g *= scale
    if case["state"] == "f32":
        m, v = s["m"].double(), s["v"].double()
    else:
        m = s["m"].double() * s["m_scale"].double().repeat_interleave(BLOCK)
        v = (s["v"].double() * s["v_scale"].double().repeat_interleave(BLOCK)).pow(2)
    m = m + (1 - b1) * (g - m)
    v = v + (1 - b2) * (g.pow(2) - v)
    del g
    p = s["master"].double()
    p[:s["vec_at"]] -= lr * HYPER["weight_decay"] * p[:s["vec_at"]]
    p -= lr * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + eps)
    out = dict(master=p)
    if case["state"] == "f32":
        out.update(m=m, v=v)
    else:
        s["step"] = t
        rnd = _random_bits(s)
        for name, val, r in (("m", m, rnd & 0xFFFF), ("v", v.sqrt(), rnd >> 16)):
            top = val.view(-1, BLOCK).abs().amax(1)
            inv = torch.where(top > 0, E4M3_MAX / top, 0.0).repeat_interleave(BLOCK)
            a = val.abs() * inv
            # spacing of the e4m3 values around a: 2^-9 below 2^-6, an eighth of the binade above
            ulp = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
            out[name] = torch.floor(a / ulp + r.double() / 65536).mul(ulp).clamp(max=E4M3_MAX) * torch.sign(val)
            out[name + "_scale"] = top / E4M3_MAX
    if "weight" in s:
        out["weight"] = p
    if case["ema"]:
        out["ema"] = HYPER["ema_decay"] * s["ema"].double() + (1 - HYPER["ema_decay"]) * p
    if case["max_norm"] > 0:
        out.update(clip)
    return out


def _exact_balance(s):
    c = s["case"]
    T, E, K, B = c["T"], c["E"], c["K"], c["seqs"]
    x, wg = s["x"].double(), s["wg"].double()
    P = torch.softmax(x @ wg.t() + s["bias"].double(), 1)
    off = s["offsets"].tolist()
    full = sum(1 for a, b in zip(off, off[1:]) if b > a)
    slots = torch.arange(s["idx"].shape[1], device=DEV)[None] < s["n_sel"][:, None]
    sel = torch.zeros((T, E + 1), dtype=torch.float64, device=DEV)
    sel.scatter_(1, torch.where(slots, s["idx"].long(), E), 1.0)
    sel = sel[:, :E]
    counts = torch.zeros((B, E), dtype=torch.float64, device=DEV)
    seq_loss = torch.zeros(B, dtype=torch.float64, device=DEV)
    dP = torch.zeros((T, E), dtype=torch.float64, device=DEV)
    for b, (lo, hi) in enumerate(zip(off, off[1:])):
        if hi > lo:
            n = hi - lo
            counts[b] = sel[lo:hi].sum(0)
            f = E * counts[b] / (K * n)
            seq_loss[b] = 0.01 * (f * P[lo:hi].mean(0)).sum()
            dP[lo:hi] = 0.01 * f / n / full
    out = dict(counts=counts.to(torch.int32), seq_loss=seq_loss, loss=(seq_loss.sum() / max(full, 1)).view(1))
    if not c["grads"]:
        return out
    if s["dgate"] is not None:
        up = torch.zeros((T, E + 1), dtype=torch.float64, device=DEV)
        up.scatter_(1, torch.where(slots, s["idx"].long(), E), s["dgate"].double())
        dP += up[:, :E]
    dl = P * dP - P * (P * dP).sum(1, keepdim=True)
    dl[:off[0]] = 0
    dl[off[-1]:] = 0
    dx = dl @ wg + (s["dx"].double() if c["accumulate"] else 0)
    dx[:off[0]] = s["dx"][:off[0]].double()
    dx[off[-1]:] = s["dx"][off[-1]:].double()
    out.update(dwg=dl.t() @ x, dbias=dl.sum(0), dx=dx)
    return out
