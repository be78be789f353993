"""The operators of a training step around the BitLinear layers, as a program calls them, with their plain forms.

Four operators: the embedding lookup with scaling that makes the first layer's x, its gradient from the layers' dx,
the gradient of the MLGRU recurrence, and the AdamW step over many tensors at once (states in 32 or in 8 bits).
``own`` chooses between elementary torch operations and the library's kernels; both take what ``prepare`` gives.

Widths and batch shapes follow the workloads of the 1.3B and 2.7B widths (2048/5632 and 2560/6912, sequences of 2048
tokens); vocabularies are generic.
"""
import math
import random

import torch

own = False

BLOCK = 256  # elements that share the scales of 8-bit states
_GOLDEN = 0x9E3779B97F4A7C15
_M1 = 0xBF58476D1CE4E5B9
_M2 = 0x94D049BB133111EB
_MASK64 = (1 << 64) - 1


# -- cases -----------------------------------------------------------------------


def listed():
    return [
        # a token just drawn: one row, where only latency counts
        {"name": "lookup-1", "op": "lookup", "M": 1, "K": 2560, "V": 32000, "table": "bf16", "ids": 32, "padded": 0},
        # a prefill of 8192 tokens from the fp32 master table, the last 100 places of the batch padded
        {"name": "lookup-8192-fp32", "op": "lookup", "M": 8192, "K": 2560, "V": 32000, "table": "fp32", "ids": 64, "padded": 100},
        # a quarter of the training batch from the bf16 copy of the table
        {"name": "lookup-131072-bf16", "op": "lookup", "M": 131072, "K": 2048, "V": 50257, "table": "bf16", "ids": 64, "padded": 0},
        # one more short micro-batch added to a gradient that is there already
        {"name": "lookup-grad-511-add", "op": "lookup_grad", "M": 511, "K": 1024, "V": 32000, "ids": 32, "padded": 0, "add": True},
        # a batch of 4 x 2048 tokens, padded at its end
        {"name": "lookup-grad-8192", "op": "lookup_grad", "M": 8192, "K": 2560, "V": 32000, "ids": 64, "padded": 100, "add": False},
        # a quarter of the training batch: the most frequent words have thousands of tokens each
        {"name": "lookup-grad-131072", "op": "lookup_grad", "M": 131072, "K": 2048, "V": 50257, "ids": 64, "padded": 0, "add": False},
        # a short sequence of odd length and width
        {"name": "scan-grad-1x37x1022", "op": "scan_grad", "B": 1, "T": 37, "D": 1022, "carry": True},
        # the recurrence workload: 4 sequences of 2048 tokens at the 1.3B width
        {"name": "scan-grad-4x2048x2048", "op": "scan_grad", "B": 4, "T": 2048, "D": 2048, "carry": False},
        # a larger batch whose sequences go on from an earlier call and into a later one
        {"name": "scan-grad-16x2048x2048", "op": "scan_grad", "B": 16, "T": 2048, "D": 2048, "carry": True},
        # 24 small tensors of ragged sizes, every other one with 8-bit states: launches count
        {"name": "adamw-ragged-24", "op": "adamw", "tensors": "ragged", "count": 24, "most": 70000, "sizes_seed": 3, "bits": 0, "grad": "fp32", "copy": False},
        # one layer set of the 1.3B width with its gains, 32-bit states
        {"name": "adamw-32bit-1.3b", "op": "adamw", "tensors": "layers", "d": 2048, "f": 5632, "layers": 1, "bits": 32, "grad": "fp32", "copy": False},
        # two layer sets of the 2.7B width, 8-bit states, gradients reduced in bf16, the bf16 copy written too
        {"name": "adamw-8bit-2.7b", "op": "adamw", "tensors": "layers", "d": 2560, "f": 6912, "layers": 2, "bits": 8, "grad": "bf16", "copy": True},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("lookup", "lookup_grad", "scan_grad", "adamw"))
    if op in ("lookup", "lookup_grad"):
        K = 8 * _log(rng, 8, 320)
        M = _log(rng, 1, min(131072, 131072 * 2048 // K))
        case = {"op": op, "M": M, "K": K, "V": _log(rng, 1000, 50257), "ids": rng.choice((32, 64)), "padded": rng.choice((0, M // 9))}
        if op == "lookup":
            return dict(case, table=rng.choice(("fp32", "bf16")))
        return dict(case, add=rng.random() < 0.5)
    if op == "scan_grad":
        B, T = _log(rng, 1, 16), _log(rng, 1, 4096)
        return {"op": op, "B": B, "T": T, "D": 2 * _log(rng, 1, min(1280, 8 * 2048 * 2048 // (B * T))), "carry": rng.random() < 0.5}
    case = {"op": op, "bits": rng.choice((32, 8)), "grad": rng.choice(("fp32", "bf16")), "copy": rng.random() < 0.3}
    if rng.random() < 0.5:
        return dict(case, tensors="ragged", count=rng.randint(1, 40), most=_log(rng, 100, 2000000), sizes_seed=rng.randrange(1 << 20))
    d = 8 * _log(rng, 16, 224)
    return dict(case, tensors="layers", d=d, f=8 * ((d * 11 // 4 + 4) // 8), layers=rng.randint(1, 2))


def _sizes(case):
    """Elements of each tensor of an AdamW case: a layer set has four d x d matrices, gate, up and down, and their gains."""
    if case["tensors"] == "ragged":
        r = random.Random(case["sizes_seed"])
        return [_log(r, 1, case["most"]) for _ in range(case["count"])]
    d, f = case["d"], case["f"]
    return ([d * d] * 4 + [d * f] * 3 + [d, d, d, f]) * case["layers"]


def _bits(case, i):
    """The bits of tensor i's states; gains keep 32, they are few and small."""
    if case["tensors"] == "layers" and i % 11 > 6:
        return 32
    return case["bits"] or (32, 8)[i % 2]


# -- inputs ----------------------------------------------------------------------


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _ids(case, gen):
    """Words by Zipf's law, the frequent ones anywhere in the table; a padded place holds -1."""
    M, V = case["M"], case["V"]
    u = torch.rand(M, generator=gen, device="cuda", dtype=torch.float64)
    rank = (10.0 * torch.expm1(u * math.log1p(V / 10.0))).long().clamp(max=V - 1)  # rank r with weight log((r + 11) / (r + 10))
    ids = torch.randperm(V, generator=gen, device="cuda")[rank]
    ids[M - case["padded"]:] = -1
    return ids.to(torch.int32 if case["ids"] == 32 else torch.int64)


def _power(values, low):
    """The exponent e of each block's largest value, 2^e <= largest < 2^(e+1), and 2^(e - low) as fp32."""
    e = torch.frexp(values.abs().amax(1))[1] - 1
    e = torch.where(values.abs().amax(1) > 0, e, -90).clamp(min=-90)
    return e, ((127 + e - low) << 23).to(torch.int32).view(torch.float32)


def _prepare_adamw(case, gen, seed):
    sizes = _sizes(case)
    state = {"op": "adamw", "tensors": [], "outputs": {}, "step": 1000, "lr": 3e-4, "beta1": 0.9, "beta2": 0.95,
             "eps": 1e-8, "grad_scale": 0.5, "seed": seed}
    for bits in (32, 8):
        mine = [i for i in range(len(sizes)) if _bits(case, i) == bits]
        if not mine:
            continue
        # all tensors of a kind in one allocation each, at places that are multiples of four blocks
        starts, total = {}, 0
        for i in mine:
            starts[i] = total
            total += -(-sizes[i] // (4 * BLOCK)) * 4 * BLOCK  # scales start on 16 bytes
        inside = torch.zeros(total, device="cuda")
        for i in mine:
            inside[starts[i]:starts[i] + sizes[i]] = 1.0
        flat = {"p": 0.02 * _normal(gen, total) * inside,
                "g": (2e-3 * _normal(gen, total) * inside).to(torch.bfloat16 if case["grad"] == "bf16" else torch.float32)}
        m, v = 3e-4 * _normal(gen, total) * inside, (1e-3 * _normal(gen, total)).square() * inside
        if bits == 8:
            em, flat["m_scale"] = _power(m.view(-1, BLOCK), 7)
            ev, flat["v_scale"] = _power(v.view(-1, BLOCK), 14)
            m = m.view(-1, BLOCK) / flat["m_scale"][:, None]
            v = v.view(-1, BLOCK) / flat["v_scale"][:, None]
            flat["m"] = torch.where(m.abs() < 2.0**-6, 0.0, m).reshape(-1).to(torch.float8_e4m3fn)
            flat["v"] = torch.where(v > 0, v.clamp(min=2.0**-14), v).reshape(-1).to(torch.float8_e5m2)
        else:
            flat["m"], flat["v"] = m, v
        if case["copy"]:
            flat["p_bf16"] = flat["p"].to(torch.bfloat16)
        for i in mine:
            a, n = starts[i], sizes[i]
            t = {k: x[a // BLOCK:a // BLOCK - (-n // BLOCK)] if k.endswith("scale") else x[a:a + n] for k, x in flat.items()}
            t["weight_decay"] = 0.1 if case["tensors"] == "ragged" or i % 11 <= 6 else 0.0
            state["tensors"].append((i, t))
        state["outputs"].update({"%s_%d" % (k, bits): x for k, x in flat.items() if k != "g"})
    state["tensors"] = [t for _, t in sorted(state["tensors"], key=lambda x: x[0])]
    return state


def prepare(case, seed):
    gen = _generator(seed)
    op = case["op"]
    if op == "adamw":
        return _prepare_adamw(case, gen, seed)
    if op == "scan_grad":
        shape = (case["B"], case["T"], case["D"])
        state = {"op": op, "f": (_normal(gen, *shape) + 0.5).to(torch.bfloat16), "c": _normal(gen, *shape).to(torch.bfloat16),
                 "g": _normal(gen, *shape).to(torch.bfloat16), "do": (1e-2 * _normal(gen, *shape)).to(torch.bfloat16),
                 "h0": None, "dh_last": None}
        if case["carry"]:
            state["h0"] = 0.5 * _normal(gen, shape[0], shape[2])
            state["dh_last"] = 1e-2 * _normal(gen, shape[0], shape[2])
        return state
    state = {"op": op, "ids": _ids(case, gen), "scale": math.sqrt(case["K"]), "V": case["V"]}
    if op == "lookup":
        table = 0.02 * _normal(gen, case["V"], case["K"])
        state["table"] = table.to(torch.bfloat16) if case["table"] == "bf16" else table
    else:
        state["dx"] = (1e-2 * _normal(gen, case["M"], case["K"])).to(torch.bfloat16)
        state["dtable"] = 1e-2 * _normal(gen, case["V"], case["K"]) if case["add"] else None
    return state


# -- plain forms -----------------------------------------------------------------


def _lookup_plain(s):
    there = (s["ids"] >= 0) & (s["ids"] < s["V"])
    rows = s["table"][torch.where(there, s["ids"], 0).long()].float() * s["scale"]
    return torch.where(there[:, None], rows, 0.0).to(torch.bfloat16)


def _lookup_grad_plain(s):
    there = (s["ids"] >= 0) & (s["ids"] < s["V"])
    rows = torch.where(there[:, None], s["dx"].float() * s["scale"], 0.0)
    out = s["dtable"] if s["dtable"] is not None else torch.zeros(s["V"], rows.shape[1], device=rows.device)
    return out.index_add_(0, torch.where(there, s["ids"], 0).long(), rows)


def _recurrence(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from h = 0: pairs of steps are one step, so half the length gives every other h."""
    T = b.shape[1]
    if T == 1:
        return b
    n = T // 2
    a2 = a[:, 1::2] * a[:, 0:2 * n:2]
    b2 = a[:, 1::2] * b[:, 0:2 * n:2] + b[:, 1::2]
    odd = _recurrence(a2, b2)
    h = torch.empty_like(b)
    h[:, 1::2] = odd
    h[:, 0] = b[:, 0]
    h[:, 2::2] = a[:, 2::2] * odd[:, :(T - 1) // 2] + b[:, 2::2]
    return h


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _scan_grad_plain(s):
    fp, cp, gp, do = (s[k].float() for k in ("f", "c", "g", "do"))
    f, keep, sc, g = _sigmoid(fp), _sigmoid(-fp), _sigmoid(cp), _sigmoid(gp)  # keep = 1 - f
    c = cp * sc
    first = torch.zeros_like(c[:, 0]) if s["h0"] is None else s["h0"]
    b = keep * c
    b[:, 0] += f[:, 0] * first
    h = _recurrence(f, b)
    before = torch.cat((first[:, None], h[:, :-1]), 1)
    b = do * g
    if s["dh_last"] is not None:
        b[:, -1] += s["dh_last"]
    a = torch.cat((f[:, 1:], torch.ones_like(f[:, :1])), 1)
    dh = _recurrence(a.flip(1), b.flip(1)).flip(1)
    df = dh * (before - c) * f * keep
    dc = dh * keep * sc * (1.0 + cp * (1.0 - sc))
    dg = do * h * g * (1.0 - g)
    return [df.to(torch.bfloat16), dc.to(torch.bfloat16), dg.to(torch.bfloat16), f[:, 0] * dh[:, 0]]


def _signed(v):
    return v - (1 << 64) if v >= (1 << 63) else v


def _shift(z, s):
    return (z >> s) & ((1 << (64 - s)) - 1)


def _key(seed, stream):
    z = ((seed << 32) + stream) & _MASK64
    z = ((z ^ (z >> 30)) * _M1) & _MASK64
    z = ((z ^ (z >> 27)) * _M2) & _MASK64
    return z ^ (z >> 31)


def _noise(seed, ordinal, n, device):
    """16 random bits for m and 16 for v of each element: draw j of the SplitMix64 stream (seed, ordinal) serves elements 2j, 2j + 1."""
    z = torch.arange(1, (n + 1) // 2 + 1, dtype=torch.int64, device=device) * _signed(_GOLDEN) + _signed(_key(seed, ordinal))
    z = (z ^ _shift(z, 30)) * _signed(_M1)
    z = (z ^ _shift(z, 27)) * _signed(_M2)
    z = z ^ _shift(z, 31)
    z = torch.stack((z, _shift(z, 32)), 1).view(-1)[:n]
    return (z & 0xFFFF).int(), ((z >> 16) & 0xFFFF).int()


def _blocks(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).view(-1, BLOCK)


def _encode(x, noise, low, drop, kind):
    """8-bit codes of x and their blocks' scales: 2^(e - low) for a largest value in [2^e, 2^(e+1)), rounded up or down by the noise."""
    x, n = _blocks(x), x.numel()
    top = (x.view(torch.int32) & 0x7FFFFFFF).amax(1)
    lost = top >= 0x7F000000  # 2^127 and more, infinities, NaN
    e = ((top >> 23) - 127).clamp(min=-90)
    scale = torch.where(lost, torch.nan, ((127 + e - low) << 23).view(torch.float32))
    y = (x * ((127 + low - e) << 23).view(torch.float32)[:, None]).view(torch.int32)
    least = 8 if drop == 20 else 4  # the smallest normal number's code
    c = (((y & 0x7FFFFFFF) + (_blocks(noise) << (drop - 16)) + (1 << (drop - 17))) >> drop) - (960 if drop == 20 else 448)
    c = torch.where(c < least, 0, c) if drop == 20 else torch.where(x > 0, c.clamp(min=least), 0)
    c = torch.where(lost[:, None], 0, c | (torch.where(y < 0, 128, 0) if drop == 20 else 0))
    return c.to(torch.uint8).view(-1)[:n].view(kind), scale


def _decode(codes, scale):
    return (_blocks(codes.float()) * scale[:, None]).view(-1)[:codes.numel()]


def _adamw_plain(s, ordinal, t):
    g = t["g"].float() * s["grad_scale"]
    eight = "m_scale" in t
    m = _decode(t["m"], t["m_scale"]) if eight else t["m"]
    v = _decode(t["v"], t["v_scale"]) if eight else t["v"]
    m = m * s["beta1"] + g * (1.0 - s["beta1"])
    v = v * s["beta2"] + (g * g) * (1.0 - s["beta2"])
    root = torch.sqrt(v) * (1.0 / math.sqrt(1.0 - s["beta2"] ** s["step"])) + s["eps"]
    p = t["p"] * (1.0 - s["lr"] * t["weight_decay"]) - (m / root) * (s["lr"] / (1.0 - s["beta1"] ** s["step"]))
    t["p"].copy_(p)
    if "p_bf16" in t:
        t["p_bf16"].copy_(p)
    if eight:
        rm, rv = _noise(s["seed"], ordinal, p.numel(), p.device)
        m, sm = _encode(m, rm, 7, 20, torch.float8_e4m3fn)
        v, sv = _encode(v, rv, 14, 21, torch.float8_e5m2)
        t["m_scale"].copy_(sm)
        t["v_scale"].copy_(sv)
    t["m"].copy_(m)
    t["v"].copy_(v)


def run(state):
    s = state
    if own:
        from bitlinear_rmsnorm_quant_b200 import mmf

        if s["op"] == "lookup":
            return mmf.embed_fwd(s["ids"], s["table"], scale=s["scale"])
        if s["op"] == "lookup_grad":
            return mmf.embed_bwd(s["ids"], s["dx"], s["V"], scale=s["scale"], out=s["dtable"], accumulate=s["dtable"] is not None)
        if s["op"] == "scan_grad":
            return mmf.mlgru_scan_bwd(s["f"], s["c"], s["g"], s["do"], h0=s["h0"], dh_last=s["dh_last"])
        mmf.adamw_step([mmf.AdamWTensor(**t) for t in s["tensors"]], step=s["step"], lr=s["lr"], beta1=s["beta1"],
                       beta2=s["beta2"], eps=s["eps"], grad_scale=s["grad_scale"], seed=s["seed"])
        return s["outputs"]
    if s["op"] == "lookup":
        return _lookup_plain(s)
    if s["op"] == "lookup_grad":
        return _lookup_grad_plain(s)
    if s["op"] == "scan_grad":
        return _scan_grad_plain(s)
    [_adamw_plain(s, i, t) for i, t in enumerate(s["tensors"])]
    return s["outputs"]


# -- in 64 bits ------------------------------------------------------------------


def _exact_lookup(s):
    there = (s["ids"] >= 0) & (s["ids"] < s["V"])
    out = torch.zeros(s["ids"].numel(), s["table"].shape[1], dtype=torch.float64, device="cuda")
    out[there] = s["table"].index_select(0, s["ids"][there].long()).double().mul_(s["scale"])
    return out


def _exact_lookup_grad(s):
    there = (s["ids"] >= 0) & (s["ids"] < s["V"])
    out = s["dtable"].double() if s["dtable"] is not None else torch.zeros(s["V"], s["dx"].shape[1], dtype=torch.float64, device="cuda")
    return out.index_put_((s["ids"][there].long(),), s["dx"][there].double() * s["scale"], accumulate=True)


def _exact_scan_grad(s):
    """Token by token, forward and back, each derivative from its own definition."""
    B, T, D = s["f"].shape
    zero = torch.zeros(B, D, dtype=torch.float64, device="cuda")
    h = [zero if s["h0"] is None else s["h0"].double()]
    for t in range(T):
        f = torch.sigmoid(s["f"][:, t].double())
        h.append(f * h[-1] + (1 - f) * torch.nn.functional.silu(s["c"][:, t].double()))
    grads = [torch.empty(B, T, D, dtype=torch.float32 if B * T * D > 1 << 24 else torch.float64, device="cuda") for _ in range(3)]
    dh = zero if s["dh_last"] is None else s["dh_last"].double()
    for t in reversed(range(T)):
        f, g, x, do = torch.sigmoid(s["f"][:, t].double()), torch.sigmoid(s["g"][:, t].double()), s["c"][:, t].double(), s["do"][:, t].double()
        sx = torch.sigmoid(x)
        grads[2][:, t] = do * h[t + 1] * (g - g * g)
        dh = dh + do * g
        grads[0][:, t] = dh * (h[t] - x * sx) * torch.sigmoid(-s["f"][:, t].double()) * f
        grads[1][:, t] = dh * torch.sigmoid(-s["f"][:, t].double()) * (sx + x * sx * torch.sigmoid(-x))
        dh = dh * f
    return grads + [dh]


def _exact_adamw(s):
    out = {k: (x.double() if x.dtype in (torch.float32, torch.bfloat16) else None) for k, x in s["outputs"].items()}
    for k in ("m_scale_8", "v_scale_8"):  # decided by roundings, as the codes are
        if k in out:
            out[k] = None
    where = {x.untyped_storage().data_ptr(): k for k, x in s["outputs"].items()}

    def place(x):
        k = where[x.untyped_storage().data_ptr()]
        return None if out[k] is None else out[k][x.storage_offset():x.storage_offset() + x.numel()]

    for t in s["tensors"]:
        g, m, v = t["g"].double() * s["grad_scale"], t["m"].double(), t["v"].double()
        if "m_scale" in t:
            m = m * t["m_scale"].double().repeat_interleave(BLOCK)[:m.numel()]
            v = v * t["v_scale"].double().repeat_interleave(BLOCK)[:v.numel()]
        m.add_((g - m) * (1 - s["beta1"]))
        v.add_((g * g - v) * (1 - s["beta2"]))
        up = m / (1 - s["beta1"] ** s["step"]) / ((v / (1 - s["beta2"] ** s["step"])).sqrt() + s["eps"])
        p = t["p"].double()
        p = p - s["lr"] * (up + t["weight_decay"] * p)
        place(t["p"]).copy_(p)
        if "p_bf16" in t:
            place(t["p_bf16"]).copy_(p)
        if "m_scale" not in t:
            place(t["m"]).copy_(m)
            place(t["v"]).copy_(v)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "lookup":
        return _exact_lookup(s)
    if s["op"] == "lookup_grad":
        return _exact_lookup_grad(s)
    return _exact_scan_grad(s) if s["op"] == "scan_grad" else _exact_adamw(s)


# -- work ------------------------------------------------------------------------


def _distinct(case):
    """How many different words the batch is expected to hold."""
    n = case["M"] - case["padded"]
    total = math.log1p(case["V"] / 10.0)
    return sum(-math.expm1(n * math.log1p(-math.log1p(1.0 / (r + 10.0)) / total)) for r in range(case["V"])) if n else 0.0


def work(case):
    op = case["op"]
    if op == "lookup":
        M, K = case["M"], case["K"]
        return {"bytes": 2 * M * K + _distinct(case) * K * (2 if case["table"] == "bf16" else 4) + M * case["ids"] // 8, "flops": M * K}
    if op == "lookup_grad":
        M, K = case["M"] - case["padded"], case["K"]
        table = _distinct(case) * K * 8 if case["add"] else 4 * case["V"] * K
        return {"bytes": 2 * M * K + case["M"] * case["ids"] // 8 + table, "flops": 2 * M * K}
    if op == "scan_grad":
        E, states = case["B"] * case["T"] * case["D"], case["B"] * case["D"]
        return {"bytes": 14 * E + 4 * states * (3 if case["carry"] else 1), "flops": 40 * E}
    sizes = _sizes(case)
    grad, copy = (2 if case["grad"] == "bf16" else 4), (2 if case["copy"] else 0)
    return {"bytes": sum(n * (8 + grad + copy + (16 if _bits(case, i) == 32 else 4)) for i, n in enumerate(sizes)), "flops": 15 * sum(sizes)}
