"""Plain 64-bit forms of the training-step operators (embedding, gradient of
the MLGRU recurrence, AdamW), written from their formulas for the tests, with
the error bounds the tests hold the kernels to.

U is half a step of fp32 relative to the value, 2^-24; UB that of bf16, 2^-8."""
from __future__ import annotations

import numpy as np
import torch

from bitlinear_rmsnorm_quant_b200 import inputs as I

U = torch.finfo(torch.float32).eps / 2
UB = torch.finfo(torch.bfloat16).eps / 2
BLOCK = 256


def sigmoid(v):
    return 1.0 / (1.0 + np.exp(-v))


# -- embedding -------------------------------------------------------------------

def embed_bwd(ids: np.ndarray, dx: np.ndarray, V: int, scale: float, base=None):
    """(dtable, bound) in fp64.  A row's tokens are added in fp32 in groups of at
    most 256 (each addition off by at most U of the partial sum, itself at most
    the sum of magnitudes), the groups in fp64 and rounded once, the product
    with the scale rounded once, and the sum with `base` once."""
    K = dx.shape[1]
    out, mag, n = np.zeros((V, K)), np.zeros((V, K)), np.zeros(V)
    for m, v in enumerate(ids):
        if 0 <= v < V:
            out[v] += dx[m]
            mag[v] += np.abs(dx[m])
            n[v] += 1
    out *= scale
    mag *= abs(scale)
    bound = (np.minimum(n, 256)[:, None] + 3) * U * mag
    if base is not None:
        out = out + base
        bound = bound + U * np.abs(out)
    return out, bound * 1.001


# -- gradient of the recurrence ----------------------------------------------------

def scan_bwd(fp, cp, gp, do, h0=None, dh_last=None):
    """fp64 arrays [B, T, D] -> dict of df, dc, dg, dh0 and the states h [B, T + 1, D] (h[:, 0] = h0)."""
    B, T, D = fp.shape
    h = np.zeros((B, T + 1, D))
    if h0 is not None:
        h[:, 0] = h0
    f, s, g = sigmoid(fp), sigmoid(cp), sigmoid(gp)
    k = sigmoid(-fp)
    for t in range(T):
        h[:, t + 1] = f[:, t] * h[:, t] + k[:, t] * cp[:, t] * s[:, t]
    dh = np.zeros((B, T + 1, D))     # dh[:, t]: gradient of the state before token t, through later tokens
    dh[:, T] = 0 if dh_last is None else dh_last
    full = np.zeros((B, T, D))       # gradient of h_t, its own output included
    for t in reversed(range(T)):
        full[:, t] = do[:, t] * g[:, t] + dh[:, t + 1]
        dh[:, t] = full[:, t] * f[:, t]
    c = cp * s
    return {"df": full * (h[:, :-1] - c) * f * k, "dc": full * k * s * (1 + cp * sigmoid(-cp)),
            "dg": do * h[:, 1:] * g * sigmoid(-gp), "dh0": dh[:, 0], "h": h, "full": full, "f": f, "k": k, "c": c,
            "s": s, "g": g}


def scan_bwd_bounds(r, fp, cp, gp, do):
    """Bounds on the kernel's distance from `r` by a running error analysis.  A
    gate comes from an exponential (2 ulp, and |v| U relative from rounding its
    argument), a reciprocal (1 ulp) and at most six products and sums: within
    (16 + |v|) U of its value, and so are the products of a token's gates with
    each other taken together.  The states carry their errors on."""
    B, T, D = fp.shape
    C = 16 + max(np.abs(v).max() if v.size else 0.0 for v in (fp, cp, gp))
    eh = np.zeros((B, T + 1, D))
    h, f, k, c, g, full = (r[n] for n in ("h", "f", "k", "c", "g", "full"))
    for t in range(T):
        eh[:, t + 1] = f[:, t] * eh[:, t] + 2 * C * U * (np.abs(f[:, t] * h[:, t]) + np.abs(k[:, t] * c[:, t]))
    ed = np.zeros((B, T + 1, D))
    efull = np.zeros((B, T, D))
    for t in reversed(range(T)):
        efull[:, t] = ed[:, t + 1] + 2 * C * U * (np.abs(do[:, t] * g[:, t]) + np.abs(full[:, t]))
        ed[:, t] = f[:, t] * (efull[:, t] + 2 * C * U * np.abs(full[:, t]))
    fk = f * k
    raw = {"df": fk * (efull * np.abs(h[:, :-1] - c) + np.abs(full) * (eh[:, :-1] + 2 * C * U * (np.abs(h[:, :-1]) + np.abs(c)))),
           "dc": efull * np.abs(r["k"] * r["s"]) * (1 + np.abs(cp)) + 4 * C * U * np.abs(full * r["k"] * r["s"]) * (1 + np.abs(cp)),
           "dg": np.abs(do) * g * sigmoid(-gp) * (eh[:, 1:] + 4 * C * U * np.abs(h[:, 1:]))}
    out = {n: v + 4 * C * U * np.abs(r[n]) + UB * (np.abs(r[n]) + v) for n, v in raw.items()}
    out["dh0"] = ed[:, 0] + 2 * C * U * np.abs(r["dh0"])
    tiny = 2.0 ** -126  # results below fp32's normal range
    return {n: 1.01 * v + tiny for n, v in out.items()}


# -- AdamW -------------------------------------------------------------------------

def noise(seed: int, tensor: int, n: int):
    """The 16 random bits of m and of v for each element."""
    z = I.raw_u64(seed, tensor, 0, (n + 1) // 2).numpy().view(np.uint64)
    both = np.stack([z & np.uint64(0xFFFFFFFF), z >> np.uint64(32)], 1).reshape(-1)[:n].astype(np.int64)
    return both & 0xFFFF, both >> 16


def quantise(x: np.ndarray, bits16: np.ndarray, low: int, mant: int, bias: int, keep_positive: bool):
    """fp32 x -> (codes uint8, scales fp32): each block's power of two, and the
    value between two neighbours of the 8-bit grid taken up when its place
    between them plus the random fraction reaches 1."""
    n = x.size
    codes, scales = np.zeros(n, np.uint8), []
    for b in range(0, n, BLOCK):
        v = x[b:b + BLOCK].astype(np.float64)
        top = np.abs(v).max() if not np.isnan(v).any() else np.inf
        if not top < 2.0 ** 127:
            scales.append(np.nan)
            continue
        e = max(int(np.frexp(top)[1]) - 1, -90) if top > 0 else -90
        scale = 2.0 ** (e - low)
        scales.append(scale)
        y = np.abs(v) / scale
        with np.errstate(divide="ignore"):
            ex = np.where(y > 0, np.frexp(np.where(y > 0, y, 1.0))[1] - 1, -200)
        place = (y / 2.0 ** ex - 1) * 2 ** mant
        k = np.floor(place)
        up = (place - k) * 65536 + bits16[b:b + BLOCK] + 0.5 >= 65536
        c = ((ex + bias) << mant) + k.astype(np.int64) + up
        least = 1 << mant
        if keep_positive:
            c = np.where(y > 0, np.maximum(c, least), 0)
        else:
            c = np.where((y > 0) & (c >= least), c, 0) | np.where(np.signbit(v), 128, 0)
        codes[b:b + BLOCK] = c
    return codes, np.asarray(scales, np.float32)


def adamw(t: dict, ordinal: int, step, lr, beta1, beta2, eps, grad_scale, seed):
    """One tensor (numpy, moments as fp32 values) -> new p in fp64 and its bound, m and v in fp32 as the
    elementwise operations round them, and for 8-bit moments the codes and scales."""
    f = np.float32
    with np.errstate(invalid="ignore", over="ignore"):
        g = (t["g"].astype(f) * f(grad_scale)).astype(f)
        m = (t["m"] * f(beta1) + g * f(1 - beta1)).astype(f)
        v = (t["v"] * f(beta2) + (g * g) * f(1 - beta2)).astype(f)
        m64, v64 = m.astype(np.float64), v.astype(np.float64)
        upd = lr / (1 - beta1 ** step) * m64 / (np.sqrt(v64 / (1 - beta2 ** step)) + eps)
        kept = t["p"].astype(np.float64) * (1 - lr * t["weight_decay"])
    out = {"p": kept - upd, "m": m, "v": v}
    # lr, weight decay, their product and 1 minus it each rounded once, two more products and the sum; the update
    # from a square root and a division of at most 2 ulp each and six roundings
    out["bound"] = U * (6 * np.abs(kept) + 16 * np.abs(upd)) + 2.0 ** -126
    if t["eight"]:
        rm, rv = noise(seed, ordinal, m.size)
        out["m_code"], out["m_scale"] = quantise(m, rm, 7, 3, 7, False)
        out["v_code"], out["v_scale"] = quantise(v, rv, 14, 2, 15, True)
    return out
