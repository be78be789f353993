"""The training-step operators without a GPU: the plain forms the GPU tests
compare with (against differences, and worked cases), and what the C ABI and
the binding refuse before any CUDA call."""
import ctypes as C

import numpy as np
import pytest
import torch

import training_plain as P
from bitlinear_rmsnorm_quant_b200 import mmf

A = 0x10000
MIS = 0x10008
BIG = 1 << 62


@pytest.fixture(scope="module")
def L():
    from bitlinear_rmsnorm_quant_b200 import build
    build.build()
    return mmf.lib()


# -- the plain forms ---------------------------------------------------------------

def _scan_loss(fp, cp, gp, do, h0, dh_last):
    h, loss = h0, 0.0
    for t in range(fp.shape[1]):
        f = P.sigmoid(fp[:, t])
        h = f * h + (1 - f) * cp[:, t] * P.sigmoid(cp[:, t])
        loss += (do[:, t] * P.sigmoid(gp[:, t]) * h).sum()
    return loss + (dh_last * h).sum()


@pytest.mark.parametrize("B,T,D", [(1, 1, 2), (2, 7, 4)])
def test_scan_gradient_matches_differences(B, T, D):
    r = np.random.default_rng(T)
    fp, cp, gp, do = (r.standard_normal((B, T, D)) for _ in range(4))
    h0, dh_last = r.standard_normal((B, D)), r.standard_normal((B, D))
    got = P.scan_bwd(fp, cp, gp, do, h0, dh_last)
    step = 1e-5  # central differences: error of step^2 times a third derivative of a few units, and 1e-16 / step
    for name, x in (("df", fp), ("dc", cp), ("dg", gp), ("dh0", h0)):
        diff = np.zeros_like(x)
        for i in np.ndindex(*x.shape):
            old = x[i]
            x[i] = old + step
            up = _scan_loss(fp, cp, gp, do, h0, dh_last)
            x[i] = old - step
            down = _scan_loss(fp, cp, gp, do, h0, dh_last)
            x[i] = old
            diff[i] = (up - down) / (2 * step)
        assert np.abs(diff - got[name]).max() < 1e-8


def test_embed_gradient_matches_definition():
    ids, V, K = np.array([3, -1, 0, 3, 9, 3]), 5, 8
    dx = np.random.default_rng(0).standard_normal((6, K))
    d, _ = P.embed_bwd(ids, dx, V, 2.0)
    assert np.allclose(d[3], 2 * (dx[0] + dx[3] + dx[5])) and np.allclose(d[0], 2 * dx[2])
    assert not d[[1, 2, 4]].any()


def test_adamw_worked_step():
    t = {"p": np.float32([1.0]), "g": np.float32([0.5]), "m": np.float32([0.0]), "v": np.float32([0.0]),
         "weight_decay": 0.1, "eight": False}
    r = P.adamw(t, 0, 1, 0.01, 0.9, 0.99, 1e-8, 1.0, 0)
    # the first step moves by lr against the gradient's sign, after the decay
    assert abs(r["p"][0] - (1.0 * (1 - 0.001) - 0.01)) < 1e-7


def test_quantise_grid_and_mean():
    # values on the grid stay; a value between two neighbours goes up in proportion to its place between them
    x = np.zeros(256, np.float32)
    x[:4] = [128.0, -80.0, 17.0, 0.0]
    codes, scale = P.quantise(x, np.full(256, 65535), 7, 3, 7, False)
    val = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy() * scale[0]
    assert scale[0] == 1.0 and val[0] == 128 and val[1] == -80 and val[2] == 18 and val[3] == 0
    codes, _ = P.quantise(x, np.zeros(256, np.int64), 7, 3, 7, False)
    assert torch.from_numpy(codes).view(torch.float8_e4m3fn).float()[2] == 16
    x[:] = 16.5
    x[0] = 128
    codes, _ = P.quantise(x, np.arange(256) * 256, 7, 3, 7, False)
    val = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()[1:]
    assert (val == 18).mean() == pytest.approx(0.25, abs=1 / 128)   # a quarter of the way from 16 to 18


# -- refusals ----------------------------------------------------------------------

def test_embed_argument_errors(L):
    f = L.mmf_embed_fwd
    nan = float("nan")
    assert f(A, A, 1.0, 100, 4, 64, A, 8, None) == 1           # unknown flag
    assert f(A, A, 1.0, 100, 4, 64, A, 4, None) == 1           # accumulate is the gradient's
    assert f(A, A, nan, 100, 4, 64, A, 0, None) == 1
    assert f(A, A, 1.0, -1, 4, 64, A, 0, None) == 1
    assert f(A, None, 1.0, 100, 4, 64, A, 0, None) == 1
    for K in (0, 4, 12, 65544):
        assert f(A, A, 1.0, 100, 4, K, A, 0, None) == 2
    assert f(A, A, 1.0, 100, 65535 * 256 + 1, 64, A, 0, None) == 2
    assert f(A, A, 1.0, (1 << 31) - 1, 4, 64, A, 0, None) == 2
    assert f(A, A, 1.0, 1 << 30, 4, 65536, A, 0, None) == 2    # V * K beyond 2^40
    assert f(MIS, A, 1.0, 100, 4, 64, A, 0, None) == 3
    assert f(None, None, 1.0, 100, 0, 64, None, 0, None) == 0  # no tokens
    g = L.mmf_embed_bwd
    need = L.mmf_embed_bwd_workspace_bytes(100, 2000, 64)
    assert need > 0 and L.mmf_embed_bwd_workspace_bytes(100, 0, 64) == 0
    assert L.mmf_embed_bwd_workspace_bytes(100, 2000, 12) == 0
    assert g(A, A, 1.0, 100, 4, 64, A, A, need, 2, None) == 1  # the table's type is the lookup's
    assert g(A, A, float("inf"), 100, 4, 64, A, A, need, 0, None) == 1
    assert g(A, None, 1.0, 100, 4, 64, A, A, need, 0, None) == 1
    assert g(A, A, 1.0, 100, 4, 64, None, A, need, 0, None) == 1
    assert g(A, A, 1.0, 100, 4, 65, A, A, need, 0, None) == 2
    assert g(A, A, 1.0, 100, 4, 64, MIS, A, need, 0, None) == 3
    assert g(A, A, 1.0, 100, 2000, 64, A, A, need - 1, 0, None) == 4
    assert g(A, A, 1.0, 100, 2000, 64, A, None, need, 0, None) == 4
    assert g(None, None, 1.0, 100, 0, 64, None, None, 0, 4, None) == 0   # nothing to add
    assert g(None, None, 1.0, 0, 4, 64, None, None, 0, 0, None) == 0     # an empty table
    if not torch.cuda.is_available():
        assert g(None, None, 1.0, 100, 0, 64, A, None, 0, 0, None) == 7  # no tokens: zeros, on a device


def test_workspace_of_the_largest_batch_serves_all(L):
    """A workspace made for the most tokens is enough for any fewer of them."""
    for V, K in ((50, 8), (32000, 2048), (100, 65536)):
        marks = [0, 1, 1023, 1024, 1025, 3999]
        for edge in (4096, 16384, 32768, 1 << 20):
            marks += [edge - 1, edge, edge + 1, edge + edge // 2]
        sizes = [L.mmf_embed_bwd_workspace_bytes(V, M, K) for M in marks]
        assert sizes == sorted(sizes) and sizes[3] == 0 < sizes[4]
    batches = (1, 2, 3, 4, 5, 7, 8, 16, 31, 64, 300, 1000)
    for D in (2, 64, 1022, 2048):
        for T in (1, 7, 8, 63, 64, 65, 1000, 4097):
            sizes = [L.mmf_mlgru_scan_bwd_workspace_bytes(B, T, D) for B in batches]
            assert sizes == sorted(sizes), (D, T)
        for B in batches:
            sizes = [L.mmf_mlgru_scan_bwd_workspace_bytes(B, T, D) for T in [*range(1, 300), 512, 1000, 2047, 2048, 9001]]
            assert sizes == sorted(sizes), (D, B)


def test_overlaps_are_refused(L):
    """Outputs over inputs, over one another or over the workspace; buffers next to one another are apart."""
    apart = 0 if torch.cuda.is_available() else 7
    if apart == 0:
        pytest.skip("the addresses below are no memory")
    at = [0x10000000 * (i + 1) for i in range(12)]
    fwd, bwd, scan = L.mmf_embed_fwd, L.mmf_embed_bwd, L.mmf_mlgru_scan_bwd
    ids, table, x = at[:3]
    assert fwd(ids, table, 1.0, 100, 2000, 64, x, 0, None) == apart
    assert fwd(ids, table, 1.0, 100, 2000, 64, table + 4 * 100 * 64, 0, None) == apart      # behind the table
    assert fwd(ids, table, 1.0, 100, 2000, 64, table + 4 * 100 * 64 - 16, 0, None) == 1
    assert fwd(ids, table, 1.0, 100, 2000, 64, ids + 4 * 2000 - 16, 0, None) == 1
    assert fwd(ids, table, 1.0, 100, 2000, 64, ids + 8 * 2000 - 16, 0, None) == apart
    assert fwd(ids, table, 1.0, 100, 2000, 64, ids + 8 * 2000 - 16, 1, None) == 1           # int64 ids are longer
    dx, d, ws = at[1:4]
    need = L.mmf_embed_bwd_workspace_bytes(100, 2000, 64)
    assert bwd(ids, dx, 1.0, 100, 2000, 64, d, ws, need, 0, None) == apart
    for d_at, ws_at in ((dx, ws), (ids, ws), (ws, ws), (ws + need - 16, ws), (d, dx + 2 * 2000 * 64 - 16), (d, ids)):
        assert bwd(ids, dx, 1.0, 100, 2000, 64, d_at, ws_at, need, 0, None) == 1
    assert bwd(ids, dx, 1.0, 100, 2000, 64, ws + need, ws, need, 0, None) == apart
    need = L.mmf_mlgru_scan_bwd_workspace_bytes(2, 4000, 64)
    ok = [*at[:6], 2, 4000, 64, *at[6:11], need, None]
    pointers = (0, 1, 2, 3, 4, 5, 9, 10, 11, 12, 13)
    assert scan(*ok) == apart
    for w in (9, 10, 11, 12, 13):
        for other in pointers:
            if other != w:
                a = list(ok)
                a[w] = a[other]
                assert scan(*a) == 1, (w, other)


def test_scan_bwd_argument_errors(L):
    f = L.mmf_mlgru_scan_bwd
    need = L.mmf_mlgru_scan_bwd_workspace_bytes(1, 4000, 64)
    assert need > 0 and L.mmf_mlgru_scan_bwd_workspace_bytes(1, 0, 64) == 0
    ok = [A, A, A, A, None, None, 1, 4000, 64, A, A, A, None, A, need, None]

    def but(**at):
        a = list(ok)
        for i, v in at.items():
            a[int(i[1:])] = v
        return f(*a)

    assert but(_8=65) == 2
    assert but(_6=65536) == 2 and but(_7=1 << 31) == 2
    assert but(_6=65535, _7=(1 << 31) - 1, _8=(1 << 31) - 2) == 2   # a product beyond 64 bits
    assert but(_6=-1) == 1 and but(_7=-1) == 1
    for i in (0, 1, 2, 3, 9, 10, 11):
        assert but(**{f"_{i}": None}) == 1
        assert but(**{f"_{i}": MIS}) == 3
    for i in (4, 5, 12, 13):
        assert but(**{f"_{i}": MIS}) == 3
    assert but(_13=None) == 4 and but(_14=need - 1) == 4
    assert but(_6=0) == 0 and but(_8=0) == 0
    assert but(_7=0) == 0                                         # no tokens and no dh0 wanted


def _tensors(*descs):
    buf = bytearray(72 * len(descs))
    for i, d in enumerate(descs):
        mmf._ADAMW_DESC.pack_into(buf, 72 * i, *d)
    return (C.c_char * len(buf)).from_buffer(buf)


def _hyper(**k):
    v = dict(step=1, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, grad_scale=1.0, seed=0)
    v.update(k)
    return mmf._adamw_hyper(**v)


def _desc(p=0x100000, g=0x200000, m=0x300000, v=0x400000, ms=0, vs=0, pb=0, n=100, wd=0.0, flags=0):
    return (p, g, m, v, ms, vs, pb, n, wd, flags)


def test_adamw_argument_errors(L):
    def go(*descs, scalars=None, **k):
        tensors = _tensors(*descs)
        return L.mmf_adamw_step(C.addressof(tensors), len(descs), C.byref(_hyper(**k)), scalars, None)

    for bad in (dict(step=0), dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0), dict(beta1=-0.1),
                dict(beta2=1.0), dict(beta2=1 - 1e-12), dict(eps=0.0), dict(eps=1e-60), dict(eps=float("inf")),
                dict(grad_scale=float("inf")), dict(lr=1e300)):
        assert go(_desc(), **bad) == 1, bad
        out = (C.c_char * 32)()
        assert L.mmf_adamw_scalars_at(C.byref(_hyper(**bad)), out) == 1, bad
    assert L.mmf_adamw_scalars_at(None, None) == 1
    assert L.mmf_adamw_step(None, 1, C.byref(_hyper()), None, None) == 1
    assert L.mmf_adamw_step(None, 0, C.byref(_hyper()), None, None) == 0
    assert L.mmf_adamw_step(None, -1, C.byref(_hyper()), None, None) == 1
    assert go(_desc(n=-1)) == 1
    assert go(_desc(n=(1 << 40) + 1)) == 2
    assert go(_desc(flags=4)) == 1
    assert go(_desc(wd=-0.1)) == 1 and go(_desc(wd=float("nan"))) == 1
    for k in ("p", "g", "m", "v"):
        assert go(_desc(**{k: 0})) == 1
        assert go(_desc(**{k: _desc()[("p", "g", "m", "v").index(k)] + 8})) == 3
    assert go(_desc(pb=MIS)) == 3
    assert go(_desc(), scalars=MIS) == 3
    assert go(_desc(ms=0x500000, vs=0x600000)) == 1              # scales without 8-bit moments
    assert go(_desc(flags=1)) == 1 and go(_desc(flags=1, ms=0x500000)) == 1
    # overlaps: one tensor twice, a moment inside another's weights, a gradient that is a moment
    assert go(_desc(), _desc()) == 1
    assert go(_desc(), _desc(p=0x700000, g=0x800000, m=0x100000 + 96 * 4, v=0x900000)) == 1
    assert go(_desc(g=0x300000)) == 1
    assert go(_desc(pb=0x100000)) == 1
    two = (_desc(), _desc(p=0x700000, m=0x800000, v=0x900000))   # one gradient for two tensors is read twice
    if not torch.cuda.is_available():
        assert go(*two) == 7
        assert go(_desc(), _desc(p=0x100000 + 400, g=0x200000, m=0x700000, v=0x800000)) == 7   # next to one another
        assert go(_desc(p=0, g=0, m=0, v=0, n=0)) == 7


def test_adamw_scalars():
    s = mmf.adamw_scalars(step=10, lr=1e-3, beta1=0.9, beta2=0.99, grad_scale=0.5, seed=7)
    f = s[:16].view(torch.float32)
    assert f[0] == np.float32(1e-3) and f[3] == 0.5
    assert f[1].item() == pytest.approx(1e-3 / (1 - 0.9 ** 10), rel=1e-6)
    assert f[2].item() == pytest.approx((1 - 0.99 ** 10) ** -0.5, rel=1e-6)
    assert s[16:24].view(torch.int64).item() == 7


def test_binding_refuses_cpu_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        mmf.embed_fwd(torch.zeros(3, dtype=torch.int64), torch.zeros(4, 8))
    with pytest.raises(TypeError, match="ids"):
        mmf.embed_fwd(torch.zeros(3, dtype=torch.int16), torch.zeros(4, 8))
    with pytest.raises(ValueError, match="CUDA"):
        mmf.mlgru_scan_bwd(*[torch.zeros(1, 2, 4, dtype=torch.bfloat16)] * 4)
    p = torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        mmf.adamw_step([mmf.AdamWTensor(p, p, **mmf.adamw_state(p))], step=1, lr=1e-3)
    with pytest.raises(ValueError, match="bits"):
        mmf.adamw_state(p, 16)
    s = mmf.adamw_state(torch.zeros(257), 8)
    assert s["m"].dtype == torch.float8_e4m3fn and s["m_scale"].numel() == 2
