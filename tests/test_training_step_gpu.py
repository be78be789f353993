"""The training-step operators on the GPU against their plain 64-bit forms:
embedding lookup and its gradient, the gradient of the MLGRU recurrence, the
AdamW step, and a run of them together with the layers."""
import numpy as np
import pytest
import torch

import training_plain as P
from bitlinear_rmsnorm_quant_b200 import mmf

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True, scope="module")
def _built():
    from bitlinear_rmsnorm_quant_b200 import build
    build.build()
    torch.cuda.set_device(0)


def bf(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


# -- embedding -------------------------------------------------------------------

def make_ids(rng, M, V, kind):
    if kind == "one":
        ids = np.full(M, V // 2)
    elif kind == "outside":
        ids = rng.choice([-1, -2, V, V + 7, -(1 << 31), (1 << 31) - 1], M)
    else:
        ids = np.minimum((10 * np.expm1(rng.random(M) * np.log1p(V / 10))).astype(np.int64), V - 1)
        ids = rng.permutation(V)[ids]
        ids[rng.random(M) < 0.05] = -1
    return ids.astype(np.int64)


@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,V,K,kind", [(1, 100, 2560, "mixed"), (37, 1000, 8, "mixed"), (300, 50, 1000, "mixed"),
                                        (2000, 32000, 264, "mixed"), (5, 7, 4104, "mixed"), (64, 10, 64, "outside"),
                                        (3, 1, 16, "one")])
def test_embed_fwd(M, V, K, kind, dtype, idt):
    rng = np.random.default_rng(M + K)
    ids = torch.from_numpy(make_ids(rng, M, V, kind)).to(idt)
    table = torch.from_numpy(rng.standard_normal((V, K)).astype(np.float32)).to(dtype)
    x = mmf.embed_fwd(ids.to(DEV), table.to(DEV), scale=3.3)
    want = torch.zeros(M, K, dtype=torch.bfloat16)
    there = (ids >= 0) & (ids < V)
    want[there] = (table[ids[there].long()].float() * 3.3).to(torch.bfloat16)
    assert torch.equal(x.cpu(), want)


def test_embed_fwd_int64_ids_beyond_32_bits():
    """An id whose low 32 bits name a row is still outside the table."""
    ids = torch.tensor([(1 << 32) + 1, 1, -(1 << 32) + 1], device=DEV)
    table = torch.ones(4, 8, device=DEV)
    assert mmf.embed_fwd(ids, table).float().sum(1).tolist() == [0.0, 8.0, 0.0]
    d = mmf.embed_bwd(ids, torch.ones(3, 8, dtype=torch.bfloat16, device=DEV), 4)
    assert d.sum(1).tolist() == [0.0, 8.0, 0.0, 0.0]


@pytest.mark.parametrize("M,V,K,kind", [
    (1, 100, 2560, "mixed"), (37, 1000, 8, "mixed"), (300, 50, 1000, "mixed"), (2000, 32000, 264, "mixed"),
    (5, 7, 4104, "mixed"), (64, 10, 64, "outside"), (3, 1, 16, "one"),
    # the most tokens of one launch, and one more
    (1024, 100, 72, "mixed"), (1024, 9, 136, "one"), (1025, 100, 72, "mixed"), (1030, 9, 2056, "one"),
    # one word for all tokens: a run over every summing CTA; more than one sorting CTA and round
    (1000, 300, 40, "one"), (9000, 70000, 64, "mixed"), (40000, 3, 16, "mixed"), (140000, 1000, 8, "mixed"),
    (140000, 20, 8, "one"),
    # the most tokens of the one-launch sort, one more, and three passes of each sort
    (16384, 3000, 16, "mixed"), (16385, 3000, 16, "mixed"), (8193, 1 << 17, 8, "mixed"), (17000, 1 << 17, 8, "mixed"),
    # keys of one digit, of exactly 8 and 16 bits, of three digits
    (1500, 255, 16, "mixed"), (1500, 256, 16, "mixed"), (1500, 65535, 8, "mixed"), (1500, 65536, 8, "mixed"),
    (1700, 1 << 20, 8, "mixed"), (2000, 5, 16, "outside"), (1200, (1 << 24) + 5, 8, "mixed")])
@pytest.mark.parametrize("add", [False, True])
def test_embed_bwd(M, V, K, kind, add):
    rng = np.random.default_rng(M + K)
    ids = make_ids(rng, M, V, kind)
    dx = bf(rng.standard_normal((M, K)))
    base = rng.standard_normal((V, K)).astype(np.float32) if add else None
    idt = torch.int32 if kind != "outside" and M % 2 else torch.int64
    out = torch.from_numpy(base).to(DEV) if add else torch.full((V, K), float("nan"), device=DEV)
    ids_d, dx_d = torch.from_numpy(ids).to(idt).to(DEV), dx.to(DEV)
    got = mmf.embed_bwd(ids_d, dx_d, V, scale=-1.7, out=out, accumulate=add)
    scale = float(np.float32(-1.7))
    want, bound = P.embed_bwd(ids, f64(dx), V, scale, base)
    assert got is out
    assert (np.abs(f64(got) - want) <= bound).all()
    absent = np.setdiff1d(np.arange(V), ids)
    assert np.array_equal(got.cpu().numpy()[absent], base[absent] if add else np.zeros((absent.size, K), np.float32))
    again = mmf.embed_bwd(ids_d, dx_d, V, scale=-1.7, out=torch.from_numpy(base).to(DEV) if add else None, accumulate=add)
    assert torch.equal(again, got)


@pytest.mark.parametrize("M,V,K", [
    # one launch: lists that one slice adds, lists divided among 2, 4 and 8 slices, with columns left over
    (60, 40, 24), (700, 40, 1032), (1024, 500, 2064), (900, 300, 264), (512, 90, 520),
    # runs over many summing CTAs, 256 columns and fewer or more, some behind the CTA's last join warp
    (3000, 900, 264), (4096, 50, 1000), (4097, 50, 256), (9000, 2000, 520), (20000, 30, 248), (40000, 100, 16)])
@pytest.mark.parametrize("frequent", ["first", "last", "two"])
def test_embed_bwd_of_frequent_ids(M, V, K, frequent):
    """Padded batches: most tokens of one or two ids."""
    rng = np.random.default_rng(M + K)
    ids = make_ids(rng, M, V, "mixed")
    at = rng.random(M)
    if frequent == "two":
        ids[at < 0.35] = V // 3
        ids[at > 0.6] = V // 3 + 1
    else:
        ids[at < 0.8] = 0 if frequent == "first" else V - 1
    dx = bf(rng.standard_normal((M, K)))
    base = rng.standard_normal((V, K)).astype(np.float32)
    ids_d, dx_d = torch.from_numpy(ids).to(DEV), dx.to(DEV)
    for add in (False, True):
        want, bound = P.embed_bwd(ids, f64(dx), V, 0.5, base if add else None)
        outs = [torch.from_numpy(base).to(DEV) for _ in range(2)]
        for out in outs:
            mmf.embed_bwd(ids_d, dx_d, V, scale=0.5, out=out, accumulate=add)
        assert (np.abs(f64(outs[0]) - want) <= bound).all()
        assert torch.equal(*outs)


def test_embed_bwd_empty():
    d = mmf.embed_bwd(torch.zeros(0, dtype=torch.int64, device=DEV), torch.zeros(0, 16, dtype=torch.bfloat16, device=DEV),
                      5, out=torch.ones(5, 16, device=DEV))
    assert not d.any()
    d = mmf.embed_bwd(torch.zeros(0, dtype=torch.int64, device=DEV), torch.zeros(0, 16, dtype=torch.bfloat16, device=DEV),
                      5, out=torch.ones(5, 16, device=DEV), accumulate=True)
    assert (d == 1).all()
    assert mmf.embed_fwd(torch.zeros(0, dtype=torch.int32, device=DEV), torch.ones(3, 16, device=DEV)).shape == (0, 16)


def test_embed_infinities_stay_in_their_rows():
    ids = torch.tensor([1, 2, 1], device=DEV)
    dx = torch.ones(3, 8, dtype=torch.bfloat16, device=DEV)
    dx[1, 3] = float("inf")
    dx[2, 0] = float("nan")
    d = mmf.embed_bwd(ids, dx, 4).cpu()
    assert torch.isnan(d[1, 0]) and (d[1, 1:] == 2).all() and d[2, 3] == float("inf") and not d[0].any() and not d[3].any()


# -- gradient of the recurrence ----------------------------------------------------

SCAN_SHAPES = [(1, 2048, 64), (2, 2049, 72), (3, 130, 640), (1, 2600, 264), (2, 3000, 192), (1, 8200, 64), (1, 1, 2), (1, 1, 2560), (2, 37, 128), (3, 100, 66), (1, 37, 1022), (2, 5, 64), (3, 8, 62), (1, 300, 200),
               (2, 16, 4104), (2, 129, 512), (5, 70, 34), (1, 1000, 72), (2, 2048, 8), (1, 4099, 24), (70, 3, 6),
               # the most tokens of one launch, and one more; short sequences of more channels than it takes; single steps
               (1, 40, 96), (1, 41, 96), (1, 64, 96), (1, 65, 96), (600, 7, 264), (600, 8, 264), (4100, 7, 64), (4100, 8, 64), (2400, 5, 6), (2400, 9, 64), (600, 64, 264),
               # enough segments for both walks in one launch, at each width of its CTAs
               (41, 1003, 256), (30, 1001, 264), (75, 1027, 72), (160, 968, 64)]


@pytest.mark.parametrize("B,T,D", SCAN_SHAPES)
@pytest.mark.parametrize("carry", [False, True])
def test_mlgru_scan_bwd(B, T, D, carry):
    rng = np.random.default_rng(B * 1000 + T + D)
    fp, cp, gp, do = (bf(2 * rng.standard_normal((B, T, D))) for _ in range(4))
    h0 = torch.from_numpy(rng.standard_normal((B, D)).astype(np.float32)) if carry else None
    dl = torch.from_numpy(rng.standard_normal((B, D)).astype(np.float32)) if carry else None
    got = mmf.mlgru_scan_bwd(*(t.to(DEV) for t in (fp, cp, gp, do)), h0=h0.to(DEV) if carry else None,
                             dh_last=dl.to(DEV) if carry else None)
    a = [f64(t) for t in (fp, cp, gp, do)]
    want = P.scan_bwd(*a, f64(h0) if carry else None, f64(dl) if carry else None)
    bound = P.scan_bwd_bounds(want, *a)
    for n, t in zip(("df", "dc", "dg", "dh0"), got):
        assert (np.abs(f64(t) - want[n]) <= bound[n]).all(), n


@pytest.mark.parametrize("T,D", [(300, 64), (70, 66)])
def test_mlgru_scan_bwd_saturated_gates(T, D):
    """Pre-activations of +-60 among ordinary ones.  The kernel clamps them below
    at -28 before the exponential: a gate of e^-60 comes out as e^-28 < 7e-13, so
    beside the running bound each output may be off by 1e-11 of the state's and
    the gradient's size times the pre-activation (60)."""
    rng = np.random.default_rng(T)
    a = [2 * rng.standard_normal((2, T, D)) for _ in range(4)]
    for x in a[:3]:
        x[rng.random(x.shape) < 0.1] = 60.0
        x[rng.random(x.shape) < 0.1] = -60.0
    t = [bf(x) for x in a]
    a = [f64(x) for x in t]
    got = mmf.mlgru_scan_bwd(*(x.to(DEV) for x in t))
    want = P.scan_bwd(*a)
    bound = P.scan_bwd_bounds(want, *a)
    size = 60 * (1 + np.abs(want["h"]).max()) * (1 + np.abs(want["full"]).max())
    for n, x in zip(("df", "dc", "dg", "dh0"), got):
        assert np.isfinite(f64(x)).all()
        assert (np.abs(f64(x) - want[n]) <= bound[n] + 1e-11 * size).all(), n


def test_mlgru_scan_bwd_no_tokens():
    e = torch.zeros(2, 0, 8, dtype=torch.bfloat16, device=DEV)
    dl = torch.randn(2, 8, device=DEV)
    assert torch.equal(mmf.mlgru_scan_bwd(e, e, e, e, dh_last=dl)[3], dl)
    assert not mmf.mlgru_scan_bwd(e, e, e, e)[3].any()


def test_mlgru_scan_bwd_continues_across_calls():
    """The halves of a sequence, the state carried forward and its gradient back, give the whole's gradients."""
    rng = np.random.default_rng(3)
    B, T, D, cut = 2, 300, 96, 133
    fp, cp, gp, do = (bf(rng.standard_normal((B, T, D))).to(DEV) for _ in range(4))
    whole = mmf.mlgru_scan_bwd(fp, cp, gp, do)
    lo, hi = ([t[:, s].contiguous() for t in (fp, cp, gp, do)] for s in (slice(0, cut), slice(cut, T)))
    _, h = mmf.mlgru_scan(*lo[:3])
    second = mmf.mlgru_scan_bwd(*hi, h0=h)
    first = mmf.mlgru_scan_bwd(*lo, dh_last=second[3])
    a = [f64(t) for t in (fp, cp, gp, do)]
    bound = P.scan_bwd_bounds(P.scan_bwd(*a), *a)
    for i, n in enumerate(("df", "dc", "dg")):
        # both sides are within the bound of the same gradients, and the forward's state is a few ulp off besides
        assert (np.abs(f64(torch.cat((first[i], second[i]), 1)) - f64(whole[i])) <= 4 * bound[n] + 1e-6).all(), n
    assert (np.abs(f64(first[3]) - f64(whole[3])) <= 4 * bound["dh0"] + 1e-6).all()


def test_mlgru_scan_bwd_nan_stays_in_its_channel():
    fp, cp, gp, do = (bf(np.ones((2, 20, 64))).to(DEV) for _ in range(4))
    cp[1, 10, 5] = float("nan")
    out = mmf.mlgru_scan_bwd(fp, cp, gp, do)
    bad = torch.zeros(2, 64, dtype=torch.bool, device=DEV)
    for t in out[:3]:
        bad |= torch.isnan(t).any(1)
    assert bad[1, 5] and bad.sum() == 1
    assert torch.isnan(out[2][1, 10:, 5]).all() and not torch.isnan(out[2][1, :10, 5]).any()


def test_mlgru_scan_bwd_repeats_its_bits():
    rng = np.random.default_rng(9)
    t = [bf(rng.standard_normal((3, 1000, 320))).to(DEV) for _ in range(4)]
    a, b = mmf.mlgru_scan_bwd(*t), mmf.mlgru_scan_bwd(*t)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


# -- AdamW -------------------------------------------------------------------------

HYPER = dict(step=7, lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, grad_scale=0.7, seed=123)


def adam_tensor(rng, n, eight, grad_bf16, copy, wd):
    """(AdamWTensor on the GPU with guard elements behind every buffer, numpy description)."""
    g = rng.standard_normal(n).astype(np.float32) * 10.0 ** rng.integers(-6, 2, n)
    gt = torch.from_numpy(g.astype(np.float32))
    gt = gt.to(torch.bfloat16) if grad_bf16 else gt
    p = rng.standard_normal(n).astype(np.float32)
    blocks = -(-n // 256)
    m, v = (rng.standard_normal(n) * 1e-2).astype(np.float32), (rng.random(n) * 1e-3).astype(np.float32)
    d = {"p": p, "g": gt.float().numpy(), "weight_decay": wd, "eight": eight, "n": n}

    def guarded(x):
        full = torch.zeros(x.numel() + 64, dtype=torch.uint8, device=DEV) if x.element_size() == 1 else \
            torch.full((x.numel() + 64,), 7.0, dtype=x.dtype, device=DEV)
        if x.element_size() == 1:
            full.fill_(85)
            full[:x.numel()] = x.view(torch.uint8).to(DEV)
            return full.view(x.dtype)[:x.numel()]
        full[:x.numel()] = x.to(DEV)
        return full[:x.numel()]

    args = {"p": guarded(torch.from_numpy(p)), "g": gt.to(DEV), "weight_decay": wd}
    if eight:
        mc, ms = P.quantise(m, np.zeros(n, np.int64), 7, 3, 7, False)
        vc, vs = P.quantise(v, np.zeros(n, np.int64), 14, 2, 15, True)
        mt, vt = torch.from_numpy(mc).view(torch.float8_e4m3fn), torch.from_numpy(vc).view(torch.float8_e5m2)
        m = mt.float().numpy() * np.repeat(ms, 256)[:n]
        v = vt.float().numpy() * np.repeat(vs, 256)[:n]
        args.update(m=guarded(mt), v=guarded(vt), m_scale=guarded(torch.from_numpy(ms)), v_scale=guarded(torch.from_numpy(vs)))
        assert len(ms) == blocks
    else:
        args.update(m=guarded(torch.from_numpy(m)), v=guarded(torch.from_numpy(v)))
    if copy:
        args["p_bf16"] = guarded(torch.zeros(n, dtype=torch.bfloat16))
    d.update(m=m, v=v)
    return mmf.AdamWTensor(**args), d


def check_adam(t, want):
    assert (np.abs(f64(t.p) - want["p"]) <= want["bound"]).all()
    if want.get("m_code") is not None:
        assert np.array_equal(t.m.view(torch.uint8).cpu().numpy(), want["m_code"])
        assert np.array_equal(t.v.view(torch.uint8).cpu().numpy(), want["v_code"])
        assert np.array_equal(t.m_scale.cpu().numpy(), want["m_scale"], equal_nan=True)
        assert np.array_equal(t.v_scale.cpu().numpy(), want["v_scale"], equal_nan=True)
    else:
        assert np.array_equal(t.m.cpu().numpy(), want["m"], equal_nan=True)
        assert np.array_equal(t.v.cpu().numpy(), want["v"], equal_nan=True)
    if t.p_bf16 is not None:
        assert torch.equal(t.p_bf16, t.p.to(torch.bfloat16))
    for x in (t.p, t.m, t.v, t.m_scale, t.v_scale, t.p_bf16):   # nothing behind a buffer's end is written
        if x is not None:
            full = torch.as_strided(x.view(torch.uint8) if x.element_size() == 1 else x, (x.numel() + 64,), (1,))
            assert (full[x.numel():] == (85 if x.element_size() == 1 else 7)).all()


@pytest.mark.parametrize("grad_bf16", [False, True])
@pytest.mark.parametrize("eight", [False, True])
def test_adamw_sizes(eight, grad_bf16):
    rng = np.random.default_rng(1 + eight)
    sizes = [1, 2, 3, 4, 5, 127, 128, 129, 131, 255, 256, 257, 511, 4095, 4096, 4097, 9999, 70001]
    made = [adam_tensor(rng, n, eight, grad_bf16, i % 3 == 0, 0.1 * (i % 2)) for i, n in enumerate(sizes)]
    want = [P.adamw(d, i, **HYPER) for i, (_, d) in enumerate(made)]
    mmf.adamw_step([t for t, _ in made], **HYPER)
    for (t, _), w in zip(made, want):
        check_adam(t, w)


def test_adamw_more_tensors_than_a_launch_takes():
    rng = np.random.default_rng(4)
    made = [adam_tensor(rng, int(rng.integers(1, 600)), bool(i % 2), bool(i % 3 == 0), bool(i % 5 == 0), 0.01 * (i % 4))
            for i in range(523)]
    empty = torch.empty(0, device=DEV)
    made[100] = made[256] = made[522] = (mmf.AdamWTensor(empty, empty, empty, empty), None)
    want = [P.adamw(d, i, **HYPER) if d else None for i, (_, d) in enumerate(made)]
    mmf.adamw_step([t for t, _ in made], **HYPER)
    for (t, _), w in zip(made, want):
        if w:
            check_adam(t, w)


def test_adamw_steps_from_fresh_states():
    """Three steps in a row, the noise of each from its own seed; the first update is lr against the sign."""
    rng = np.random.default_rng(5)
    for eight in (False, True):
        p0 = rng.standard_normal(1000).astype(np.float32)
        p = torch.from_numpy(p0).to(DEV)
        state = mmf.adamw_state(p, 8 if eight else 32)
        d = {"p": p0, "m": np.zeros(1000, np.float32), "v": np.zeros(1000, np.float32), "weight_decay": 0.0, "eight": eight}
        for step in (1, 2, 3):
            g = rng.standard_normal(1000).astype(np.float32)
            k = dict(HYPER, step=step, seed=1000 + step)
            t = mmf.AdamWTensor(p, torch.from_numpy(g).to(DEV), **state)
            d["g"] = g
            w = P.adamw(d, 0, **k)
            mmf.adamw_step([t], **k)
            check = {n: x for n, x in w.items()}
            assert (np.abs(f64(t.p) - check["p"]) <= check["bound"]).all()
            if step == 1:
                assert np.allclose(p.cpu().numpy(), p0 - 3e-3 * np.sign(g), atol=2e-5)
            d["p"] = p.cpu().numpy()
            if eight:
                assert np.array_equal(t.m.view(torch.uint8).cpu().numpy(), w["m_code"])
                assert np.array_equal(t.v.view(torch.uint8).cpu().numpy(), w["v_code"])
                d["m"] = t.m.float().cpu().numpy() * np.repeat(w["m_scale"], 256)[:1000]
                d["v"] = t.v.float().cpu().numpy() * np.repeat(w["v_scale"], 256)[:1000]
            else:
                d["m"], d["v"] = w["m"], w["v"]


def test_adamw_rounding_has_the_right_mean():
    """Over N seeds the mean of a code's value is within 5 standard errors of the moment (a rounding's deviation is
    at most half the grid's step, an eighth of the value for m and a quarter for v) plus the 2^-17 of a step by
    which 16 random bits can miss."""
    N, n = 400, 512
    rng = np.random.default_rng(6)
    g = torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(DEV)
    sm, sv = torch.zeros(n, dtype=torch.float64, device=DEV), torch.zeros(n, dtype=torch.float64, device=DEV)
    for seed in range(N):
        p = torch.zeros(n, device=DEV)
        t = mmf.AdamWTensor(p, g, **mmf.adamw_state(p, 8))
        mmf.adamw_step([t], step=1, lr=1e-3, beta1=0.9, beta2=0.95, seed=seed)
        sm += t.m.double() * t.m_scale.double().repeat_interleave(256)
        sv += t.v.double() * t.v_scale.double().repeat_interleave(256)
    m, v = 0.1 * g.double(), 0.05 * g.double().square()
    top = m.abs().view(-1, 256).amax(1).repeat_interleave(256)
    held = m.abs() > top * 2.0 ** -13     # below the smallest normal code m is dropped
    assert held.float().mean() > 0.9
    assert ((sm / N - m).abs() <= (5 * 0.5 / N ** 0.5 + 2.0 ** -16) * m.abs() / 8 + 1e-7 * m.abs())[held].all()
    assert ((sv / N - v).abs() <= (5 * 0.5 / N ** 0.5 + 2.0 ** -16) * v / 4 + 1e-7 * v)[held].all()


def test_adamw_range_of_the_blocks():
    """Moments of any size in a block: tiny ones, zeros, one large; v never reads as 0 where it is not."""
    n = 768
    g = np.zeros(n, np.float32)
    g[:256] = 10.0 ** np.linspace(-18, 3, 256)          # far below the block's largest: m drops out, v stays at the floor
    g[256:512] = np.float32(1e-25) * np.linspace(0, 1, 256)   # v underflows to 0 in fp32, m below 2^-90's reach too
    p = torch.zeros(n, device=DEV)
    t = mmf.AdamWTensor(p, torch.from_numpy(g).to(DEV), **mmf.adamw_state(p, 8))
    d = {"p": np.zeros(n, np.float32), "g": g, "m": np.zeros(n, np.float32), "v": np.zeros(n, np.float32),
         "weight_decay": 0.0, "eight": True}
    w = P.adamw(d, 0, **dict(HYPER, step=1))
    mmf.adamw_step([t], **dict(HYPER, step=1))
    assert np.array_equal(t.m.view(torch.uint8).cpu().numpy(), w["m_code"])
    assert np.array_equal(t.v.view(torch.uint8).cpu().numpy(), w["v_code"])
    assert np.array_equal(t.m_scale.cpu().numpy(), w["m_scale"])
    assert np.array_equal(t.v_scale.cpu().numpy(), w["v_scale"])
    v = t.v.float().cpu().numpy() * np.repeat(w["v_scale"], 256)
    assert ((v > 0) == (w["v"] > 0)).all() and (v[512:] == 0).all()


@pytest.mark.parametrize("bad", [float("inf"), float("nan"), 3e38])
def test_adamw_values_that_cannot_be_held(bad):
    """A non-finite gradient reaches its own element in fp32, and in 8 bits makes its block of 256 read as NaN;
    its neighbours' weights and the other blocks are as without it."""
    rng = np.random.default_rng(8)
    for eight in (False, True):
        t, d = adam_tensor(rng, 1000, eight, False, False, 0.0)
        t2 = mmf.AdamWTensor(**{k: (getattr(t, k).clone() if getattr(t, k) is not None else None)
                                for k in ("p", "g", "m", "v", "m_scale", "v_scale")})
        t.g[300] = bad
        mmf.adamw_step([t], **HYPER)
        mmf.adamw_step([t2], **HYPER)
        keep = torch.arange(1000, device=DEV) != 300
        assert torch.equal(t.p[keep], t2.p[keep])
        if eight:
            blocks = torch.isnan(t.v_scale).tolist()
            assert blocks == [False, True, False, False]
            same = torch.arange(1000, device=DEV) // 256 != 1
            assert torch.equal(t.v.view(torch.uint8)[same], t2.v.view(torch.uint8)[same])
            assert torch.equal(t.m.view(torch.uint8)[same], t2.m.view(torch.uint8)[same])
        else:
            assert torch.equal(t.m[keep], t2.m[keep]) and not torch.isfinite(t.v[300])


def test_adamw_scalars_from_the_device_and_graph_replays():
    """Captured once, replayed with each step's scalars copied to the device: the bits of separate calls."""
    rng = np.random.default_rng(10)
    made = [adam_tensor(rng, n, e, False, False, 0.1) for n, e in ((5000, True), (300, False), (4097, True))]
    fields = ("p", "g", "m", "v", "m_scale", "v_scale")
    copies = [mmf.AdamWTensor(**{k: (getattr(t, k).clone() if getattr(t, k) is not None else None) for k in fields},
                              weight_decay=0.1) for t, _ in made]
    tensors = [t for t, _ in made]
    per_step = [dict(HYPER, step=s, lr=1e-3 / s, grad_scale=1.0 / s, seed=50 + s) for s in (1, 2, 3)]
    dev = mmf.adamw_scalars(**per_step[0]).to(DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mmf.adamw_step(tensors, **HYPER, scalars=dev)
    for k in per_step:
        dev.copy_(mmf.adamw_scalars(**k))
        g.replay()
        mmf.adamw_step(copies, **k)
    torch.cuda.synchronize()
    for a, b in zip(tensors, copies):
        for k in ("p", "m", "v", "m_scale", "v_scale"):
            x, y = getattr(a, k), getattr(b, k)
            if x is not None:
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), k


def test_adamw_binding_refusals():
    p = torch.zeros(300, device=DEV)
    s8, s32 = mmf.adamw_state(p, 8), mmf.adamw_state(p)
    go = lambda **k: mmf.adamw_step([mmf.AdamWTensor(**{"p": p, "g": p.clone(), **s32, **k})], step=1, lr=1e-3)
    with pytest.raises(TypeError):
        go(m=s8["m"])
    with pytest.raises(TypeError):
        go(g=p.half())
    with pytest.raises(ValueError):
        go(m=s8["m"], v=s8["v"])
    with pytest.raises(ValueError):
        go(**{**s8, "m_scale": s8["m_scale"][:1]})
    with pytest.raises(ValueError):
        go(g=torch.zeros(299, device=DEV))
    with pytest.raises(ValueError):
        go(g=torch.zeros(600, device=DEV)[::2])
    with pytest.raises(ValueError):
        go(g=torch.zeros(300))
    with pytest.raises(mmf.MMFError):
        go(g=s32["m"])
    with pytest.raises(mmf.MMFError):
        mmf.adamw_step([mmf.AdamWTensor(p, p.clone(), **s32)], step=0, lr=1e-3)


# -- streams and graphs --------------------------------------------------------------

def test_side_stream_and_graph():
    """The operators on a stream given as an argument, and captured into two graphs that are replayed in turn with
    new inputs: each has the workspace it was captured with."""
    rng = np.random.default_rng(11)
    ids = [torch.from_numpy(make_ids(rng, 3000, 500, "mixed")).to(DEV) for _ in range(2)]
    dx = [bf(rng.standard_normal((3000, 64))).to(DEV) for _ in range(2)]
    scan = [[bf(rng.standard_normal((2, 200, 64))).to(DEV) for _ in range(4)] for _ in range(2)]
    want_e = [mmf.embed_bwd(i, d, 500) for i, d in zip(ids, dx)]
    want_s = [mmf.mlgru_scan_bwd(*s) for s in scan]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        e = mmf.embed_bwd(ids[0], dx[0], 500, stream=s)
        r = mmf.mlgru_scan_bwd(*scan[0], stream=s)
        side.synchronize()
        assert torch.equal(e, want_e[0]) and all(torch.equal(a, b) for a, b in zip(r, want_s[0]))
    graphs = []
    for _ in range(2):
        i, d, t = ids[0].clone(), dx[0].clone(), [x.clone() for x in scan[0]]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            e = mmf.embed_bwd(i, d, 500)
            r = mmf.mlgru_scan_bwd(*t)
        graphs.append((g, i, d, t, e, r))
    for k in (1, 0, 1):
        for n, (g, i, d, t, _, _) in enumerate(graphs):
            src = (k + n) % 2
            i.copy_(ids[src])
            d.copy_(dx[src])
            for a, b in zip(t, scan[src]):
                a.copy_(b)
            g.replay()
        torch.cuda.synchronize()
        for n, (_, _, _, _, e, r) in enumerate(graphs):
            src = (k + n) % 2
            assert torch.equal(e, want_e[src]) and all(torch.equal(a, b) for a, b in zip(r, want_s[src]))


# -- together ------------------------------------------------------------------------

def test_training_steps_of_a_token_mixer():
    """Embedding, the f, c, g projections, the recurrence and the o projection, then all of it backwards and an
    AdamW step whose weights are packed again, twice over: every operator against its plain form on the inputs it
    got, and the second step's forward on the first step's weights."""
    rng = np.random.default_rng(12)
    B, T, V, D = 2, 33, 50, 128
    M = B * T
    W = {n: torch.from_numpy((0.02 * rng.standard_normal((D, D))).astype(np.float32)).to(DEV) for n in "fcgo"}
    gamma = {n: torch.ones(D, device=DEV) for n in ("in", "o")}
    table = torch.from_numpy((0.02 * rng.standard_normal((V, D))).astype(np.float32)).to(DEV)
    table_bf16 = table.to(torch.bfloat16)
    params = {**W, **{"gamma_" + k: v for k, v in gamma.items()}, "table": table}
    state = {n: mmf.adamw_state(p, 8 if n in W else 32) for n, p in params.items()}
    ids = torch.from_numpy(make_ids(rng, M, V, "mixed")).to(DEV)
    d_y = bf(rng.standard_normal((M, D))).to(DEV)
    for step in (1, 2):
        packed = {n: mmf.pack_ternary(w) for n, w in W.items()}
        x = mmf.embed_fwd(ids, table_bf16, scale=8.0)
        pre = mmf.bitlinear_fwd_group(x, gamma["in"], [(*packed[n], D) for n in "fcg"])
        pre = [t.view(B, T, D) for t in pre]
        o, _ = mmf.mlgru_scan(*pre)
        y = mmf.bitlinear_fwd(o.view(M, D), gamma["o"], *packed["o"], D)
        assert torch.isfinite(y.float()).all()
        d_o, dg_o, dW_o = mmf.bitlinear_bwd(d_y, o.view(M, D), gamma["o"], *packed["o"])
        got = mmf.mlgru_scan_bwd(*pre, d_o.view(B, T, D))
        a = [f64(t) for t in (*pre, d_o.view(B, T, D))]
        want = P.scan_bwd(*a)
        bound = P.scan_bwd_bounds(want, *a)
        for n, t in zip(("df", "dc", "dg", "dh0"), got):
            assert (np.abs(f64(t) - want[n]) <= bound[n]).all(), n
        grads, dxs, dgs = {"o": dW_o, "gamma_o": dg_o}, [], []
        for n, t in zip("fcg", got):
            dx, dg, grads[n] = mmf.bitlinear_bwd(t.view(M, D), x, gamma["in"], *packed[n])
            dxs.append(dx.float())
            dgs.append(dg)
        grads["gamma_in"] = dgs[0] + dgs[1] + dgs[2]
        dx = (dxs[0] + dxs[1] + dxs[2]).to(torch.bfloat16)
        grads["table"] = mmf.embed_bwd(ids, dx, V, scale=8.0)
        e, eb = P.embed_bwd(ids.cpu().numpy(), f64(dx), V, 8.0)
        assert (np.abs(f64(grads["table"]) - e) <= eb).all()
        k = dict(HYPER, step=step, seed=step)
        descs, tensors = [], []
        for n, p in params.items():
            s = state[n]
            t = mmf.AdamWTensor(p, grads[n], **s, p_bf16=table_bf16 if n == "table" else None,
                                weight_decay=0.1 if n in W else 0.0)
            eight = "m_scale" in s
            val = lambda c, sc: (c.float() * sc.repeat_interleave(256)[:c.numel()].view(c.shape)).cpu().numpy().ravel()
            descs.append({"p": p.cpu().numpy().ravel(), "g": grads[n].cpu().numpy().ravel(), "eight": eight,
                          "m": val(s["m"], s["m_scale"]) if eight else s["m"].cpu().numpy().ravel(),
                          "v": val(s["v"], s["v_scale"]) if eight else s["v"].cpu().numpy().ravel(),
                          "weight_decay": t.weight_decay})
            tensors.append(t)
        mmf.adamw_step(tensors, **k)
        for i, (t, d) in enumerate(zip(tensors, descs)):
            w = P.adamw(d, i, **k)
            assert (np.abs(f64(t.p).ravel() - w["p"]) <= w["bound"]).all()
            if d["eight"]:
                assert np.array_equal(t.m.view(torch.uint8).cpu().numpy().ravel(), w["m_code"])
                assert np.array_equal(t.v.view(torch.uint8).cpu().numpy().ravel(), w["v_code"])
        assert torch.equal(table_bf16, table.to(torch.bfloat16))
        before = x
    assert not torch.equal(before, mmf.embed_fwd(ids, table_bf16, scale=8.0))


def test_two_calls_at_once_and_stream_handles():
    """Calls that overlap on two streams, each with its own buffers, and streams given as handles, 0 among them."""
    rng = np.random.default_rng(13)
    ids = [torch.from_numpy(make_ids(rng, 5000, 3000, "mixed")).to(DEV) for _ in range(2)]
    dx = [bf(rng.standard_normal((5000, 512))).to(DEV) for _ in range(2)]
    scan = [[bf(rng.standard_normal((4, 700, 512))).to(DEV) for _ in range(4)] for _ in range(2)]
    table = torch.randn(3000, 512, device=DEV)
    want = [(mmf.embed_bwd(i, d, 3000), mmf.mlgru_scan_bwd(*s), mmf.embed_fwd(i, table)) for i, d, s in zip(ids, dx, scan)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [None, None]
        for k, s in enumerate(streams):
            got[k] = (mmf.embed_bwd(ids[k], dx[k], 3000, stream=s), mmf.mlgru_scan_bwd(*scan[k], stream=s),
                      mmf.embed_fwd(ids[k], table, stream=s))
        torch.cuda.synchronize()
        for (e, r, x), (we, wr, wx) in zip(got, want):
            assert torch.equal(e, we) and torch.equal(x, wx) and all(torch.equal(a, b) for a, b in zip(r, wr))
    x = mmf.embed_fwd(ids[0], table, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(x, want[0][2])


def test_given_buffers():
    """Outputs and workspaces of the caller's; a short workspace and wrong shapes are refused."""
    rng = np.random.default_rng(14)
    t = [bf(rng.standard_normal((2, 2500, 64))).to(DEV) for _ in range(4)]
    want = mmf.mlgru_scan_bwd(*t)
    outs = [torch.empty_like(t[0]) for _ in range(3)]
    dh0 = torch.empty(2, 64, device=DEV)
    ws = torch.empty(mmf.mlgru_scan_bwd_workspace_bytes(2, 2500, 64), dtype=torch.uint8, device=DEV)
    got = mmf.mlgru_scan_bwd(*t, outs=outs, dh0=dh0, workspace=ws)
    assert got[3] is dh0 and all(a is b for a, b in zip(got, outs))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(ValueError, match="workspace"):
        mmf.mlgru_scan_bwd(*t, workspace=ws[:-256])
    with pytest.raises(ValueError):
        mmf.mlgru_scan_bwd(t[0], t[1], t[2], t[3][:, :-1])
    with pytest.raises(ValueError):
        mmf.mlgru_scan_bwd(*t, h0=torch.zeros(2, 63, device=DEV))
    with pytest.raises(TypeError):
        mmf.mlgru_scan_bwd(*t[:3], t[3].float())
    ids = torch.from_numpy(make_ids(rng, 2000, 50, "mixed")).to(DEV)
    dx = bf(rng.standard_normal((2000, 64))).to(DEV)
    ws = torch.empty(mmf.embed_bwd_workspace_bytes(50, 2000, 64), dtype=torch.uint8, device=DEV)
    assert torch.equal(mmf.embed_bwd(ids, dx, 50, workspace=ws), mmf.embed_bwd(ids, dx, 50))
    with pytest.raises(ValueError, match="workspace"):
        mmf.embed_bwd(ids, dx, 50, workspace=ws[:-256])
    with pytest.raises(ValueError, match="out"):
        mmf.embed_bwd(ids, dx, 50, accumulate=True)
    with pytest.raises(ValueError):
        mmf.embed_bwd(ids, dx[:-1], 50)
    with pytest.raises(ValueError):
        mmf.embed_bwd(ids, dx, 50, out=torch.zeros(51, 64, device=DEV))
    with pytest.raises(mmf.MMFError):
        mmf.embed_fwd(ids[1:], torch.zeros(50, 64, device=DEV))     # not on 16 bytes
    two_d = ids.view(40, 50)
    assert mmf.embed_fwd(two_d, torch.zeros(50, 64, device=DEV)).shape == (40, 50, 64)
    assert torch.equal(mmf.embed_bwd(two_d, dx.view(40, 50, 64), 50), mmf.embed_bwd(ids, dx, 50))


def test_embed_offsets_beyond_32_bits():
    """The most tokens a call takes, with more than 2^32 elements in x and dx."""
    M, K, V = 65535 * 256, 264, 1000
    g = torch.Generator(device=DEV).manual_seed(1)
    ids = torch.randint(0, V, (M,), device=DEV, dtype=torch.int32, generator=g)
    table = torch.randn(V, K, device=DEV, generator=g)
    x = mmf.embed_fwd(ids, table, scale=2.0)
    for a in (0, M // 2, M - 1000):
        assert torch.equal(x[a:a + 1000], (table[ids[a:a + 1000].long()] * 2.0).to(torch.bfloat16))
    d = mmf.embed_bwd(ids, x, V)
    for v in (0, V // 2, V - 1):
        n = int((ids == v).sum())
        row = x[M - 1 - int((ids.flip(0) == v).int().argmax())].double()   # all of a word's rows are the same here
        assert ((d[v].double() - n * row).abs() <= (256 + 3) * P.U * n * row.abs()).all()
