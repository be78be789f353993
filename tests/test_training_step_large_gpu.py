"""The training-step operators at sizes whose offsets pass 32 bits, and at the
widest tables: slices of the results against their plain forms."""
import numpy as np
import pytest
import torch

import training_plain as P
from bitlinear_rmsnorm_quant_b200 import inputs as I
from bitlinear_rmsnorm_quant_b200 import mmf

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _built():
    from bitlinear_rmsnorm_quant_b200 import build
    build.build()
    torch.cuda.set_device(0)
    yield
    torch.cuda.empty_cache()   # tens of GB a test


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("D", [16392, 16390])   # with tensor copies and without
def test_scan_bwd_offsets_beyond_32_bits(D):
    """More than 2^32 elements: the first and the last sequence's outer channels."""
    B, T = 32, 8192
    gen = torch.Generator(device=DEV).manual_seed(D)
    x = [torch.randn(B, T, D, dtype=torch.bfloat16, device=DEV, generator=gen) for _ in range(4)]
    got = mmf.mlgru_scan_bwd(*x)
    for b in (0, B - 1):
        for k in (slice(0, 32), slice(D - 32, D)):
            a = [f64(t[b:b + 1, :, k]) for t in x]
            want = P.scan_bwd(*a)
            bound = P.scan_bwd_bounds(want, *a)
            for n, t in zip(("df", "dc", "dg"), got):
                assert (np.abs(f64(t[b:b + 1, :, k]) - want[n]) <= bound[n]).all(), n
            assert (np.abs(f64(got[3][b:b + 1, k]) - want["dh0"]) <= bound["dh0"]).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_offsets_beyond_32_bits(bits):
    """One tensor of more than 2^32 elements: its first, last and middle blocks."""
    n, count = (1 << 32) + 1003, 4096
    hyper = dict(step=1, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, grad_scale=1.0, seed=77)
    gen = torch.Generator(device=DEV).manual_seed(bits)
    g = torch.randn(n, dtype=torch.bfloat16, device=DEV, generator=gen)
    p = torch.zeros(n, device=DEV)
    t = mmf.AdamWTensor(p, g, **mmf.adamw_state(p, bits))
    mmf.adamw_step([t], **hyper)
    for at in (0, 1 << 31, 1 << 32, (1 << 32) - count):
        s = slice(at, min(n, at + count))
        zero = np.zeros(s.stop - at, np.float32)
        w = P.adamw({"p": zero, "g": g[s].float().cpu().numpy(), "m": zero, "v": zero, "weight_decay": 0.0, "eight": False},
                    0, **hyper)
        assert (np.abs(f64(p[s]) - w["p"]) <= w["bound"]).all()
        if bits == 32:
            assert np.array_equal(t.m[s].cpu().numpy(), w["m"]) and np.array_equal(t.v[s].cpu().numpy(), w["v"])
            continue
        z = I.raw_u64(77, 0, at // 2, (zero.size + 1) // 2).numpy().view(np.uint64)
        z = np.stack([z & np.uint64(0xFFFFFFFF), z >> np.uint64(32)], 1).reshape(-1)[:zero.size].astype(np.int64)
        blocks = slice(at // 256, at // 256 - (-zero.size // 256))
        for code, scale, (c, sc) in ((t.m, t.m_scale, P.quantise(w["m"], z & 0xFFFF, 7, 3, 7, False)),
                                     (t.v, t.v_scale, P.quantise(w["v"], z >> 16, 14, 2, 15, True))):
            assert np.array_equal(code[s].view(torch.uint8).cpu().numpy(), c)
            assert np.array_equal(scale[blocks].cpu().numpy(), sc)


@pytest.mark.parametrize("M,V,K", [(1300, 3000, 8200), (1100, 150, 65536), (17000, 2000, 8192), (700, 400, 16400)])
@pytest.mark.parametrize("add", [False, True])
def test_embed_bwd_of_wide_tables(M, V, K, add):
    """Many column tiles, with rows to zero beside them."""
    rng = np.random.default_rng(M + K)
    ids = np.minimum((V * rng.random(M) ** 3).astype(np.int64), V - 1) * 2 % V   # frequent and absent ids
    gen = torch.Generator(device=DEV).manual_seed(K)
    dx = torch.randn(M, K, dtype=torch.bfloat16, device=DEV, generator=gen)
    base = torch.randn(V, K, device=DEV, generator=gen) if add else torch.full((V, K), float("nan"), device=DEV)
    out = base.clone()
    mmf.embed_bwd(torch.from_numpy(ids).to(DEV), dx, V, scale=0.5, out=out, accumulate=add)
    columns = torch.cat([torch.arange(0, 40), torch.arange(K // 2 - 20, K // 2 + 20), torch.arange(K - 40, K)])
    columns = torch.cat([columns, torch.arange(1, K, max(1, K // 64))]).to(DEV)
    want, bound = P.embed_bwd(ids, f64(dx[:, columns]), V, 0.5, f64(base[:, columns]) if add else None)
    assert (np.abs(f64(out[:, columns]) - want) <= bound).all()
    absent = torch.from_numpy(np.setdiff1d(np.arange(V), ids)).to(DEV)
    assert absent.numel() > V // 4
    assert torch.equal(out[absent], base[absent] if add else torch.zeros_like(out[absent]))
