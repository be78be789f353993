"""Where a NaN among the recurrence gradient's inputs goes: to the outputs that
the formulas make of it, and to no other token."""
import numpy as np
import pytest
import torch

import training_plain as P
from bitlinear_rmsnorm_quant_b200 import mmf

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NAMES = ("df", "dc", "dg", "dh0")


@pytest.fixture(autouse=True, scope="module")
def _built():
    from bitlinear_rmsnorm_quant_b200 import build
    build.build()
    torch.cuda.set_device(0)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


# one launch; segments with tensor copies, of one to four warps' channels; segments without
SHAPES = [(2, 20, 64), (2, 2048, 64), (1, 1003, 128), (1, 1003, 192), (2, 1003, 256), (2, 515, 66), (1, 900, 34)]


@pytest.mark.parametrize("B,T,D", SHAPES)
@pytest.mark.parametrize("which", ["f", "c", "g", "do"])
def test_nan_reaches_what_the_formulas_say(B, T, D, which):
    """One NaN at the first, a middle or the last token of a channel, each in a
    channel of its own; pairs of channels share a lane, so their neighbours are
    looked at too.  An output is NaN where the formulas give NaN, and elsewhere
    as close to them as without the NaN, on which it does not depend."""
    rng = np.random.default_rng(T + D)
    clean = [torch.from_numpy(2 * rng.standard_normal((B, T, D)).astype(np.float32)).to(torch.bfloat16) for _ in range(4)]
    bad = [t.clone() for t in clean]
    at = [(B - 1, 0, 1), (0, T // 2, 4), (0, T // 2 + 3, 7), (B - 1, T - 1, D - 1), (0, T - 1, D - 2), (0, 8, 11)]
    for b, t, k in at:
        bad[("f", "c", "g", "do").index(which)][b, t, k] = float("nan")
    h0, dl = (torch.from_numpy(rng.standard_normal((B, D)).astype(np.float32)) for _ in range(2))
    got = mmf.mlgru_scan_bwd(*(t.to(DEV) for t in bad), h0=h0.to(DEV), dh_last=dl.to(DEV))
    with np.errstate(invalid="ignore"):
        mask = P.scan_bwd(*(f64(t) for t in bad), f64(h0), f64(dl))
    a = [f64(t) for t in clean]
    want = P.scan_bwd(*a, f64(h0), f64(dl))
    bound = P.scan_bwd_bounds(want, *a)
    for n, t in zip(NAMES, got):
        nan = np.isnan(mask[n])
        assert np.array_equal(np.isnan(f64(t)), nan), n
        assert (np.abs(f64(t) - want[n]) <= bound[n])[~nan].all(), n
