"""8-bit moments over many steps: they follow the 32-bit ones in the mean as
long as the rounding noise is new at every step, which it is by default."""
import numpy as np
import pytest
import torch

import training_plain as P
from bitlinear_rmsnorm_quant_b200 import inputs as I
from bitlinear_rmsnorm_quant_b200 import mmf

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True, scope="module")
def _built():
    from bitlinear_rmsnorm_quant_b200 import build
    build.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("path", ["arguments", "scalars"])
def test_8bit_moments_follow_the_32bit_ones(path):
    """400 steps without a seed given, the gradients halved midway.

    Rounding an e5m2 code at random moves v by a variance of at most a quarter
    of the grid's step squared, the step a quarter of the value at most: 1/64 of
    the value squared.  The variance V (relative to v squared) that the moving
    average holds is then at most V = beta2^2 V (1 + 1/64) + 1/64, 0.19 at
    beta2 = 0.95, and of m (e4m3, an eighth of the value, beta1 = 0.9) 0.021.
    Over n elements the mean of the ratio to the exact moment is off by
    sqrt(V / n) a standard deviation, here taken six times; what is left of the
    moments before the halving (3 * 0.95^200 < 2e-4) and the 2^-17 of a step by
    which 16 random bits miss are far below.  1 / sqrt(v) is convex, so the mean
    step of p is at least the exact one's less the sampling's deviation: v is
    never below 0.05 of its limit, so 1 / sqrt(v) is at most 4.5 of its, a
    deviation of at most 2.3 / sqrt(n) of the mean.
    """
    n, steps, beta1, beta2 = 4096, 400, 0.9, 0.95
    gen = torch.Generator(device=DEV).manual_seed(1)
    size = torch.empty(n, device=DEV).uniform_(0.5, 2.0, generator=gen)
    sign = torch.where(torch.rand(n, device=DEV, generator=gen) < 0.5, -1.0, 1.0)
    p = {bits: torch.zeros(n, device=DEV) for bits in (8, 32)}
    g = torch.empty(n, device=DEV)
    tensors = {bits: mmf.AdamWTensor(p[bits], g, **mmf.adamw_state(p[bits], bits)) for bits in p}
    for step in range(1, steps + 1):
        g.copy_(size * sign * (1.0 if step <= steps // 2 else 0.5))
        for t in tensors.values():
            if path == "scalars":
                mmf.adamw_step([t], step=1, lr=1.0, beta1=beta1, beta2=beta2,
                               scalars=mmf.adamw_scalars(step=step, lr=1e-3, beta1=beta1, beta2=beta2).to(DEV))
            else:
                mmf.adamw_step([t], step=step, lr=1e-3, beta1=beta1, beta2=beta2)
    eight, full = tensors[8], tensors[32]
    m = eight.m.double() * eight.m_scale.double().repeat_interleave(256)
    v = eight.v.double() * eight.v_scale.double().repeat_interleave(256)
    for got, want, beta, grid in ((m, full.m, beta1, 1 / 8), (v, full.v, beta2, 1 / 4)):
        once = grid * grid / 4
        var = once / (1 - beta * beta * (1 + once))
        assert abs((got / want.double()).mean().item() - 1) <= 6 * (var / n) ** 0.5 + 1e-3
    moved = (p[8].double() / p[32].double()).mean().item()
    assert moved >= 1 - 6 * 2.3 / n ** 0.5


def plain_codes(g, seed, tensor):
    """The codes of m and v after a first step with beta 0.9 and 0.95 (0.1 g and 0.05 g^2 in fp32), by the draws of
    the stream whose key takes the seed's lower half as the input streams do and its upper half mixed."""
    key = I.mix_int(((seed & 0xFFFFFFFF) << 32) + tensor + I.mix_int(seed >> 32))
    z = I._mix(torch.arange(1, (g.size + 1) // 2 + 1) * I._s64(I._GOLDEN) + I._s64(key)).numpy().view(np.uint64)
    bits = np.stack([z & np.uint64(0xFFFFFFFF), z >> np.uint64(32)], 1).reshape(-1)[:g.size].astype(np.int64)
    m, v = g * np.float32(1 - 0.9), (g * g) * np.float32(1 - 0.95)
    return P.quantise(m, bits & 0xFFFF, 7, 3, 7, False)[0], P.quantise(v, bits >> 16, 14, 2, 15, True)[0]


@pytest.mark.parametrize("path", ["arguments", "scalars"])
def test_all_bits_of_the_seed_count(path):
    """Seeds that differ in their upper half alone give other codes, those of their own streams."""
    g = np.random.default_rng(2).standard_normal(2049).astype(np.float32)
    gd = torch.from_numpy(g).to(DEV)
    seen = []
    for seed in (5, 5 + (1 << 32), 5 + (1 << 33), 5 + (1 << 63), (1 << 64) - 1):
        ps = [torch.zeros(g.size, device=DEV) for _ in range(2)]
        ts = [mmf.AdamWTensor(p, gd, **mmf.adamw_state(p, 8)) for p in ps]
        if path == "scalars":
            mmf.adamw_step(ts, step=1, lr=1e-3, scalars=mmf.adamw_scalars(step=1, lr=1e-3, seed=seed).to(DEV))
        else:
            mmf.adamw_step(ts, step=1, lr=1e-3, seed=seed)
        for i, t in enumerate(ts):
            m, v = plain_codes(g, seed, i)
            assert np.array_equal(t.m.view(torch.uint8).cpu().numpy(), m)
            assert np.array_equal(t.v.view(torch.uint8).cpu().numpy(), v)
            seen.append(m)
    # two independent draws round a value apart a third of the time in the mean
    assert all((a != b).mean() > 0.1 for i, a in enumerate(seen) for b in seen[:i])
