"""The seed of the AdamW step's rounding noise, without a GPU."""
import pytest
import torch

from bitlinear_rmsnorm_quant_b200 import mmf


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bitlinear_rmsnorm_quant_b200 import build
    build.build()


def _seed(**k):
    return mmf.adamw_scalars(lr=1e-3, **k)[16:24].view(torch.int64).item()


def test_default_seed_is_the_step():
    """A seed that stays from step to step would give every element the same threshold at each of them."""
    assert [_seed(step=s) for s in (1, 2, 300)] == [1, 2, 300]
    assert _seed(step=5, seed=0) == 0 and _seed(step=5, seed=9) == 9


def test_seed_beyond_64_bits_is_refused():
    assert _seed(step=1, seed=(1 << 64) - 1) == -1 and _seed(step=1, seed=-1) == -1
    for seed in (1 << 64, -(1 << 63) - 1):
        with pytest.raises(ValueError, match="seed"):
            _seed(step=1, seed=seed)
