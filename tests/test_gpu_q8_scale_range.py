"""Attention over block scales at the ends of what the append makes, 2^-64 and
2^120, against the bound of tests/q8_reference.py: weights that spread over many
binades count in the sums whatever their V scale is."""
import numpy as np
import pytest
import torch

from test_gpu_q8 import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_455_b200 import pa as mod
    return mod


def _case(seed, lens, hq, hkv, d, bs, chunks, v_exp):
    c = Case(seed, lens, hq, hkv, d, bs, chunks=chunks, spread=0.0)
    held = c.vp != 0x7F
    rng = np.random.default_rng(seed)
    # V codes from -2 to 2, so that no output leaves bf16; logits of some units
    codes = torch.from_numpy(rng.uniform(-2, 2, c.vp.shape).astype(np.float32))
    codes = codes.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    c.vp[held] = codes[held]
    c.vs[:] = np.exp2(v_exp(rng, c.vs.shape)).astype(np.float32)
    c.scale *= 2.0
    return c


RANGES = {
    "lowest": lambda rng, s: np.full(s, -64.0),
    "highest": lambda rng, s: np.full(s, 120.0),
    "near the highest": lambda rng, s: rng.integers(108, 121, s).astype(np.float64),
    "near the lowest": lambda rng, s: rng.integers(-64, -51, s).astype(np.float64),
    "all": lambda rng, s: rng.integers(-64, 121, s).astype(np.float64),
}


@pytest.mark.parametrize("name", list(RANGES))
@pytest.mark.parametrize("lens,hq,hkv,d,bs", [([300, 1, 40, 2000], 16, 4, 256, 16),
                                              ([1500, 90], 8, 1, 128, 32), ([700, 33], 4, 4, 128, 16)])
def test_decode(pa, name, lens, hq, hkv, d, bs):
    c = _case(81, lens, hq, hkv, d, bs, None, RANGES[name])
    c.check(c.decode(pa), False)
    c.check(c.decode(pa, workspace=False), False)


@pytest.mark.parametrize("name", list(RANGES))
@pytest.mark.parametrize("lens,chunks,hq,hkv,d,bs", [([300, 1, 40], [130, 1, 5], 16, 4, 256, 16),
                                                     ([2500], [4], 8, 1, 128, 32)])
def test_prefill(pa, name, lens, chunks, hq, hkv, d, bs):
    c = _case(82, lens, hq, hkv, d, bs, chunks, RANGES[name])
    c.check(c.prefill(pa), True)
