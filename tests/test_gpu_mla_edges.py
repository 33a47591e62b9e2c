"""The ends of the e4m3 cache's range."""
import math

import pytest
import torch

from gated_delta_rule_127_b200 import kda
from mla_ref import LATENT, PE, Cache

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
E4M3, BF16 = torch.float8_e4m3fn, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_127_b200 import build
    build.build()
    kda.load_library()


@pytest.mark.parametrize("source", [BF16, torch.float32])
def test_the_largest_values_through_an_e4m3_cache(source):
    top = torch.finfo(source).max
    rows = [top, 247 * 2.0 ** 120, 240 * 2.0 ** 120, 448 * 2.0 ** 119, math.inf, 1.5 * 2.0 ** 100]
    latent = torch.zeros(len(rows), LATENT, dtype=source, device=DEV)
    latent[:, 7] = torch.tensor(rows, dtype=torch.float64).to(source).to(DEV)
    latent[:, 8] = -latent[:, 7]
    pe = torch.zeros(len(rows), PE, dtype=source, device=DEV)
    cache = Cache([len(rows)], 16, E4M3, DEV)
    kda.kda_mla_cache_write(latent, pe, cache.latent, cache.pe, cache.table, cache.seq_lens, cache_scale=cache.scale)
    at = cache.rows(0, 0, len(rows))
    codes = cache.latent.view(torch.uint8).view(-1, LATENT)[at].view(E4M3).float()[:, 7]
    # e4m3 has 240, 256 and no value between: 247 goes down, the largest values up
    assert codes.tolist() == [256.0, 240.0, 240.0, 448.0, 448.0, 384.0]
    assert torch.log2(cache.scale.view(-1)[at]).tolist() == [120.0, 120.0, 120.0, 119.0, 120.0, 92.0]
    for dtype_o in (BF16, torch.float32):
        got, _ = kda.kda_mla_cache_read(cache.latent, cache.pe, cache.table, None, len(rows), cache_scale=cache.scale,
                                        dtype_o=dtype_o)
        want = [math.inf, 240 * 2.0 ** 120, 240 * 2.0 ** 120, 448 * 2.0 ** 119, math.inf, 1.5 * 2.0 ** 100]
        assert got[:, 7].double().tolist() == want and got[:, 8].double().tolist() == [-x for x in want]
    assert kda.kda_get_device_status() == (kda.KDA_OK, 0)
