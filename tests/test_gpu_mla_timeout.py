"""The timeout path of the latent-attention kernels, without hanging or faulting the GPU: with the roles' waits bounded at a
few polls (include/kda_testing.h) some of them give up in the middle of a tile.  All roles then leave their loops,
drain what they have in flight (those waits keep their default bound) and meet at the kernel's end: the call comes back
promptly, and the next normal one gives the same bits as one made before."""
import math
import time

import pytest
import torch

from gated_delta_rule_127_b200 import kda
from mla_ref import LATENT, PE, Cache, cu_of

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16
SCALE = 1.0 / math.sqrt(192)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_127_b200 import build
    build.build()
    kda.load_library()


def _decode(dtype, S, H):
    cache = Cache([2000, 65, 700, 0], 32, dtype, DEV).fill(2)
    g = torch.Generator(device=DEV).manual_seed(5)
    q = torch.randn(4, S, H, LATENT, generator=g, device=DEV).to(BF16)
    qp = torch.randn(4, S, H, PE, generator=g, device=DEV).to(BF16)
    return lambda: kda.kda_mla_decode(q, qp, cache.latent, cache.pe, cache.table, cache.seq_lens, softmax_scale=SCALE,
                                      cache_scale=cache.scale, output_lse=True)


def _prefill(causal):
    nq, nk = [600, 130, 40], [900, 130, 20]
    g = torch.Generator(device=DEV).manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF16)  # noqa: E731
    q, kv, kp = r(sum(nq), 3, 192), r(sum(nk), 3, 256), r(sum(nk), 64)
    cq, ck = cu_of(nq, DEV), cu_of(nk, DEV)
    return lambda: kda.kda_mla_prefill(q, kv, kp, cq, ck, causal=causal, softmax_scale=SCALE, output_lse=True)


CASES = {"decode_bf16": lambda: _decode(BF16, 1, 32), "decode_bf16_64_rows": lambda: _decode(BF16, 2, 32),
         "decode_e4m3": lambda: _decode(torch.float8_e4m3fn, 1, 32), "prefill_causal": lambda: _prefill(True),
         "prefill_full": lambda: _prefill(False)}


@pytest.mark.parametrize("polls", [0, 1, 2, 4])
@pytest.mark.parametrize("case", sorted(CASES))
def test_small_wait_bound_ends_promptly_and_leaves_the_context_usable(case, polls):
    call = CASES[case]()
    ref = call()
    assert kda.kda_get_device_status() == (kda.KDA_OK, 0)
    kda.kda_testing_set_wait_limit(polls)
    try:
        t0 = time.monotonic()
        call()
        st, flags = kda.kda_get_device_status()  # synchronises the stream
        elapsed = time.monotonic() - t0
    finally:
        kda.kda_testing_set_wait_limit(-1)
    if polls == 0:  # with some polls a wait may still be met in time
        assert st == kda.KDA_ERR_TIMEOUT
    assert flags in (0, kda.KDA_DEVFLAG_TIMEOUT) and elapsed < 1.0, (flags, elapsed)
    again = call()
    assert kda.kda_get_device_status() == (kda.KDA_OK, 0)
    assert torch.equal(again[0], ref[0]) and torch.equal(again[1], ref[1])
