"""Streams given as raw handles: another stream's, and the runtime's names for the default ones (0 and 1 the legacy
default stream, 2 the thread's own), as every entry point of the binding takes them."""
import pytest
import torch

from gated_delta_rule_127_b200 import inputs as gen
from gated_delta_rule_127_b200 import kda
from mla_ref import LATENT, PE, Cache

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_127_b200 import build
    build.build()
    kda.load_library()


@pytest.mark.parametrize("which", ["none", "stream", "handle", 0, 1, 2])
def test_stream_handles(which):
    side = torch.cuda.Stream()
    stream = {"none": None, "stream": side, "handle": side.cuda_stream}.get(which, which)
    r = lambda *s: torch.randn(*s, device=DEV).to(BF16)  # noqa: E731
    n = [130, 7]
    cache = Cache(n, 64, BF16, DEV)
    cu = torch.tensor([0, 130, 137], dtype=torch.int32, device=DEV)
    lat, pe, q, qp = r(137, LATENT), r(137, PE), r(2, 1, 8, LATENT), r(2, 1, 8, PE)
    Q, KV = r(137, 4, 192), r(137, 4, 256)
    state = gen.make_decode_state(2, 2, 128, 128, seed=0, device=DEV)
    x = gen.make_decode_step(0, 2, 2, 128, 128, seed=0, device=DEV)

    def calls(**kw):
        kda.kda_mla_cache_write(lat, pe, cache.latent, cache.pe, cache.table, cache.seq_lens, cu, **kw)
        got = kda.kda_mla_cache_read(cache.latent, cache.pe, cache.table, cu, 137, **kw)
        dec = kda.kda_mla_decode(q, qp, cache.latent, cache.pe, cache.table, cache.seq_lens, softmax_scale=0.07,
                                 output_lse=True, **kw)
        pre = kda.kda_mla_prefill(Q, KV, pe, cu, cu, softmax_scale=0.07, output_lse=True, **kw)
        torch.cuda.synchronize()
        return (*got, *dec, *pre)

    want = calls()
    torch.cuda.synchronize()
    got = calls(stream=stream)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    kda.kda_decode_step(x.q, x.k, x.v, x.log_alpha, x.beta, state, stream=stream)
    torch.cuda.synchronize()
    assert kda.kda_get_device_status() == (kda.KDA_OK, 0)
