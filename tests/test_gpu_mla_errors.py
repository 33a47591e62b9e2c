"""A call that fails on the host (here: on a stream whose capture has become invalid, so that nothing is launched) reports
it once: the next call, of any entry point, is not refused for it."""
import ctypes

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


class _InvalidCapture:
    """A stream in a capture that a synchronisation has made invalid (the driver's interface, so that the runtime that
    torch uses keeps no error of it)."""

    def __enter__(self):
        self.drv = ctypes.CDLL("libcuda.so.1")
        self.stream = torch.cuda.Stream()
        h = ctypes.c_void_p(self.stream.cuda_stream)
        assert self.drv.cuStreamBeginCapture_v2(h, 2) == 0          # CU_STREAM_CAPTURE_MODE_RELAXED
        assert self.drv.cuStreamSynchronize(h) != 0
        return self.stream.cuda_stream

    def __exit__(self, *_):
        graph = ctypes.c_void_p()
        assert self.drv.cuStreamEndCapture(ctypes.c_void_p(self.stream.cuda_stream), ctypes.byref(graph)) != 0


def _calls(stream):
    """The latent-attention entry points on prepared arrays, as calls of the library on `stream`."""
    lib = kda.load_library()
    cache = Cache([100], 64, BF16, DEV).fill(2)
    q, qp = torch.zeros(1, 1, 4, LATENT, dtype=BF16, device=DEV), torch.zeros(1, 1, 4, PE, dtype=BF16, device=DEV)
    o = torch.zeros_like(q)
    lat, pe = torch.zeros(100, LATENT, dtype=BF16, device=DEV), torch.zeros(100, PE, dtype=BF16, device=DEV)
    Q, KV = torch.zeros(8, 4, 192, dtype=BF16, device=DEV), torch.zeros(8, 4, 256, dtype=BF16, device=DEV)
    O = torch.zeros(8, 4, 128, dtype=BF16, device=DEV)
    ws = torch.zeros(kda.kda_mla_decode_workspace_size(1, 1, 4), dtype=torch.uint8, device=DEV)
    keep = (cache, q, qp, o, lat, pe, Q, KV, O, ws)
    p = lambda t: t.data_ptr()  # noqa: E731
    pages, width = cache.pages, cache.table.shape[1]
    return keep, {
        "write": lambda: lib.kda_mla_cache_write(p(lat), p(pe), None, p(cache.seq_lens), 100, 1, 512, 64, 0, 0, p(cache.latent),
                                                 p(cache.pe), None, p(cache.table), pages, 64, width, stream),
        "read": lambda: lib.kda_mla_cache_read(p(cache.latent), p(cache.pe), None, p(cache.table), None, None, 100, 1, 512, 64,
                                               pages, 64, width, 0, 0, p(lat), p(pe), stream),
        "decode": lambda: lib.kda_mla_decode(p(q), p(qp), p(cache.latent), p(cache.pe), None, p(cache.table), p(cache.seq_lens),
                                             1, 1, 4, 512, 64, pages, 64, width, 0.1, 0, 0, 0, p(o), None, p(ws), ws.numel(),
                                             stream),
        "prefill": lambda: lib.kda_mla_prefill(p(Q), p(KV), p(pe), None, None, 8, 8, 1, 4, 128, 64, 128, 1, 0.1, 0, 0, p(O),
                                               None, stream),
        "status": lambda: lib.kda_get_device_status(stream, None),
    }


@pytest.mark.parametrize("name", ["write", "read", "decode", "prefill", "status"])
def test_a_failed_call_is_reported_once(name):
    state = gen.make_decode_state(2, 2, 128, 128, seed=0, device=DEV)
    x = gen.make_decode_step(0, 2, 2, 128, 128, seed=0, device=DEV)
    kda.kda_decode_step(x.q, x.k, x.v, x.log_alpha, x.beta, state)
    keep, good = _calls(torch.cuda.current_stream().cuda_stream)
    assert good[name]() == kda.KDA_OK
    torch.cuda.synchronize()
    with _InvalidCapture() as stream:
        keep_bad, bad = _calls(stream)
        assert bad[name]() == kda.KDA_ERR_CUDA
    kda.kda_decode_step(x.q, x.k, x.v, x.log_alpha, x.beta, state)  # raises where the old error is taken for its own
    assert good["prefill"]() == kda.KDA_OK
    assert kda.kda_get_device_status() == (kda.KDA_OK, 0)
