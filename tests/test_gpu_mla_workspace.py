"""The workspace's size as the library itself checks it: a call that is right but for its workspace."""
import pytest
import torch

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


def test_a_workspace_of_too_few_bytes_is_refused():
    cache = Cache([100], 64, BF16, DEV).fill(2)
    q = torch.randn(1, 1, 32, LATENT, device=DEV).to(BF16)
    qp = torch.randn(1, 1, 32, PE, device=DEV).to(BF16)
    o = torch.zeros_like(q)
    need = kda.kda_mla_decode_workspace_size(1, 1, 32)
    assert need > 0
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    lib = kda.load_library()

    def call(size):
        return lib.kda_mla_decode(q.data_ptr(), qp.data_ptr(), cache.latent.data_ptr(), cache.pe.data_ptr(), None,
                                  cache.table.data_ptr(), cache.seq_lens.data_ptr(), 1, 1, 32, 512, 64, cache.pages, 64,
                                  cache.table.shape[1], 0.1, 0, 0, 0, o.data_ptr(), None, ws.data_ptr(), size, None)

    assert call(need) == kda.KDA_OK
    assert call(need - 16) == kda.KDA_ERR_INVALID_ARG
    assert call(1) == kda.KDA_ERR_INVALID_ARG
    assert call(0) == kda.KDA_OK       # none given
    assert kda.kda_get_device_status() == (kda.KDA_OK, 0)
