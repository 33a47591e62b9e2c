"""The latent-attention entry points' refusals, each from a call that is right but for the one altered argument: its arrays
lie apart, and without a GPU it gets as far as the launch (KDA_ERR_CUDA).  The addresses are made up, so machines with a GPU
do not make these calls."""
import pytest
import torch

from gated_delta_rule_127_b200 import build as kbuild
from gated_delta_rule_127_b200 import kda
from test_mla_host import CACHE_REFUSALS, FAKE, INV, OK, UNS, _decode, _far, _prefill, _read, _write

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses")
E4M3 = kda.KDA_E4M3


@pytest.fixture(scope="module", autouse=True)
def lib():
    kbuild.build()
    return kda.load_library()


WRITE = dict(latent=_far(0), pe=_far(1), cl=_far(2), cp=_far(3), table=_far(4), lens=_far(5))
READ = dict(latent=_far(0), pe=_far(1), cl=_far(2), cp=_far(3), table=_far(4), starts=_far(5))
DECODE = dict(q=_far(0), qp=_far(1), cl=_far(2), cp=_far(3), table=_far(4), lens=_far(5), o=_far(6), lse=_far(7))
PREFILL = dict(q=_far(0), kv=_far(1), kp=_far(2), cq=_far(3), ck=_far(4), o=_far(5), lse=_far(6))


def _refused(call, lib, right, kw, expect):
    assert call(lib, **right) == kda.KDA_ERR_CUDA
    assert call(lib, **{**right, **kw}) == expect


@pytest.mark.parametrize("kw,expect", CACHE_REFUSALS + [(dict(lens=None), INV), (dict(lens=FAKE + 1), INV), (dict(din=E4M3), INV),
                                                        (dict(pe=FAKE + 8), INV), (dict(cl=FAKE + 4), INV), (dict(cp=None), INV)])
def test_cache_write(lib, kw, expect):
    _refused(_write, lib, WRITE, kw, expect)


@pytest.mark.parametrize("kw,expect", CACHE_REFUSALS + [(dict(starts=FAKE + 1), INV), (dict(do=E4M3), INV), (dict(pe=FAKE + 8), INV),
                                                        (dict(cl=FAKE + 4), INV), (dict(cp=None), INV)])
def test_cache_read(lib, kw, expect):
    _refused(_read, lib, READ, kw, expect)


@pytest.mark.parametrize("kw,expect", [
    (dict(dl=576), UNS), (dict(dl=0), INV), (dict(dp=32), UNS), (dict(page=48), UNS), (dict(page=8), UNS), (dict(page=2048), UNS),
    (dict(pages=-1), INV), (dict(pages=1 << 26), UNS), (dict(width=-1), INV), (dict(width=1 << 26), UNS),
    (dict(dc=kda.KDA_FP32), UNS), (dict(dc=7), INV), (dict(dc=E4M3), INV), (dict(dc=E4M3, cs=FAKE + 4), INV),
    (dict(dq=kda.KDA_FP32), UNS), (dict(dq=E4M3), INV), (dict(do=5), INV), (dict(do=E4M3), INV), (dict(B=-1), INV),
    (dict(S=0), INV), (dict(H=0), INV), (dict(S=300, H=300), UNS), (dict(B=1 << 30, H=4), UNS),
    (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(q=None), INV), (dict(q=FAKE + 8), INV),
    (dict(qp=None), INV), (dict(qp=FAKE + 2), INV), (dict(o=None), INV), (dict(o=FAKE + 8), INV), (dict(lse=FAKE + 2), INV),
    (dict(lens=None), INV), (dict(lens=FAKE + 2), INV), (dict(table=None), INV), (dict(table=FAKE + 2), INV), (dict(cl=None), INV),
    (dict(cl=FAKE + 8), INV), (dict(cp=None), INV), (dict(cp=FAKE + 8), INV), (dict(ws=FAKE + 4, wsb=1 << 24), INV),
    (dict(ws=_far(9), wsb=16), INV), (dict(B=0, q=None, o=None, lse=None), OK),
])
def test_decode(lib, kw, expect):
    _refused(_decode, lib, DECODE, kw, expect)


@pytest.mark.parametrize("kw,expect", [
    (dict(dn=64), UNS), (dict(dn=0), INV), (dict(dp=32), UNS), (dict(dv=64), UNS), (dict(dt=kda.KDA_FP32), UNS),
    (dict(dt=E4M3), INV), (dict(do=E4M3), INV), (dict(H=65536), UNS), (dict(H=0), INV), (dict(causal=2), INV),
    (dict(scale=float("-inf")), INV), (dict(scale=float("nan")), INV), (dict(Tq=-1), INV), (dict(Tk=-1), INV),
    (dict(Tq=1 << 31), UNS), (dict(Tk=1 << 31), UNS), (dict(B=0), INV), (dict(Tq=7, cq=None), INV), (dict(Tk=7, ck=None), INV),
    (dict(q=None), INV), (dict(q=FAKE + 2), INV), (dict(kv=None), INV), (dict(kv=FAKE + 8), INV), (dict(kp=None), INV),
    (dict(kp=FAKE + 4), INV), (dict(o=None), INV), (dict(o=FAKE + 4), INV), (dict(lse=FAKE + 1), INV), (dict(cq=FAKE + 2), INV),
    (dict(ck=FAKE + 2), INV), (dict(Tq=0, q=None, o=None, lse=None), OK),
])
def test_prefill(lib, kw, expect):
    _refused(_prefill, lib, PREFILL, kw, expect)


def test_calls_that_are_right(lib):
    # the arguments that the altered calls leave out: they are no reason to refuse
    for call, right, kws in (
            (_write, WRITE, [dict(cu=_far(8)), dict(T=9, cu=_far(8)), dict(din=kda.KDA_FP32), dict(dc=E4M3, cs=_far(9))]),
            (_read, READ, [dict(starts=None), dict(cu=_far(8), T=9), dict(do=kda.KDA_FP32), dict(dc=E4M3, cs=_far(9))]),
            (_decode, DECODE, [dict(lse=None), dict(do=kda.KDA_FP32), dict(dc=E4M3, cs=_far(9)), dict(scale=0.0), dict(scale=-1.0),
                               dict(ws=_far(9), wsb=lib.kda_mla_decode_workspace_size(2, 1, 32, 512, 64))]),
            (_prefill, PREFILL, [dict(cq=None, ck=None), dict(lse=None), dict(do=kda.KDA_FP32), dict(causal=0), dict(Tq=7),
                                 dict(Tk=0, kv=None, kp=None)])):
        for kw in kws:
            assert call(lib, **{**right, **kw}) == kda.KDA_ERR_CUDA, kw
