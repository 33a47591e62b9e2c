"""The latent-attention entry points without a GPU: sizes, types, pointers and shapes are refused on the host."""
import pytest
import torch

from gated_delta_rule_127_b200 import build as kbuild
from gated_delta_rule_127_b200 import kda

FAKE = 1 << 20  # 16-byte aligned fake device address: never dereferenced, validation fails first
INV, UNS, OK = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_OK


@pytest.fixture(scope="module", autouse=True)
def lib():
    kbuild.build()
    return kda.load_library()


def test_entry_points_are_declared():
    assert {"kda_mla_cache_write", "kda_mla_cache_read", "kda_mla_decode", "kda_mla_decode_workspace_size",
            "kda_mla_prefill"} <= set(kda.header_symbols())


def _write(lib, **kw):
    a = dict(latent=FAKE, pe=FAKE, cu=None, lens=FAKE, T=8, B=2, dl=512, dp=64, din=kda.KDA_BF16, dc=kda.KDA_BF16,
             cl=FAKE, cp=FAKE, cs=None, table=FAKE, pages=4, page=64, width=2)
    a.update(kw)
    return lib.kda_mla_cache_write(a["latent"], a["pe"], a["cu"], a["lens"], a["T"], a["B"], a["dl"], a["dp"], a["din"],
                                   a["dc"], a["cl"], a["cp"], a["cs"], a["table"], a["pages"], a["page"], a["width"], None)


def _read(lib, **kw):
    a = dict(latent=FAKE, pe=FAKE, cu=None, starts=None, T=8, B=2, dl=512, dp=64, do=kda.KDA_BF16, dc=kda.KDA_BF16,
             cl=FAKE, cp=FAKE, cs=None, table=FAKE, pages=4, page=64, width=2)
    a.update(kw)
    return lib.kda_mla_cache_read(a["cl"], a["cp"], a["cs"], a["table"], a["cu"], a["starts"], a["T"], a["B"], a["dl"],
                                  a["dp"], a["pages"], a["page"], a["width"], a["dc"], a["do"], a["latent"], a["pe"], None)


CACHE_REFUSALS = [
    (dict(dl=256), UNS), (dict(dp=32), UNS), (dict(dl=0), INV), (dict(page=24), UNS), (dict(page=8), UNS),
    (dict(page=2048), UNS), (dict(page=0), INV), (dict(pages=-1), INV), (dict(pages=1 << 26), UNS),
    (dict(width=-1), INV), (dict(dc=kda.KDA_FP32), UNS), (dict(dc=9), INV), (dict(cl=None), INV), (dict(cp=FAKE + 8), INV),
    (dict(dc=kda.KDA_E4M3), INV),                    # no scale
    (dict(dc=kda.KDA_E4M3, cs=FAKE + 4), INV), (dict(table=None), INV), (dict(table=FAKE + 2), INV), (dict(B=0), INV),
    (dict(T=-1), INV), (dict(T=9), INV),             # no cu_seqlens: equal lengths
    (dict(latent=None), INV), (dict(latent=FAKE + 2), INV), (dict(pe=None), INV), (dict(cu=FAKE + 1), INV),
    (dict(T=1 << 31), UNS), (dict(T=0), OK), (dict(T=0, latent=None, cl=None, table=None), OK),
]


@pytest.mark.parametrize("kw,expect", CACHE_REFUSALS + [(dict(lens=None), INV), (dict(lens=FAKE + 1), INV),
                                                        (dict(din=kda.KDA_E4M3), INV)])
def test_cache_write_rejects_on_host(lib, kw, expect):
    assert _write(lib, **kw) == expect


@pytest.mark.parametrize("kw,expect", CACHE_REFUSALS + [(dict(starts=FAKE + 1), INV), (dict(do=kda.KDA_E4M3), INV)])
def test_cache_read_rejects_on_host(lib, kw, expect):
    assert _read(lib, **kw) == expect


def _decode(lib, **kw):
    a = dict(q=FAKE, qp=FAKE, cl=FAKE, cp=FAKE, cs=None, table=FAKE, lens=FAKE, B=2, S=1, H=32, dl=512, dp=64, pages=4,
             page=64, width=2, scale=0.1, dq=kda.KDA_BF16, dc=kda.KDA_BF16, do=kda.KDA_BF16, o=FAKE, lse=None, ws=None, wsb=0)
    a.update(kw)
    return lib.kda_mla_decode(a["q"], a["qp"], a["cl"], a["cp"], a["cs"], a["table"], a["lens"], a["B"], a["S"], a["H"],
                              a["dl"], a["dp"], a["pages"], a["page"], a["width"], a["scale"], a["dq"], a["dc"], a["do"],
                              a["o"], a["lse"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dl=576), UNS), (dict(page=48), UNS), (dict(dc=kda.KDA_FP32), UNS), (dict(dc=kda.KDA_E4M3), INV),
    (dict(dq=kda.KDA_FP32), UNS), (dict(dq=kda.KDA_E4M3), INV), (dict(do=5), INV), (dict(B=-1), INV), (dict(S=0), INV),
    (dict(H=0), INV), (dict(S=300, H=300), UNS), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
    (dict(q=None), INV), (dict(qp=FAKE + 2), INV), (dict(o=FAKE + 8), INV), (dict(lse=FAKE + 2), INV),
    (dict(lens=None), INV), (dict(ws=FAKE + 4, wsb=1 << 40), INV), (dict(B=0, q=None, o=None), OK),
])
def test_decode_rejects_on_host(lib, kw, expect):
    assert _decode(lib, **kw) == expect


def _prefill(lib, **kw):
    a = dict(q=FAKE, kv=FAKE, kp=FAKE, cq=None, ck=None, Tq=8, Tk=8, B=2, H=4, dn=128, dp=64, dv=128, causal=1, scale=0.1,
             dt=kda.KDA_BF16, do=kda.KDA_BF16, o=FAKE, lse=None)
    a.update(kw)
    return lib.kda_mla_prefill(a["q"], a["kv"], a["kp"], a["cq"], a["ck"], a["Tq"], a["Tk"], a["B"], a["H"], a["dn"],
                               a["dp"], a["dv"], a["causal"], a["scale"], a["dt"], a["do"], a["o"], a["lse"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dn=64), UNS), (dict(dp=32), UNS), (dict(dv=64), UNS), (dict(dt=kda.KDA_FP32), UNS), (dict(H=65536), UNS),
    (dict(dt=kda.KDA_E4M3), INV), (dict(do=kda.KDA_E4M3), INV), (dict(causal=2), INV), (dict(scale=float("-inf")), INV),
    (dict(Tq=-1), INV), (dict(B=0), INV), (dict(H=0), INV), (dict(Tq=7), INV), (dict(Tk=7), INV), (dict(q=FAKE + 2), INV),
    (dict(kv=None), INV), (dict(kp=FAKE + 4), INV), (dict(o=None), INV), (dict(lse=FAKE + 1), INV), (dict(cq=FAKE + 2), INV),
    (dict(Tq=0, q=None, o=None), OK),
])
def test_prefill_rejects_on_host(lib, kw, expect):
    assert _prefill(lib, **kw) == expect


def test_workspace_size_is_a_pure_host_function(lib):
    for args in ((0, 1, 32), (4, 0, 32), (4, 1, 0), (4, 300, 300)):
        assert kda.kda_mla_decode_workspace_size(*args) == 0
    assert kda.kda_mla_decode_workspace_size(4, 1, 32, 256, 64) == 0


# ---- the binding
def _tensors(dtype=torch.bfloat16):
    cl = torch.zeros(4, 64, 512, dtype=dtype)
    return dict(cache_latent=cl, cache_pe=torch.zeros(4, 64, 64, dtype=torch.bfloat16),
                page_table=torch.zeros(2, 2, dtype=torch.int32)), torch.ones(2, dtype=torch.int32)


def test_binding_refuses_shapes_and_types():
    c, lens = _tensors()
    q, qp = torch.zeros(2, 1, 4, 512, dtype=torch.bfloat16), torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16)
    dec = lambda q=q, qp=qp, lens=lens, **kw: kda.kda_mla_decode(q, qp, **{**c, **kw}, seq_lens=lens, softmax_scale=0.1)  # noqa: E731
    with pytest.raises(ValueError, match="q_latent"):
        dec(q=q[:1])
    with pytest.raises(ValueError, match="seq_lens"):
        dec(lens=lens.long())
    with pytest.raises(ValueError, match="page_table"):
        dec(page_table=c["page_table"].long())
    with pytest.raises(TypeError, match="cache_latent"):
        dec(cache_latent=c["cache_latent"].half())
    with pytest.raises(ValueError, match="cache_scale"):
        dec(cache_latent=c["cache_latent"].to(torch.float8_e4m3fn))
    with pytest.raises(ValueError, match="cache_scale"):
        dec(cache_scale=torch.ones(4, 64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        dec()
    with pytest.raises(ValueError, match="cu_seqlens"):
        kda.kda_mla_cache_write(torch.zeros(4, 512), torch.zeros(4, 64), **c, seq_lens=lens, cu_seqlens=torch.zeros(2))
    with pytest.raises(TypeError, match="share"):
        kda.kda_mla_cache_write(torch.zeros(4, 512), torch.zeros(4, 64).bfloat16(), **c, seq_lens=lens)
    with pytest.raises(ValueError, match="latent"):
        kda.kda_mla_cache_read(**c, cu_seqlens=None, T=4, latent=torch.zeros(3, 512))
    q, kv, kp = torch.zeros(8, 4, 192).bfloat16(), torch.zeros(8, 4, 256).bfloat16(), torch.zeros(8, 64).bfloat16()
    with pytest.raises(ValueError, match="k_pe"):
        kda.kda_mla_prefill(q, kv, kp[:7], softmax_scale=0.1)
    with pytest.raises(TypeError, match="share"):
        kda.kda_mla_prefill(q, kv, kp.float(), softmax_scale=0.1)
    with pytest.raises(ValueError, match="lse"):
        kda.kda_mla_prefill(q, kv, kp, softmax_scale=0.1, lse=torch.zeros(8))
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.kda_mla_prefill(q, kv, kp, softmax_scale=0.1)


# Calls whose arrays lie apart but for one pair.  They are refused before anything is launched; where that failed they
# would run on fake addresses, so only machines without a GPU make them.
def _far(k):
    return (k + 1) << 36


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses")
@pytest.mark.parametrize("kw", [
    dict(o=_far(0)), dict(o=_far(0) + 2 * 32 * 512 * 2 - 16), dict(o=_far(1)), dict(o=_far(2) + 16), dict(o=_far(3)),
    dict(lse=_far(0) + 64), dict(lse=_far(4)), dict(lse=_far(5)), dict(lse=_far(6) + 64),
    dict(ws=_far(0), wsb=1 << 30), dict(ws=_far(6) - 1024, wsb=1 << 30),
    dict(dc=kda.KDA_E4M3, cs=_far(9), lse=_far(9) + 4 * 64 * 4 - 4),
])
def test_decode_refuses_outputs_over_other_arrays(lib, kw):
    apart = dict(q=_far(0), qp=_far(1), cl=_far(2), cp=_far(3), table=_far(4), lens=_far(5), o=_far(6), lse=_far(7))
    assert _decode(lib, **{**apart, **kw}) == INV
    assert _decode(lib, **apart) == kda.KDA_ERR_CUDA  # apart: refused only for want of a GPU


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses")
@pytest.mark.parametrize("kw", [dict(o=_far(0)), dict(o=_far(0) + 8 * 4 * 192 * 2 - 16), dict(o=_far(1)), dict(o=_far(2)),
                                dict(lse=_far(0)), dict(lse=_far(5)), dict(lse=_far(3), cq=_far(3)), dict(o=_far(4), ck=_far(4), cq=_far(3))])
def test_prefill_refuses_outputs_over_other_arrays(lib, kw):
    apart = dict(q=_far(0), kv=_far(1), kp=_far(2), o=_far(5), lse=_far(6))
    assert _prefill(lib, **{**apart, **kw}) == INV
    assert _prefill(lib, **apart) == kda.KDA_ERR_CUDA


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses")
@pytest.mark.parametrize("kw", [dict(latent=_far(2)), dict(pe=_far(3) + 4 * 64 * 128 - 16), dict(latent=_far(3)),
                                dict(dc=kda.KDA_E4M3, cs=_far(0) + 16), dict(table=_far(2)), dict(cl=_far(3) - 16)])
def test_cache_calls_refuse_outputs_over_other_arrays(lib, kw):
    apart = dict(latent=_far(0), pe=_far(1), cl=_far(2), cp=_far(3), table=_far(4))
    assert _write(lib, **{**apart, "lens": _far(5), **kw}) == INV
    assert _write(lib, **{**apart, "lens": _far(5)}) == kda.KDA_ERR_CUDA
    if "table" not in kw and "cl" not in kw:
        assert _read(lib, **{**apart, "starts": _far(5), **kw}) == INV
    assert _read(lib, **{**apart, "starts": _far(5)}) == kda.KDA_ERR_CUDA
