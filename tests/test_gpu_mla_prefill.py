"""Expanded latent attention over packed batches against the 64-bit definition, with elementwise bounds."""
import math

import pytest
import torch

import mla_ref
from gated_delta_rule_127_b200 import kda
from mla_ref import DV, check, cu_of

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16
SCALE = 1.0 / math.sqrt(192)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_127_b200 import build
    build.build()
    kda.load_library()


def _inputs(Tq, Tk, H, seed=7):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF16)  # noqa: E731
    return r(Tq, H, 192), r(Tk, H, 256), r(Tk, 64)


def _run(q, kv, kp, nq, nk, causal=True, scale=SCALE, **kw):
    o, lse = kda.kda_mla_prefill(q, kv, kp, cu_of(nq, DEV), cu_of(nk, DEV), causal=causal, softmax_scale=scale,
                                 output_lse=True, **kw)
    assert kda.kda_get_device_status() == (kda.KDA_OK, 0)
    return o, lse


CASES = [  # queries and keys of each sequence, heads
    ([1], [1], 1), ([1], [300], 4), ([200], [200], 4), ([128], [128], 2), ([129], [129], 2), ([256], [256], 2),
    ([257, 1, 127], [257, 1, 127], 3), ([5, 0, 130], [5, 0, 130], 2), ([64, 300], [1000, 333], 2),
    ([0, 0], [0, 4], 2), ([40], [17], 2), ([300, 10], [40, 0], 2), ([3], [0], 1), ([600], [1500], 2), ([700], [700], 5),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk,H", CASES)
def test_prefill_matches_the_definition(nq, nk, H, causal):
    q, kv, kp = _inputs(sum(nq), sum(nk), H)
    for dtype_o in (torch.float32, BF16):
        o, lse = _run(q, kv, kp, nq, nk, causal, dtype_o=dtype_o)
        assert o.dtype == dtype_o
        want, tol, wl, lt = mla_ref.prefill(q, kv, kp, nq, nk, causal, SCALE, dtype_o)
        check(o, want, tol, "o")
        check(lse, wl, lt, "lse")


def test_longer_sequences():
    nq, nk = [2000, 1025], [2000, 4100]
    q, kv, kp = _inputs(sum(nq), sum(nk), 2)
    o, lse = _run(q, kv, kp, nq, nk, dtype_o=torch.float32)
    want, tol, wl, lt = mla_ref.prefill(q, kv, kp, nq, nk, True, SCALE, torch.float32)
    check(o, want, tol, "o")
    check(lse, wl, lt, "lse")


@pytest.mark.parametrize("rising", [True, False])
def test_scores_that_rise_or_fall_by_hundreds(rising):
    n = 900
    q, kv, kp = _inputs(n, n, 2)
    ramp = torch.linspace(0, 400, n, device=DEV)
    kp.zero_()
    kp[:, 0] = (ramp if rising else ramp.flip(0)).to(BF16)
    q[..., 128:] = 0
    q[:, 0, 128] = 1 / SCALE
    q[:, 1, 128] = -1 / SCALE
    o, lse = _run(q, kv, kp, [n], [n], dtype_o=torch.float32)
    want, tol, wl, lt = mla_ref.prefill(q, kv, kp, [n], [n], True, SCALE, torch.float32)
    check(o, want, tol, "o")
    check(lse, wl, lt, "lse")


def test_many_short_sequences():
    # more sequences than threads in a block, most of a few queries
    g = torch.Generator().manual_seed(5)
    nq = [int(x) for x in torch.randint(0, 9, (700,), generator=g)]
    nk = [n + int(x) for n, x in zip(nq, torch.randint(0, 9, (700,), generator=g))]
    nq[300], nk[300] = 400, 431
    q, kv, kp = _inputs(sum(nq), sum(nk), 1)
    o, lse = _run(q, kv, kp, nq, nk, dtype_o=torch.float32)
    want, tol, wl, lt = mla_ref.prefill(q, kv, kp, nq, nk, True, SCALE, torch.float32)
    check(o, want, tol, "o")
    check(lse, wl, lt, "lse")


def test_negative_and_zero_scale():
    q, kv, kp = _inputs(150, 150, 2)
    for scale in (0.0, -0.05):
        o, lse = _run(q, kv, kp, [150], [150], scale=scale, dtype_o=torch.float32)
        want, tol, wl, lt = mla_ref.prefill(q, kv, kp, [150], [150], True, scale, torch.float32)
        check(o, want, tol, "o")
        check(lse, wl, lt, "lse")


@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_neighbours_and_padding_do_not_leak(poison):
    # poisoned rows behind the last sequence and a poisoned second sequence: the others' results keep their bits
    nq = [100, 70, 130]
    q, kv, kp = _inputs(sum(nq) + 50, sum(nq) + 50, 2)
    cu = cu_of(nq, DEV)
    want = [torch.full((sum(nq) + 50, 2, DV), 7.0, device=DEV), torch.full((sum(nq) + 50, 2), 7.0, device=DEV)]
    got = [w.clone() for w in want]
    kda.kda_mla_prefill(q, kv, kp, cu, cu, softmax_scale=SCALE, o=want[0], lse=want[1])
    for t in (q, kv, kp):
        t[100:170] = poison
        t[300:] = poison
    kda.kda_mla_prefill(q, kv, kp, cu, cu, softmax_scale=SCALE, o=got[0], lse=got[1])
    assert kda.kda_get_device_status() == (kda.KDA_OK, 0)
    for g, w in zip(got, want):
        assert torch.equal(g[:100], w[:100]) and torch.equal(g[170:], w[170:])
        assert bool((g[300:] == 7).all())


def test_equal_lengths_without_cu_seqlens():
    q, kv, kp = _inputs(120, 360, 2)
    o, lse = kda.kda_mla_prefill(q, kv, kp, num_seqs=3, softmax_scale=SCALE, output_lse=True)
    ref = _run(q, kv, kp, [40] * 3, [120] * 3)
    assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


def test_device_checks_skip_and_flag():
    q, kv, kp = _inputs(60, 60, 2)
    good, _ = _run(q, kv, kp, [20] * 3, [20] * 3)
    cu = cu_of([20] * 3, DEV)
    for bad in ([0, 20, 10, 60], [0, 20, 40, 61], [3, 20, 40, 60]):
        bad = torch.tensor(bad, dtype=torch.int32, device=DEV)
        o = torch.full((60, 2, DV), 7.0, dtype=BF16, device=DEV)
        kda.kda_mla_prefill(q, kv, kp, bad, cu, softmax_scale=SCALE, o=o)
        assert kda.kda_get_device_status() == (kda.KDA_ERR_DEVICE_CHECK, kda.KDA_DEVFLAG_CU_SEQLENS)
        o2, lse = kda.kda_mla_prefill(q, kv, kp, cu, bad, softmax_scale=SCALE, output_lse=True)
        assert kda.kda_get_device_status() == (kda.KDA_ERR_DEVICE_CHECK, kda.KDA_DEVFLAG_CU_SEQLENS)
        assert bool((lse == -math.inf).any())
    assert torch.equal(o2[20:], good[20:]) and not bool(o2[:20].any())


def test_streams_and_graphs():
    nq = [300, 20]
    q, kv, kp = _inputs(320, 320, 4)
    o1, l1 = _run(q, kv, kp, nq, nq)
    cu = cu_of(nq, DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, l2 = kda.kda_mla_prefill(q, kv, kp, cu, cu, softmax_scale=SCALE, output_lse=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o3, l3 = kda.kda_mla_prefill(q, kv, kp, cu, cu, softmax_scale=SCALE, output_lse=True)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o1, o3) and torch.equal(l1, l3)


def test_no_queries():
    q, kv, kp = _inputs(0, 10, 2)
    o, lse = _run(q, kv, kp, [0], [10])
    assert o.shape == (0, 2, DV) and lse.shape == (0, 2)


@pytest.mark.parametrize("causal", [True, False])
def test_more_sequences_than_are_ordered_at_once(causal):
    # the work is ordered by size 32 sequences at a time: lengths from 0 to several tiles, keys fewer and more than
    # queries, on both sides of that boundary; a result nobody wrote would stay NaN
    g = torch.Generator().manual_seed(13)
    nq = torch.randint(0, 300, (70,), generator=g).tolist()
    nk = [max(0, n + int(x)) for n, x in zip(nq, torch.randint(-150, 250, (70,), generator=g))]
    nq[5], nk[5], nq[31], nk[31], nq[32], nk[32], nq[69], nk[69] = 900, 900, 600, 2000, 257, 0, 700, 1500
    q, kv, kp = _inputs(sum(nq), sum(nk), 3)
    o = torch.full((sum(nq), 3, DV), float("nan"), device=DEV)
    lse = torch.full((sum(nq), 3), float("nan"), device=DEV)
    kda.kda_mla_prefill(q, kv, kp, cu_of(nq, DEV), cu_of(nk, DEV), causal=causal, softmax_scale=SCALE, o=o, lse=lse)
    want, tol, wl, lt = mla_ref.prefill(q, kv, kp, nq, nk, causal, SCALE, torch.float32)
    check(o, want, tol, "o")
    check(lse, wl, lt, "lse")
