"""Absorbed latent attention over the paged cache against the 64-bit definition, with elementwise bounds."""
import math

import pytest
import torch

import mla_ref
from gated_delta_rule_127_b200 import kda
from mla_ref import LATENT, PE, Cache, check

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
E4M3, BF16 = torch.float8_e4m3fn, torch.bfloat16
SCALE = 1.0 / math.sqrt(192)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_127_b200 import build
    build.build()
    kda.load_library()


def _queries(B, S, H, seed=5, size=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randn(B, S, H, LATENT, generator=g, device=DEV) * size
    return q.to(BF16), (torch.randn(B, S, H, PE, generator=g, device=DEV) * size).to(BF16)


def _run(cache, q, qp, scale=SCALE, **kw):
    o, lse = kda.kda_mla_decode(q, qp, cache.latent, cache.pe, cache.table, cache.seq_lens, softmax_scale=scale,
                                cache_scale=cache.scale, output_lse=True, **kw)
    assert kda.kda_get_device_status() == (kda.KDA_OK, 0)
    return o, lse


def _check(cache, q, qp, o, lse, scale=SCALE):
    want, tol, wl, lt = mla_ref.decode(q, qp, cache, scale, o.dtype)
    check(o, want, tol, "o")
    check(lse, wl, lt, "lse")


CASES = [  # lengths, S, H, page
    ([1], 1, 32, 64), ([0, 1, 2, 63], 1, 32, 64), ([64, 65, 0, 128], 1, 32, 64), ([300], 1, 32, 16),
    ([127, 129, 191, 5], 1, 8, 32), ([1000, 1, 70], 2, 16, 16), ([3, 0, 1, 2], 4, 12, 16), ([513, 77], 1, 64, 128),
    ([200, 64], 1, 128, 256), ([90, 1], 3, 20, 1024), ([50], 1, 1, 16), ([2, 700], 5, 40, 64), ([40000], 1, 32, 64),
    ([9000, 13, 5000], 1, 33, 32),
]


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("lengths,S,H,page", CASES)
def test_decode_matches_the_definition(dtype, lengths, S, H, page):
    cache = Cache(lengths, page, dtype, DEV).fill(2)
    q, qp = _queries(len(lengths), S, H)
    for dtype_o in (torch.float32, BF16):
        o, lse = _run(cache, q, qp, dtype_o=dtype_o)
        assert o.dtype == dtype_o
        _check(cache, q, qp, o, lse)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("lengths,S,H", [([70, 3], 40, 128), ([100], 1, 300), ([0, 130, 1], 37, 7)])
def test_many_rows_per_sequence(dtype, lengths, S, H):
    # from a few row tiles to more of them than SMs (then no sequence is split)
    cache = Cache(lengths, 64, dtype, DEV).fill(2)
    q, qp = _queries(len(lengths), S, H)
    o, lse = _run(cache, q, qp, dtype_o=torch.float32)
    _check(cache, q, qp, o, lse)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_without_workspace(dtype):
    cache = Cache([3000, 0, 65, 129], 64, dtype, DEV).fill(2)
    q, qp = _queries(4, 1, 32)
    o, lse = _run(cache, q, qp, dtype_o=torch.float32, use_workspace=False)
    _check(cache, q, qp, o, lse)


@pytest.mark.parametrize("workspace", [True, False])
def test_more_sequences_than_threads(workspace):
    g = torch.Generator().manual_seed(5)
    lengths = [int(x) for x in torch.randint(0, 130, (1500,), generator=g)]
    cache = Cache(lengths, 64, BF16, DEV).fill(4)
    q, qp = _queries(1500, 1, 4)
    o, lse = _run(cache, q, qp, dtype_o=torch.float32, use_workspace=workspace)
    _check(cache, q, qp, o, lse)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_many_ragged_sequences(dtype):
    # more sequences than SMs, most of them short, lengths around tile borders
    g = torch.Generator().manual_seed(3)
    lengths = [int(x) for x in torch.randint(0, 200, (317,), generator=g)]
    lengths[100], lengths[101], lengths[316] = 5000, 0, 64
    cache = Cache(lengths, 32, dtype, DEV).fill(4)
    q, qp = _queries(317, 1, 16)
    o, lse = _run(cache, q, qp, dtype_o=torch.float32)
    _check(cache, q, qp, o, lse)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("rising", [True, False])
def test_scores_that_rise_or_fall_by_hundreds(dtype, rising):
    # the running maximum moves at every tile (or never): the accumulated output is rescaled each time
    n = 700
    cache = Cache([n], 64, dtype, DEV).fill(2, spread=0.0)
    ramp = torch.linspace(0, 300, n, device=DEV)
    if not rising:
        ramp = ramp.flip(0)
    at = cache.rows(0, 0, n)
    cache.pe.view(-1, PE)[at] = 0
    cache.pe.view(-1, PE)[at, 0] = ramp.to(BF16)
    q, qp = _queries(1, 1, 32)
    qp.zero_()
    qp[..., 0] = (1 / SCALE)
    qp[..., ::2, 0] *= -1
    o, lse = _run(cache, q, qp, dtype_o=torch.float32)
    _check(cache, q, qp, o, lse)


def test_negative_and_zero_scale():
    cache = Cache([333], 64, BF16, DEV).fill(2)
    q, qp = _queries(1, 2, 16)
    for scale in (0.0, -0.05):
        o, lse = _run(cache, q, qp, scale=scale, dtype_o=torch.float32)
        _check(cache, q, qp, o, lse, scale=scale)


def test_tokens_of_very_different_size():
    # scales over the whole e4m3 range of tokens: 2^-40 .. 2^20
    n = 200
    cache = Cache([n], 64, E4M3, DEV).fill(2, spread=0.0)
    at = cache.rows(0, 0, n)
    g = torch.Generator().manual_seed(1)
    cache.scale.view(-1)[at] = torch.exp2(torch.randint(-40, -5, (n,), generator=g).float()).to(DEV)
    cache.scale.view(-1)[at[0]] = 2.0 ** -64
    q, qp = _queries(1, 1, 32)
    o, lse = _run(cache, q, qp, dtype_o=torch.float32)
    _check(cache, q, qp, o, lse)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_nan_in_a_visible_token_stays_in_its_sequence(dtype):
    cache = Cache([100, 100], 64, dtype, DEV).fill(2)
    cache.pe.view(-1, PE)[cache.rows(0, 50, 51)] = float("nan")
    q, qp = _queries(2, 1, 32)
    o, lse = _run(cache, q, qp, dtype_o=torch.float32)
    assert bool(torch.isnan(o[0]).all()) and bool(torch.isnan(lse[0]).all())
    cache.lengths[0] = 0
    want, tol, wl, lt = mla_ref.decode(q, qp, cache, SCALE, torch.float32)
    check(o[1], want[1], tol[1], "o")
    check(lse[1], wl[1], lt[1], "lse")


def test_shared_pages():
    # two sequences with a common prefix given the same pages
    cache = Cache([128, 256], 64, BF16, DEV).fill(2)
    cache.table[0, :2] = cache.table[1, :2]
    q, qp = _queries(2, 1, 32)
    o, lse = _run(cache, q, qp, dtype_o=torch.float32)
    _check(cache, q, qp, o, lse)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_cache_past_four_gigabytes(dtype):
    first = 70000 if dtype == BF16 else 135000
    cache = Cache([1000], 64, dtype, DEV, first_page=first, poison=False).fill(2)
    assert cache.latent.numel() * cache.latent.element_size() > 1 << 32
    q, qp = _queries(1, 1, 32)
    o, lse = _run(cache, q, qp, dtype_o=torch.float32)
    _check(cache, q, qp, o, lse)


def test_device_checks_skip_and_flag():
    cache = Cache([100, 100, 100], 64, BF16, DEV).fill(2)
    q, qp = _queries(3, 1, 32)
    good = _run(cache, q, qp, dtype_o=torch.float32)
    args = (q, qp, cache.latent, cache.pe)
    kw = dict(softmax_scale=SCALE, output_lse=True, dtype_o=torch.float32)
    lens = torch.tensor([-1, 100, 1 << 20], dtype=torch.int32, device=DEV)
    o, lse = kda.kda_mla_decode(*args, cache.table, lens, **kw)
    assert kda.kda_get_device_status() == (kda.KDA_ERR_DEVICE_CHECK, kda.KDA_DEVFLAG_SEQ_LENS)
    assert not bool(o[0].any()) and not bool(o[2].any()) and bool((lse[[0, 2]] == -math.inf).all())
    tol = mla_ref.decode(q, qp, cache, SCALE, torch.float32)
    check(o[1], tol[0][1], tol[1][1], "o")
    # a bad page number: its 64 tokens count as absent
    table = cache.table.clone()
    table[0, 0], table[2, 0] = cache.pages, -1
    o, lse = kda.kda_mla_decode(*args, table, cache.seq_lens, **kw)
    assert kda.kda_get_device_status() == (kda.KDA_ERR_DEVICE_CHECK, kda.KDA_DEVFLAG_PAGE_TABLE)
    check(o[1], tol[0][1], tol[1][1], "o")
    short = Cache([36, 100, 36], 64, BF16, DEV)
    short.table, short.latent, short.pe = cache.table.clone(), cache.latent, cache.pe
    short.table[:, 0] = torch.where(torch.tensor([True, False, True], device=DEV), cache.table[:, 1], cache.table[:, 0])
    want, t, wl, lt = mla_ref.decode(q, qp, short, SCALE, torch.float32)
    check(o, want, t, "o")
    check(lse, wl, lt, "lse")
    again = _run(cache, q, qp, dtype_o=torch.float32)
    assert torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_given_buffers_streams_and_graphs(dtype):
    lengths = [3000, 100, 64, 0]
    cache = Cache(lengths, 64, dtype, DEV).fill(2)
    q, qp = _queries(4, 1, 32)
    o1, l1 = _run(cache, q, qp)
    ws = torch.empty(kda.kda_mla_decode_workspace_size(4, 1, 32), dtype=torch.uint8, device=DEV)
    ws.fill_(0xFF)  # its contents on entry do not matter
    o = torch.full((4, 1, 32, LATENT), 7.0, dtype=BF16, device=DEV)
    lse = torch.full((4, 1, 32), 7.0, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call = lambda **kw: kda.kda_mla_decode(q, qp, cache.latent, cache.pe, cache.table, cache.seq_lens,  # noqa: E731
                                           softmax_scale=SCALE, cache_scale=cache.scale, **kw)
    got = call(o=o, lse=lse, workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert got[0] is o and got[1] is lse
    assert torch.equal(o, o1) and torch.equal(lse, l1)   # a fixed order of sums: the same bits
    # one captured call, replayed after the lengths and the cache have changed
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go, gl = call(output_lse=True)
    cache.seq_lens.copy_(torch.tensor([2500, 17, 0, 0], dtype=torch.int32))
    g.replay()
    ref = call(output_lse=True)
    assert torch.equal(go, ref[0]) and torch.equal(gl, ref[1])
    # two calls at once, a workspace each
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [call(stream=s, output_lse=True) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(x[0], ref[0]) and torch.equal(x[1], ref[1]) for x in outs)


def test_a_workspace_that_is_too_small_is_refused_by_the_library():
    cache = Cache([100], 64, BF16, DEV).fill(2)
    q, qp = _queries(1, 1, 32)
    need = kda.kda_mla_decode_workspace_size(1, 1, 32)
    if need:
        lib = kda.load_library()
        st = lib.kda_mla_decode(q.data_ptr(), qp.data_ptr(), cache.latent.data_ptr(), cache.pe.data_ptr(), None,
                                cache.table.data_ptr(), cache.seq_lens.data_ptr(), 1, 1, 32, 512, 64, cache.pages, 64,
                                cache.table.shape[1], 0.1, 0, 0, 0, q.data_ptr(), None, q.data_ptr(), need - 16, None)
        assert st == kda.KDA_ERR_INVALID_ARG


def test_empty_batch():
    cache = Cache([], 64, BF16, DEV)
    q, qp = _queries(0, 1, 32)
    o, lse = _run(cache, q, qp)
    assert o.shape == (0, 1, 32, LATENT) and lse.shape == (0, 1, 32)
