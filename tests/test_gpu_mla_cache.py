"""The paged latent cache on the GPU: what is written equals the 64-bit definition bit for bit (powers of two and one
rounding leave nothing open), what is read back equals what was written, and nothing else is touched."""
import pytest
import torch

from gated_delta_rule_127_b200 import kda
from mla_ref import LATENT, PE, Cache, cu_of, quantise

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_127_b200 import build
    build.build()
    kda.load_library()


def _bits(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def _new(total, dtype, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = torch.randn(total, LATENT, generator=g, device=DEV) * torch.exp(2 * torch.randn(total, 1, generator=g, device=DEV))
    return c.to(dtype), torch.randn(total, PE, generator=g, device=DEV).to(dtype)


def _write(cache, latent, pe, new, **kw):
    kda.kda_mla_cache_write(latent, pe, cache.latent, cache.pe, cache.table, cache.seq_lens, cu_of(new, DEV),
                            cache_scale=cache.scale, **kw)


def _expect(cache, latent, pe, new):
    """The cache's tensors after the write, from copies of those before it."""
    lat, p = cache.latent.clone(), cache.pe.clone()
    sc = None if cache.scale is None else cache.scale.clone()
    at = 0
    for b, n in enumerate(new):
        rows = cache.rows(b, cache.lengths[b] - n, cache.lengths[b])
        c = latent[at:at + n]
        if sc is None:
            lat.view(-1, LATENT)[rows] = c.to(torch.bfloat16)
        else:
            codes, s = quantise(c.double())
            lat.view(torch.uint8).view(-1, LATENT)[rows] = codes.view(torch.uint8)
            sc.view(-1)[rows] = s.float()
        p.view(-1, PE)[rows] = pe[at:at + n].to(torch.bfloat16)
        at += n
    return lat, p, sc


def _same(cache, want):
    assert torch.equal(_bits(cache.latent), _bits(want[0]))
    assert torch.equal(_bits(cache.pe), _bits(want[1]))
    if cache.scale is not None:
        assert torch.equal(_bits(cache.scale), _bits(want[2]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, E4M3])
@pytest.mark.parametrize("source", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,total,new", [
    (16, [1], [1]), (16, [0, 17, 33], [0, 1, 33]), (64, [64, 65, 200, 3], [64, 1, 100, 0]), (1024, [1500, 7], [1100, 7]),
])
def test_write_and_read_back(dtype, source, page, total, new):
    cache = Cache(total, page, dtype, DEV)
    latent, pe = _new(sum(new), source)
    want = _expect(cache, latent, pe, new)
    _write(cache, latent, pe, new)
    assert kda.kda_get_device_status() == (kda.KDA_OK, 0)
    _same(cache, want)
    starts = torch.tensor([t - n for t, n in zip(total, new)], dtype=torch.int32, device=DEV)
    for dtype_o in (torch.bfloat16, torch.float32):
        got, gp = kda.kda_mla_cache_read(cache.latent, cache.pe, cache.table, cu_of(new, DEV), sum(new), starts=starts,
                                         cache_scale=cache.scale, dtype_o=dtype_o)
        assert got.dtype == dtype_o
        ref = [cache.tokens(b, t - n, t) for b, (t, n) in enumerate(zip(total, new))]
        assert torch.equal(got.double(), torch.cat([r[0] for r in ref]))   # exact in bf16 too: 4 bits times 2^k
        assert torch.equal(gp.double(), torch.cat([r[1] for r in ref]))


def test_scale_edges():
    # exact powers, one step above, the range's ends, zeros, infinities and NaN
    rows = [448.0, 448.0 * 2, 449.0, 3.5, 3.5 * (1 + 2.0 ** -20), 0.0, 1e-30, 3.0e38, float("inf"), 2.0 ** -126]
    latent = torch.zeros(len(rows) + 1, LATENT, device=DEV)
    for i, a in enumerate(rows):
        latent[i, 5] = -a
        latent[i, 6] = a / 3
    latent[-1, 3], latent[-1, 4] = float("nan"), 1.0
    n = len(rows) + 1
    cache = Cache([n], 16, E4M3, DEV)
    pe = torch.zeros(n, PE, device=DEV)
    want = _expect(cache, latent, pe, [n])
    _write(cache, latent, pe, [n])
    nan = torch.isnan(want[0].float())
    assert torch.equal(torch.isnan(cache.latent.float()), nan)
    assert torch.equal(cache.latent.float()[~nan], want[0].float()[~nan])
    at = cache.rows(0, 0, n)
    s = cache.scale.view(-1)[at]
    assert torch.equal(s, want[2].view(-1)[at])
    assert s[5] == 2.0 ** -64 and s[8] == 2.0 ** 120 and s[0] == 1 and s[1] == 2 and s[2] == 2
    assert torch.isnan(cache.latent.view(torch.uint8).view(-1, LATENT)[at[-1]].view(E4M3).float()[3])


def test_padded_batch_leaves_rows_behind_the_last_sequence():
    new, pad = [3, 5], 4
    for dtype in (torch.bfloat16, E4M3):
        cache = Cache([10, 5], 16, dtype, DEV)
        latent, pe = _new(sum(new) + pad, torch.bfloat16)
        latent[sum(new):] = float("nan")
        want = _expect(cache, latent, pe, new)
        _write(cache, latent, pe, new)
        _same(cache, want)
        got = torch.full((sum(new) + pad, LATENT), 7.0, device=DEV, dtype=torch.bfloat16)
        gp = torch.full((sum(new) + pad, PE), 7.0, device=DEV, dtype=torch.bfloat16)
        cache.fill(3)
        kda.kda_mla_cache_read(cache.latent, cache.pe, cache.table, cu_of(new, DEV), sum(new) + pad,
                               cache_scale=cache.scale, latent=got, pe=gp)
        assert bool((got[sum(new):] == 7).all()) and bool((gp[sum(new):] == 7).all())
        assert torch.equal(got[:3].double(), cache.tokens(0, 0, 3)[0])
        assert kda.kda_get_device_status() == (kda.KDA_OK, 0)


def test_device_checks_skip_and_flag():
    cache = Cache([20, 20], 16, torch.bfloat16, DEV)
    latent, pe = _new(8, torch.bfloat16)
    before = cache.latent.clone()

    def write(cu, lens=(20, 20), table=None):
        kda.kda_mla_cache_write(latent, pe, cache.latent, cache.pe, cache.table if table is None else table,
                                torch.tensor(lens, dtype=torch.int32, device=DEV),
                                torch.tensor(cu, dtype=torch.int32, device=DEV))
        return kda.kda_get_device_status()

    bad = (kda.KDA_ERR_DEVICE_CHECK, kda.KDA_DEVFLAG_CU_SEQLENS)
    assert write([0, 4, 9]) == bad        # beyond T (the first sequence is written)
    assert write([0, 9, 8]) == bad
    assert write([0, 5, 3]) == bad
    assert write([2, 1, 8])[0] == kda.KDA_ERR_DEVICE_CHECK
    cache.latent.copy_(before)
    assert write([0, 4, 8], lens=(3, 3)) == (kda.KDA_ERR_DEVICE_CHECK, kda.KDA_DEVFLAG_SEQ_LENS)
    assert write([0, 4, 8], lens=(-1, 1 << 30)) == (kda.KDA_ERR_DEVICE_CHECK, kda.KDA_DEVFLAG_SEQ_LENS)
    assert torch.equal(_bits(before), _bits(cache.latent))
    table = cache.table.clone()
    table[:, 1] = torch.tensor([cache.pages, -1], dtype=torch.int32, device=DEV)
    assert write([0, 4, 8], table=table) == (kda.KDA_ERR_DEVICE_CHECK, kda.KDA_DEVFLAG_PAGE_TABLE)
    assert torch.equal(_bits(before), _bits(cache.latent))
    out = torch.full((8, LATENT), 7.0, device=DEV, dtype=torch.bfloat16)
    po = torch.full((8, PE), 7.0, device=DEV, dtype=torch.bfloat16)
    for starts, tab, flag in (([-1, 100], cache.table, kda.KDA_DEVFLAG_SEQ_LENS), ([16, 16], table, kda.KDA_DEVFLAG_PAGE_TABLE)):
        kda.kda_mla_cache_read(cache.latent, cache.pe, tab, None, 8, latent=out, pe=po,
                               starts=torch.tensor(starts, dtype=torch.int32, device=DEV))
        assert kda.kda_get_device_status() == (kda.KDA_ERR_DEVICE_CHECK, flag)
        assert bool((out == 7).all()) and bool((po == 7).all())


def test_rows_past_four_gigabytes():
    # the pool's last pages: byte offsets beyond 2^32
    first = 70000
    cache = Cache([100], 64, torch.bfloat16, DEV, first_page=first, poison=False)
    assert cache.latent.numel() * 2 > 1 << 32
    latent, pe = _new(100, torch.bfloat16)
    _write(cache, latent, pe, [100])
    got, gp = kda.kda_mla_cache_read(cache.latent, cache.pe, cache.table, None, 100)
    assert torch.equal(got, latent) and torch.equal(gp, pe)
    assert not bool(cache.latent[:first].any())


def test_stream_and_graph():
    cache = Cache([130, 7], 64, E4M3, DEV)
    latent, pe = _new(137, torch.bfloat16)
    want = _expect(cache, latent, pe, [130, 7])
    cu = cu_of([130, 7], DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kda.kda_mla_cache_write(latent, pe, cache.latent, cache.pe, cache.table, cache.seq_lens, cu, cache_scale=cache.scale,
                            stream=side)
    got, _ = kda.kda_mla_cache_read(cache.latent, cache.pe, cache.table, cu, 137, cache_scale=cache.scale, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _same(cache, want)
    cache.latent.view(torch.uint8).fill_(0x7F)  # as it was before the write
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.kda_mla_cache_write(latent, pe, cache.latent, cache.pe, cache.table, cache.seq_lens, cu,
                                cache_scale=cache.scale)
        again, _ = kda.kda_mla_cache_read(cache.latent, cache.pe, cache.table, cu, 137, cache_scale=cache.scale)
    g.replay()
    torch.cuda.synchronize()
    _same(cache, want)
    assert torch.equal(again, got)
