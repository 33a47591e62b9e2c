"""Absorbed decode where a few tokens carry weights far above those of a long tail whose mass still counts (an attention
sink over a long context): every weight has to enter the output, however far below the row's largest one it is.

The bound of o, per row and channel, counts what include/kda.h promises.  With w the normalised weights, c the cached
values, and for an e4m3 cache s the tokens' scales and e = c / s their codes:
  scores    2^-20 sum |q||k| scale + 2^-22 |x| (two channels that are not 0; the products of the others are exact)
  weights   2^-8 of each (bf16, or two e4m3 parts of 2^-4 each)
  sums      keys / 32 additions of 2^-23 each, relative to sum w |c|
  e4m3      a weight times its scale that is small beside the row's reference is off by at most half of 2^-13, a reference at
            which the row's largest w s is 2^4 or more: 2^-18 of it.  Every 512 tokens the reference follows what the
            tokens weigh (once they weigh less than 2^3, to a quarter or less, by 20 binades in all at most).  So with E
            the largest sum of |e| over 512 tokens:
              2^-14 / 2^3 sum w s E       where 512 tokens weigh 2^3 or more,
              2^-18 E sum (over windows of 512 tokens) max w s    for those at whose end the reference falls, 4/3 of that
                with those after it (each fall leaves a quarter), as much again for a last window without an end,
                and twice all that for windows that lie across the kernel's: less than 5,
              2^-38 max w s sum |e|       below the reference's lowest place
  output    half a step of its type
None of it grows with the length but the sums' 2^-28 a key."""
import math

import pytest
import torch

from gated_delta_rule_127_b200 import kda
from mla_ref import LATENT, PE, U, Cache, check, quantise

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
E4M3, BF16 = torch.float8_e4m3fn, torch.bfloat16
SCALE = 1.0 / math.sqrt(192)
H, WIN = 8, 512
GAIN = torch.linspace(0.7, 1.2, H, dtype=torch.float64)  # per head: how far the scores are spread


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_127_b200 import build
    build.build()
    kda.load_library()


def _cache(lengths, dtype, scores, size=None, page=64, seed=3):
    """A cache whose tokens' scores are `scores` (nats, in one positional channel) plus noise from a second channel; the
    latents have a common mean as large as their spread."""
    cache = Cache(lengths, page, dtype, DEV)
    g = torch.Generator(device=DEV).manual_seed(seed)
    for b, n in enumerate(lengths):
        at = cache.rows(b, 0, n)
        c = torch.randn(n, LATENT, generator=g, device=DEV) + 1.0
        if size is not None:
            c = c * size[b][:, None]
        if cache.scale is None:
            cache.latent.view(-1, LATENT)[at] = c.to(BF16)
        else:
            codes, s = quantise(c.double())
            cache.latent.view(torch.uint8).view(-1, LATENT)[at] = codes.view(torch.uint8)
            cache.scale.view(-1)[at] = s.float()
        pe = torch.zeros(n, PE, device=DEV)
        pe[:, 0] = scores[b]
        pe[:, 1] = torch.randn(n, generator=g, device=DEV)
        cache.pe.view(-1, PE)[at] = pe.to(BF16)
    return cache


def _queries(B, noise):
    q = torch.zeros(B, 1, H, LATENT, dtype=BF16, device=DEV)
    qp = torch.zeros(B, 1, H, PE, dtype=BF16, device=DEV)
    qp[..., 0] = (GAIN / SCALE).to(BF16).to(DEV)
    qp[..., 1] = noise / SCALE
    return q, qp


def _want(cache, b, qp, out_dtype):
    """(o, tol) [H, LATENT] of sequence b."""
    n = cache.lengths[b]
    c, p, s = cache.tokens(b, 0, n)
    Q = qp[b, 0].double()
    x = SCALE * (Q @ p.T)
    d = (2.0 ** -20 * SCALE * (Q.abs() @ p.abs().T) + 2.0 ** -22 * x.abs()).amax(1, keepdim=True)
    w = torch.softmax(x, 1)
    o = w @ c
    rel = torch.expm1(2 * d) + 2.0 ** -8 + n / 32 * 2.0 ** -23 + 2.0 ** -16
    tol = rel * (w @ c.abs())
    if s is not None:
        e = (c / s[:, None]).abs()
        pad = -n % WIN
        win = torch.nn.functional.pad(e, (0, 0, 0, pad)).view(-1, WIN, LATENT).sum(1).amax(0)   # E
        ws = w * s
        top = torch.nn.functional.pad(ws, (0, pad)).view(H, -1, WIN).amax(2)
        tol += 2.0 ** -17 * ws.sum(1, keepdim=True) * win + 5 * 2.0 ** -18 * top.sum(1, keepdim=True) * win
        tol += 2.0 ** -38 * ws.amax(1, keepdim=True) * e.sum(0)
    return o, tol + U[out_dtype] * o.abs() * (1 + rel) + 1e-30


def _run(cache, q, qp, **kw):
    o, _ = kda.kda_mla_decode(q, qp, cache.latent, cache.pe, cache.table, cache.seq_lens, softmax_scale=SCALE,
                              cache_scale=cache.scale, dtype_o=torch.float32, **kw)
    assert kda.kda_get_device_status() == (kda.KDA_OK, 0)
    return o


def _check(cache, qp, o, seqs):
    for b in seqs:
        want, tol = _want(cache, b, qp, o.dtype)
        check(o[b, 0], want, tol, "o of sequence %d" % b)


def _sink(n, nats, at):
    x = torch.zeros(n, device=DEV)
    x[at] = nats
    return x


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("n,nats,at", [(8192, 11.0, 0), (32768, 12.75, 0), (32768, 14.0, 64 * 100 + 5), (131072, 13.0, 0),
                                       (131072, 12.0, 70000), (500001, 13.0, 0), (500001, 15.0, 250000)])
def test_a_sink_over_a_long_tail(dtype, n, nats, at):
    cache = _cache([n], dtype, [_sink(n, nats, at)])
    q, qp = _queries(1, 1.0)
    _check(cache, qp, _run(cache, q, qp), [0])
    if n <= 131072:
        _check(cache, qp, _run(cache, q, qp, use_workspace=False), [0])


@pytest.mark.parametrize("nats", [9.0, 12.5, 14.0])
def test_a_sink_over_equal_scores(nats):
    # every weight of the tail is rounded the same way, so no two errors cancel
    n = 40000
    cache = _cache([n], E4M3, [_sink(n, nats, 0)])
    q, qp = _queries(1, 0.0)
    for ws in (True, False):
        _check(cache, qp, _run(cache, q, qp, use_workspace=ws), [0])


def test_the_same_sequence_alone_and_in_a_batch():
    # 200 sequences, the first and the last one the same long one: there one CTA has much more of it than alone
    n = 32768
    alone = _cache([n], E4M3, [_sink(n, 13.0, 0)])
    q, qp = _queries(200, 1.0)
    _check(alone, qp, _run(alone, q[:1], qp[:1]), [0])
    lens = [n] + [4096] * 198 + [n]
    table = alone.table.expand(200, -1).contiguous()
    o, _ = kda.kda_mla_decode(q, qp, alone.latent, alone.pe, table, torch.tensor(lens, dtype=torch.int32, device=DEV),
                              softmax_scale=SCALE, cache_scale=alone.scale, dtype_o=torch.float32)
    assert kda.kda_get_device_status() == (kda.KDA_OK, 0)
    want, tol = _want(alone, 0, qp, o.dtype)
    check(o[0, 0], want, tol, "the first")
    check(o[199, 0], want, tol, "the last")


@pytest.mark.parametrize("dtype", [E4M3, BF16])
@pytest.mark.parametrize("period,height", [(700, 12.0), (3000, 20.0), (9000, 40.0)])
def test_scores_that_go_up_and_down(dtype, period, height):
    # the reference rises and falls again and again; with the tallest waves beyond the 20 binades that it may fall
    n = 30000
    wave = height * torch.cos(torch.arange(n, device=DEV) * (2 * math.pi / period))
    cache = _cache([n, 5000], dtype, [wave, wave[2000:7000]], page=16)
    q, qp = _queries(2, 1.0)
    for ws in (True, False):
        _check(cache, qp, _run(cache, q, qp, use_workspace=ws), [0, 1])


@pytest.mark.parametrize("falling", [True, False])
def test_a_long_slope(falling):
    # tens of thousands of tokens, each a little lighter (or heavier) than the one before
    n = 30000
    slope = torch.linspace(30, 0, n, device=DEV)
    cache = _cache([n], E4M3, [slope if falling else slope.flip(0)])
    q, qp = _queries(1, 0.5)
    for ws in (True, False):
        _check(cache, qp, _run(cache, q, qp, use_workspace=ws), [0])


def test_tokens_of_very_different_size():
    # a sink without a value (scale 2^-64), one with a large one, tails of small and large latents
    n = 20000
    g = torch.Generator(device=DEV).manual_seed(9)
    size = torch.exp2(torch.randint(-12, 13, (n,), generator=g, device=DEV).float())
    size[0], size[1] = 0.0, 2.0 ** 20
    x = _sink(n, 14.0, 0)
    x[1] = 6.0
    cache = _cache([n], E4M3, [x], size=[size])
    assert cache.scale.view(-1)[cache.rows(0, 0, 1)] == 2.0 ** -64
    q, qp = _queries(1, 1.0)
    for ws in (True, False):
        _check(cache, qp, _run(cache, q, qp, use_workspace=ws), [0])


def test_the_tail_after_absent_pages_and_short_sequences():
    # pages out of range count as absent: tokens that weigh nothing for a whole window, then a tail
    n = 4096
    cache = _cache([n, 70], E4M3, [_sink(n, 12.0, 3), _sink(70, 12.0, 69)])
    table = cache.table.clone()
    gone = list(range(8, 40))
    table[0, gone] = -1
    q, qp = _queries(2, 1.0)
    for ws in (True, False):
        o, _ = kda.kda_mla_decode(q, qp, cache.latent, cache.pe, table, cache.seq_lens, softmax_scale=SCALE,
                                  cache_scale=cache.scale, dtype_o=torch.float32, use_workspace=ws)
        assert kda.kda_get_device_status() == (kda.KDA_ERR_DEVICE_CHECK, kda.KDA_DEVFLAG_PAGE_TABLE)
        keep = [i for i in range(n // 64) if i not in gone]
        short = Cache([len(keep) * 64, 70], 64, E4M3, DEV)
        short.table = cache.table.clone()
        short.table[0, :len(keep)] = cache.table[0, keep]
        short.latent, short.scale, short.pe, short.page = cache.latent, cache.scale, cache.pe, cache.page
        _check(short, qp, o, [0, 1])
