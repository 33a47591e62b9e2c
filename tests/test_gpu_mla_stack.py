"""The operators together, as a hybrid stack uses them: prompts go through KDA prefill and latent-attention prefill,
their latents into the paged cache; then tokens are decoded one (or two) at a time by the KDA step and the absorbed
form over the cache.  Every token's output of the decoded form equals the expanded form's over the whole sequence."""
import math

import pytest
import torch

import mla_ref
from gated_delta_rule_127_b200 import inputs as gen
from gated_delta_rule_127_b200 import kda
from mla_ref import DV, LATENT, NOPE, PE, Cache, cu_of

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16
SCALE = 1.0 / math.sqrt(192)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gated_delta_rule_127_b200 import build
    build.build()
    kda.load_library()


@pytest.mark.parametrize("dtype", [BF16, torch.float8_e4m3fn])
def test_prefill_then_decode(dtype):
    H, prompts, steps, S = 4, [70, 1, 200], 3, 2
    B = len(prompts)
    full = [n + steps * S for n in prompts]
    g = torch.Generator(device=DEV).manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    w_k, w_v = r(H, NOPE, LATENT) / math.sqrt(LATENT), r(H, DV, LATENT) / math.sqrt(LATENT)
    c = [r(n, LATENT).to(BF16) for n in full]
    p = [r(n, PE).to(BF16) for n in full]
    q = [r(n, H, 192).to(BF16) for n in full]
    cache = Cache(full, 16, dtype, DEV)
    if dtype != BF16:  # what the cache holds is the layer's input to both forms
        for i in range(B):
            codes, s = mla_ref.quantise(c[i].double())
            c[i] = (codes.double() * s[:, None]).to(BF16)

    # the prompt: cache write, read back, expansion, prefill; the KDA layer beside it carries its state
    lens = torch.tensor(prompts, dtype=torch.int32, device=DEV)
    cu = cu_of(prompts, DEV)
    kda.kda_mla_cache_write(torch.cat([x[:n] for x, n in zip(c, prompts)]), torch.cat([x[:n] for x, n in zip(p, prompts)]),
                            cache.latent, cache.pe, cache.table, lens, cu, cache_scale=cache.scale)
    lat, pe = kda.kda_mla_cache_read(cache.latent, cache.pe, cache.table, cu, sum(prompts), cache_scale=cache.scale)
    assert torch.equal(lat, torch.cat([x[:n] for x, n in zip(c, prompts)]))
    kv = torch.einsum("tc,hdc->thd", lat.float(), torch.cat([w_k, w_v], 1)).to(BF16)
    qs = torch.cat([x[:n] for x, n in zip(q, prompts)])
    o, _ = kda.kda_mla_prefill(qs, kv.contiguous(), pe, cu, cu, softmax_scale=SCALE, dtype_o=torch.float32)
    x = gen.make_prefill(prompts, H, 128, 128, dtype=BF16, seed=3, device=DEV)
    _, state = kda.kda_chunk_fwd(x.q, x.k, x.v, x.log_alpha, x.beta, None, x.cu_seqlens)

    def exact(b, lo, hi):  # rows lo..hi of sequence b from the definition, 64 bits, weights as given
        kv64 = torch.einsum("tc,hdc->thd", c[b][:hi].double(), torch.cat([w_k, w_v], 1).double())
        out = torch.zeros(hi - lo, H, DV, dtype=torch.float64, device=DEV)
        for h in range(H):
            K = torch.cat([kv64[:, h, :NOPE], p[b][:hi].double()], 1)
            s = SCALE * (q[b][lo:hi, h].double() @ K.T)
            s = s.masked_fill(torch.ones_like(s, dtype=torch.bool).triu(1 + lo), -math.inf)
            out[:, h] = torch.softmax(s, 1) @ kv64[:, h, NOPE:]
        return out

    # keys and values (expanded) or queries (absorbed) are rounded to bf16 (2^-8 each), weights too; the logits here are
    # sums of 192 terms of size about 1 times SCALE, so their rounding errors stay below 2^-8 * sqrt(192) * SCALE * 8
    # (eight standard deviations): relative 0.032 in the weights, and 2^-7 more for the values and the weights
    tol = 0.032 + 2.0 ** -7
    at = 0
    for b, n in enumerate(prompts):
        want = exact(b, 0, n)
        assert float((o[at:at + n].double() - want).abs().max()) <= tol * 6
        assert float((o[at:at + n].double() - want).norm() / want.norm()) <= tol
        at += n

    for step in range(steps):
        lens = lens + S
        new_c = torch.cat([x[n + step * S:n + (step + 1) * S] for x, n in zip(c, prompts)])
        new_p = torch.cat([x[n + step * S:n + (step + 1) * S] for x, n in zip(p, prompts)])
        kda.kda_mla_cache_write(new_c, new_p, cache.latent, cache.pe, cache.table, lens, cache_scale=cache.scale)
        qn = torch.stack([x[n + step * S:n + (step + 1) * S] for x, n in zip(q, prompts)])       # [B, S, H, 192]
        ql = torch.einsum("bshd,hdc->bshc", qn[..., :NOPE].float(), w_k).to(BF16).contiguous()
        ol, _ = kda.kda_mla_decode(ql, qn[..., NOPE:].contiguous(), cache.latent, cache.pe, cache.table, lens,
                                   softmax_scale=SCALE, cache_scale=cache.scale, dtype_o=torch.float32)
        got = torch.einsum("bshc,hdc->bshd", ol.double(), w_v.double())
        for b, n in enumerate(prompts):
            lo = n + step * S
            want = exact(b, lo, lo + S)
            assert float((got[b] - want).norm() / want.norm()) <= tol
        y = gen.make_decode_step(step, B, H, 128, 128, seed=0, device=DEV)
        kda.kda_decode_step(y.q, y.k, y.v, y.log_alpha, y.beta, state)
    assert kda.kda_get_device_status() == (kda.KDA_OK, 0)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("last", ["kernel", "copy", "set", "join"])
def test_calls_wait_for_what_comes_before(last, captured):
    # write, read and decode may start while the work before them ends; its results are theirs all the same.  The slow
    # work ends in the new tokens, the lengths and the queries; what comes last before the calls is a kernel, a copy, a
    # memory set or another stream's event.
    n, H = 40, 32
    cache = Cache([n] * 8, 64, BF16, DEV).fill(3)
    g = torch.Generator(device=DEV).manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF16)  # noqa: E731
    new = [(r(8, LATENT), r(8, PE), r(8, 1, H, LATENT), r(8, 1, H, PE)) for _ in range(3)]
    lens = torch.full((8,), n, dtype=torch.int32, device=DEV)
    cu = cu_of([1] * 8, DEV)
    starts = lens - 1
    now = [torch.zeros_like(t) for t in new[0]]
    source = [torch.zeros_like(t) for t in new[0]]
    out = [torch.zeros(8, 1, H, LATENT, dtype=BF16, device=DEV), torch.zeros(8, LATENT, dtype=BF16, device=DEV)]
    big, spare = torch.randn(2048, 2048, generator=g, device=DEV), torch.ones(1 << 20, device=DEV)
    lat, pe = torch.zeros(8, LATENT, dtype=BF16, device=DEV), torch.zeros(8, PE, dtype=BF16, device=DEV)
    ws = torch.empty(kda.kda_mla_decode_workspace_size(8, 1, H), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()

    def work():
        def slow():
            x = big
            for _ in range(8):
                x = (x @ big) * 0.02
            zero = x[0, 0] * 0.0
            for t, s in zip(now, source):
                t.copy_(s + zero.to(BF16))
        if last == "join":
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                slow()
            spare.add_(1)
            torch.cuda.current_stream().wait_stream(side)
        else:
            slow()
            if last == "copy":
                now[2].copy_(source[2])
            elif last == "set":
                spare.zero_()
        kda.kda_mla_cache_write(now[0], now[1], cache.latent, cache.pe, cache.table, lens, cu)
        kda.kda_mla_cache_read(cache.latent, cache.pe, cache.table, cu, 8, starts=starts, latent=lat, pe=pe)
        out[1].copy_(lat)
        kda.kda_mla_decode(now[2], now[3], cache.latent, cache.pe, cache.table, lens, softmax_scale=SCALE, o=out[0],
                           workspace=ws)

    def set_inputs(i):
        for s, t in zip(source, new[i]):
            s.copy_(t)

    set_inputs(0)
    work()
    torch.cuda.synchronize()
    run = work
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            work()
        run = graph.replay
    for i in (1, 2, 0, 1):
        set_inputs(i)
        run()
        got = out[0].clone()
        torch.cuda.synchronize()
        assert torch.equal(out[1], new[i][0]) and torch.equal(pe, new[i][1])
        want, tol, _, _ = mla_ref.decode(new[i][2], new[i][3], cache, SCALE, BF16)
        mla_ref.check(got, want, tol, "o")


def test_two_streams_at_once():
    # two caches and two workspaces, each call's results as when it ran alone
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    caches = [Cache([700, 1, 90], 64, BF16, DEV, seed=1).fill(5), Cache([33, 2000], 16, torch.float8_e4m3fn, DEV, seed=2).fill(6)]
    g = torch.Generator(device=DEV).manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF16)  # noqa: E731
    work = []
    for c in caches:
        B = len(c.lengths)
        work.append(dict(q=[r(B, 1, 32, LATENT) for _ in range(10)], p=[r(B, 1, 32, PE) for _ in range(10)],
                         lat=r(B, LATENT), pe=r(B, PE), cu=cu_of([1] * B, DEV)))

    def run(c, w):
        kda.kda_mla_cache_write(w["lat"], w["pe"], c.latent, c.pe, c.table, c.seq_lens, w["cu"], cache_scale=c.scale)
        return [kda.kda_mla_decode(q, p, c.latent, c.pe, c.table, c.seq_lens, softmax_scale=SCALE, cache_scale=c.scale,
                                   output_lse=True) for q, p in zip(w["q"], w["p"])]

    alone = [run(c, w) for c, w in zip(caches, work)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [None, None]
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got[i] = run(caches[i], work[i])
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            for (o1, l1), (o2, l2) in zip(a, b):
                assert torch.equal(o1, o2) and torch.equal(l1, l2)
