"""Workloads of the latent-attention operators: the paged latent cache (write and read back), the absorbed form over that
cache (decode) and the expanded form (prefill), as the callers of libkda meet them.

A hybrid stack of KDA layers and latent-attention layers keeps, for each latent-attention layer, one latent vector of
512 channels and one positional key of 64 channels per token, in pages of a pool shared by the sequences.  Sizes: 32
heads and packed ragged batches as in this repository's KDA workloads, page sizes 16 to 128.

`own` False: the operators in elementary torch operations, in 32 bits, rounded once at the end.
`own` True: the calls of the library's binding.
"""
import math
import random

import torch

own = False

LATENT, PE = 512, 64          # cached channels per token
NOPE, DV = 128, 128           # per-head channels of the expanded form (queries and keys 128 + 64, values 128)
SCALE = 1.0 / math.sqrt(NOPE + PE)
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
DEV = "cuda"


# ---------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user's short chat: nothing but latency
        dict(name="decode_one_short", op="decode", batch=1, q_tokens=1, heads=32, min_len=300, max_len=300, page=64,
             cache="bf16"),
        # a served batch with ragged contexts
        dict(name="decode_batch_ragged", op="decode", batch=64, q_tokens=1, heads=32, min_len=1024, max_len=16384,
             page=64, cache="bf16"),
        # a large batch from a quantised cache, two tokens a sequence (one of them drafted), small pages
        dict(name="decode_batch_e4m3", op="decode", batch=128, q_tokens=2, heads=16, min_len=1, max_len=8000, page=16,
             cache="e4m3"),
        # one very long context: the split over the key axis
        dict(name="decode_long", op="decode", batch=1, q_tokens=1, heads=32, min_len=1000001, max_len=1000001, page=128,
             cache="bf16"),
        # a short prompt
        dict(name="prefill_short", op="prefill", batch=1, heads=32, min_q=200, max_q=200, max_prefix=0, causal=True),
        # a packed batch of ragged prompts
        dict(name="prefill_packed", op="prefill", batch=8, heads=32, min_q=63, max_q=2500, max_prefix=0, causal=True),
        # one long prompt
        dict(name="prefill_long", op="prefill", batch=1, heads=32, min_q=8192, max_q=8192, max_prefix=0, causal=True),
        # one chunk of a chunked prefill: its queries see the whole cached prefix
        dict(name="prefill_chunk", op="prefill", batch=1, heads=32, min_q=2048, max_q=2048, max_prefix=30000,
             causal=True),
        # the new tokens of one decode step of a large batch
        dict(name="write_step", op="write", batch=256, min_new=1, max_new=1, max_past=4000, page=64, source="bf16",
             cache="e4m3"),
        # the tokens of a packed prefill
        dict(name="write_prompts", op="write", batch=16, min_new=1024, max_new=8192, max_past=0, page=64, source="bf16",
             cache="e4m3"),
        # prefixes brought back for a chunked prefill, from either kind of cache
        dict(name="read_prefixes_e4m3", op="read", batch=16, min_len=1000, max_len=8000, page=64, cache="e4m3",
             out="bf16"),
        dict(name="read_one_bf16", op="read", batch=1, min_len=777, max_len=777, page=16, cache="bf16", out="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "write", "read"])
    page = rng.choice([16, 32, 64, 128])
    if op == "decode":
        batch = _log_uniform(rng, 1, 256)
        q_tokens = rng.choice([1, 1, 1, 2, 3, 4])
        heads = rng.choice([8, 12, 16, 20, 32, 32, 64, 128])
        most = min(1000000, 32000000 // (batch * q_tokens * heads), 1000000 // batch)
        max_len = _log_uniform(rng, 1, max(1, most))
        return dict(op=op, batch=batch, q_tokens=q_tokens, heads=heads, min_len=rng.randint(1, max_len),
                    max_len=max_len, page=page, cache=rng.choice(["bf16", "e4m3"]))
    if op == "prefill":
        batch = rng.choice([1, 1, 2, 3, 5, 8])
        heads = rng.choice([8, 12, 16, 32, 32, 64])
        pairs = 32 * 8192 * 8192 // (batch * heads)
        max_q = _log_uniform(rng, 1, min(16384, int(math.sqrt(pairs))))
        prefix = rng.choice([0, 0, 1]) * _log_uniform(rng, 1, max(1, min(32768, pairs // max_q - max_q)))
        return dict(op=op, batch=batch, heads=heads, min_q=rng.randint(1, max_q), max_q=max_q, max_prefix=prefix,
                    causal=rng.random() < 0.8)
    batch = _log_uniform(rng, 1, 256)
    if op == "write":
        max_new = _log_uniform(rng, 1, max(1, 70000 // batch))
        return dict(op=op, batch=batch, min_new=rng.randint(1, max_new), max_new=max_new,
                    max_past=rng.choice([0, 100, 60000 // batch]), page=page, source=rng.choice(["bf16", "bf16", "fp32"]),
                    cache=rng.choice(["bf16", "e4m3"]))
    max_len = _log_uniform(rng, 1, max(1, 70000 // batch))
    return dict(op=op, batch=batch, min_len=rng.randint(1, max_len), max_len=max_len, page=page,
                cache=rng.choice(["bf16", "e4m3"]), out=rng.choice(["bf16", "bf16", "fp32"]))


def _lengths(case, lo, hi, salt):
    """One length a sequence: the case's own, whatever the seed of the data; the first one is the longest."""
    key = ",".join("%s=%s" % (k, case[k]) for k in sorted(case) if k != "name")
    rng = random.Random(key + salt)
    return [hi if i == 0 else rng.randint(lo, hi) for i in range(case["batch"])]


def _cu(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu


# ---------------------------------------------------------------------------------------------------- inputs
def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pool(case, lengths, gen):
    """A pool of pages in random order with some left over, filled as a pool in use is, and the sequences' page table."""
    page = case["page"]
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + max(4, sum(need) // 16)
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    width = max(max(need), 1)
    col = torch.arange(width, device=DEV)
    first = torch.tensor(_cu(need)[:-1], device=DEV)[:, None]
    used = col[None] < torch.tensor(need, device=DEV)[:, None]
    table = torch.where(used, order[(first + col).clamp(max=pages - 1)], torch.full((), -1, dtype=torch.int32, device=DEV))
    latent = torch.randn(pages, page, LATENT, generator=gen, device=DEV, dtype=torch.bfloat16)
    pe = torch.randn(pages, page, PE, generator=gen, device=DEV, dtype=torch.bfloat16)
    scale = None
    if case["cache"] == "e4m3":  # a token's largest value of 512 is around 3 to 4: scales of 2^-7 mostly, some others
        scale = torch.exp2(torch.randint(-8, -5, (pages, page), generator=gen, device=DEV).float())
        latent = (latent.float() / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return dict(cache_latent=latent, cache_pe=pe, cache_scale=scale, page_table=table.contiguous())


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device=DEV, dtype=dtype)

    op, batch = case["op"], case["batch"]
    if op == "decode":
        lengths = _lengths(case, case["min_len"], case["max_len"], "len")
        s = _pool(case, lengths, gen)
        rows = (batch, case["q_tokens"], case["heads"])
        s |= dict(q_latent=normal(*rows, LATENT), q_pe=normal(*rows, PE), seq_lens=_int32(lengths))
    elif op == "prefill":
        nq = _lengths(case, case["min_q"], case["max_q"], "q")
        nk = [a + b for a, b in zip(nq, _lengths(case, 0, case["max_prefix"], "prefix"))]
        h = case["heads"]
        s = dict(q=normal(sum(nq), h, NOPE + PE), kv=normal(sum(nk), h, NOPE + DV), k_pe=normal(sum(nk), PE),
                 cu_q=_int32(_cu(nq)), cu_k=_int32(_cu(nk)), max_q=max(nq), max_k=max(nk), causal=case["causal"])
    elif op == "write":
        new = _lengths(case, case["min_new"], case["max_new"], "new")
        total = [a + b for a, b in zip(new, _lengths(case, 0, case["max_past"], "past"))]
        s = _pool(case, total, gen)
        # normalised latents differ in size from token to token, by their norm's weights
        size = torch.exp(torch.randn(sum(new), 1, generator=gen, device=DEV) * 0.5)
        dt = DTYPES[case["source"]]
        s |= dict(latent=(torch.randn(sum(new), LATENT, generator=gen, device=DEV) * size).to(dt),
                  pe=normal(sum(new), PE, dtype=dt), cu=_int32(_cu(new)), seq_lens=_int32(total))
    else:
        lengths = _lengths(case, case["min_len"], case["max_len"], "len")
        s = _pool(case, lengths, gen)
        s |= dict(cu=_int32(_cu(lengths)), total=sum(lengths), out=DTYPES[case["out"]])
    s["op"] = op
    return s


# ---------------------------------------------------------------------------------------------------- plain forms
def _slots(table, page, seq, pos):
    """Rows of the pool, flattened over pages, of the positions `pos` of the sequences `seq`."""
    return table[seq, pos // page].long().clamp(min=0) * page + pos % page


def _cached(s, slots):
    """The cached latents and positional keys of these rows, in 32 bits."""
    latent = s["cache_latent"]
    if s["cache_scale"] is not None:
        codes = latent.view(torch.uint8).reshape(-1, LATENT)[slots].view(torch.float8_e4m3fn)
        c = codes.float() * s["cache_scale"].reshape(-1)[slots][..., None]
    else:
        c = latent.reshape(-1, LATENT)[slots].float()
    return c, s["cache_pe"].reshape(-1, PE)[slots].float()


def _softmax(x, seen):
    """softmax over the last axis of the places `seen`, and log sum exp; a row that sees nothing gives 0 and -inf."""
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = x.sum(-1, keepdim=True)
    lse = (total.log() + top).squeeze(-1)
    return x.div_(torch.where(total == 0, torch.ones_like(total), total)), lse


def _decode(s):
    b, n, h, _ = s["q_latent"].shape
    page = s["cache_latent"].shape[1]
    lens, width = s["seq_lens"].long(), s["page_table"].shape[1] * page
    pos = torch.arange(width, device=DEV)
    c, p = _cached(s, _slots(s["page_table"], page, torch.arange(b, device=DEV)[:, None], pos[None]))
    q, qp = s["q_latent"].float().reshape(b, n * h, LATENT), s["q_pe"].float().reshape(b, n * h, PE)
    x = (q @ c.transpose(1, 2) + qp @ p.transpose(1, 2)).mul_(SCALE).reshape(b, n, h, width)
    last = lens[:, None] - (n - 1 - torch.arange(n, device=DEV))[None]
    w, lse = _softmax(x, (pos < last[..., None])[:, :, None])
    o = (w.reshape(b, n * h, width) @ c).reshape(b, n, h, LATENT)
    return o.to(torch.bfloat16), lse


def _prefill(s):
    h, batch = s["q"].shape[1], s["cu_q"].numel() - 1
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    nq, nk = cq[1:] - cq[:-1], ck[1:] - ck[:-1]
    iq, ik = torch.arange(s["max_q"], device=DEV), torch.arange(s["max_k"], device=DEV)
    at_q = (cq[:-1, None] + iq).clamp(max=s["q"].shape[0] - 1)       # [batch, max_q]
    at_k = (ck[:-1, None] + ik).clamp(max=s["kv"].shape[0] - 1)
    q = s["q"][at_q].float().transpose(1, 2)                         # [batch, heads, max_q, 192]
    kv = s["kv"][at_k].float().transpose(1, 2)
    p = s["k_pe"][at_k].float()[:, None]
    x = q[..., :NOPE] @ kv[..., :NOPE].transpose(2, 3)
    x += q[..., NOPE:] @ p.transpose(2, 3)
    x.mul_(SCALE)
    seen = (ik < nk[:, None])[:, None, None]
    if s["causal"]:
        seen = seen & (ik <= (iq + (nk - nq)[:, None])[..., None])[:, None]
    w, lse = _softmax(x, seen)
    o = (w @ kv[..., NOPE:]).transpose(1, 2).to(torch.bfloat16)      # [batch, max_q, heads, 128]
    t = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(cq[1:], t, right=True).clamp(max=batch - 1)
    return o[seq, t - cq[seq]], lse.transpose(1, 2)[seq, t - cq[seq]]


def _quantised(latent):
    """e4m3 codes of each token's latent, and its scale: the least power of two that brings the token into e4m3's range."""
    m, e = torch.frexp(latent.abs().amax(-1))
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(-64, 120)       # 448 = 0.875 * 2^9
    k = torch.where(m == 0, torch.full_like(k, -64), k)
    return torch.ldexp(latent, -k[:, None]).to(torch.float8_e4m3fn), torch.ldexp(torch.ones_like(m), k)


def _write(s):
    page = s["cache_latent"].shape[1]
    cu, lens = s["cu"].long(), s["seq_lens"].long()
    t = torch.arange(s["latent"].shape[0], device=DEV)
    seq = torch.searchsorted(cu[1:], t, right=True)
    at = _slots(s["page_table"], page, seq, lens[seq] - (cu[seq + 1] - t))
    latent = s["latent"].float()
    if s["cache_scale"] is not None:
        codes, scale = _quantised(latent)
        s["cache_latent"].view(torch.uint8).view(-1, LATENT)[at] = codes.view(torch.uint8)
        s["cache_scale"].view(-1)[at] = scale
    else:
        s["cache_latent"].view(-1, LATENT)[at] = latent.to(torch.bfloat16)
    s["cache_pe"].view(-1, PE)[at] = s["pe"].float().to(torch.bfloat16)
    return s["cache_latent"], s["cache_pe"], s["cache_scale"]


def _read(s):
    page, cu = s["cache_latent"].shape[1], s["cu"].long()
    t = torch.arange(s["total"], device=DEV)
    seq = torch.searchsorted(cu[1:], t, right=True)
    c, p = _cached(s, _slots(s["page_table"], page, seq, t - cu[seq]))
    return c.to(s["out"]), p.to(s["out"])


def run(s):
    if own:
        return _own(s)
    return {"decode": _decode, "prefill": _prefill, "write": _write, "read": _read}[s["op"]](s)


def _own(s):
    from gated_delta_rule_127_b200 import kda
    if s["op"] == "decode":
        return kda.kda_mla_decode(s["q_latent"], s["q_pe"], s["cache_latent"], s["cache_pe"], s["page_table"], s["seq_lens"],
                                  softmax_scale=SCALE, cache_scale=s["cache_scale"], output_lse=True)
    if s["op"] == "prefill":
        return kda.kda_mla_prefill(s["q"], s["kv"], s["k_pe"], s["cu_q"], s["cu_k"], causal=s["causal"],
                                   softmax_scale=SCALE, output_lse=True)
    if s["op"] == "write":
        kda.kda_mla_cache_write(s["latent"], s["pe"], s["cache_latent"], s["cache_pe"], s["page_table"], s["seq_lens"],
                                s["cu"], cache_scale=s["cache_scale"])
        return s["cache_latent"], s["cache_pe"], s["cache_scale"]
    return kda.kda_mla_cache_read(s["cache_latent"], s["cache_pe"], s["page_table"], s["cu"], s["total"],
                                  cache_scale=s["cache_scale"], dtype_o=s["out"])


# ---------------------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "prefill":
        nq = _lengths(case, case["min_q"], case["max_q"], "q")
        nk = [a + b for a, b in zip(nq, _lengths(case, 0, case["max_prefix"], "prefix"))]
        h = case["heads"]
        pairs = sum(a * b - (a * (a - 1) // 2 if case["causal"] else 0) for a, b in zip(nq, nk))
        moved = sum(nq) * h * ((NOPE + PE + DV) * 2 + 4) + sum(nk) * (h * (NOPE + DV) + PE) * 2
        return {"bytes": moved, "flops": 2 * h * pairs * (NOPE + PE + DV)}
    row = (LATENT + 4 if case["cache"] == "e4m3" else 2 * LATENT) + 2 * PE
    if op == "decode":
        lengths = _lengths(case, case["min_len"], case["max_len"], "len")
        rows = case["q_tokens"] * case["heads"]
        moved = sum(lengths) * row + case["batch"] * rows * ((2 * LATENT + PE) * 2 + 4)
        return {"bytes": moved, "flops": 2 * rows * sum(lengths) * (2 * LATENT + PE)}
    if op == "write":
        n = sum(_lengths(case, case["min_new"], case["max_new"], "new"))
        return {"bytes": n * (row + (LATENT + PE) * DTYPES[case["source"]].itemsize), "flops": n * LATENT}
    n = sum(_lengths(case, case["min_len"], case["max_len"], "len"))
    return {"bytes": n * (row + (LATENT + PE) * DTYPES[case["out"]].itemsize), "flops": n * LATENT}


# ---------------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The operators' definitions in 64 bits, one sequence (and head) at a time."""
    s = prepare(case, seed)
    if s["op"] == "prefill":
        return _exact_prefill(s)
    page, table = s["cache_latent"].shape[1], s["page_table"]

    def rows(b, first, count):  # the pool's rows of `count` positions of sequence b
        pos = torch.arange(first, first + count, device=DEV)
        return table[b].long()[torch.div(pos, page, rounding_mode="floor")] * page + torch.remainder(pos, page)

    flat_c, flat_p = s["cache_latent"].view(-1, LATENT), s["cache_pe"].view(-1, PE)
    flat_s = None if s["cache_scale"] is None else s["cache_scale"].view(-1)

    def tokens(b, first, count):
        at = rows(b, first, count)
        if flat_s is None:
            return flat_c[at].double(), flat_p[at].double()
        c = flat_c.view(torch.uint8)[at].view(torch.float8_e4m3fn).double()
        return torch.einsum("tc,t->tc", c, flat_s[at].double()), flat_p[at].double()

    if s["op"] == "decode":
        batch, n, h, _ = s["q_latent"].shape
        o = torch.zeros(batch, n, h, LATENT, dtype=torch.float64, device=DEV)
        lse = torch.full((batch, n, h), -math.inf, dtype=torch.float64, device=DEV)
        for b, length in enumerate(s["seq_lens"].tolist()):
            c, p = tokens(b, 0, length)
            for i in range(n):
                see = length - (n - 1 - i)
                if see > 0:
                    x = torch.einsum("hc,tc->ht", s["q_latent"][b, i].double(), c[:see])
                    x = SCALE * (x + torch.einsum("hc,tc->ht", s["q_pe"][b, i].double(), p[:see]))
                    lse[b, i] = torch.logsumexp(x, 1)
                    o[b, i] = torch.einsum("ht,tc->hc", torch.exp(x - lse[b, i, :, None]), c[:see])
        return o, lse
    cu = s["cu"].tolist()
    if s["op"] == "read":
        got = [tokens(b, 0, cu[b + 1] - cu[b]) for b in range(len(cu) - 1)]
        return torch.cat([c for c, _ in got]), torch.cat([p for _, p in got])
    latent, pe = flat_c.double(), flat_p.double()
    scale = None if flat_s is None else flat_s.double()
    for b, length in enumerate(s["seq_lens"].tolist()):
        new = s["latent"][cu[b]:cu[b + 1]].double()
        at = rows(b, length - len(new), len(new))
        pe[at] = s["pe"][cu[b]:cu[b + 1]].double()
        if scale is None:
            latent[at] = new
        else:
            # the inputs have at most 24 bits, so a size that is no exact 448 * 2^k is over it by a factor of 1 + 2^-24
            size = torch.exp2(torch.ceil(torch.log2(new.abs().amax(1) / 448.0) - 1e-10).clamp(-64, 120))
            scale[at] = size
            latent[at] = new / size[:, None]
    shape = s["cache_latent"].shape
    return (latent.view(shape), pe.view(s["cache_pe"].shape), None if scale is None else scale.view(shape[:2]))


def _exact_prefill(s):
    cq, ck, h = s["cu_q"].tolist(), s["cu_k"].tolist(), s["q"].shape[1]
    o = torch.zeros(cq[-1], h, DV, dtype=torch.float64, device=DEV)
    lse = torch.full((cq[-1], h), -math.inf, dtype=torch.float64, device=DEV)
    for b in range(len(cq) - 1):
        nq, nk = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        hidden = None
        if s["causal"]:
            hidden = torch.ones(nq, nk, dtype=torch.bool, device=DEV).triu(1 + nk - nq)
        pe = s["k_pe"][ck[b]:ck[b + 1]].double()
        for i in range(h):
            q, kv = s["q"][cq[b]:cq[b + 1], i].double(), s["kv"][ck[b]:ck[b + 1], i].double()
            x = SCALE * (q @ torch.cat([kv[:, :NOPE], pe], 1).T)
            if hidden is not None:
                x = x.masked_fill(hidden, -math.inf)
            row = torch.logsumexp(x, 1)
            lse[cq[b]:cq[b + 1], i] = row
            o[cq[b]:cq[b + 1], i] = torch.exp(x - row[:, None]) @ kv[:, NOPE:]
    return o, lse
