"""Plain 64-bit forms of the latent-attention operators for the tests, with elementwise error bounds.

The bounds count every rounding of the documented arithmetic (u = half a step relative to the value: 2^-8 for bf16,
2^-24 for fp32, 2^-4 for e4m3):
  scores    sums of n products in fp32: n 2^-23 sum |q||k| (a factor 2 for the tensor core's own adder), and a
            relative 2^-22 for scaling and the change of the exponent's base
  weights   e^{dx} for a score error dx, then 2^-8 for their rounding (bf16, or two e4m3 parts: 2^-4 * 2^-4)
  sums      n 2^-23 sum w |v| in fp32
  output    half a step of its type
"""
import math

import torch

LATENT, PE, NOPE, DV = 512, 64, 128, 128
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def cu_of(lengths, device):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=device)


def attend(x, dx, v, out_dtype, extra=0.0):
    """softmax(x) v over the last axis of x [rows, keys] with score errors dx: (o, bound of o, lse, bound of lse).
    `extra`: a further absolute error of each weight, per row [rows, 1], in units of the largest weight's e^x."""
    rows, keys = x.shape
    if keys == 0:
        z = torch.zeros(rows, v.shape[1], dtype=torch.float64, device=x.device)
        return z, z, torch.full((rows,), -math.inf, dtype=torch.float64, device=x.device), torch.zeros_like(x.sum(1))
    lse = torch.logsumexp(x, 1)
    w = torch.exp(x - lse[:, None])
    o = w @ v
    d = dx.amax(1, keepdim=True)                     # one score error for the row
    rel = torch.expm1(2 * d) + 2.0 ** -8 + keys * 2.0 ** -23 + 2.0 ** -20
    a = w @ v.abs()
    tol = rel * a + extra + U[out_dtype] * o.abs() * (1 + rel) + 1e-30
    return o, tol, lse, d[:, 0] + (keys * 2.0 ** -23) + 2.0 ** -20 * (1 + lse.abs())


def score_error(q, k, scale, x):
    n = q.shape[-1]
    return abs(scale) * n * 2.0 ** -23 * (q.abs() @ k.abs().T) + 2.0 ** -22 * x.abs()


def prefill(q, kv, k_pe, nq, nk, causal, scale, out_dtype):
    """(o, tol, lse, lse tol), packed, for sequences of nq queries and nk keys each."""
    H = q.shape[1]
    got = [[], [], [], []]
    q0 = k0 = 0
    for a, b in zip(nq, nk):
        per = [[], [], [], []]
        for h in range(H):
            Q = q[q0:q0 + a, h].double()
            KV = kv[k0:k0 + b, h].double()
            K = torch.cat([KV[:, :NOPE], k_pe[k0:k0 + b].double()], 1)
            x = scale * (Q @ K.T)
            dx = score_error(Q, K, scale, x)
            if causal and b > 0:
                see = torch.arange(b, device=q.device)[None] <= (torch.arange(a, device=q.device)[:, None] + b - a)
                x = x.masked_fill(~see, -math.inf)
                dx = dx.masked_fill(~see, 0.0)
                seen = see.any(1)
            else:
                seen = torch.full((a,), b > 0, device=q.device)
            o = torch.zeros(a, DV, dtype=torch.float64, device=q.device)
            tol, lse = torch.zeros_like(o), torch.full((a,), -math.inf, dtype=torch.float64, device=q.device)
            lt = torch.zeros_like(lse)
            if bool(seen.any()):
                o[seen], tol[seen], lse[seen], lt[seen] = attend(x[seen], dx[seen], KV[:, NOPE:], out_dtype)
            for lst, t in zip(per, (o, tol, lse, lt)):
                lst.append(t)
        for lst, p in zip(got, per):
            lst.append(torch.stack(p, 1))
        q0, k0 = q0 + a, k0 + b
    return [torch.cat(g) for g in got]


class Cache:
    """A pool of pages in random order; unused rows, unused pages and unused table entries hold poison."""

    def __init__(self, lengths, page, dtype, device, seed=0, spare=3, poison=True, width_extra=2, first_page=0):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lengths]
        self.pages, self.page, self.dtype = first_page + sum(need) + spare, page, dtype
        order = (first_page + torch.randperm(sum(need) + spare, generator=g)).tolist()
        width = max(need + [0]) + width_extra
        table = torch.full((len(lengths), width), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.table = table.to(device)
        self.lengths, self.device = list(lengths), device
        bad = float("nan") if poison else 0.0
        self.latent = torch.empty(self.pages, page, LATENT, dtype=dtype, device=device)
        if dtype == torch.float8_e4m3fn:
            self.latent.view(torch.uint8).fill_(0x7F if poison else 0)
            self.scale = torch.full((self.pages, page), bad, device=device)
        else:
            self.latent.fill_(bad)
            self.scale = None
        self.pe = torch.full((self.pages, page, PE), bad, dtype=torch.bfloat16, device=device)
        self.seq_lens = torch.tensor(self.lengths, dtype=torch.int32, device=device)

    def rows(self, b, lo, hi):
        pos = torch.arange(lo, hi, device=self.device)
        return self.table[b, pos // self.page].long() * self.page + pos % self.page

    def fill(self, seed, spread=0.5):
        """Values for every used row, set directly (not through the library)."""
        g = torch.Generator(device=self.device).manual_seed(seed)
        for b, n in enumerate(self.lengths):
            at = self.rows(b, 0, n)
            c = torch.randn(n, LATENT, generator=g, device=self.device)
            c *= torch.exp(spread * torch.randn(n, 1, generator=g, device=self.device))
            if self.scale is None:
                self.latent.view(-1, LATENT)[at] = c.to(torch.bfloat16)
            else:
                codes, s = quantise(c.double())
                self.latent.view(torch.uint8).view(-1, LATENT)[at] = codes.view(torch.uint8)
                self.scale.view(-1)[at] = s.float()
            self.pe.view(-1, PE)[at] = torch.randn(n, PE, generator=g, device=self.device).to(torch.bfloat16)
        return self

    def tokens(self, b, lo, hi):
        at = self.rows(b, lo, hi)
        if self.scale is None:
            return self.latent.view(-1, LATENT)[at].double(), self.pe.view(-1, PE)[at].double(), None
        codes = self.latent.view(torch.uint8).view(-1, LATENT)[at].view(torch.float8_e4m3fn).double()
        s = self.scale.view(-1)[at].double()
        return codes * s[:, None], self.pe.view(-1, PE)[at].double(), s


def quantise(c):
    """e4m3 codes and power-of-two scales of rows c (64 bits), by trying exponents: the least k with max|c| <= 448 2^k."""
    a = c.abs().nan_to_num(nan=0.0).amax(1)
    k = torch.full_like(a, -64)
    for e in range(-64, 120):
        k = torch.where(a > 448 * 2.0 ** e, torch.full_like(k, e + 1), k)
    s = 2.0 ** k
    return (c / s[:, None]).clamp(-448, 448).float().to(torch.float8_e4m3fn), s


def decode(q_latent, q_pe, cache, scale, out_dtype):
    """(o, tol, lse, lse tol) [B, S, H, ...] of the absorbed form."""
    B, S, H, _ = q_latent.shape
    dev = q_latent.device
    o = torch.zeros(B, S, H, LATENT, dtype=torch.float64, device=dev)
    tol = torch.zeros_like(o)
    lse = torch.full((B, S, H), -math.inf, dtype=torch.float64, device=dev)
    lt = torch.zeros_like(lse)
    for b, n in enumerate(cache.lengths):
        c, p, s = cache.tokens(b, 0, n)
        for i in range(S):
            see = n - (S - 1 - i)
            if see <= 0:
                continue
            Q = torch.cat([q_latent[b, i].double(), q_pe[b, i].double()], 1)
            K = torch.cat([c[:see], p[:see]], 1)
            x = scale * (Q @ K.T)
            dx = score_error(Q, K, scale, x)
            extra = 0.0
            if s is not None:
                # e4m3 parts below their normal range: a query value is off by at most half of 2^-9 in units that put
                # the largest above 224, a weight times its scale by half of 2^-9 in units that put the largest
                # above 2^-1 (2^8 in the kernel's worst case of an old maximum 2^8 above it)
                dx = dx + abs(scale) * (Q[:, :LATENT].abs().amax(1, keepdim=True) * 2.0 ** -10 / 224) * c[:see].abs().sum(1)
                w = torch.exp(x - torch.logsumexp(x, 1)[:, None])
                top = (w * s[:see]).amax(1, keepdim=True)
                extra = 2.0 ** -9 * top * ((c[:see] / s[:see, None]).abs().sum(0)[None]) * 2.0 ** -8
            o[b, i], tol[b, i], lse[b, i], lt[b, i] = attend(x, dx, c[:see], out_dtype, extra)
    return o, tol, lse, lt


def check(got, want, tol, what):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), what + ": infinities"
    off = (got - want).abs()[~inf]
    over = off > tol[~inf]
    assert not bool(over.any()), "%s: %d of %d beyond the bound, worst %.3g of it" % (
        what, int(over.sum()), over.numel(), float((off / tol[~inf]).nan_to_num(posinf=1e30).max()))
