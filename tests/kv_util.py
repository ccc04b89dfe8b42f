"""Helpers for the tests of the 4-bit key/value cache: caches filled through q4.kv_write,
and attention in 64 bits over what q4.kv_read gives (which has its own tests against the
oracle), with the error that the arithmetic of the kernels allows."""
from __future__ import annotations

import math

import torch

from quantized_decode_q4_b200 import q4

INF = math.inf


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


class Filled:
    """A cache whose sequences hold `lens` random tokens, in pages in random order, with
    pages to spare; the places behind each sequence's end hold scales that are NaN."""

    def __init__(self, lens, heads, dim, page=32, seed=0, k_std=1.0, v_std=1.0, spare=2, stale_nan=True, pages=None,
                 tail=0):
        g = torch.Generator().manual_seed(seed)
        each = max(1, -(-max(max(lens), 1) // page)) + tail  # table entries behind the longest sequence too
        n = len(lens)
        pages = pages or n * each + spare
        self.cache = q4.KVCache(pages, heads, dim, page)
        self.table = torch.randperm(pages, generator=g)[: n * each].view(n, each).to(torch.int32).cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32).cuda()
        top = each * page
        gg = torch.Generator(device="cuda").manual_seed(seed + 1)
        k = torch.randn(n, top, heads, dim, generator=gg, device="cuda") * k_std
        v = torch.randn(n, top, heads, dim, generator=gg, device="cuda") * v_std
        if stale_nan:
            stale = torch.arange(top, device="cuda") >= self.lens[:, None]
            k[stale] = float("nan")
            v[stale] = float("nan")
        q4.kv_write(self.cache, k, v, self.table, torch.full_like(self.lens, top))

    def read(self, count=None):
        count = self.table.shape[1] * self.cache.page_size if count is None else count
        return q4.kv_read(self.cache, self.table, self.lens, count)


def attention64(f: Filled, q, new_lens=None, scale=None, window=0, softcap=0.0, alibi=None):
    """(out, lse, bound) in binary64. bound: what the kernels' arithmetic may be off by, before
    the result is rounded to its type. With x the scores and w their softmax, B = sum of
    |scale q k| and V = sum of w |v|, each with 24 |d| in place of |d (q - 8)| since codes and
    their offset of 8 are summed apart (15 + 8 < 24), u = 2^-23 (a tensor core's binary32 sum
    truncates):
      scores   |dx| <= 8 u B (q as two binary16 parts, 22 bits of the row's largest element;
               at most four sums a block) + 4 u |x| (scale, cap, bias, base-2 argument)
      weights  2 max |dx| + 8 u (exponential), and P rounded: rho
      sums     n / 16 + 8 truncations in V, and P below binary16's range: n 2^-30
    rho = 2 * 2^-11 where P is one binary16 number times a binary16 scale (bfloat16 results),
    4 u where it is two. The kernel chooses by q's type."""
    k, v = (t.double() for t in f.read(max(1, int(f.lens.max()))))
    s, t, hq, dim = q.shape
    h = f.cache.heads
    n = k.shape[1]
    kd, vd = (_scales(f, x, n) for x in "kv")
    scale = dim ** -0.5 if scale is None else scale
    q64 = q.double().reshape(s, t, h, hq // h, dim)
    x = torch.einsum("sthgd,snhd->sthgn", q64, k) * scale
    top = q64.abs().amax(-1, keepdim=True)
    big = torch.einsum("sthgd,snhd->sthgn", q64.abs() + top * 2.0 ** -1, kd) * scale
    u = 2.0 ** -23
    mag = x.abs()
    if softcap:
        x = softcap * torch.tanh(x / softcap)
        mag = mag + softcap  # tanh to a relative 2u
    nl = torch.full((s,), t, device="cuda") if new_lens is None else new_lens.long().clamp(0, t)
    i = torch.arange(t, device="cuda")
    pos = torch.where(i < nl[:, None], f.lens.long().clamp(min=0)[:, None] - nl[:, None] + i, -1)[:, :, None, None, None]
    key = torch.arange(n, device="cuda")
    if alibi is not None:
        a = alibi.double().view(1, 1, h, hq // h, 1) * (key - pos)
        x = x + a
        mag = mag + a.abs()
    seen = (key <= pos) & (pos >= 0)
    if window:
        seen = seen & (key > pos - window)
    x = x.masked_fill(~seen, -INF)
    m = x.amax(-1, keepdim=True)
    w = torch.exp(x - torch.where(m == -INF, 0.0, m))
    z = w.sum(-1, keepdim=True)
    w = w / torch.where(z > 0, z, 1.0)
    out = torch.einsum("sthgn,snhd->sthgd", w, v)
    lse = (m + torch.log(z)).squeeze(-1)
    dx = torch.where(seen, 8 * u * big + 4 * u * mag, 0.0).amax(-1, keepdim=True)
    vv = torch.einsum("sthgn,snhd->sthgd", w, vd)
    va = torch.einsum("sthgn,snhd->sthgd", w, v.abs())
    rho = 2 * 2.0 ** -11 if q.dtype == torch.bfloat16 else 4 * u
    bound = vv * (2 * dx + 8 * u + (n / 16 + 8) * u) + va * rho + n * 2.0 ** -30
    lse_bound = dx.squeeze(-1) + (n / 8 + 16) * u + 2 * u * lse.abs().nan_to_num(0, 0, 0)
    return out.reshape(s, t, hq, dim), lse.reshape(s, t, hq), bound.reshape(s, t, hq, dim), lse_bound.reshape(s, t, hq)


def _scales(f: Filled, which, n):
    """24 |d| of every value, spread over its block, [seqs, n, heads, dim]: from the largest
    magnitude of the block, which its scale makes 8 |d| exactly."""
    x = f.read(n)[0 if which == "k" else 1].double()
    b = x.view(*x.shape[:-1], -1, 32).abs().amax(-1, keepdim=True)
    return (b * 3).expand(*x.shape[:-1], -1, 32).reshape(x.shape)


def check_attention(f: Filled, q, out_dtype=None, got=None, **kw):
    """Runs q4.kv_attention (or takes `got` = (out, lse)) and compares it with attention64."""
    if got is None:
        lse = torch.full(q.shape[:3], float("nan"), device="cuda")
        out = torch.full(q.shape, float("nan"), dtype=out_dtype or q.dtype, device="cuda")
        args = {k: v for k, v in kw.items()}
        r = q4.kv_attention(f.cache, q, f.table, f.lens, out=out, lse=lse, **args)
        assert r is out
    else:
        out, lse = got
    ref, ref_lse, bound, lse_bound = attention64(f, q, **{k: v for k, v in kw.items() if k not in ("ws", "stream")})
    empty = ref_lse == -INF
    assert bool((out[empty] == 0).all()) and bool((lse[empty] == -INF).all())
    err = (out.double() - ref).abs()
    tol = bound + half_step(out.dtype) * (ref.abs() + bound) + 2.0 ** -25 * (out.dtype == torch.float16)
    bad = ~(err <= tol)
    assert not bool(bad.any()), (f"{int(bad.sum())} of {bad.numel()} outside; worst {float((err / tol).nan_to_num(1e9).max()):.3g} "
                                 f"at {torch.nonzero(bad)[0].tolist()}")
    lerr = (lse.double() - ref_lse).abs()
    lbad = ~(lerr <= lse_bound) & ~empty
    assert not bool(lbad.any()), f"lse off by {float(lerr[lbad].max()):.3g}, allowed {float(lse_bound[lbad].min()):.3g}"
    return out, lse
