"""The measured calls of the 4-bit key/value cache: writing new tokens into it, reading
tokens back, and decode attention over it.

The cache holds keys and values as Q4_0 blocks along the head dimension (32 values, one
binary16 scale d, codes q in 0..15, value d * (q - 8)) in pages of a multiple of 32
tokens. `run` computes each operator in plain torch when `own` is false and calls the
library when it is true; both work on the same bytes. `exact` gives the same outputs from
the definitions in 64 bits, from the drawn codes and scales, not from the bytes.

Bytes of one record (32 tokens of one key/value head, 36 * head_dim bytes; NB = head_dim / 32
blocks a token, in chunks of C = min(NB, 4)):
  keys    [NB/C][32 tokens][4 words][C blocks] 32-bit words: word c of a block holds its
          bytes 4c .. 4c+3 (byte j: code j in the low nibble, code j + 16 in the high one)
  values  [NB/C][2][2][4][8][2][C] 16-bit halves: token 16 u + 8 j + 2 c + e, half g
          (bytes 2g, 2g+1) of a block at [chunk][u][j][c][g][e][block]
  scales  of the keys, then of the values: binary16 [32 tokens][NB]
Record (page, head, group of 32 tokens) starts at ((page * heads + head) * groups + group) * 36 * head_dim.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one decode step of 16 sequences appends its keys and values, ragged contexts
        {"name": "write decode 16", "op": "write", "seqs": 16, "new": 1, "len": 2048, "ragged": True, "heads": 8, "dim": 128, "page": 64, "type": "f32"},
        # a prompt's keys and values in one call
        {"name": "write prompt 8192", "op": "write", "seqs": 1, "new": 8192, "len": 8192, "ragged": False, "heads": 8, "dim": 128, "page": 64, "type": "bf16"},
        # five prompts of different lengths in one padded call, odd sizes, small heads
        {"name": "write padded 5x333", "op": "write", "seqs": 5, "new": 333, "len": 901, "ragged": True, "heads": 3, "dim": 64, "page": 32, "type": "f16"},
        # a long context read back whole, as a prefill over a cached prefix does
        {"name": "read 32768", "op": "read", "seqs": 1, "new": 32768, "len": 32768, "ragged": False, "heads": 8, "dim": 128, "page": 64, "type": "bf16"},
        # four ragged sequences read back in binary32
        {"name": "read 4x1111", "op": "read", "seqs": 4, "new": 1111, "len": 1111, "ragged": True, "heads": 5, "dim": 64, "page": 32, "type": "f32"},
        # the smallest call: one token, one short sequence
        {"name": "attend 1x777", "op": "attend", "seqs": 1, "new": 1, "len": 777, "ragged": False, "q_heads": 9, "heads": 3, "dim": 64, "page": 32, "type": "f32", "window": 0, "softcap": 0.0, "alibi": False, "lse": False},
        # one token of an 8B-class layer over a long context
        {"name": "attend 1x8192", "op": "attend", "seqs": 1, "new": 1, "len": 8192, "ragged": False, "q_heads": 32, "heads": 8, "dim": 128, "page": 64, "type": "f32", "window": 0, "softcap": 0.0, "alibi": False, "lse": False},
        # a serving batch of a small model, lengths ragged, one slot empty
        {"name": "attend 24x3000", "op": "attend", "seqs": 24, "new": 1, "len": 3000, "ragged": True, "q_heads": 15, "heads": 5, "dim": 64, "page": 64, "type": "bf16", "window": 0, "softcap": 0.0, "alibi": False, "lse": True},
        # the largest: a long-context serving batch of an 8B-class layer
        {"name": "attend 16x32768", "op": "attend", "seqs": 16, "new": 1, "len": 32768, "ragged": True, "q_heads": 32, "heads": 8, "dim": 128, "page": 128, "type": "bf16", "window": 0, "softcap": 0.0, "alibi": False, "lse": False},
        # several tokens a sequence (checked drafts), causal among themselves
        {"name": "attend 4x8 of 6000", "op": "attend", "seqs": 4, "new": 8, "len": 6000, "ragged": True, "q_heads": 32, "heads": 8, "dim": 128, "page": 64, "type": "bf16", "window": 0, "softcap": 0.0, "alibi": False, "lse": False},
        # a layer with a sliding window and capped scores, wide heads
        {"name": "attend window softcap", "op": "attend", "seqs": 12, "new": 1, "len": 9001, "ragged": True, "q_heads": 16, "heads": 8, "dim": 256, "page": 64, "type": "f16", "window": 4096, "softcap": 50.0, "alibi": False, "lse": False},
        # a bias by distance, one key/value head a query head, two tokens
        {"name": "attend alibi", "op": "attend", "seqs": 8, "new": 2, "len": 1024, "ragged": True, "q_heads": 12, "heads": 12, "dim": 64, "page": 32, "type": "f32", "window": 0, "softcap": 0.0, "alibi": True, "lse": True},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even in its logarithm."""
    return min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend", "attend"])
    dim = rng.choice([64, 128, 128, 256])
    heads = rng.choice([1, 2, 3, 4, 5, 8, 12])
    case = {"op": op, "page": rng.choice([32, 64, 96, 128, 256]), "type": rng.choice(["f32", "f16", "bf16"]), "ragged": rng.random() < 0.75}
    if op == "attend":
        length = _spread(rng, 1, 32768)
        room = 200_000_000 // (length * heads * dim)  # values of the keys: no more than the largest listed case
        seqs = max(1, min(_spread(rng, 1, 64), room))
        new = rng.choice([1, 1, 1, 2, 3, 4, 5, 8, 16])
        group = rng.choice([1, 2, 3, 4, 5, 7, 8])
        if seqs * length * heads * dim * group * new > 8_000_000_000:
            new = 1
        case |= {"seqs": seqs, "new": new, "len": length, "q_heads": heads * group, "heads": heads, "dim": dim,
                 "window": rng.choice([0, 0, _spread(rng, 1, 8192)]), "softcap": rng.choice([0.0, 0.0, 30.0]), "alibi": rng.random() < 0.25, "lse": rng.random() < 0.5}
    else:
        new = _spread(rng, 1, 32768)
        room = 32_000_000 // (new * heads * dim)
        seqs = max(1, min(_spread(rng, 1, 64), room))
        case |= {"seqs": seqs, "new": new, "len": new + (_spread(rng, 1, 2048) if op == "write" else 0), "heads": heads, "dim": dim}
    return case


def _lengths(case):
    """Tokens each sequence holds, and how many of them are new: by the case alone."""
    s, n, t = case["seqs"], case["len"], case["new"]
    if not case["ragged"]:
        return [n] * s, [t] * s
    r = random.Random("%d %d %d" % (s, n, t))
    lens = [n] + [r.randint(max(1, n // 8), n) for _ in range(s - 1)]
    new = [t] * s
    if case["op"] == "attend" and s >= 8:
        lens[s // 2] = 0  # a slot of the batch that holds no sequence
    if case["op"] == "write":
        new = [min(t, m) if i % 2 else max(1, min(t, m) * 2 // 3) for i, m in enumerate(lens)]
    return lens, new


def _quantise(w):
    """Q4_0 codes and scales of binary32 blocks along the last dimension."""
    b = w.view(*w.shape[:-1], -1, 32)
    at = b.abs().max(-1, keepdim=True).indices
    d = b.gather(-1, at) * -0.125
    inv = torch.where(d != 0, 1.0 / d, torch.zeros_like(d))
    q = torch.floor(b * inv + 8.5).clamp_(0, 15).to(torch.uint8)
    return q.view(w.shape), d.squeeze(-1).to(torch.float16)


def _records(kq, kd, vq, vd):
    """Bytes of records from codes [n, 32, dim] and scales [n, 32, NB]."""
    n, _, dim = kq.shape
    nb = dim // 32
    c = min(nb, 4)

    def joined(q):
        q = q.view(n, 32, nb, 2, 16)
        return q[:, :, :, 0] | (q[:, :, :, 1] << 4)

    k = joined(kq).view(n, 32, nb // c, c, 4, 4).permute(0, 2, 1, 4, 3, 5).reshape(n, 16 * dim)
    v = joined(vq).view(n, 2, 2, 4, 2, nb // c, c, 8, 2).permute(0, 5, 1, 2, 3, 7, 4, 6, 8).reshape(n, 16 * dim)
    s = [x.contiguous().view(n, 32 * nb).view(torch.uint8) for x in (kd, vd)]
    return torch.cat([k, v, *s], 1)


def _values(rec, dim):
    """Keys and values [n, 32, dim] in binary32 from the bytes of records [n, 36 * dim]."""
    n = rec.shape[0]
    nb = dim // 32
    c = min(nb, 4)
    k = rec[:, :16 * dim].reshape(n, nb // c, 32, 4, c, 4).permute(0, 2, 1, 4, 3, 5).reshape(n, 32, nb, 16)
    v = rec[:, 16 * dim:32 * dim].reshape(n, nb // c, 2, 2, 4, 8, 2, c, 2).permute(0, 2, 3, 4, 6, 1, 7, 5, 8).reshape(n, 32, nb, 16)
    s = rec[:, 32 * dim:].contiguous().view(torch.float16).view(n, 2, 32, nb, 1).float()
    k = torch.cat([k & 15, k >> 4], -1).float().sub_(8).mul_(s[:, 0]).view(n, 32, dim)
    v = torch.cat([v & 15, v >> 4], -1).float().sub_(8).mul_(s[:, 1]).view(n, 32, dim)
    return k, v


def _inputs(case, seed):
    """Everything that is drawn, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    s, h, dim, page = case["seqs"], case["heads"], case["dim"], case["page"]
    lens, new = _lengths(case)
    each = -(-max(lens) // page)  # pages of the longest sequence
    pages = s * each + 3
    x = {"lens": torch.tensor(lens, dtype=torch.int32, device="cuda"), "new": torch.tensor(new, dtype=torch.int32, device="cuda"), "pages": pages,
         "table": torch.randperm(pages, generator=g, device="cuda")[: s * each].view(s, each).to(torch.int32)}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "write":
        x["k"], x["v"] = (normal(s, case["new"], h, dim).to(TYPES[case["type"]]) for _ in "kv")
        return x
    # a page of keys has a few large channels, as keys after rotary positions do
    scale = 1 + 3 * (torch.rand(h, 1, dim, generator=g, device="cuda") > 0.97)
    shape = (pages, h, page // 32, 32)
    for name in "kv":
        q = torch.empty(*shape, dim, dtype=torch.uint8, device="cuda")
        d = torch.empty(*shape, dim // 32, dtype=torch.float16, device="cuda")
        step = max(1, 50_000_000 // (h * page * dim))
        for p in range(0, pages, step):
            m = min(step, pages - p)
            w = normal(m, h, page, dim) * (scale if name == "k" else 0.7)
            a, b = _quantise(w)
            q[p:p + m], d[p:p + m] = a.view(m, *shape[1:], dim), b.view(m, *shape[1:], dim // 32)
        x[name + "q"], x[name + "d"] = q, d
    if case["op"] == "attend":
        x["q"] = (normal(s, case["new"], case["q_heads"], dim) * (0.5 + torch.rand(case["q_heads"], 1, generator=g, device="cuda"))).to(TYPES[case["type"]])
        x["slopes"] = 2.0 ** (-8.0 * torch.arange(1, case["q_heads"] + 1, device="cuda") / case["q_heads"]) if case["alibi"] else None
    return x


def prepare(case, seed):
    x = _inputs(case, seed)
    h, dim, page = case["heads"], case["dim"], case["page"]
    state = {"case": case, "lens": x["lens"], "table": x["table"]}
    if case["op"] == "write":
        state["data"] = torch.zeros(x["pages"], h, page // 32, 36 * dim, dtype=torch.uint8, device="cuda")
        state |= {"k": x["k"], "v": x["v"], "new": x["new"], "starts": x["lens"] - x["new"]}
    else:
        n = x["pages"] * h * (page // 32)
        parts = [x[m].view(n, 32, -1) for m in ("kq", "kd", "vq", "vd")]
        step = max(1, 100_000_000 // (32 * dim))
        state["data"] = torch.cat([_records(*(p[i:i + step] for p in parts)) for i in range(0, n, step)]).view(x["pages"], h, page // 32, 36 * dim)
        if case["op"] == "attend":
            state |= {"q": x["q"], "slopes": x["slopes"]}
    if own:  # the handle of the same bytes, and the workspace, that a program keeps
        from quantized_decode_q4_b200 import q4
        state["cache"] = q4.KVCache(x["pages"], h, dim, page, data=state["data"])
        if case["op"] == "attend":
            state["ws"] = q4.workspace(q4.kv_attention_workspace_bytes(dim))
    return state


def run(state):
    case = state["case"]
    if own:
        from quantized_decode_q4_b200 import q4
        if case["op"] == "write":
            q4.kv_write(state["cache"], state["k"], state["v"], state["table"], state["lens"], state["new"])
            return q4.kv_read(state["cache"], state["table"], state["lens"], case["new"], state["starts"], dtype=torch.float32)
        if case["op"] == "read":
            return q4.kv_read(state["cache"], state["table"], state["lens"], case["new"], dtype=TYPES[case["type"]])
        lse = torch.empty(state["q"].shape[:3], dtype=torch.float32, device="cuda") if case["lse"] else None
        out = q4.kv_attention(state["cache"], state["q"], state["table"], state["lens"], window=case["window"], softcap=case["softcap"],
                              alibi=state["slopes"], lse=lse, ws=state["ws"])
        return {"out": out, "lse": lse} if case["lse"] else {"out": out}
    if case["op"] == "write":
        return _plain_write(state)
    if case["op"] == "read":
        k, v = _plain_read(state, case["new"])
        return k.to(TYPES[case["type"]]), v.to(TYPES[case["type"]])
    return _plain_attend(state)


def _plain_write(state):
    """The new tokens' records are read, their tokens replaced, and written back."""
    case = state["case"]
    s, t, h, dim, page = case["seqs"], case["new"], case["heads"], case["dim"], case["page"]
    i = torch.arange(t, device="cuda")
    there = i < state["new"][:, None]
    pos = torch.where(there, state["starts"][:, None] + i, 0).long()
    slot = (state["table"].gather(1, pos // page).long() * page + pos % page)[there]  # [new tokens]
    (kq, kd), (vq, vd) = (_quantise(state[m][there].float()) for m in "kv")  # [new tokens, h, ...]
    groups = state["data"].view(-1, h, page // 32, 36 * dim).transpose(1, 2).reshape(-1, h, 36 * dim)  # by group of 32 tokens
    at, inverse = torch.unique(slot // 32, return_inverse=True)
    n = at.numel()
    nb = dim // 32
    # codes and scales of the touched records, then the new tokens' in their places
    old = groups[at].view(n * h, 36 * dim)
    k0, v0 = _codes(old, dim)
    s0 = old[:, 32 * dim:].contiguous().view(torch.float16).view(n, h, 2, 32, nb)
    k0, v0 = k0.view(n, h, 32, dim), v0.view(n, h, 32, dim)
    k0[inverse, :, slot % 32], v0[inverse, :, slot % 32] = kq, vq
    s0[inverse, :, 0, slot % 32], s0[inverse, :, 1, slot % 32] = kd, vd
    rec = _records(k0.view(n * h, 32, dim), s0[:, :, 0].reshape(n * h, 32, nb), v0.view(n * h, 32, dim), s0[:, :, 1].reshape(n * h, 32, nb))
    state["data"].view(-1, h, page // 32, 36 * dim)[at // (page // 32), :, at % (page // 32)] = rec.view(n, h, 36 * dim)
    out = []
    for q, d in ((kq, kd), (vq, vd)):
        o = torch.zeros(s, t, h, dim, device="cuda")
        o[there] = ((q.float() - 8).view(-1, h, nb, 32) * d.float()[..., None]).view(-1, h, dim)
        out.append(o)
    return tuple(out)


def _codes(rec, dim):
    n = rec.shape[0]
    nb = dim // 32
    c = min(nb, 4)
    k = rec[:, :16 * dim].reshape(n, nb // c, 32, 4, c, 4).permute(0, 2, 1, 4, 3, 5).reshape(n, 32, nb, 16)
    v = rec[:, 16 * dim:32 * dim].reshape(n, nb // c, 2, 2, 4, 8, 2, c, 2).permute(0, 2, 3, 4, 6, 1, 7, 5, 8).reshape(n, 32, nb, 16)
    return torch.cat([k & 15, k >> 4], -1).view(n, 32, dim), torch.cat([v & 15, v >> 4], -1).view(n, 32, dim)


def _plain_read(state, count):
    """Keys and values [seqs, count, heads, dim] in binary32, zero behind each sequence's end."""
    case = state["case"]
    s, h, dim, page = case["seqs"], case["heads"], case["dim"], case["page"]
    rec = state["data"][state["table"].long()]  # [s, pages, h, groups, bytes]
    rec = rec.transpose(2, 3).reshape(-1, 36 * dim)
    there = (torch.arange(count, device="cuda") < state["lens"][:, None])[..., None, None]
    k, v = (x.view(s, -1, h, 32, dim).transpose(2, 3).reshape(s, -1, h, dim)[:, :count] for x in _values(rec, dim))
    return torch.where(there, k, 0), torch.where(there, v, 0)


def _plain_attend(state):
    case = state["case"]
    s, t, hq, h, dim, n = case["seqs"], case["new"], case["q_heads"], case["heads"], case["dim"], case["len"]
    k, v = _plain_read(state, n)
    q = state["q"].float().view(s, t, h, hq // h, dim).permute(0, 2, 1, 3, 4).reshape(s, h, -1, dim)
    w = (q @ k.permute(0, 2, 3, 1)).view(s, h, t, hq // h, n) / math.sqrt(dim)
    if case["softcap"]:
        w = torch.tanh(w / case["softcap"]) * case["softcap"]
    key = torch.arange(n, device="cuda")
    row = (state["lens"][:, None] - t + torch.arange(t, device="cuda"))[:, None, :, None, None]  # position of each query token
    if case["alibi"]:
        w = w + state["slopes"].view(1, h, 1, hq // h, 1) * (key - row)
    seen = (key <= row) & (row >= 0)
    if case["window"]:
        seen = seen & (key > row - case["window"])
    w = w.masked_fill(~seen, -math.inf)
    m = w.amax(-1, keepdim=True)
    e = torch.exp(w - torch.where(m == -math.inf, 0.0, m))
    z = e.sum(-1, keepdim=True)
    o = (e.view(s, h, -1, n) @ v.transpose(1, 2)).view(s, h, t, hq // h, dim) / torch.where(z > 0, z, 1.0)
    out = {"out": o.permute(0, 2, 1, 3, 4).reshape(s, t, hq, dim).to(TYPES[case["type"]])}
    if case["lse"]:
        out["lse"] = (m + torch.log(z)).squeeze(-1).permute(0, 2, 1, 3).reshape(s, t, hq)
    return out


def work(case):
    lens, new = _lengths(case)
    h, dim, s, t = case["heads"], case["dim"], case["seqs"], case["new"]
    token = 2 * h * dim * 18 // 32  # bytes of a token in the cache
    wide = 2 * h * dim  # values of a token's key and value
    if case["op"] == "write":
        # the new tokens in, their blocks out; then the blocks in again and binary32 out
        return {"bytes": sum(new) * (wide * SIZE[case["type"]] + 2 * token) + s * t * wide * 4, "flops": sum(new) * wide * 4}
    if case["op"] == "read":
        return {"bytes": sum(min(t, n) for n in lens) * token + s * t * wide * SIZE[case["type"]], "flops": s * t * wide}
    seen = pairs = 0
    for n in lens:
        rows = [n - t + i for i in range(t) if n - t + i >= 0]
        low = [max(0, r - case["window"] + 1) if case["window"] else 0 for r in rows]
        seen += n - min(low) if rows else 0
        pairs += sum(r + 1 - a for r, a in zip(rows, low))
    q = s * t * case["q_heads"]
    return {"bytes": seen * token + q * (2 * dim * SIZE[case["type"]] + 4 * case["lse"]) + 8 * s, "flops": 4 * pairs * case["q_heads"] * dim}


def exact(case, seed):
    """The outputs of `run` in binary64, from the definitions: sequence by sequence, from the drawn codes and scales."""
    x = _inputs(case, seed)
    lens, new = _lengths(case)
    s, t, h, dim, page = case["seqs"], case["new"], case["heads"], case["dim"], case["page"]
    f64 = torch.float64
    if case["op"] == "write":
        outs = []
        for name in "kv":
            w = x[name].double().reshape(s, t, h, dim // 32, 32)
            # the block's value of largest magnitude, the first of equal ones
            big = w.abs().amax(-1, keepdim=True)
            first = (w.abs() == big).double().cumsum(-1) == 1
            first &= w.abs() == big
            m = (w * first).sum(-1, keepdim=True)
            d = m / -8
            # each step of the rule rounds to binary32: the reciprocal, the product, the sum
            inv = torch.where(d == 0, 0.0, 1 / torch.where(d == 0, 1.0, d)).float().double()
            code = torch.floor(((w * inv).float().double() + 8.5).float().double()).clamp(0, 15)
            value = (code - 8) * d.float().half().double()
            there = torch.arange(t, device="cuda") < x["new"][:, None]
            outs.append((value.reshape(s, t, h, dim) * there[..., None, None]))
        return tuple(outs)

    def of(name, i, n):
        """Keys or values of sequence i's first n tokens, [n, h, dim]."""
        p = x["table"][i, : -(-n // page)].long()
        q, d = (x[name + e][p].movedim(1, 3).reshape(-1, h, x[name + e].shape[-1])[:n].double() for e in "qd")
        return (q - 8) * d.repeat_interleave(32, -1)

    if case["op"] == "read":
        outs = [torch.zeros(s, t, h, dim, dtype=f64, device="cuda") for _ in "kv"]
        for o, name in zip(outs, "kv"):
            for i, n in enumerate(lens):
                o[i, : min(n, t)] = of(name, i, min(n, t))
        return tuple(outs)
    hq = case["q_heads"]
    out = torch.zeros(s, t, hq, dim, dtype=f64, device="cuda")
    lse = torch.full((s, t, hq), -math.inf, dtype=f64, device="cuda")
    for i, n in enumerate(lens):
        if not n:
            continue
        k, v = of("k", i, n), of("v", i, n)
        for j in range(max(0, t - n), t):
            row = n - t + j
            low = max(0, row - case["window"] + 1) if case["window"] else 0
            q = x["q"][i, j].double().reshape(h, hq // h, dim)
            w = torch.einsum("hgd,nhd->hgn", q, k[low:row + 1]) / math.sqrt(dim)
            if case["softcap"]:
                w = case["softcap"] * torch.tanh(w / case["softcap"])
            if case["alibi"]:
                w = w + x["slopes"].double().reshape(h, -1, 1) * torch.arange(low - row, 1, device="cuda")
            lse[i, j] = torch.logsumexp(w, -1).reshape(hq)
            out[i, j] = torch.einsum("hgn,nhd->hgd", torch.softmax(w, -1), v[low:row + 1]).reshape(hq, dim)
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
