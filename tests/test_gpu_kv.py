"""The 4-bit key/value cache on the GPU: writing and reading back against the oracle's
Q4_0 blocks, bit for bit."""
import numpy as np
import pytest
import torch

import oracle
from quantized_decode_q4_b200 import q4

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def oracle_values(x: torch.Tensor) -> torch.Tensor:
    """x [..., dim] through the oracle's pack and dequant, binary32 on the CPU."""
    w = x.detach().float().cpu().reshape(-1, x.shape[-1]).numpy()
    return torch.from_numpy(oracle.q4_dequant(oracle.q4_pack(w), *w.shape)).view(x.shape)


def tables(n, each, extra=3, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(n * each + extra, generator=g)[: n * each].view(n, each).to(torch.int32).cuda(), n * each + extra


def rows(*shape, seed=0, dtype=torch.float32, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,heads,page", [(64, 3, 32), (128, 8, 64), (256, 2, 96)])
def test_write_then_read_is_the_oracle(dim, heads, page, dtype):
    lens, new = [150, 1, 97, 40], [150, 1, 33, 0]
    t = max(new)
    table, pages = tables(4, -(-150 // page))
    cache = q4.KVCache(pages, heads, dim, page)
    k, v = rows(4, t, heads, dim, seed=1, dtype=dtype), rows(4, t, heads, dim, seed=2, dtype=dtype, std=0.03)
    tl, tn = torch.tensor(lens, dtype=torch.int32).cuda(), torch.tensor(new, dtype=torch.int32).cuda()
    q4.kv_write(cache, k, v, table, tl, tn)
    for out_dtype in TYPES:
        gk, gv = q4.kv_read(cache, table, tl, t, tl - tn, dtype=out_dtype)
        for got, x in ((gk, k), (gv, v)):
            ref = oracle_values(x)
            for s in range(4):
                ref[s, new[s]:] = 0
            assert got.dtype == out_dtype and torch.equal(got.cpu(), ref.to(out_dtype))
    # before the new tokens of sequence 2 the cache is still empty
    k0, _ = q4.kv_read(cache, table, tl, 64)
    assert not bool(k0[2].any()) and not bool(k0[3].any())


def test_bytes_follow_the_documented_layout():
    """The record's bytes, from q4_pack's planes of the same rows and the layout's formula."""
    for dim in (64, 128, 256):
        heads, page, n = 2, 64, 64
        cache = q4.KVCache(2, heads, dim, page)
        table = torch.tensor([[1]], dtype=torch.int32).cuda()
        k, v = rows(1, n, heads, dim, seed=3), rows(1, n, heads, dim, seed=4)
        q4.kv_write(cache, k, v, table, torch.tensor([n], dtype=torch.int32).cuda())
        nb, c = dim // 32, min(dim // 32, 4)
        data = cache.data.cpu().view(2, heads, page // 32, 36 * dim)
        assert not bool(data[0].any())
        planes = []
        for x in (k, v):
            m = q4.pack(x.view(n * heads, dim))
            planes.append((m.qs_plane().cpu().view(n, heads, nb, 16), m.d_plane().cpu().view(n, heads, nb)))
        for h in range(heads):
            for r in range(page // 32):
                rec = data[1, h, r]
                kw = rec[: 16 * dim].view(nb // c, 32, 4, c, 4)
                vh = rec[16 * dim: 32 * dim].view(nb // c, 2, 2, 4, 8, 2, c, 2)
                sc = rec[32 * dim:].view(torch.int16).view(2, 32, nb)
                for t in range(32):
                    kq, vq = planes[0][0][32 * r + t, h], planes[1][0][32 * r + t, h]
                    for b in range(nb):
                        assert torch.equal(kw[b // c, t, :, b % c].reshape(16), kq[b])
                        got = vh[b // c, t >> 4, t >> 3 & 1, t >> 1 & 3, :, t & 1, b % c].reshape(16)
                        assert torch.equal(got, vq[b])
                        assert sc[0, t, b] == planes[0][1][32 * r + t, h, b]
                        assert sc[1, t, b] == planes[1][1][32 * r + t, h, b]


def test_one_token_at_a_time_equals_one_call():
    """Decode appends leave the same bytes as one call, across a page and a record border."""
    dim, heads, page, n = 128, 2, 32, 70
    table, pages = tables(1, 3)
    k, v = rows(1, n, heads, dim, seed=5), rows(1, n, heads, dim, seed=6)
    a, b = q4.KVCache(pages, heads, dim, page), q4.KVCache(pages, heads, dim, page)
    q4.kv_write(a, k, v, table, torch.tensor([n], dtype=torch.int32).cuda())
    for i in range(n):
        q4.kv_write(b, k[:, i:i + 1], v[:, i:i + 1], table, torch.tensor([i + 1], dtype=torch.int32).cuda())
    assert torch.equal(a.data, b.data)


def test_tokens_without_a_place_are_skipped():
    dim, heads, page = 64, 2, 32
    cache = q4.KVCache(4, heads, dim, page)
    cache.data.fill_(0x5A)
    before = cache.data.clone()
    k, v = rows(3, 5, heads, dim, seed=7), rows(3, 5, heads, dim, seed=8)
    # a negative page, one behind the cache; lengths that end behind the table and before 0
    table = torch.tensor([[-1, 4], [1000000, -2147483648], [0, 1]], dtype=torch.int32).cuda()
    for lens in ([5, 40, 0], [33, 5, -7], [64, 64, 2000000000]):
        q4.kv_write(cache, k, v, table, torch.tensor(lens, dtype=torch.int32).cuda())
        torch.cuda.synchronize()
        assert torch.equal(cache.data, before)
    # two of five tokens have positions 0 and 1
    q4.kv_write(cache, k, v, table, torch.tensor([0, 0, 2], dtype=torch.int32).cuda())
    gk, gv = q4.kv_read(cache, table, torch.tensor([0, 0, 2], dtype=torch.int32).cuda(), 2)
    assert torch.equal(gk[2].cpu(), oracle_values(k[2, 3:])) and torch.equal(gv[2].cpu(), oracle_values(v[2, 3:]))
    changed = (cache.data.view(4, -1) != before.view(4, -1)).any(1).tolist()
    assert changed == [True, False, False, False]
    # reads of the same bad pages give zeros
    gk, gv = q4.kv_read(cache, table, torch.tensor([64, 64, 0], dtype=torch.int32).cuda(), 70,
                        torch.tensor([-3, 0, 0], dtype=torch.int32).cuda())
    assert not bool(gk.any()) and not bool(gv.any())


def test_blocks_that_are_not_finite_read_back_as_nan():
    dim, heads, page = 128, 1, 32
    cache = q4.KVCache(1, heads, dim, page)
    table, lens = torch.zeros(1, 1, dtype=torch.int32).cuda(), torch.tensor([4], dtype=torch.int32).cuda()
    k, v = rows(1, 4, heads, dim, seed=9), rows(1, 4, heads, dim, seed=10)
    k[0, 0, 0, 5], k[0, 1, 0, 40], v[0, 2, 0, 127] = float("nan"), float("inf"), -float("inf")
    q4.kv_write(cache, k, v, table, lens)
    gk, gv = (x.isnan().view(4, 4, 32).all(-1).tolist() for x in q4.kv_read(cache, table, lens, 4))
    want = [[False] * 4 for _ in range(4)]
    wk = [r[:] for r in want]
    wk[0][0] = wk[1][1] = True
    wv = [r[:] for r in want]
    wv[2][3] = True
    assert gk == wk and gv == wv
    assert int(q4.kv_read(cache, table, lens, 4)[0].isnan().sum()) == 64


def test_zero_blocks_ties_and_ranges():
    """All-zero blocks, equal magnitudes of both signs, subnormal and large scales."""
    dim = 64
    x = torch.zeros(1, 32, 1, dim)
    x[0, 1, 0, ::2], x[0, 1, 0, 1::2] = 1.5, -1.5
    x[0, 2, 0, ::2], x[0, 2, 0, 1::2] = -1.5, 1.5
    x[0, 3] = torch.linspace(-1e-7, 1e-7, dim)
    x[0, 4] = torch.linspace(-4e5, 5e5, dim)
    x[0, 5] = -0.0
    x[0, 6, 0, 31], x[0, 6, 0, 32] = 3.0, -3.0
    x[0, 7:] = torch.randn(25, 1, dim, generator=torch.Generator().manual_seed(1)) * torch.logspace(-6, 4, 25)[:, None, None]
    cache = q4.KVCache(1, 1, dim, 32)
    table, lens = torch.zeros(1, 1, dtype=torch.int32).cuda(), torch.tensor([32], dtype=torch.int32).cuda()
    q4.kv_write(cache, x.cuda(), x.cuda().flip(1), table, lens)
    k, v = q4.kv_read(cache, table, lens, 32)
    assert np.array_equal(k.cpu().numpy(), oracle_values(x).numpy())
    assert np.array_equal(v.cpu().numpy(), oracle_values(x.flip(1)).numpy())


@pytest.mark.parametrize("dtype", TYPES)
def test_ties_and_tiny_values_of_every_type(dtype):
    """Equal magnitudes of both signs at every distance, and blocks whose 1 / d overflows."""
    dim, n = 128, 40
    g = torch.Generator().manual_seed(21)
    x = torch.randint(-3, 4, (1, n, 2, dim), generator=g).float() * 0.75  # many ties
    x[0, 3] = torch.randn(2, dim, generator=g) * 2.0 ** -130
    x[0, 4] = torch.randn(2, dim, generator=g) * 2.0 ** -127
    x[0, 5, 0, 7], x[0, 5, 1, 31] = 2.0 ** -133, -(2.0 ** -24)
    x[0, 6] = 0
    x[0, 6, 0, 64], x[0, 6, 0, 95] = -1.0, 1.0
    x = x.to(dtype)
    cache = q4.KVCache(2, 2, dim, 32)
    table, lens = torch.tensor([[1, 0]], dtype=torch.int32).cuda(), torch.tensor([n], dtype=torch.int32).cuda()
    q4.kv_write(cache, x.cuda(), x.cuda().flip(1), table, lens)
    k, v = q4.kv_read(cache, table, lens, n)
    assert torch.equal(k.cpu(), oracle_values(x)) and torch.equal(v.cpu(), oracle_values(x.flip(1)))
    # rows of two types in one call
    other = {torch.float32: torch.bfloat16, torch.float16: torch.float32, torch.bfloat16: torch.float16}[dtype]
    q4.kv_write(cache, x.cuda(), x.to(other).cuda(), table, lens)
    out = (torch.empty(1, n, 2, dim, dtype=other, device="cuda"), torch.empty(1, n, 2, dim, dtype=dtype, device="cuda"))
    q4.kv_read(cache, table, lens, n, out=out)
    assert torch.equal(out[0].cpu(), oracle_values(x).to(other)) and torch.equal(out[1].cpu(), oracle_values(x.to(other)).to(dtype))


def test_strides_and_unaligned_rows():
    dim, heads, n, s = 128, 4, 9, 3
    table, pages = tables(s, 1)
    lens = torch.tensor([9, 9, 9], dtype=torch.int32).cuda()
    for dtype in TYPES:
        base = rows(s, heads, n, dim, seed=11, dtype=dtype)
        k = base.transpose(1, 2)  # heads outside tokens
        flat = rows(s * n * heads * dim + 1, seed=12, dtype=dtype)
        v = flat[1:].view(s, n, heads, dim)  # an element off every alignment
        cache = q4.KVCache(pages, heads, dim, 32)
        q4.kv_write(cache, k, v, table, lens)
        room = [torch.full((s * n * heads * dim + 1,), 7.0, dtype=dtype, device="cuda"),
                torch.full((s, heads, n, dim), 7.0, dtype=dtype, device="cuda")]
        out = (room[0][1:].view(s, n, heads, dim), room[1].transpose(1, 2))
        q4.kv_read(cache, table, lens, n, out=out)
        assert torch.equal(out[0].cpu(), oracle_values(k).to(dtype)) and torch.equal(out[1].cpu(), oracle_values(v).to(dtype))
        assert room[0][0] == 7.0
    # one token's rows broadcast to every sequence, a table with wider rows
    wide = torch.full((s, 5), -1, dtype=torch.int32, device="cuda")
    wide[:, :1] = table
    one = rows(1, 1, heads, dim, seed=13)
    q4.kv_write(cache, one.expand(s, 2, heads, dim), one.expand(s, 2, heads, dim), wide[:, :1], lens)
    k, _ = q4.kv_read(cache, wide, lens, 2, lens - 2)
    assert torch.equal(k.cpu(), oracle_values(one).expand(s, 2, heads, dim))


def test_cache_beyond_two_and_four_gigabytes():
    dim, heads, page = 256, 8, 64
    per_page = 9216 * 2 * heads
    pages = (9 << 29) // per_page  # 4.8 GB
    cache = q4.KVCache(pages, heads, dim, page)
    at = [0, (1 << 31) // per_page, (1 << 32) // per_page, pages - 1]
    table = torch.tensor(at, dtype=torch.int32).cuda()[:, None]
    lens = torch.tensor([64, 64, 64, 64], dtype=torch.int32).cuda()
    k, v = rows(4, 64, heads, dim, seed=14, dtype=torch.bfloat16), rows(4, 64, heads, dim, seed=15, dtype=torch.bfloat16)
    q4.kv_write(cache, k, v, table, lens)
    gk, gv = q4.kv_read(cache, table, lens, 64)
    assert torch.equal(gk.cpu(), oracle_values(k)) and torch.equal(gv.cpu(), oracle_values(v))


def test_zero_tokens_and_sequences():
    cache = q4.KVCache(1, 1, 64, 32)
    table, lens = torch.zeros(2, 1, dtype=torch.int32).cuda(), torch.zeros(2, dtype=torch.int32).cuda()
    none = torch.empty(2, 0, 1, 64, device="cuda")
    before = q4.launch_count()
    q4.kv_write(cache, none, none, table, lens)
    assert q4.kv_read(cache, table, lens, 0)[0].shape == (2, 0, 1, 64)
    assert q4.kv_read(cache, table[:0], lens[:0], 3)[1].shape == (0, 3, 1, 64)
    assert q4.kv_attention(cache, none, table, lens).shape == (2, 0, 1, 64)
    assert q4.kv_attention(cache, torch.empty(0, 1, 1, 64, device="cuda"), table[:0], lens[:0]).shape == (0, 1, 1, 64)
    assert q4.launch_count() == before


def test_binding_refuses():
    cache = q4.KVCache(2, 2, 64, 32)
    table, lens = torch.zeros(1, 1, dtype=torch.int32).cuda(), torch.ones(1, dtype=torch.int32).cuda()
    x = torch.zeros(1, 1, 2, 64, device="cuda")
    q = torch.zeros(1, 1, 4, 64, device="cuda")

    def refused(call, status=1):
        with pytest.raises(q4.Q4Error) as e:
            call()
        assert e.value.status == status

    refused(lambda: q4.KVCache(0, 2, 64, 32))
    refused(lambda: q4.KVCache(2, 2, 96, 32))
    refused(lambda: q4.KVCache(2, 2, 64, 48))
    refused(lambda: q4.KVCache(2, 2, 64, 32, data=torch.zeros(10, dtype=torch.uint8, device="cuda")))
    refused(lambda: q4.KVCache(2, 2, 64, 32, data=cache.data.cpu()))
    refused(lambda: q4.kv_write(cache, x.double(), x, table, lens))
    refused(lambda: q4.kv_write(cache, x.cpu(), x, table, lens))
    refused(lambda: q4.kv_write(cache, x, x[:, :, :1], table, lens))
    refused(lambda: q4.kv_write(cache, x, torch.zeros(1, 2, 2, 64, device="cuda"), table, lens))
    refused(lambda: q4.kv_write(cache, x.transpose(2, 3).contiguous().transpose(2, 3), x, table, lens))
    refused(lambda: q4.kv_write(cache, x, x, table.long(), lens))
    refused(lambda: q4.kv_write(cache, x, x, table, lens.cpu()))
    refused(lambda: q4.kv_write(cache, x, x, table, lens, lens.long()))
    refused(lambda: q4.kv_read(cache, table, lens, 2, out=(x, x)))
    refused(lambda: q4.kv_read(cache, table, lens, 2, dtype=torch.float64))
    wide = x.expand(1, 3, 2, 64)
    refused(lambda: q4.kv_read(cache, table, lens, 3, out=(wide, wide)))  # rows that overlap
    refused(lambda: q4.kv_attention(cache, torch.zeros(1, 17, 4, 64, device="cuda"), table, lens), 4)
    refused(lambda: q4.kv_attention(cache, torch.zeros(1, 1, 3, 64, device="cuda"), table, lens))
    refused(lambda: q4.kv_attention(cache, q, table, lens, scale=0.0))
    refused(lambda: q4.kv_attention(cache, q, table, lens, scale=float("nan")))
    refused(lambda: q4.kv_attention(cache, q, table, lens, softcap=-1.0))
    refused(lambda: q4.kv_attention(cache, q, table, lens, window=-1))
    refused(lambda: q4.kv_attention(cache, q, table, lens, alibi=torch.zeros(3, device="cuda")))
    refused(lambda: q4.kv_attention(cache, q, table, lens, lse=torch.zeros(1, 4, 1, device="cuda")))
    refused(lambda: q4.kv_attention(cache, q, table, lens, out=torch.zeros(1, 1, 4, 128, device="cuda")))
    refused(lambda: q4.kv_attention(cache, q, table, lens, ws=torch.zeros(16, dtype=torch.uint8, device="cuda")), 3)
    with pytest.raises(q4.Q4Error):
        q4.kv_attention_workspace_bytes(96)


def test_the_memory_of_a_cache_is_not_exchanged():
    cache = q4.KVCache(1, 1, 64, 32)
    with pytest.raises(AttributeError):
        cache.data = torch.zeros_like(cache.data)
    assert cache.data.data_ptr() == cache.c.data and cache.data.numel() == cache.nbytes
