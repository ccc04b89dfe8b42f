"""Attention over the 4-bit key/value cache against the same in 64 bits."""
import math

import pytest
import torch

from kv_util import Filled, check_attention
from quantized_decode_q4_b200 import q4

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def queries(s, t, heads, dim, dtype, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(s, t, heads, dim, generator=g) * std).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("dim,heads,group,page", [(64, 3, 3, 32), (128, 2, 4, 64), (256, 2, 2, 32), (128, 1, 1, 96)])
def test_lengths(dim, heads, group, page, dtype):
    """From no token to several pages: ends inside and at the borders of records and pages."""
    lens = [0, 1, 2, 31, 32, 33, 63, 64, 65, 95, 96, 97, 128, 200, 257, 300]
    f = Filled(lens, heads, dim, page, seed=dim + heads)
    check_attention(f, queries(len(lens), 1, heads * group, dim, dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 7, 8, 9, 16, 33])
def test_groups(group, dtype):
    f = Filled([77, 300], 2, 64, 64, seed=group)
    check_attention(f, queries(2, 1, 2 * group, 64, dtype, seed=group))


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("tokens,group,dim", [(2, 4, 128), (3, 3, 64), (5, 1, 256), (8, 4, 128), (16, 2, 64), (16, 7, 128)])
def test_several_tokens_are_causal(tokens, group, dim, dtype):
    """Sequences shorter than the call's tokens leave the first rows without a position."""
    f = Filled([tokens + 40, 1, tokens - 1, tokens, 0, 333], 2, dim, 32, seed=tokens)
    check_attention(f, queries(6, tokens, 2 * group, dim, dtype, seed=tokens))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_new_lens(dtype):
    """Padded batches: rows behind a sequence's new tokens, counts outside 0 .. tokens."""
    f = Filled([50, 50, 50, 3, 100, 0], 2, 128, 32, seed=5)
    new = torch.tensor([4, 1, 0, 4, 9, -3], dtype=torch.int32).cuda()
    check_attention(f, queries(6, 4, 8, 128, dtype), new_lens=new)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("window,tokens", [(1, 1), (1, 5), (7, 3), (32, 1), (33, 2), (100, 16), (5000, 2)])
def test_windows(window, tokens, dtype):
    f = Filled([1, 30, 64, 257, 600], 2, 64, 32, seed=window)
    check_attention(f, queries(5, tokens, 6, 64, dtype, seed=window), window=window)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_softcap_alibi_scale(dim, dtype):
    f = Filled([5, 64, 333], 2, dim, 64, seed=dim, k_std=2.0)
    q = queries(3, 2, 8, dim, dtype, seed=3, std=2.0)
    slopes = (2.0 ** -torch.arange(1, 9).float()).cuda()
    check_attention(f, q, softcap=30.0)
    check_attention(f, q, alibi=slopes)
    check_attention(f, q, softcap=5.0, alibi=slopes, window=100, scale=0.3)
    check_attention(f, q, scale=1e-3)
    check_attention(f, q, scale=2.0)
    check_attention(f, q, alibi=-slopes)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_magnitudes(dtype):
    """Large and tiny values, large scores (one key takes everything), keys far apart in size."""
    for k_std, v_std, q_std in ((1.0, 1e-2, 1.0), (1.0, 3e3, 1.0), (8.0, 1.0, 8.0), (1e-3, 1.0, 1.0), (100.0, 1.0, 1e-3)):
        f = Filled([400, 37], 2, 128, 64, seed=7, k_std=k_std, v_std=v_std)
        out, _ = check_attention(f, queries(2, 1, 8, 128, dtype, seed=8, std=q_std), out_dtype=F32)
        assert bool(out.isfinite().all())


def test_growing_values():
    """Values and scores that grow along the sequence, so that every running maximum rises."""
    f = Filled([700], 1, 64, 32, seed=9, stale_nan=False)
    k, v = (x.clone() for x in f.read(700))
    ramp = torch.arange(700, device="cuda").view(1, -1, 1, 1) / 70
    for grow in (lambda k, v: (k * ramp, v), (lambda k, v: (k, v * 2 ** ramp)), (lambda k, v: (k * ramp, v * 2 ** ramp)),
                 (lambda k, v: (k.abs() * ramp, v * 2 ** -ramp))):
        q4.kv_write(f.cache, *grow(k, v), f.table, f.lens)
        for dtype in (F32, BF16):
            check_attention(f, queries(1, 1, 4, 64, dtype, seed=10, std=3.0), out_dtype=F32)
            check_attention(f, queries(1, 1, 4, 64, dtype, seed=11).abs(), out_dtype=F32)


def test_queries_of_zero_and_outliers():
    f = Filled([100], 2, 128, 32, seed=12)
    for dtype in (F32, F16, BF16):
        q = queries(1, 2, 8, 128, dtype, seed=13)
        q[0, 0, 0] = 0
        q[0, 0, 1] *= 1e-4
        q[0, 0, 2, 5] = 300.0
        q[0, 1, 3] = 0
        q[0, 1, 3, 127] = 1.0
        check_attention(f, q, out_dtype=F32)


def test_what_is_not_finite_stays_in_its_row():
    f = Filled([100, 60], 2, 64, 32, seed=14)
    for dtype in (F32, BF16):
        q = queries(2, 2, 8, 64, dtype, seed=15)
        want, want_lse = check_attention(f, q)
        q[0, 1, 3, 7], q[1, 0, 6, 0] = float("nan"), float("inf")
        lse = torch.empty(2, 2, 8, device="cuda")
        out = q4.kv_attention(f.cache, q, f.table, f.lens, lse=lse)
        hit = torch.zeros(2, 2, 8, dtype=torch.bool, device="cuda")
        hit[0, 1, 3] = hit[1, 0, 6] = True
        assert bool(out[hit].isnan().all()) and bool(lse[hit].isnan().all())
        assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])
    # a key that is not finite is seen by the rows behind it and by nobody before it
    k, v = q4.kv_read(f.cache, f.table, f.lens, 100)
    k[0, 99, 1, 3] = float("nan")
    q4.kv_write(f.cache, k, v, f.table, torch.full_like(f.lens, 100))
    out = q4.kv_attention(f.cache, queries(2, 2, 8, 64, F32, seed=15), f.table, f.lens)
    assert bool(out[0, 1, 4:].isnan().all()) and not bool(out[0, 0].isnan().any()) and not bool(out[0, 1, :4].isnan().any())


def test_bad_pages_are_masked_and_recorded():
    f = Filled([100, 100], 1, 64, 32, seed=16)
    q = queries(2, 1, 2, 64, F32, seed=17)
    ws = q4.workspace(q4.kv_attention_workspace_bytes(64))
    good = q4.kv_attention(f.cache, q, f.table, f.lens, ws=ws)
    assert q4.workspace_status(ws) == 0
    for bad in (-1, f.cache.pages, 2 ** 31 - 1):
        table = f.table.clone()
        table[1, 1] = bad
        out = q4.kv_attention(f.cache, q, table, f.lens, ws=ws)
        assert q4.workspace_status(ws) == 1
        q4.workspace_init(ws)
        assert torch.equal(out[0], good[0])
        # without positions 32 .. 63
        k, v = (x.double()[1, :100, 0] for x in f.read(100))
        keep = torch.cat([torch.arange(32), torch.arange(64, 100)]).cuda()
        w = torch.softmax(q[1, 0].double() @ k[keep].T / 8, -1)
        assert torch.allclose(out[1, 0].double(), w @ v[keep], rtol=0, atol=1e-4)
    # all of a sequence's pages: nothing is seen
    table[1] = -1
    out = q4.kv_attention(f.cache, q, table, f.lens, ws=ws)
    assert not bool(out[1].any()) and torch.equal(out[0], good[0])


def test_lengths_behind_the_table_count_as_its_reach():
    f = Filled([96], 1, 64, 32, seed=18)
    q = queries(1, 2, 2, 64, F32, seed=19)
    a = q4.kv_attention(f.cache, q, f.table, f.lens)
    b = q4.kv_attention(f.cache, q, f.table, torch.tensor([2 ** 31 - 1], dtype=torch.int32).cuda())
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides_and_unaligned_rows(dtype):
    f = Filled([45, 130], 2, 128, 64, seed=20)
    q = queries(2, 8, 3, 128, dtype, seed=21).transpose(1, 2)  # [2, 3 tokens, 8 heads, dim], heads outside
    want, _ = check_attention(f, q.contiguous())
    assert torch.equal(q4.kv_attention(f.cache, q, f.table, f.lens), want)
    flat = torch.zeros(q.numel() + 1, dtype=dtype, device="cuda")
    off = flat[1:].view(q.shape)
    off.copy_(q)
    room = torch.full((q.numel() + 2,), 7.0, dtype=dtype, device="cuda")
    out = room[1:-1].view(q.shape)
    q4.kv_attention(f.cache, off, f.table, f.lens, out=out)
    assert torch.equal(out, want) and room[0] == 7.0 and room[-1] == 7.0
    wide = torch.zeros(2, 3, 8, 2, 128, dtype=dtype, device="cuda")
    q4.kv_attention(f.cache, q, f.table, f.lens, out=wide[:, :, :, 1])
    assert torch.equal(wide[:, :, :, 1], want) and not bool(wide[:, :, :, 0].any())
    one = q[:1, :1]
    got = q4.kv_attention(f.cache, one.expand(2, 2, 8, 128), f.table, f.lens)
    assert torch.equal(got, q4.kv_attention(f.cache, one.expand(2, 2, 8, 128).contiguous(), f.table, f.lens))


@pytest.mark.parametrize("q_dtype,out_dtype", [(BF16, F32), (F32, BF16), (F16, F32), (BF16, F16)])
def test_result_of_another_type(q_dtype, out_dtype):
    f = Filled([45, 130], 2, 128, 64, seed=22)
    check_attention(f, queries(2, 1, 8, 128, q_dtype, seed=23), out_dtype=out_dtype)


def test_long_sequence():
    f = Filled([70001], 1, 64, 128, seed=24)
    for dtype in (F32, BF16):
        check_attention(f, queries(1, 1, 4, 64, dtype, seed=25))


def test_many_short_sequences():
    lens = [(7 * i) % 90 for i in range(1500)]
    f = Filled(lens, 2, 64, 32, seed=26)
    for dtype in (F32, BF16):
        check_attention(f, queries(1500, 1, 4, 64, dtype, seed=27))


def test_one_long_among_short():
    f = Filled([3, 9000, 12, 0, 40], 4, 128, 64, seed=28)
    for dtype in (F32, BF16):
        check_attention(f, queries(5, 1, 16, 128, dtype, seed=29))
        check_attention(f, queries(5, 4, 16, 128, dtype, seed=29))


def test_pages_behind_the_sequence_may_be_anything():
    f = Filled([40, 10], 1, 64, 32, seed=30, tail=3)
    q = queries(2, 1, 2, 64, F32, seed=31)
    want, _ = check_attention(f, q)
    table = f.table.clone()
    table[0, 2:], table[1, 1:] = -5, 1 << 30
    ws = q4.workspace(q4.kv_attention_workspace_bytes(64))
    assert torch.equal(q4.kv_attention(f.cache, q, table, f.lens, ws=ws), want) and q4.workspace_status(ws) == 0


def test_same_bits_every_time_and_with_a_shared_workspace():
    """Repeated calls, other calls of the library in the same workspace between them."""
    f = Filled([5000, 300, 2222], 2, 128, 64, seed=32)
    w = q4.pack(torch.randn(3, 28672, device="cuda"))  # its K is split: tickets and partial sums
    x = torch.randn(28672, device="cuda")
    ws = q4.workspace(max(q4.kv_attention_workspace_bytes(128), q4.workspace_bytes(3, 28672)))
    y0 = q4.gemv(w, x)
    for dtype in (F32, BF16):
        q = queries(3, 2, 8, 128, dtype, seed=33)
        want, _ = check_attention(f, q)
        for _ in range(20):
            y = q4.gemv(w, x, ws=ws)
            out = q4.kv_attention(f.cache, q, f.table, f.lens, ws=ws)
            assert torch.equal(out, want) and torch.equal(y, y0)
    assert q4.workspace_status(ws) == 0


def test_other_streams():
    """Each stream with its own workspace; results and allocations belong to the stream."""
    f = Filled([3000, 1000], 2, 128, 64, seed=34)
    qs = [queries(2, 1, 8, 128, F32, seed=35 + i) for i in range(4)]
    want = [q4.kv_attention(f.cache, q, f.table, f.lens) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], [], [], []]
    for _ in range(10):
        for i, (q, s) in enumerate(zip(qs, streams)):
            got[i].append(q4.kv_attention(f.cache, q, f.table, f.lens, stream=s))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(a, x) for x in b)


def test_decode_steps_in_a_captured_graph():
    """What a decode step does: project, write the token, attend, project; captured once and
    replayed with new inputs and lengths in place, against eager calls."""
    d, heads, kv, dim, page, steps = 512, 8, 2, 64, 32, 40
    g = torch.Generator(device="cuda").manual_seed(36)
    wq, wk, wv, wo = (q4.pack(torch.randn(n, k, generator=g, device="cuda") * k ** -0.5)
                      for n, k in ((heads * dim, d), (kv * dim, d), (kv * dim, d), (d, heads * dim)))
    batch = 3
    xs = torch.randn(steps, batch, d, generator=g, device="cuda")
    table = torch.randperm(batch * 4, generator=torch.Generator().manual_seed(37)).view(batch, 4).to(torch.int32).cuda()
    start = torch.tensor([0, 17, 60], dtype=torch.int32).cuda()

    def program(captured):
        cache = q4.KVCache(batch * 4, kv, dim, page)
        k, v = (torch.randn(batch, 60, kv, dim, generator=torch.Generator(device="cuda").manual_seed(38 + i), device="cuda") for i in (0, 1))
        q4.kv_write(cache, k, v, table, start, start)
        x, lens = torch.empty(batch, d, device="cuda"), start.clone()
        ws = q4.workspace(max(q4.kv_attention_workspace_bytes(dim), *(q4.workspace_bytes(m.n, m.k, batch) for m in (wq, wk, wo))))

        def step():
            lens.add_(1)
            q, k, v = (q4.gemv_batched(m, x, ws=ws).view(batch, 1, -1, dim) for m in (wq, wk, wv))
            q4.kv_write(cache, k, v, table, lens)
            a = q4.kv_attention(cache, q, table, lens, ws=ws)
            return q4.gemv_batched(wo, a.view(batch, -1), ws=ws)

        outs = []
        if captured:
            x.copy_(xs[0])
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                y = step()
            torch.cuda.synchronize()
        for i in range(steps):
            x.copy_(xs[i])
            if captured:
                graph.replay()
                outs.append(y.clone())
            else:
                outs.append(step())
        torch.cuda.synchronize()
        assert q4.workspace_status(ws) == 0
        return torch.stack(outs), cache.data

    (a, ca), (b, cb) = program(False), program(True)
    assert torch.equal(a, b) and torch.equal(ca, cb) and bool(a.isfinite().all())


def test_capture_without_a_workspace():
    """A call that makes its own workspace may be captured; two such graphs run at once."""
    f = Filled([900, 31], 2, 64, 32, seed=40)
    graphs, outs, want = [], [], []
    for i in range(2):
        q = queries(2, 1, 8, 64, F32, seed=41 + i)
        want.append(q4.kv_attention(f.cache, q, f.table, f.lens))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(q4.kv_attention(f.cache, q, f.table, f.lens))
        graphs.append((graph, q, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, _, s in graphs:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("dim,dtype", [(64, F32), (128, BF16), (256, F16)])
def test_waits_run_out_and_the_device_stays_usable(dim, dtype):
    """Barriers that expect more than comes: the kernel gives up, records it, and ends; the
    same workspace, cleared, serves a normal call."""
    import ctypes
    f = Filled([700, 0, 40], 2, dim, 32, seed=50)
    q = queries(3, 1, 4, dim, dtype, seed=51)
    ws = q4.workspace(q4.kv_attention_workspace_bytes(dim))
    out = torch.empty_like(q)
    r = ctypes.byref
    seqs = q4._kv_seqs(f.cache, f.table, f.lens, None)
    rows = [q4._kv_rows(f.cache, t, tuple(q.shape), "q") for t in (q, out)]
    call = q4.lib().q4_debug_kv_attention_stall
    call.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32] + [ctypes.c_void_p] * 4 + [ctypes.c_size_t, ctypes.c_void_p]
    call.restype = ctypes.c_int
    scores = q4.q4_kv_scores(0.1, 0.0, 0, None)
    assert call(r(f.cache.c), r(seqs), 1, 4, r(rows[0]), r(scores), r(rows[1]), ws.data_ptr(), ws.numel(), None) == 0
    torch.cuda.synchronize()
    assert q4.workspace_status(ws) == 6
    q4.workspace_init(ws)
    check_attention(f, q, ws=ws)
    assert q4.workspace_status(ws) == 0


@pytest.mark.parametrize("count,dim,tokens", [(32, 128, 1), (33, 64, 3), (200, 128, 1), (513, 256, 2)])
def test_batches_of_every_kind_of_count(count, dim, tokens):
    """Up to 32 sequences each warp finds its work by itself, above that the CTA does, a
    thread a sequence or several; every third holds nothing."""
    g = torch.Generator().manual_seed(count)
    lens = [0 if i % 3 == 1 else int(v) for i, v in enumerate(torch.randint(0, 200, (count,), generator=g))]
    f = Filled(lens, 2, dim, 32, seed=count)
    for dtype in (F32, BF16):
        check_attention(f, queries(count, tokens, 6, dim, dtype, seed=count))


@pytest.mark.parametrize("window,visible", [(0, True), (2**31 - 1, True), (2**31 - 32, True), (2**31 - 33, False)])
def test_the_longest_sequence(window, visible):
    """2^31 - 32 tokens, nearly all of them one page's: token 0 outweighs the others wherever the
    window shows it."""
    cache = q4.KVCache(2, 1, 64, 32)
    one = torch.ones(1, 32, 1, 64, device="cuda")
    q4.kv_write(cache, 0 * one, one, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                torch.tensor([32], dtype=torch.int32, device="cuda"))
    q4.kv_write(cache, one[:, :1], 2 * one[:, :1], torch.ones(1, 1, dtype=torch.int32, device="cuda"),
                torch.tensor([1], dtype=torch.int32, device="cuda"))
    table = torch.zeros(1, 2**26 - 1, dtype=torch.int32, device="cuda")
    table[0, 0] = 1
    lens = torch.tensor([2**31 - 32], dtype=torch.int32, device="cuda")
    lse = torch.empty(1, 1, 1, device="cuda")
    out = q4.kv_attention(cache, one[:, :1] * (100 / 64), table, lens, scale=1.0, window=window, lse=lse)
    # hidden: scores of 0, values of 1 but for 31 of 0. Joins add 160 partial sums at most, of
    # the outputs and of the weights, each to 2^-24: 2e-5
    assert (out - (2.0 if visible else 1.0)).abs().max().item() < 2 * 2e-5
    assert abs(lse.item() - (100.0 if visible else math.log(2**31 - 33))) < 2e-5 + 100 * 2**-23
