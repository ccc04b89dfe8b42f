"""The 4-bit key/value cache on the CPU: sizes, refusals before any CUDA call, and the
record layout."""
import ctypes
import random

import numpy as np
import pytest

from quantized_decode_q4_b200 import q4

INVALID, MISALIGNED, WORKSPACE, UNSUPPORTED = 1, 2, 3, 4


def cache(data=256, pages=4, heads=2, dim=64, page=32):
    return q4.q4_kv_cache(data, pages, heads, dim, page)


def seqs(table=256, stride=4, pages=4, count=2, lens=256, new=None):
    return q4.q4_kv_seqs(table, stride, pages, count, lens, new)


def rows(data=256, type=0, s=1024, t=512, h=64):
    return q4.q4_rows(data, type, s, t, h)


def ref(x):
    return None if x is None else ctypes.byref(x)


def test_cache_bytes():
    f = q4.lib().q4_kv_cache_bytes
    assert f(3, 5, 64, 32) == 3 * 5 * 36 * 64
    assert f(10, 8, 128, 128) == 10 * 8 * 4 * 4608
    assert f(2 ** 31 - 1, 65535, 256, 32) == (2 ** 31 - 1) * 65535 * 9216
    for bad in ((0, 1, 64, 32), (-1, 1, 64, 32), (2 ** 31, 1, 64, 32), (1, 0, 64, 32), (1, 65536, 64, 32), (1, 1, 96, 32),
                (1, 1, 0, 32), (1, 1, 64, 0), (1, 1, 64, 48), (1, 1, 64, 65568), (2 ** 31 - 1, 65535, 256, 65536)):
        assert f(*bad) == 0, bad


@pytest.mark.parametrize("name", ["q4_kv_write", "q4_kv_read"])
def test_move_refusals(name):
    L = q4.lib()

    def call(c=cache(), s=seqs(), tokens=2, k=rows(), v=rows()):
        args = (ref(c), ref(s), *([None] if name == "q4_kv_read" else []), tokens, ref(k), ref(v), None)
        return getattr(L, name)(*args)

    for c in (None, cache(data=None), cache(pages=0), cache(heads=0), cache(page=31), cache(page=48)):
        assert call(c=c) == INVALID
    assert call(c=cache(dim=80)) == UNSUPPORTED and call(c=cache(data=192)) == MISALIGNED
    for s in (None, seqs(table=None), seqs(lens=None), seqs(count=-1), seqs(pages=0), seqs(stride=-1), seqs(pages=1 << 26)):
        assert call(s=s) == INVALID
    for s in (seqs(table=258), seqs(lens=257), seqs(new=254 + 1)):
        assert call(s=s) == MISALIGNED
    assert call(tokens=-1) == INVALID
    for bad, status in ((None, INVALID), (rows(data=None), INVALID), (rows(type=3), UNSUPPORTED), (rows(type=-1), UNSUPPORTED),
                        (rows(s=-1), INVALID), (rows(t=-64), INVALID), (rows(h=1 << 47), INVALID), (rows(data=258), MISALIGNED),
                        (rows(data=257, type=2), MISALIGNED)):
        assert call(k=bad) == status and call(v=bad) == status
    # inputs may broadcast, outputs may not overlap
    wide = rows(t=0)
    if name == "q4_kv_read":
        assert call(k=wide) == INVALID and call(v=rows(h=32)) == INVALID
    assert call(s=seqs(count=1 << 20), tokens=1 << 20, k=rows(s=1 << 30, t=1024)) == INVALID
    assert call(tokens=0) == 0 and call(s=seqs(count=0)) == 0


def test_attention_refusals():
    L = q4.lib()
    need = q4.kv_attention_workspace_bytes(64)
    assert need >= 256 and L.q4_kv_attention_workspace_bytes(96) == 0

    def call(c=cache(), s=seqs(), tokens=2, heads=4, q=rows(t=256, s=512), scores=(0.125, 0.0, 0, None), out=rows(t=256, s=512), lse=None,
             ws=256, ws_bytes=need):
        sc = None if scores is None else q4.q4_kv_scores(*scores)
        return L.q4_kv_attention(ref(c), ref(s), tokens, heads, ref(q), ref(sc), ref(out), lse, ws, ws_bytes, None)

    assert call(tokens=0) == 0 and call(s=seqs(count=0)) == 0
    assert call(c=None) == INVALID and call(s=None) == INVALID and call(c=cache(dim=32)) == UNSUPPORTED
    assert call(tokens=-1) == UNSUPPORTED and call(tokens=17) == UNSUPPORTED
    for h in (0, -2, 3, 65536):
        assert call(heads=h) == INVALID
    inf, nan = float("inf"), float("nan")
    for sc in (None, (0.0, 0, 0, None), (-1.0, 0, 0, None), (nan, 0, 0, None), (inf, 0, 0, None), (1, nan, 0, None), (1, -1, 0, None),
               (1, inf, 0, None), (1, 0, -1, None)):
        assert call(scores=sc) == INVALID, sc
    # more query heads a key/value head, or more tiles, than the kernel counts
    assert call(heads=2 * 4097) == INVALID
    assert call(s=seqs(pages=(1 << 26) - 1, count=17)) == INVALID and call(s=seqs(pages=1 << 20, count=1 << 10), tokens=16) == INVALID
    assert call(scores=(1, 0, 0, 258)) == MISALIGNED and call(lse=258) == MISALIGNED
    assert call(q=None) == INVALID and call(out=None) == INVALID and call(q=rows(type=7)) == UNSUPPORTED
    assert call(out=rows(h=0)) == INVALID and call(out=rows(t=0)) == INVALID
    assert call(ws=None) == WORKSPACE and call(ws_bytes=need - 1) == WORKSPACE and call(ws=320) == MISALIGNED


def test_python_sizes():
    for bad in ((1 << 40, 1, 64, 32), (1, 1 << 32, 64, 32), (1, 1, 1 << 35, 32), (0, 1, 64, 32), (1, 1, 64, (1 << 32) + 32)):
        with pytest.raises(q4.Q4Error):
            q4.kv_cache_bytes(*bad)
    assert q4.kv_cache_bytes(2, 3, 128, 64) == 2 * 3 * 2 * 4608


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_record_layout(dim):
    f = q4.lib().q4_debug_check_kv_layout
    f.argtypes, f.restype = [ctypes.c_int], ctypes.c_int
    assert f(dim) == 0
    assert f(96) != 0


def test_attention_plans_replay_on_host():
    """Every tile is covered once and every cut unit is joined once: one sequence and many,
    empty ones, windows, lengths behind the table, fewer tiles than warps and far more."""
    f = q4.lib().q4_debug_check_kv_plan
    i32p = ctypes.POINTER(ctypes.c_int32)
    f.argtypes, f.restype = [i32p, i32p] + [ctypes.c_int] * 7, ctypes.c_int
    rng = np.random.default_rng(11)

    def check(lens, new, tokens, window, reach, units, warps, grid):
        n = len(lens)
        a = (ctypes.c_int32 * n)(*lens)
        b = None if new is None else (ctypes.c_int32 * n)(*new)
        r = f(a, b, n, tokens, window, reach, units, warps, grid)
        assert r == 0, (r, lens[:8], tokens, window, reach, units, warps, grid)

    for warps in (8, 12, 16):
        for grid in (148, 132, 1, 7, 252):
            check([0], None, 1, 0, 32, 1, warps, grid)
            check([777], None, 1, 0, 800, 3, warps, grid)
            check([8192], None, 1, 0, 8192, 8, warps, grid)
            check([2 ** 31 - 1], None, 16, 0, 2 ** 31 - 32, 2, warps, grid)
            check([2 ** 31 - 1, -5, 9], [3, 9, -1], 4, 4096, 2 ** 31 - 32, 9, warps, grid)
    for _ in range(400):
        n = int(rng.integers(1, 200)) if rng.random() < 0.7 else int(rng.integers(500, 2000))
        top = int(2 ** rng.uniform(0, 16))
        lens = [int(v) for v in rng.integers(-2, top + 1, n)]
        tokens = int(rng.integers(1, 17))
        new = None if rng.random() < 0.5 else [int(v) for v in rng.integers(-1, 20, n)]
        window = 0 if rng.random() < 0.5 else int(2 ** rng.uniform(0, 14))
        reach = -(-max(1, top if rng.random() < 0.8 else top // 2) // 32) * 32
        check(lens, new, tokens, window, reach, int(rng.integers(1, 40)), int(rng.choice([8, 12, 16])), int(rng.choice([148, 3, 252])))


def test_packed_arguments_are_the_structure():
    """q4_kv_call takes what the binding packs: the calls' own refusals come back."""
    import struct

    L = q4.lib()

    class Args(ctypes.Structure):
        _fields_ = [("cache", q4.q4_kv_cache), ("seqs", q4.q4_kv_seqs), ("a", q4.q4_rows), ("b", q4.q4_rows), ("scores", q4.q4_kv_scores),
                    ("extra", ctypes.c_void_p), ("ws", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t), ("tokens", ctypes.c_int32),
                    ("q_heads", ctypes.c_int32)]

    head = struct.pack("@Pqiii4x", 1, 2, 3, 4, 5)
    rest = q4._ARGS.pack(6, 7, 8, 9, 10, 11, 12, 2, 13, 14, 15, 16, 1, 17, 18, 19, 0.5, 0.25, 20, 21, 22, 23, 24, 25, 26)
    assert len(head) + len(rest) == ctypes.sizeof(Args)
    a = Args.from_buffer_copy(head + rest)
    assert (a.cache.data, a.cache.pages, a.cache.heads, a.cache.dim, a.cache.page_size) == (1, 2, 3, 4, 5)
    assert (a.seqs.table, a.seqs.table_stride, a.seqs.table_pages, a.seqs.count, a.seqs.lens, a.seqs.new_lens) == (6, 7, 8, 9, 10, 11)
    assert [(r.data, r.type, r.seq_stride, r.token_stride, r.head_stride) for r in (a.a, a.b)] == [(12, 2, 13, 14, 15), (16, 1, 17, 18, 19)]
    assert (a.scores.scale, a.scores.softcap, a.scores.window, a.scores.alibi) == (0.5, 0.25, 20, 21)
    assert (a.extra, a.ws, a.ws_bytes, a.tokens, a.q_heads) == (22, 23, 24, 25, 26)

    def call(which, c=(256, 4, 2, 64, 32), tokens=2, ws=256, null=False):
        need = q4.kv_attention_workspace_bytes(64)
        b = struct.pack("@Pqiii4x", *c) + q4._ARGS.pack(256, 4, 4, 2, 256, 0, 256, 0, 512, 256, 64, 256, 0, 512, 256, 64, 0.125, 0.0, 0, 0,
                                                        0, ws, need, tokens, 4)
        return L.q4_kv_call(which, None if null else b, None)

    for which in (0, 1, 2):
        assert call(which, null=True) == INVALID and call(which, tokens=0) == 0
        assert call(which, c=(256, 0, 2, 64, 32)) == INVALID and call(which, c=(192, 4, 2, 64, 32)) == MISALIGNED
    assert call(2, tokens=17) == UNSUPPORTED and call(2, ws=0) == WORKSPACE and call(3) == INVALID and call(-1) == INVALID


def test_quotients():
    f = q4.lib().q4_debug_kv_quotient
    top = 2**31 - 1
    g = random.Random(3)
    divisors = [1, 2, 3, 5, 7, 8, 32, 96, 127, 128, 65535, 65536, 2**30 - 1, 2**30, 2**30 + 1, top - 1, top]
    for d in divisors + [int(2**g.uniform(0, 31)) for _ in range(200)]:
        near = [m * d + e for m in (1, 2, top // d // 2, top // d) for e in (-1, 0, 1)]
        for n in [0, 1, top - 1, top] + near + [g.randrange(2**31) for _ in range(20)]:
            if 0 <= n <= top:
                assert f(n, d) == n // d, (n, d)
