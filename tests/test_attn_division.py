"""The division of the multi-query attention's work among CTAs, on the CPU,
walked by the kernels' own code: every key of every item is taken once, parts
follow one another, and the places of partial results and counters are
distinct, over random launches and contexts up to the longest accepted."""
import ctypes
import random

import numpy as np
import pytest

from test_abi import pk  # noqa: F401

FIELDS = ("cta", "seq", "row", "ntok", "pos", "first", "kv0", "kv1", "g", "part", "nparts", "keys", "per_key", "owner0",
          "owner", "slot")
LONGEST = 2 ** 31 - 1 - 1024


def items(pk, rows, seqs, kv_heads, group_log2, grid=None, max_context=LONGEST):  # noqa: F811
    fn = pk.lib.pkv_internal_attn_items
    fn.restype = ctypes.c_longlong
    fn.argtypes = [ctypes.c_int] + [ctypes.c_void_p] * 2 + [ctypes.c_int] * 6 + [ctypes.c_void_p, ctypes.c_longlong]
    start = np.concatenate([[0], np.cumsum([n for n, _ in seqs])]).astype(np.int32)
    ctx = np.array([c for _, c in seqs], dtype=np.int32)
    grid = grid or (148 if rows == 256 else 296)
    cap = 1 << 17
    out = np.zeros((cap, len(FIELDS)), dtype=np.int64)
    n = fn(rows, start.ctypes.data, ctx.ctypes.data, len(seqs), int(start[-1]), kv_heads, group_log2, max_context, grid,
           out.ctypes.data, cap)
    assert n <= cap
    return start, grid, [dict(zip(FIELDS, r.tolist())) for r in out[:n]]


def check(pk, rows, seqs, kv_heads, group_log2, **kw):  # noqa: F811
    start, grid, got = items(pk, rows, seqs, kv_heads, group_log2, **kw)
    tt = rows >> group_log2
    want = {}
    for s, (n, c) in enumerate(seqs):
        for t in range(-(-n // tt)):
            for g in range(kv_heads):
                ok = n <= c <= kw.get("max_context", LONGEST)
                want[(s, int(start[s]) + t * tt, g)] = (min(tt, n - t * tt), c - n + min((t + 1) * tt, n) if ok else 0)
    seen, slots, counters = {}, set(), {}
    for it in got:
        key = (it["seq"], it["row"], it["g"])
        ntok, keys = want[key]
        assert it["ntok"] == ntok and it["keys"] == keys
        seen.setdefault(key, []).append(it)
    assert set(seen) == set(want)
    for key, parts in seen.items():
        keys = want[key][1]
        assert [p["part"] for p in parts] == list(range(len(parts)))
        assert all(p["nparts"] == len(parts) for p in parts)
        at = 0
        for p in parts:
            assert p["kv0"] == at and (p["kv1"] > at or keys == 0)
            at = p["kv1"]
            if p["kv1"] != keys:
                assert p["kv1"] % (64 if rows < 256 else 128) == 0
        assert at == keys
        if len(parts) > 1:
            assert counters.setdefault(parts[0]["owner0"], key) == key
            for p in parts:
                assert p["owner"] == p["cta"] and 0 <= p["owner0"] < grid and p["owner0"] == parts[0]["cta"]
                assert 0 <= p["slot"] < 2 * grid and p["slot"] not in slots
                slots.add(p["slot"])


def draw(rng, rows, group_log2):
    seqs, left = [], 4000
    for _ in range(rng.choice([1, 1, 2, 5, 40, 300])):
        n = rng.choice([0, 1, rng.randint(1, 9), rng.randint(1, 3 * rows >> group_log2), rng.randint(1, 700)])
        n = min(n, left)
        left -= n
        c = rng.choice([n, n + rng.randint(0, 100), n + rng.randint(0, 5000), n + rng.randint(0, 10 ** 5),
                        rng.randint(n, LONGEST), max(0, n - 1)])
        seqs.append((n, c))
    return seqs


@pytest.mark.parametrize("rows", [256, 64, 16])
def test_random_launches(pk, rows):  # noqa: F811
    rng = random.Random(rows)
    for _ in range(400):
        gl = rng.randint(0, 3)
        kw = {"max_context": 4096} if rng.random() < 0.2 else {}
        check(pk, rows, draw(rng, rows, gl), rng.choice([1, 1, 2, 3, 8]), gl, **kw)


@pytest.mark.parametrize("rows", [256, 64, 16])
@pytest.mark.parametrize("group_log2", [0, 3])
@pytest.mark.parametrize("n", [1, 7, 16, 17, 300])
@pytest.mark.parametrize("ctx", [715_827_883, 715_900_000, 2 ** 30 + 1, 1_200_000_000, LONGEST])
def test_longest_contexts(pk, rows, group_log2, n, ctx):  # noqa: F811
    """Contexts whose work (keys times the work per key) passes 31 bits."""
    check(pk, rows, [(n, ctx)], 1, group_log2)
    check(pk, rows, [(1, 300), (n, ctx), (3, 3)], 2, group_log2)
