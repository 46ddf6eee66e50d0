"""Prompt and drafted-tree attention where a row's sums leave the ordinary
range: cache scales that are not finite, scores that step up late in the
context, values that are not finite in long contexts.  Compared with the plain
64-bit form; none of it may run into the kernels' time limit."""
import copy
import math

import pytest
import torch

from attn_reference import Batch, attend, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_323_b200 import build as pkv_build

    pkv_build.build()
    from paged_kv_cache_323_b200 import pagedkv

    return pagedkv


def finish(pk, code=0):
    torch.cuda.synchronize()
    assert pk.get_device_error() == code


@pytest.mark.parametrize("tree", [False, True], ids=["prefill", "tree"])
@pytest.mark.parametrize("which,value", [("ks", math.nan), ("vs", math.nan), ("vs", math.inf), ("ks", math.inf)])
@pytest.mark.parametrize("head_dim", [128, 64])
def test_cache_scales_that_are_not_finite(pk, tree, which, value, head_dim):
    """A scale of one kv head that is not finite: its rows are what the formula gives, the others keep their bits."""
    b = Batch([(40, 300), (150, 150), (5, 3000)], dtype="fp8", heads=8, kv_heads=2, head_dim=head_dim, seed=60)
    b.poison()
    good = b.call(pk, tree).clone()
    getattr(b, which)[1] = value
    got = b.call(pk, tree)
    finish(pk)
    assert torch.equal(got[:, :4], good[:, :4])
    if (which, value) == ("ks", math.inf):
        return  # rows of one score of -inf are zeros here, NaN in the 64-bit form
    ref, bound = attend(b, tree)
    assert not bool(torch.isfinite(ref[:, 4:]).any())
    close(got, ref, bound)


def steps_up(b, at, unit=50.0):
    """Scores near 0 for the first keys, `unit` more (powers of two of a weight) from each position of `at` on."""
    b.q[..., 0] = 128.0
    for s, (_, c) in enumerate(b.seqs):
        pos = torch.arange(c, device="cuda")
        blk = b.tables[s].long()[pos // b.bs]
        level = sum((pos >= (a if a >= 0 else c + a)).float() for a in at) * unit
        x = level / (128.0 * b.scale * 1.4426950408889634)
        for h in range(b.G):
            v = x / (b.ks[h] if b.ks is not None else 1.0)
            cache = b.kc.view(torch.uint8) if b.dtype == "fp8" else b.kc
            v = v.to(b.kc.dtype)
            cache[blk, h, pos % b.bs, 0] = v.view(torch.uint8) if b.dtype == "fp8" else v


@pytest.mark.parametrize("tree", [False, True], ids=["prefill", "tree"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("unit", [45.0, 120.0, 300.0])
@pytest.mark.parametrize("seqs,heads,kv_heads,head_dim", [
    ([(300, 1500), (257, 257)], 2, 1, 128),     # two tiles of rows at once
    ([(40, 900), (9, 1200), (1, 400)], 4, 2, 128),  # even and odd steps of one tile
    ([(5, 9000), (64, 3000)], 8, 2, 64),        # items in many and in few parts
    ([(70, 700)] * 40, 4, 4, 64),               # whole items, several a CTA
])
def test_scores_that_step_up(pk, tree, dtype, unit, seqs, heads, kv_heads, head_dim):
    """The reference of a row's weights, taken from its first keys, has to follow: by less and by more than
    a weight can hold, in the first and in the second half of a step, in steps with and without masks."""
    if dtype == "fp8" and unit == 300.0:
        pytest.skip("past what e4m3 times its scale can hold")
    for at in ((150,), (330,), (40, 650), (-30,), (100, -70)):
        if dtype == "fp8" and unit == 120.0 and len(at) > 1:
            continue
        b = Batch(seqs, dtype=dtype, heads=heads, kv_heads=kv_heads, head_dim=head_dim, seed=61)
        b.poison()
        steps_up(b, at, unit)
        got = b.call(pk, tree)
        finish(pk)
        ref, bound = attend(b, tree)
        close(got, ref, bound, str(at))


SHAPES = [([(300, 700), (9, 60), (33, 33)], 4, 2), ([(5, 9000), (64, 3000)], 8, 2), ([(70, 700)] * 40, 4, 4),
          ([(3, 200)] * 9, 8, 1)]


@pytest.mark.parametrize("tree", [False, True], ids=["prefill", "tree"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("head_dim,block_size", [(128, 16), (64, 8), (128, 32)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_values_that_are_not_finite(pk, tree, dtype, head_dim, block_size, shape):
    """One value of v that is not finite, in a committed or a new token of some sequences: it reaches its dim of the
    rows that see it; whole items, items in few and in many parts."""
    seqs, heads, kv_heads = SHAPES[shape]
    b = Batch(seqs, dtype=dtype, heads=heads, kv_heads=kv_heads, head_dim=head_dim, block_size=block_size, seed=63)
    b.poison()
    for s, (n, c) in enumerate(seqs):
        if s % 3 == 2:
            continue
        pos = c - 1 - n // 2 if s % 3 else c // 3
        blk, at, g = int(b.tables[s, pos // block_size]), pos % block_size, s % kv_heads
        if dtype == "fp8":
            b.vc.view(torch.uint8)[blk, g, at, 11] = 0x7F
        else:
            b.vc[blk, g, at, 11] = -math.inf if s % 2 else math.nan
    got = b.call(pk, tree)
    finish(pk)
    ref, bound = attend(b, tree)
    assert bool(torch.isfinite(ref).any()) and not bool(torch.isfinite(ref).all())
    close(got, ref, bound)


@pytest.mark.parametrize("tree", [False, True], ids=["prefill", "tree"])
@pytest.mark.parametrize("head_dim", [128, 64])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_values_near_the_largest(pk, tree, head_dim, shape):
    """Values of v whose sums with weights relative to the first keys pass what fp32 holds, the results do not."""
    seqs, heads, kv_heads = SHAPES[shape]
    b = Batch(seqs, dtype="bf16", heads=heads, kv_heads=kv_heads, head_dim=head_dim, seed=64)
    b.vc *= 2.0 ** 110
    b.poison()
    steps_up(b, (60,), 32.0)
    got = b.call(pk, tree)
    finish(pk)
    ref, bound = attend(b, tree)
    assert bool(torch.isfinite(ref).all())
    close(got, ref, bound)


@pytest.mark.parametrize("tree", [False, True], ids=["prefill", "tree"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("log2_q", [17, 20, 34, 100])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_past_their_own_rounding(pk, tree, dtype, log2_q, sign):
    """Scores so large that fp32 rounds them by more than a weight's whole range: each row is the value of the
    largest score that it sees.  Keys differ by 1/128 (fp8: by 2^-9 of the scale and more) and q is at least 2^17
    (2^27), so scores of a row by at least 2^17 2^-7 log2(e) / sqrt(128) = 130 (2^27 2^-9 2^-5 0.127 = 1000)
    powers of two."""
    seqs = [(5, 100), (100, 100), (40, 90), (3, 3000), (1, 1)]
    b = Batch(seqs, dtype=dtype, heads=4, kv_heads=2, seed=65)
    b.scale *= sign
    b.poison()
    b.q.zero_()
    b.q[..., 0] = sign * 2.0 ** (log2_q + (10 if dtype == "fp8" else 0))
    raw = b.kc.view(torch.uint8) if dtype == "fp8" else b.kc
    want = torch.empty(b.T, b.H, b.D, dtype=torch.float64, device="cuda")
    gen = torch.Generator().manual_seed(65)
    for s, (n, c) in enumerate(seqs):
        order = (torch.arange(c) * 37) % 101 if c < 101 else torch.randint(0, 100, (c,), generator=gen)
        if c >= 101:
            order[c - n - 700] = 101
        order = order.cuda()
        pos = torch.arange(c, device="cuda")
        blk, at = b.tables[s].long()[pos // b.bs], pos % b.bs
        if dtype == "fp8":  # codes rise with their bits
            raw[blk, :, at] = 0
            raw[blk, :, at, 0] = (order + 8).to(torch.uint8)[:, None]
        else:
            raw[blk, :, at] = 0
            raw[blk, :, at, 0] = (1 + order / 128.0).to(raw.dtype)[:, None]
        for i in range(n):
            seen = torch.arange(c, device="cuda") <= c - n + i
            if tree:
                seen = torch.arange(c, device="cuda") < c - n
                j = i
                while j >= 0:
                    seen[c - n + j] = True
                    j = int(b.parents[b.start_host[s] + j])
            k = int(torch.where(seen, order, -1).argmax())
            v = b.vc[blk[k], :, at[k]].double()
            if dtype == "fp8":
                v = v * b.vs.double()[:, None]
            want[b.start_host[s] + i] = v.repeat_interleave(2, 0)
    got = b.call(pk, tree).double()
    finish(pk)
    assert bool(((got - want).abs() <= 2.0 ** -7 * want.abs()).all())


@pytest.mark.parametrize("tree", [False, True], ids=["prefill", "tree"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_value_of_a_weight_that_vanishes(pk, tree, dtype):
    """A NaN value of a key that rows see with a weight below fp32's range reaches them, in steps with masks too."""
    b = Batch([(40, 60), (3, 300), (9, 9)], dtype=dtype, heads=4, kv_heads=2, seed=66)
    b.poison()
    steps_up(b, (5,), 300.0)
    for s in range(3):
        b.vc[int(b.tables[s, 0]), :, 0, 7] = math.nan
    got = b.call(pk, tree)
    finish(pk)
    ref, bound = attend(b, tree)
    close(got, ref, bound)
    assert bool(torch.isnan(got[:43, :, 7]).all())


@pytest.mark.parametrize("tree", [False, True], ids=["prefill", "tree"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("head_dim", [128, 64])
@pytest.mark.parametrize("seqs", [[(300, 900)], [(40, 900), (3, 500)], [(64, 3000)]])
def test_large_values_of_vanishing_weights(pk, tree, dtype, head_dim, seqs):
    """Values of 2^110 under weights of 2^-300: nothing of them is in the result."""
    b = Batch(seqs, dtype=dtype, heads=4, kv_heads=2, head_dim=head_dim, seed=67)
    b.poison()
    steps_up(b, (64,), -300.0)
    for s, (n, c) in enumerate(seqs):
        pos = torch.arange(128, 384, device="cuda")
        b.vc[b.tables[s].long()[pos // b.bs], :, pos % b.bs, 3] = 2.0 ** 110
    got = b.call(pk, tree)
    finish(pk)
    ref, bound = attend(b, tree)
    assert float(ref.abs().max()) < 10
    close(got, ref, bound)


def long_items(dtype, keys, heads=296, rows=256, head_dim=64):
    """One sequence whose every (tile, head) is a whole item of `keys` keys, two for a CTA: while the rows of
    one are finished its other warps wait with the next.  The table goes round 64 blocks."""
    bs = 32
    b = Batch([(rows, 64 * bs)], dtype=dtype, heads=heads, kv_heads=heads, head_dim=head_dim, block_size=bs, seed=62)
    b.tables = b.tables[:, :64].repeat(1, keys // (64 * bs)).contiguous()
    b.seqs = [(rows, keys)]
    b.ctx[0] = keys
    return b


def some_heads(b, n=2):
    """The same batch with its first heads only."""
    c = copy.copy(b)
    c.H = c.G = n
    c.q, c.kc, c.vc = b.q[:, :n], b.kc[:, :n].contiguous(), b.vc[:, :n].contiguous()
    c.ks, c.vs = (b.ks[:n], b.vs[:n]) if b.ks is not None else (None, None)
    return c


def odd_value(b):
    blk = int(b.tables[0, 0])
    if b.dtype == "fp8":
        b.vc.view(torch.uint8)[blk, :, 3, 5] = 0x7F
    else:
        b.vc[blk, :, 3, 5] = math.inf


def one_late_step(b):
    """A block of its own at the end of the table but 4 blocks, whose keys' scores are some 2^120 times the others'."""
    used = set(b.tables[0].tolist())
    spare = next(i for i in range(b.kc.shape[0]) if i not in used)
    b.tables[0, -12] = spare
    b.q[..., 0] = 128.0
    x = 120.0 / (128.0 * b.scale * 1.4426950408889634)
    raw = b.kc.view(torch.uint8) if b.dtype == "fp8" else b.kc
    raw[..., 0] = 0
    v = torch.full((b.G,), x, device="cuda") / (b.ks if b.ks is not None else 1.0)
    v = v.to(b.kc.dtype)
    raw[spare, :, :, 0] = (v.view(torch.uint8) if b.dtype == "fp8" else v)[:, None]


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("change", [odd_value, one_late_step])
@pytest.mark.parametrize("keys,limit_us", [(32768, 20000), (131072, 0)])
def test_long_items_stay_within_the_time_limit(pk, dtype, change, keys, limit_us):
    """Rows that need more work than others hold up the rest of their CTA, whose waits must not run out for it:
    under the default limit, and under one that is far above any other wait of the call."""
    b = long_items(dtype, keys)
    change(b)
    old = pk.set_wait_limit_us(limit_us)
    try:
        got = b.call(pk)
        finish(pk)
    finally:
        pk.set_wait_limit_us(old)
    c = some_heads(b)
    ref, bound = attend(c)
    close(got[:, :2], ref, bound)
    if change is odd_value:
        assert not bool(torch.isfinite(got[..., 5]).any())
        assert bool(torch.isfinite(got[..., :5]).all()) and bool(torch.isfinite(got[..., 6:]).all())
    else:
        assert bool(torch.isfinite(got).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_many_long_items_stay_within_the_time_limit(pk, dtype):
    """Six items of 4M keys for each CTA: some 50 ms each, under a limit of 10 ms for a wait.  The table goes
    round 64 blocks, so the result is that of 2048 keys; sums of 32768 steps are within 2^-9 of them each."""
    b = long_items(dtype, 1 << 22, heads=148 * 6, rows=1)
    old = pk.set_wait_limit_us(10000)
    try:
        got = b.call(pk)
        finish(pk)
    finally:
        pk.set_wait_limit_us(old)
    c = some_heads(b, 8)
    c.tables, c.seqs = b.tables[:, :64], [(1, 2048)]
    ref, bound = attend(c)
    vmax = float((c.vc.float() * (c.vs.view(1, -1, 1, 1) if c.vs is not None else 1.0)).abs().max())
    close(got[:, :8], ref, bound + 2.0 ** -8 * vmax)
    assert bool(torch.isfinite(got).all())
