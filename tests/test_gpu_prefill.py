"""Prompt attention and drafted-tree attention over the paged cache against
the plain 64-bit form, at the sizes, masks and faults where they can go wrong."""
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


def check(pk, b, tree, code=0, lost=(), **kw):
    b.poison()
    got = b.call(pk, tree, **kw)
    torch.cuda.synchronize()
    assert pk.get_device_error() == code
    ref, bound = attend(b, tree, lost)
    n = b.start_host[-1]
    close(got[:n], ref[:n], bound[:n])
    assert bool((got[n:] == -77.0).all()), "rows behind the last sequence changed"


# (queries, context): none, one, a whole short prompt, odd sizes around the
# tiles (128 and 256 rows) and the 128-key steps, chunks behind a prefix
RAGGED = [(0, 5), (1, 1), (3, 3), (1, 130), (17, 128), (127, 127), (129, 129), (0, 0), (64, 700), (257, 300)]


@pytest.mark.parametrize("tree", [False, True], ids=["prefill", "tree"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("heads,kv_heads", [(3, 3), (4, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("head_dim,block_size", [(128, 16), (64, 16), (128, 8), (64, 32), (128, 32), (64, 8)])
def test_ragged(pk, tree, dtype, heads, kv_heads, head_dim, block_size):
    b = Batch(RAGGED, dtype=dtype, heads=heads, kv_heads=kv_heads, head_dim=head_dim, block_size=block_size,
              seed=heads + head_dim + block_size, pad_rows=5)
    check(pk, b, tree)


@pytest.mark.parametrize("tree", [False, True], ids=["prefill", "tree"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("seqs,heads,kv_heads,head_dim", [
    ([(5, 9000)], 8, 1, 128),               # one sequence over all SMs: split along its keys
    ([(33, 4099), (1, 3001)], 8, 1, 128),   # two tiles, one of them of one token
    ([(200, 2500), (31, 7000)], 4, 4, 64),
    ([(1, 20000)], 1, 1, 128),
    ([(2, 40)] * 300, 2, 2, 64),            # more sequences than CTAs or threads have turns
    ([(1100, 1100)], 2, 1, 128),
])
def test_split_and_long(pk, tree, dtype, seqs, heads, kv_heads, head_dim):
    b = Batch(seqs, dtype=dtype, heads=heads, kv_heads=kv_heads, head_dim=head_dim, seed=len(seqs))
    check(pk, b, tree)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
def test_many_sequences_few_with_work(pk, dtype):
    """1500 sequences, most without queries, some without context."""
    seqs = [(0, i % 40) if i % 7 else (i % 5, 5 + i % 90) for i in range(1500)]
    check(pk, Batch(seqs, dtype=dtype, heads=4, kv_heads=2, head_dim=64, seed=3), False)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("tree", [False, True], ids=["prefill", "tree"])
def test_strided_q(pk, dtype, tree):
    b = Batch([(40, 90), (130, 130)], dtype=dtype, heads=8, kv_heads=2, head_dim=64)
    wide = torch.full((b.T, 8 + 4, 64), math.nan, device="cuda", dtype=b.q.dtype)
    wide[:, :8] = b.q
    b.q = wide[:, :8]
    check(pk, b, tree)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
def test_out_at_any_16_bytes(pk, dtype):
    """out, q and the pools at addresses that are multiples of 16 bytes and no more."""
    b = Batch([(70, 300), (130, 130), (5, 5000)], dtype=dtype, heads=8, kv_heads=2, seed=7)
    b.poison()
    ref, bound = attend(b)

    def moved(t):
        n = 16 // t.element_size()
        raw = torch.empty(t.numel() + 64, dtype=t.dtype, device="cuda")
        at = next(i for i in range(n, 64, n) if (raw.data_ptr() + i * t.element_size()) % 32)
        to = raw[at:at + t.numel()].view(t.shape)
        to.view(torch.uint8).copy_(t.contiguous().view(torch.uint8))
        return to

    b.out, b.q, b.kc, b.vc = moved(b.out), moved(b.q), moved(b.kc), moved(b.vc)
    got = b.call(pk)
    torch.cuda.synchronize()
    assert pk.get_device_error() == 0
    close(got, ref, bound)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_scales(pk, dtype, scale):
    b = Batch([(40, 300), (130, 130)], dtype=dtype, heads=8, kv_heads=2, seed=5)
    b.scale = scale
    check(pk, b, False)


@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_negative_cache_scales(pk, sign):
    """A kv head whose k scale is negative, under either sign of the softmax scale."""
    b = Batch([(40, 300), (130, 130)], dtype="fp8", heads=8, kv_heads=2, seed=5)
    b.ks[1] *= -1
    b.vs[0] *= -1
    b.scale *= sign
    check(pk, b, False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_scores(pk, dtype):
    """Scores of several hundred: the maximum moves, old sums are scaled down."""
    b = Batch([(70, 1500), (5, 2000)], dtype=dtype, heads=2, kv_heads=1, seed=6, amp=40.0)
    b.kc[:] = (b.kc.float() * torch.linspace(0.1, 1, b.bs, device="cuda").view(1, 1, -1, 1)).to(b.kc.dtype)
    b.scale = 0.1
    # a weight's relative error grows with its score's: within the bound's |q||k| term
    check(pk, b, False)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("tree", [False, True], ids=["prefill", "tree"])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_non_finite_where_masked(pk, dtype, tree, where, value):
    """A NaN or infinity in one new token reaches the rows that see it, and no other."""
    if dtype == "fp8" and value == math.inf:
        pytest.skip("e4m3 has no infinity")
    b = Batch([(150, 400), (9, 60)], dtype=dtype, heads=4, kv_heads=2, head_dim=128, seed=8)
    b.poison()
    pos = 400 - 150 + 77
    blk = int(b.tables[0, pos // b.bs])
    cache = b.kc if where == "k" else b.vc
    if dtype == "fp8":
        cache.view(torch.uint8)[blk, :, pos % b.bs, 3] = 0x7F
    else:
        cache[blk, :, pos % b.bs, 3] = value
    got = b.call(pk, tree)
    torch.cuda.synchronize()
    assert pk.get_device_error() == 0
    ref, bound = attend(b, tree)
    if where == "k":  # an infinite score may leave any non-finite or one-hot row: only rows that do not see it
        rows = torch.isfinite(ref).all(-1).all(-1)
        assert int(rows.sum()) >= 70
        close(got[rows], ref[rows], bound[rows])
    else:
        close(got, ref, bound)
        assert bool(torch.isfinite(ref).all(-1).all(-1)[:77].all())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("tree", [False, True], ids=["prefill", "tree"])
def test_bad_blocks_are_left_out(pk, dtype, tree):
    b = Batch([(20, 500), (3, 40), (2, 20)], dtype=dtype, heads=4, kv_heads=2, seed=9)
    b.poison()
    b.tables[0, 3] = b.kc.shape[0]
    b.tables[0, 17] = -1
    b.tables[2, :] = 1 << 30  # no block left: zero rows
    got = b.call(pk, tree)
    torch.cuda.synchronize()
    assert pk.get_device_error() == pk.PKV_ERR_DEVICE_BOUNDS
    ref, bound = attend(b, tree)
    close(got, ref, bound)
    assert bool((got[23:25] == 0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
def test_sequences_that_cannot_be(pk, dtype):
    """Fewer tokens than queries, a context past the table, a negative one: zeros, the others as ever."""
    b = Batch([(20, 100), (9, 20), (4, 64), (150, 160)], dtype=dtype, heads=4, kv_heads=2, seed=10, max_blocks=12)
    b.poison()
    ref, bound = attend(b)
    b.ctx[1] = 8
    b.ctx[2] = 12 * 16 + 1
    got = b.call(pk)
    torch.cuda.synchronize()
    assert pk.get_device_error() == pk.PKV_ERR_DEVICE_BOUNDS
    ref[20:33] = 0
    close(got, ref, bound)
    b.ctx[1] = -5
    b.ctx[2] = 64
    ref, bound = attend(b)
    ref[20:29] = 0
    got = b.call(pk)
    assert pk.get_device_error() == pk.PKV_ERR_DEVICE_BOUNDS
    close(got, ref, bound)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_outside_q(pk, dtype):
    """Rows that q does not have, or that run backwards, are not touched."""
    b = Batch([(20, 100), (9, 20), (30, 64)], dtype=dtype, heads=4, kv_heads=2, seed=11)
    ref, bound = attend(b)
    b.start[3] = b.T + 1
    got = b.call(pk)
    torch.cuda.synchronize()
    assert pk.get_device_error() == pk.PKV_ERR_DEVICE_BOUNDS
    close(got[:29], ref[:29], bound[:29])
    assert bool((got[29:] == -77.0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bad_parents_are_reported(pk, dtype):
    b = Batch([(20, 100), (40, 90)], dtype=dtype, heads=4, kv_heads=2, seed=12)
    good = b.call(pk, True).clone()
    assert pk.get_device_error() == 0
    for value in (7, 30, -2, 2 ** 31 - 1):
        b.parents[7] = value
        got = b.call(pk, True)
        torch.cuda.synchronize()
        assert pk.get_device_error() == pk.PKV_ERR_DEVICE_BOUNDS
        assert torch.equal(got[20:], good[20:])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
def test_chain_is_prefill_and_one_token_is_decode(pk, dtype):
    b = Batch([(1, 700), (1, 3), (1, 1999)], dtype=dtype, heads=8, kv_heads=2, seed=13)
    ref, bound = attend(b)
    tree = b.call(pk, True).clone()
    flat = b.call(pk, False)
    assert torch.equal(tree, flat)
    out = torch.empty_like(flat)
    if dtype == "fp8":
        pk.paged_attention_decode_fp8(out, b.q, b.kc, b.vc, b.ks, b.vs, b.tables, b.ctx, b.scale)
    else:
        pk.paged_attention_decode_ex(out, b.q, b.kc, b.vc, b.tables, b.ctx, b.scale)
    close(flat, ref, bound)
    close(out, ref, 4 * bound)  # the decode's own steps (weights of 8 bits, split in two terms)
    b = Batch([(37, 600), (150, 150)], dtype=dtype, heads=8, kv_heads=2, seed=14)
    for s, (n, _) in enumerate(b.seqs):
        b.parents[b.start_host[s]:b.start_host[s] + n] = torch.arange(-1, n - 1, device="cuda", dtype=torch.int32)
    assert torch.equal(b.call(pk, True).clone(), b.call(pk, False))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
def test_blocks_shared_between_sequences(pk, dtype):
    """Sequences whose tables name the same prefix blocks, one of them twice."""
    b = Batch([(33, 400), (40, 420), (7, 300)], dtype=dtype, heads=4, kv_heads=2, seed=23)
    b.tables[1, :20] = b.tables[0, :20]
    b.tables[2, :10] = b.tables[0, 0]
    ref, bound = attend(b, True)
    close(b.call(pk, True), ref, bound)
    assert pk.get_device_error() == 0


def test_every_row_of_nan(pk):
    """A cache of NaN: every row, whole and split items, comes out NaN."""
    b = Batch([(40, 90), (5, 3000)], dtype="bf16", heads=2, kv_heads=1, seed=24)
    b.vc[:] = math.nan
    assert bool(torch.isnan(b.call(pk)).all())
    b = Batch([(40, 90), (5, 3000)], dtype="bf16", heads=2, kv_heads=1, seed=24)
    b.kc[:] = math.nan
    assert bool(torch.isnan(b.call(pk)).all())
    assert pk.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
def test_same_bits_every_time_and_after_other_shapes(pk, dtype):
    """One workspace through calls of several shapes; no result depends on what ran before."""
    big = Batch([(5, 9000), (64, 3000)], dtype=dtype, heads=8, kv_heads=1, seed=15)
    small = Batch([(3, 20)] * 9, dtype=dtype, heads=4, kv_heads=4, head_dim=64, seed=16)
    first = big.call(pk, True).clone()
    for _ in range(4):
        small.call(pk)
        assert torch.equal(big.call(pk, True), first)


def test_one_workspace_for_every_kernel(pk):
    """Split calls over fp32, bf16 and fp8 caches in turn through one workspace."""
    calls = [Batch([(5, 9000), (64, 3000)], dtype=d, heads=h, kv_heads=1, head_dim=n, seed=25)
             for d, h, n in (("f32", 8, 128), ("bf16", 4, 128), ("f32", 1, 64), ("fp8", 8, 64))]
    need = max(pk.paged_attention_prefill_workspace_size(b.T, b.H, b.G, b.D, pk._dtype_code(b.kc)) for b in calls)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    refs = [attend(b) for b in calls]
    for _ in range(3):
        for b, (ref, bound) in zip(calls, refs):
            b.out.fill_(-77.0)
            close(b.call(pk, workspace=ws), ref, bound, b.dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
def test_streams_and_graphs(pk, dtype):
    """Two streams at once with workspaces of their own, and a captured call replayed on new data."""
    a = Batch([(64, 3000), (9, 500)], dtype=dtype, heads=8, kv_heads=2, seed=17)
    b = Batch([(5, 8000)], dtype=dtype, heads=8, kv_heads=1, seed=18)
    wa, wb = a.call(pk).clone(), b.call(pk, True).clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.out.zero_(), b.out.zero_()
        torch.cuda.synchronize()
        a.call(pk, stream=s1)
        b.call(pk, True, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(a.out, wa) and torch.equal(b.out, wb)
    need = pk.paged_attention_prefill_workspace_size(a.T, 8, 2, 128, pk._dtype_code(a.kc))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.call(pk, workspace=ws)
    with pytest.raises(ValueError):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            a.call(pk)
    for seed in (20, 21):
        a.q.copy_(torch.randn(a.q.shape, generator=torch.Generator().manual_seed(seed)).to(a.q.dtype))
        g.replay()
        got = a.out.clone()
        assert torch.equal(a.call(pk), got)
        ref, bound = attend(a)
        close(got, ref, bound)
    assert pk.get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_past_32_bits(pk, dtype):
    """Blocks whose elements lie past 2^31 and 2^32 of the pool."""
    free = torch.cuda.mem_get_info()[0]
    bs, G, D = 16, 8, 128
    blocks = (1 << 32) // (bs * G * D) + 64
    if free < 2.2 * blocks * bs * G * D * (4 if dtype == "f32" else 2):
        pytest.skip("not enough device memory")
    b = Batch([(9, 100), (70, 150)], dtype=dtype, heads=16, kv_heads=G, seed=19)
    ref, bound = attend(b)
    far = torch.arange(blocks - 60, blocks - 60 + b.kc.shape[0], device="cuda")
    far[1::2] -= blocks // 2
    for name in ("kc", "vc"):
        pool = torch.empty((blocks, G, bs, D), dtype=b.q.dtype, device="cuda")
        pool[far] = getattr(b, name)
        setattr(b, name, pool)
    b.tables = torch.where(b.tables >= 0, far[b.tables.clamp(min=0).long()].to(torch.int32), b.tables)
    got = b.call(pk)
    torch.cuda.synchronize()
    assert pk.get_device_error() == 0
    close(got, ref, bound)
