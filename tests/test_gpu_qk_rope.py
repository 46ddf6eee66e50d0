"""Per-head norm, rotation and append in one pass against the plain 64-bit
form, and a whole layer step (rotation and append, prompt attention, drafted
tree, decode) as an engine makes it."""
import math

import pytest
import torch

import attn_reference as ar

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_323_b200 import build as pkv_build

    pkv_build.build()
    from paged_kv_cache_323_b200 import pagedkv

    return pagedkv


class Step:
    def __init__(self, T, H, G, D, dtype, *, rotary=None, sections=None, norm="qk", interleaved=False, bs=16,
                 far=1 << 20, seed=0, pad=0, sliced=True, amp=1.7):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        act = ar.ACT[dtype]
        self.T, self.H, self.G, self.D, self.dtype, self.bs = T, H, G, D, dtype, bs
        qkv = (torch.randn(T, H + 2 * G, D, generator=gen, device="cuda") * amp).to(act)
        self.q, self.k, self.v = qkv[:, :H], qkv[:, H:H + G], qkv[:, H + G:]
        if not sliced:
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        self.q_out = torch.zeros(T, H, D, device="cuda", dtype=act)
        blocks = -(-T // bs) + 2
        self.kc, self.vc = ((torch.randn(blocks, G, bs, D, generator=gen, device="cuda")).to(ar.POOL[dtype])
                            for _ in range(2))
        self.slots = torch.randperm(blocks * bs, generator=gen, device="cuda")[:T]
        self.slots[T - pad:] = -1
        rotary = 2 * sum(sections) if sections else rotary or D
        self.sections = sections or [rotary // 2]
        pos = torch.randint(-far // 8, far, (len(self.sections), T), generator=gen, device="cuda").to(torch.int32)
        pos[:, 0] = 2 ** 31 - 1
        self.pos = pos
        i = torch.arange(0, rotary, 2, device="cuda", dtype=torch.float64)
        self.freq = (10000.0 ** (-i / rotary)).to(torch.float32)
        w = [(1 + 0.3 * torch.randn(D, generator=gen, device="cuda")).to(act) for _ in range(2)]
        self.qw, self.kw = w[0] if "q" in norm else None, w[1] if "k" in norm else None
        self.interleaved = interleaved
        self.ks, self.vs = ar.scales(G) if dtype == "fp8" else (None, None)

    def call(self, pk, q_out=None):
        fp8 = (self.ks, self.vs) if self.dtype == "fp8" else ()
        f = pk.qk_norm_rope_append_fp8 if fp8 else pk.qk_norm_rope_append
        f(self.q_out if q_out is None else q_out, self.q, self.k, self.v, self.kc, self.vc, *fp8, self.slots,
          self.pos, self.freq, q_weight=self.qw, k_weight=self.kw, eps=1e-5, sections=self.sections,
          interleaved=self.interleaved)

    def reference(self):
        def form(x, w):
            y = ar.rope(x, self.pos, self.freq, self.sections, w, 1e-5, self.interleaved)
            # a pair's values: both turn by an angle within 8 u (its reduction to [-pi, pi] and
            # rounding: 4 u, sine and cosine: 2 u each); the sum of squares of D values and the
            # root: within (D / 2 + 4) u relative; products and sums: 4 u
            n = x.double() if w is None else x.double() / (x.double().pow(2).mean(-1, keepdim=True)
                                                           + 1e-5).sqrt() * w.double()
            half = len(self.freq)
            mate = n.clone()
            if self.interleaved:
                mate[..., 0:2 * half:2], mate[..., 1:2 * half:2] = n[..., 1:2 * half:2], n[..., 0:2 * half:2]
            else:
                mate[..., :half], mate[..., half:2 * half] = n[..., half:2 * half], n[..., :half]
            return y, (n.abs() + mate.abs()) * (self.D / 2 + 16) * U
        return form(self.q, self.qw), form(self.k, self.kw)


def step_bound(y, err, dtype):
    return err + (2.0 ** -8 if dtype != "f32" else U) * (y.abs() + err) + 1e-30


CASES = [
    dict(T=1, H=1, G=1, D=64), dict(T=5, H=8, G=2, D=128), dict(T=64, H=32, G=8, D=128),
    dict(T=333, H=6, G=3, D=64, rotary=32, norm=""), dict(T=70, H=4, G=4, D=128, interleaved=True),
    dict(T=70, H=5, G=1, D=64, interleaved=True, rotary=16, norm="k"),
    dict(T=41, H=16, G=2, D=128, sections=[16, 24, 24]), dict(T=41, H=3, G=3, D=128, sections=[8, 0, 4, 20], norm="q"),
    dict(T=2000, H=2, G=1, D=64, sections=[3, 13], sliced=False, pad=7), dict(T=3, H=40, G=40, D=128, bs=8),
    dict(T=9, H=1, G=7, D=128, pad=9), dict(T=1000, H=64, G=8, D=128, bs=32, pad=3),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_rows_and_slots(pk, dtype, case):
    s = Step(dtype=dtype, seed=case, **CASES[case])
    kc0, vc0 = s.kc.clone(), s.vc.clone()
    s.call(pk)
    torch.cuda.synchronize()
    assert pk.get_device_error() == 0
    (q, eq), (k, ek) = s.reference()
    ar.close(s.q_out, q, step_bound(q, eq, s.dtype), "q")
    kept = s.slots >= 0
    at = s.slots[kept]
    raw = torch.uint8 if dtype == "fp8" else s.kc.dtype
    got_k = s.kc.view(raw)[at // s.bs, :, at % s.bs]
    got_v = s.vc.view(raw)[at // s.bs, :, at % s.bs]
    if dtype == "fp8":
        sc = s.ks.double().view(1, -1, 1)
        y, e = (k[kept] / sc).clamp(-448, 448), ek[kept] / sc
        # half a step of e4m3, subnormal ones (2^-9 apart) too
        ar.close(got_k.view(torch.float8_e4m3fn).double(), y, e + 2.0 ** -4 * (y.abs() + e) + 2.0 ** -10, "k")
        codes = (s.v[kept].float() / s.vs.view(1, -1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(got_v, codes.view(torch.uint8))
    else:
        ar.close(got_k, k[kept], step_bound(k[kept], ek[kept], dtype), "k")
        assert torch.equal(got_v, s.v[kept])
    # every other slot as it was
    for now, old in ((s.kc, kc0), (s.vc, vc0)):
        now, old = now.view(raw).clone(), old.view(raw).clone()
        now[at // s.bs, :, at % s.bs] = 0
        old[at // s.bs, :, at % s.bs] = 0
        assert torch.equal(now, old)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
def test_without_norm_and_turn_it_is_the_append(pk, dtype):
    s = Step(37, 4, 2, 128, dtype, norm="", seed=30)
    s.pos.zero_()
    other = [s.kc.clone(), s.vc.clone()]
    s.call(pk)
    k, v = s.k.contiguous(), s.v.contiguous()
    if dtype == "fp8":
        pk.kv_cache_append_fp8(*other, s.ks, s.vs, k, v, s.slots)
    else:
        pk.kv_cache_append(*other, k, v, s.slots)
    assert torch.equal(s.q_out, s.q)
    raw = torch.uint8 if dtype == "fp8" else s.kc.dtype
    assert torch.equal(s.kc.view(raw), other[0].view(raw)) and torch.equal(s.vc.view(raw), other[1].view(raw))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place_and_extremes(pk, dtype):
    s = Step(50, 8, 2, 64, dtype, seed=31)
    s.call(pk)
    q = s.q.clone()
    s.q = q
    s.call(pk, q_out=q)
    assert torch.equal(q, s.q_out)
    s = Step(6, 2, 1, 64, dtype, seed=32)
    s.q[0] = 0  # a row of zeros: eps keeps it from 0 / 0
    s.q[1] = 1e18  # squares past bf16's and near fp32's range
    s.q[2, 0, 5] = math.nan
    s.q[3, 1, 7] = math.inf
    s.call(pk)
    assert bool((s.q_out[0] == 0).all()) and bool(torch.isfinite(s.q_out[1]).all())
    assert bool(torch.isnan(s.q_out[2, 0]).all()) and bool(torch.isfinite(s.q_out[2, 1]).all())
    assert bool(torch.isfinite(s.q_out[3, 0]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
def test_slot_past_the_pool(pk, dtype):
    s = Step(20, 4, 2, 128, dtype, seed=33)
    s.slots[4] = s.kc.shape[0] * s.bs
    s.slots[9] = 1 << 40
    s.slots[11] = -(1 << 40)
    s.call(pk)
    torch.cuda.synchronize()
    assert pk.get_device_error() == pk.PKV_ERR_DEVICE_BOUNDS
    (q, eq), _ = s.reference()
    ar.close(s.q_out, q, step_bound(q, eq, dtype), "q")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("captured", [False, True])
def test_a_layer_step(pk, dtype, captured):
    """Prompts in two chunks, then a drafted tree, then a decode step, each
    preceded by its rotation and append, on one stream without a wait."""
    H, G, D, bs = 8, 2, 128, 16
    prompts, cut, drafts = [70, 9, 300], [40, 0, 129], [5, 1, 12]
    act = ar.ACT[dtype]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(40)
    bm = pk.BlockManager(200, bs)
    ids = [bm.add_sequence() for _ in prompts]
    kc, vc = (torch.zeros(200, G, bs, D, device="cuda", dtype=ar.POOL[dtype]) for _ in range(2))
    sc = ar.scales(G) if dtype == "fp8" else ()
    freq = (10000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)).to(torch.float32)
    w = [(1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(act) for _ in range(2)]
    need = pk.paged_attention_prefill_workspace_size(400, H, G, D, pk._dtype_code(kc))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    plan, done = [], [0] * len(ids)
    for new in ([c for c in cut], [p - c for p, c in zip(prompts, cut)], drafts, [1, 1, 1]):
        slots, pos, start = [], [], [0]
        for i, s in enumerate(ids):
            if new[i]:
                got, pairs = bm.append(s, new[i])
                assert len(pairs) == 0
                slots += got.tolist()
            pos += range(done[i], done[i] + new[i])
            done[i] += new[i]
            start.append(start[-1] + new[i])
        bt, lens = bm.tables(ids, 24)
        T = start[-1]
        parents = torch.tensor([x for n in new for x in [(j - 1) // 2 if j else -1 for j in range(n)]],
                               dtype=torch.int32, device="cuda")
        qkv = (torch.randn(T, H + 2 * G, D, generator=gen, device="cuda")).to(act)
        plan.append(dict(qkv=qkv, slots=torch.tensor(slots, device="cuda"), start=start,
                         pos=torch.tensor(pos, dtype=torch.int32, device="cuda"), parents=parents,
                         qs=torch.tensor(start, dtype=torch.int32, device="cuda"), bt=torch.from_numpy(bt).cuda(),
                         lens=torch.from_numpy(lens).cuda(), new=new, done=list(done),
                         qr=torch.empty(T, H, D, device="cuda", dtype=act),
                         out=torch.empty(T, H, D, device="cuda", dtype=act)))
    f8 = "_fp8" if sc else ""

    def steps():
        for i, s in enumerate(plan):
            q, k, v = s["qkv"][:, :H], s["qkv"][:, H:H + G], s["qkv"][:, H + G:]
            getattr(pk, "qk_norm_rope_append" + f8)(s["qr"], q, k, v, kc, vc, *sc, s["slots"], s["pos"], freq,
                                                    q_weight=w[0], k_weight=w[1])
            if i < 2:
                getattr(pk, "paged_attention_prefill" + f8)(s["out"], s["qr"], kc, vc, *sc, s["bt"], s["lens"],
                                                            s["qs"], D ** -0.5, workspace=ws)
            elif i == 2:
                getattr(pk, "paged_attention_tree" + f8)(s["out"], s["qr"], kc, vc, *sc, s["bt"], s["lens"],
                                                         s["qs"], s["parents"], D ** -0.5, workspace=ws)
            else:
                f = pk.paged_attention_decode_fp8 if f8 else pk.paged_attention_decode_ex
                f(s["out"], s["qr"], kc, vc, *sc, s["bt"], s["lens"], D ** -0.5, workspace=dws)

    dws = torch.zeros(pk.paged_attention_workspace_size(3, H, 24 * bs, D), dtype=torch.uint8, device="cuda")
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            steps()
        g.replay()
    else:
        steps()
    torch.cuda.synchronize()
    assert pk.get_device_error() == 0
    for i, s in enumerate(plan):
        b = ar.Batch.__new__(ar.Batch)
        b.H, b.G, b.D, b.bs, b.dtype, b.scale = H, G, D, bs, dtype, D ** -0.5
        b.seqs = list(zip(s["new"], s["done"]))
        b.start_host, b.T, b.q, b.kc, b.vc = s["start"], s["start"][-1], s["qr"], kc, vc
        b.ks, b.vs = sc if sc else (None, None)
        b.tables, b.parents = s["bt"], s["parents"]
        ref, bound = ar.attend(b, tree=i == 2)
        ar.close(s["out"], ref, bound * (4 if i == 3 else 1), f"step {i}")
        y = ar.rope(s["qkv"][:, :H], s["pos"][None], freq, [D // 2], w[0], 1e-6, False)
        ar.close(s["qr"], y, step_bound(y, (y.abs() + 8) * (D / 2 + 16) * U, dtype), f"q of step {i}")
