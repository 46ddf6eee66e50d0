"""Refusals of the operators around the paged cache, on the CPU: the C entry
points' validation and the binding's argument checks."""
import ctypes

import pytest
import torch

from test_abi import FAKE, MIS, pk as abi_pk  # noqa: F401
from test_binding_checks import Dev as HostDev, pk  # noqa: F401


class Dev(HostDev):
    def stride(self, *i):
        return self.t.stride(*i)

    def is_contiguous(self):
        return self._contiguous and self.t.is_contiguous()

    def get_device(self):
        return self.device.index if self.is_cuda else -1


@pytest.fixture(autouse=True)
def no_stream(monkeypatch):
    from paged_kv_cache_323_b200 import pagedkv

    monkeypatch.setattr(pagedkv, "_raw_stream", lambda index: 0)


def _attn(pk, name, **kw):
    a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, ctx=FAKE, qs=FAKE, par=FAKE, stride=1024,
             T=9, B=4, H=8, Hkv=2, D=128, bs=16, maxb=8, scale=0.125, nblk=64, dtype=pk.PKV_BF16, ws=FAKE,
             wsb=1 << 30)
    a.update(kw)
    args = [a["out"], a["q"], a["k"], a["v"]]
    args += [a["ks"], a["vs"]] if name.endswith("_fp8") else []
    args += [a["bt"], a["ctx"], a["qs"]] + ([a["par"]] if "tree" in name else [])
    args += [a["stride"], a["T"], a["B"], a["H"], a["Hkv"], a["D"], a["bs"], a["maxb"], a["scale"], a["nblk"]]
    args += [] if name.endswith("_fp8") else [a["dtype"]]
    return getattr(pk.lib, name)(*args, a["ws"], a["wsb"], None)


NAMES = ["paged_attention_prefill", "paged_attention_prefill_fp8", "paged_attention_tree", "paged_attention_tree_fp8"]


@pytest.mark.parametrize("name", NAMES)
def test_attention_refusals(abi_pk, name):  # noqa: F811
    pk = abi_pk
    assert _attn(pk, name, B=0, out=None) == pk.PKV_OK
    assert _attn(pk, name, T=0, q=None) == pk.PKV_OK
    assert _attn(pk, name, B=-1) == pk.PKV_ERR_INVALID
    assert _attn(pk, name, T=-1) == pk.PKV_ERR_INVALID
    for x in ("out", "q", "k", "v", "bt", "ctx", "qs") + (("ks", "vs") if "fp8" in name else ()) + \
            (("par",) if "tree" in name else ()):
        assert _attn(pk, name, **{x: None}) == pk.PKV_ERR_NULL, x
    for bad in (dict(H=6, Hkv=4), dict(Hkv=0), dict(D=0), dict(bs=0), dict(maxb=0), dict(nblk=0),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(q=MIS), dict(out=MIS), dict(k=MIS),
                dict(v=MIS), dict(stride=1023), dict(stride=1028), dict(maxb=(1 << 31) // 16)):
        assert _attn(pk, name, **bad) == pk.PKV_ERR_INVALID, bad
    for bad in (dict(D=96), dict(bs=12), dict(H=6, Hkv=2), dict(H=32)):
        assert _attn(pk, name, **bad) == pk.PKV_ERR_UNSUPPORTED, bad
    for bad in (dict(ws=None), dict(wsb=64), dict(ws=FAKE + 16)):
        assert _attn(pk, name, **bad) == pk.PKV_ERR_WORKSPACE, bad
    if not name.endswith("_fp8"):
        assert _attn(pk, name, dtype=pk.PKV_FP8_E4M3) == pk.PKV_ERR_INVALID
        assert _attn(pk, name, dtype=9) == pk.PKV_ERR_INVALID


def test_attention_workspace_size(abi_pk):  # noqa: F811
    size = abi_pk.paged_attention_prefill_workspace_size
    for code in (abi_pk.PKV_F32, abi_pk.PKV_BF16, abi_pk.PKV_FP8_E4M3):
        assert 0 < size(1, 8, 8, 64, code) < size(7, 8, 8, 64, code) < size(4096, 8, 8, 64, code)
        assert size(4096, 8, 8, 64, code) == size(1 << 30, 8, 8, 64, code)  # full tiles: no more
        assert size(0, 8, 8, 64, code) == size(5, 8, 3, 64, code) == size(5, 8, 0, 64, code) == 0
    assert size(5, 8, 8, 64, 9) == 0


def _rope(pk, fp8=False, **kw):
    a = dict(q_out=FAKE, q=FAKE, k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, slots=FAKE, pos=FAKE, freq=FAKE,
             qw=FAKE, kw=None, eps=1e-6, sections=[64], inter=0, so=1024, sq=1536, sk=1536, sv=1536, T=3, H=8, Hkv=2,
             D=128, bs=16, nblk=9, dtype=pk.PKV_BF16)
    a.update(kw)
    sec = None if a["sections"] is None else (ctypes.c_int * max(1, len(a["sections"])))(*a["sections"])
    n = 1 if a["sections"] is None else len(a["sections"])
    args = [a[x] for x in ("q_out", "q", "k", "v", "kc", "vc")] + ([a["ks"], a["vs"]] if fp8 else [])
    args += [a[x] for x in ("slots", "pos", "freq", "qw", "kw", "eps")] + [sec, n]
    args += [a[x] for x in ("inter", "so", "sq", "sk", "sv", "T", "H", "Hkv", "D", "bs", "nblk")]
    args += [] if fp8 else [a["dtype"]]
    return (pk.lib.qk_norm_rope_append_fp8 if fp8 else pk.lib.qk_norm_rope_append)(*args, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_rope_refusals(abi_pk, fp8):  # noqa: F811
    pk = abi_pk
    assert _rope(pk, fp8, T=0, q=None) == pk.PKV_OK
    assert _rope(pk, fp8, T=-1) == pk.PKV_ERR_INVALID
    for x in ("q_out", "q", "k", "v", "kc", "vc", "slots", "pos", "freq", "sections") + \
            (("ks", "vs") if fp8 else ()):
        assert _rope(pk, fp8, **{x: None}) == pk.PKV_ERR_NULL, x
    for bad in (dict(H=0), dict(Hkv=-1), dict(D=0), dict(bs=0), dict(nblk=0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(sections=[]), dict(sections=[72]), dict(sections=[-8, 16]),
                dict(sections=[0]), dict(q=MIS), dict(kc=MIS), dict(qw=MIS), dict(so=1016), dict(sq=1540),
                dict(sk=248), dict(sv=259), dict(H=1 << 30)):
        assert _rope(pk, fp8, **bad) == pk.PKV_ERR_INVALID, bad
    for bad in (dict(D=96, sections=[8]), dict(sections=[12]), dict(sections=[8] * 5)):
        assert _rope(pk, fp8, **bad) == pk.PKV_ERR_UNSUPPORTED, bad
    if not fp8:
        assert _rope(pk, dtype=pk.PKV_FP8_E4M3) == pk.PKV_ERR_INVALID


def D_(shape, dtype=torch.bfloat16, **kw):
    return Dev(torch.zeros(shape, dtype=dtype), **kw)


def attn_args(**kw):
    a = dict(out=D_((6, 8, 64)), q=D_((6, 8, 64)), kc=D_((9, 2, 16, 64)), vc=D_((9, 2, 16, 64)),
             bt=D_((3, 5), torch.int32), ctx=D_((3,), torch.int32), qs=D_((4,), torch.int32),
             par=D_((6,), torch.int32))
    a.update(kw)
    return a


def call_attn(pk, tree=False, **kw):
    a = attn_args(**kw)
    f = pk.paged_attention_tree if tree else pk.paged_attention_prefill
    more = (a["par"],) if tree else ()
    f(a["out"], a["q"], a["kc"], a["vc"], a["bt"], a["ctx"], a["qs"], *more, 0.1)


def test_attention_binding(pk):  # noqa: F811
    call_attn(pk)
    call_attn(pk, tree=True)
    wide = Dev(torch.zeros(6, 12, 64, dtype=torch.bfloat16)[:, 2:10])
    call_attn(pk, q=wide)
    sizes = [c for c in pk.fake.calls if not c[0].endswith("workspace_size")]
    assert [c[0] for c in sizes] == ["paged_attention_prefill", "paged_attention_tree", "paged_attention_prefill"]
    assert sizes[0][1][7:15] == (512, 6, 3, 8, 2, 64, 16, 5)
    assert sizes[2][1][7] == 768
    n = len(pk.fake.calls)
    for bad in (dict(out=D_((6, 4, 64))), dict(kc=D_((9, 2, 16, 128))), dict(vc=D_((8, 2, 16, 64))),
                dict(out=D_((6, 8, 64), cuda=False)), dict(out=D_((6, 8, 64), contiguous=False)),
                dict(kc=D_((9, 2, 16, 64), index=1)), dict(qs=D_((3,), torch.int32)), dict(bt=D_((2, 5), torch.int32)),
                dict(q=Dev(torch.zeros(8, 6, 64, dtype=torch.bfloat16).transpose(0, 1))),
                dict(q=Dev(torch.zeros(6, 8, 128, dtype=torch.bfloat16)[..., ::2])),
                dict(q=Dev(torch.zeros(1, 8, 64, dtype=torch.bfloat16).expand(6, 8, 64)))):
        with pytest.raises(ValueError):
            call_attn(pk, **bad)
    for bad in (dict(q=D_((6, 8, 64), torch.float32)), dict(vc=D_((9, 2, 16, 64), torch.float32)),
                dict(qs=D_((4,), torch.int64)), dict(ctx=D_((3,), torch.int64))):
        with pytest.raises(TypeError):
            call_attn(pk, **bad)
    with pytest.raises(ValueError):
        call_attn(pk, tree=True, par=D_((5,), torch.int32))
    with pytest.raises(TypeError):
        call_attn(pk, tree=True, par=D_((6,), torch.int64))
    assert all(c[0].endswith("workspace_size") for c in pk.fake.calls[n:])


def call_rope(pk, fp8=False, sections=None, **kw):
    pool = torch.float8_e4m3fn if fp8 else torch.bfloat16
    a = dict(qo=D_((6, 8, 64)), q=D_((6, 8, 64)), k=D_((6, 2, 64)), v=D_((6, 2, 64)), kc=D_((9, 2, 16, 64), pool),
             vc=D_((9, 2, 16, 64), pool), slots=D_((6,), torch.int64), pos=D_((6,), torch.int32),
             freq=D_((32,), torch.float32), qw=D_((64,)), kw=None, ks=D_((2,), torch.float32),
             vs=D_((2,), torch.float32))
    a.update(kw)
    f = pk.qk_norm_rope_append_fp8 if fp8 else pk.qk_norm_rope_append
    more = (a["ks"], a["vs"]) if fp8 else ()
    f(a["qo"], a["q"], a["k"], a["v"], a["kc"], a["vc"], *more, a["slots"], a["pos"], a["freq"], q_weight=a["qw"],
      k_weight=a["kw"], sections=sections)


def test_rope_binding(pk):  # noqa: F811
    call_rope(pk)
    call_rope(pk, fp8=True)
    call_rope(pk, sections=[8, 12, 12], pos=D_((3, 6), torch.int32))
    qkv = torch.zeros(6, 12, 64, dtype=torch.bfloat16)
    call_rope(pk, q=Dev(qkv[:, :8]), k=Dev(qkv[:, 8:10]), v=Dev(qkv[:, 10:]))
    assert [c[0] for c in pk.fake.calls] == ["qk_norm_rope_append", "qk_norm_rope_append_fp8"] + \
        ["qk_norm_rope_append"] * 2
    assert pk.fake.calls[3][1][15:19] == (512, 768, 768, 768)
    n = len(pk.fake.calls)
    for fp8 in (False, True):
        for bad in (dict(qo=D_((6, 4, 64))), dict(k=D_((6, 3, 64))), dict(v=D_((5, 2, 64))), dict(slots=D_((5,), torch.int64)),
                    dict(pos=D_((1, 7), torch.int32)), dict(qw=D_((128,))), dict(sections=[16]),
                    dict(sections=[16, 16]), dict(q=D_((6, 8, 64), index=1)), dict(freq=D_((32,), torch.float32, cuda=False)),
                    dict(q=Dev(torch.zeros(8, 6, 64, dtype=torch.bfloat16).transpose(0, 1)))):
            with pytest.raises(ValueError):
                call_rope(pk, fp8, **bad)
        for bad in (dict(q=D_((6, 8, 64), torch.float32)), dict(pos=D_((6,), torch.int64)),
                    dict(slots=D_((6,), torch.int32)), dict(freq=D_((32,))), dict(qw=D_((64,), torch.float32))):
            with pytest.raises(TypeError):
                call_rope(pk, fp8, **bad)
    assert len(pk.fake.calls) == n
