"""What is measured of the operators around the paged KV cache, next to their plain forms.

Three operators: per-head RMS norm and rotation of q and k with the append of
k and v ("rope"), causal attention of packed prompts over the paged cache
("prefill"), and attention of drafted token trees over it ("tree").

``run`` computes a case in plain torch operations, or, where ``own`` is true,
through this repository's binding.  Lengths come from the case alone, values
and the placement of blocks from the seed.
"""
import math

import numpy as np
import torch

own = False

_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.bfloat16}
_POOL = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
_ELT = {"f32": 4, "bf16": 2, "fp8": 1}


# ------------------------------------------------------------------ cases
def _rope(name, tokens, heads, kv_heads, head_dim, block_size, dtype, rotary, axes, interleaved, norm,
          far, pad):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "block_size": block_size, "dtype": dtype, "rotary": rotary,
            "axes": axes, "interleaved": interleaved, "norm": norm, "far": far, "pad": pad}


def _attn(name, op, seqs, new_lo, new_hi, ctx_lo, ctx_hi, heads, kv_heads, head_dim, block_size, dtype,
          lens=1):
    return {"name": name, "op": op, "seqs": seqs, "new_lo": new_lo, "new_hi": new_hi, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "block_size": block_size, "dtype": dtype, "lens": lens}


def listed():
    return [
        # one decode step of 64 sequences: a call whose latency counts
        _rope("rope_decode_64", 64, 32, 8, 128, 16, "bf16", 128, 1, False, True, 131072, 0),
        # image and video prompts: three position axes, an fp8 cache, the largest call
        _rope("rope_axes_fp8", 8192, 64, 8, 128, 32, "fp8", 128, 3, False, True, 32768, 64),
        # a small fp32 model: adjacent pairs, half of the head rotated, no norm, padded batch
        _rope("rope_partial_f32", 777, 4, 4, 64, 16, "f32", 32, 1, True, False, 1048576, 19),
        # four short prompts of a small fp32 model
        _attn("prefill_tiny_f32", "prefill", 4, 1, 50, 0, 0, 4, 4, 64, 16, "f32"),
        # packed prompts of mixed lengths, grouped heads: the ordinary prompt step
        _attn("prefill_packed", "prefill", 12, 40, 2048, 0, 0, 32, 8, 128, 16, "bf16"),
        # one long prompt, one query head per kv head: the largest work
        _attn("prefill_long", "prefill", 1, 8192, 8192, 0, 0, 32, 32, 128, 16, "bf16"),
        # chunks of long prompts over what earlier chunks left in an fp8 cache
        _attn("prefill_chunk_fp8", "prefill", 2, 700, 1024, 12000, 15360, 64, 8, 128, 32, "fp8"),
        # prompts behind a cached prefix, head_dim 64, the smallest blocks
        _attn("prefill_prefix_d64", "prefill", 8, 65, 999, 128, 1500, 16, 4, 64, 8, "bf16"),
        # a few drafts of one small fp32 sequence
        _attn("tree_small_f32", "tree", 2, 3, 5, 40, 300, 4, 4, 64, 16, "f32"),
        # speculative step of a 64-sequence batch, 16 drafts each
        _attn("tree_batch_64", "tree", 64, 16, 16, 128, 2048, 32, 8, 128, 16, "bf16"),
        # drafts over long contexts: the cache is read once for all of them
        _attn("tree_long", "tree", 8, 17, 33, 32768, 131072, 64, 8, 128, 32, "bf16"),
        # few drafts over an fp8 cache, one query head per kv head
        _attn("tree_mha_fp8", "tree", 24, 1, 7, 200, 2048, 32, 32, 128, 8, "fp8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "prefill", "tree"])
    dtype = rng.choice(["bf16", "bf16", "fp8", "f32"])
    head_dim = rng.choice([64, 128])
    group = rng.choice([1, 2, 4, 8])
    block_size = rng.choice([8, 16, 32])
    if op == "rope":
        kv_heads = rng.randint(1, 8)
        axes = rng.choice([1, 1, 2, 3])
        c = _rope("", _log(rng, 1, 8192 if dtype != "f32" else 4096), kv_heads * group, kv_heads, head_dim,
                  block_size, dtype, rng.choice([head_dim // 2, head_dim]), axes, rng.random() < 0.3,
                  rng.random() < 0.8, _log(rng, 1000, 1048576), rng.choice([0, 0, rng.randint(1, 9)]))
    elif op == "prefill":
        kv_heads = rng.randint(1, 8)
        if dtype == "f32":
            group, kv_heads = rng.choice([1, 2, 4]), rng.randint(1, 4)
        hi = _log(rng, 1, 4096 if dtype != "f32" else 1024)
        ctx = rng.choice([0, 0, _log(rng, 16, 8192 if dtype != "f32" else 2048)])
        most = 6e9 / (4.0 * kv_heads * group * hi * (hi + ctx))  # sequences whose scores the plain form can hold
        seqs = max(1, min(_log(rng, 1, 24), int(most)))
        c = _attn("", "prefill", seqs, rng.randint(max(1, hi // 8), hi), hi, ctx // 4, ctx, kv_heads * group,
                  kv_heads, head_dim, block_size, dtype, rng.randint(1, 10 ** 6))
    else:
        kv_heads = rng.randint(1, 8)
        hi = _log(rng, 1, 64)
        if dtype == "f32":
            group, kv_heads, hi = rng.choice([1, 2, 4]), rng.randint(1, 4), min(hi, 16)
        ctx = _log(rng, 64, 65536 if dtype != "f32" else 4096)
        most = min(6e9 / (4.0 * kv_heads * group * hi * ctx), 1e9 / (ctx * kv_heads * head_dim))
        seqs = max(1, min(_log(rng, 1, 64), int(most)))
        c = _attn("", "tree", seqs, rng.randint(1, hi), hi, ctx // 5, ctx, kv_heads * group, kv_heads, head_dim,
                  block_size, dtype, rng.randint(1, 10 ** 6))
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, context with them) of each sequence, spread over the case's ranges, both ends among them."""
    r = np.random.RandomState(case["lens"])

    def spread(lo, hi):
        x = np.exp(r.uniform(math.log(max(lo, 1)), math.log(max(hi, 1)), case["seqs"]))
        x = np.clip(np.rint(x).astype(np.int64), lo, hi)
        x[-1] = hi
        return x

    new = spread(case["new_lo"], case["new_hi"])
    before = spread(case["ctx_lo"], case["ctx_hi"]) if case["ctx_hi"] else np.zeros(case["seqs"], np.int64)
    return new, before + new


def work(case):
    h, g, d = case["heads"], case["kv_heads"], case["head_dim"]
    elt, act = _ELT[case["dtype"]], 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rope":
        t, p = case["tokens"] + case["pad"], case["tokens"]
        b = t * h * d * 2 * act + p * 2 * g * d * (act + elt) + t * (4 * case["axes"] + 8)
        return {"bytes": b, "flops": t * h * d * 7 + p * g * d * 9}
    new, ctx = _lengths(case)
    if case["op"] == "prefill":
        pairs = sum(int(n) * int(c - n) + int(n) * int(n + 1) // 2 for n, c in zip(new, ctx))
    else:  # every draft attends the committed tokens and itself at the least
        pairs = sum(int(n) * int(c - n + 1) for n, c in zip(new, ctx))
    b = int(new.sum()) * h * d * 2 * act + int(ctx.sum()) * g * d * 2 * elt
    return {"bytes": b, "flops": 4 * d * h * pairs}


# ----------------------------------------------------------------- inputs
def _sections(case):
    """Frequency pairs of each axis: all of them, or a quarter for the first axis and the rest shared."""
    pairs, axes = case["rotary"] // 2, case["axes"]
    if axes == 1:
        return [pairs]
    first = pairs // 4
    rest = [(pairs - first) // (axes - 1)] * (axes - 1)
    rest[-1] += pairs - first - sum(rest)
    return [first] + rest


def _scales(case, gen):
    g = torch.arange(case["kv_heads"], device="cuda", dtype=torch.float32)
    return (1.0 + 0.37 * g) / 32.0, (1.0 + 0.21 * g) / 24.0


def _pool(case, blocks, gen, scales):
    shape = (blocks, case["kv_heads"], case["block_size"], case["head_dim"])
    x = torch.randn(shape, generator=gen, device="cuda")
    if case["dtype"] == "fp8":
        x /= scales.view(1, -1, 1, 1)
    return x.to(_POOL[case["dtype"]])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    h, g, d, bs = case["heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    act = _TORCH[case["dtype"]]
    st = {"case": case}
    ks, vs = _scales(case, gen) if case["dtype"] == "fp8" else (None, None)
    st["k_scales"], st["v_scales"] = ks, vs
    if case["op"] == "rope":
        t, pad = case["tokens"], case["pad"]
        # the projection's output: q, k and v rows of a token next to each other
        qkv = (torch.randn(t + pad, h + 2 * g, d, generator=gen, device="cuda") * 1.7).to(act)
        st["q"], st["k"], st["v"] = qkv[:, :h], qkv[:, h:h + g], qkv[:, h + g:]
        st["q_out"] = torch.zeros(t + pad, h, d, device="cuda", dtype=act)
        blocks = -(-t // bs) + 3
        st["k_cache"], st["v_cache"] = (_pool(case, blocks, gen, s) for s in (ks, vs))
        slots = torch.randperm(blocks * bs, generator=gen, device="cuda")[:t + pad]
        slots[t:] = -1  # rows that pad the batch
        st["slots"] = slots
        pos = torch.randint(0, case["far"], (t + pad,), generator=gen, device="cuda")
        if case["axes"] > 1:  # time, then places within a frame
            pos = torch.stack([pos] + [torch.randint(0, 256, (t + pad,), generator=gen, device="cuda")
                                       for _ in range(case["axes"] - 1)])
        st["positions"] = pos.to(torch.int32)
        i = torch.arange(0, case["rotary"], 2, device="cuda", dtype=torch.float64)
        st["inv_freq"] = (500000.0 ** (-i / case["rotary"])).to(torch.float32)
        st["qw"], st["kw"] = ((1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(act)
                              if case["norm"] else None for _ in range(2))
        st["sections"] = _sections(case)
        return st
    new, ctx = _lengths(case)
    need = -(-ctx // bs)
    blocks = int(need.sum()) + 2
    table = torch.full((case["seqs"], int(need.max())), -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    used = torch.arange(int(need.max()), device="cuda") < torch.from_numpy(need).cuda()[:, None]
    table[used] = order[:int(need.sum())]
    st["tables"], st["ctx"] = table, torch.from_numpy(ctx.astype(np.int32)).cuda()
    st["start"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
    st["max_new"], st["max_ctx"], total = int(new.max()), int(ctx.max()), int(new.sum())
    st["q"] = torch.randn(total, h, d, generator=gen, device="cuda").to(act)
    st["out"] = torch.zeros(total, h, d, device="cuda", dtype=act)
    st["k_cache"], st["v_cache"] = (_pool(case, blocks, gen, s) for s in (ks, vs))
    st["scale"] = float(np.float32(1 / math.sqrt(d)))
    if case["op"] == "tree":  # each draft hangs on an earlier one; the first on the last committed token
        own_index = torch.cat([torch.arange(int(n), device="cuda") for n in new])
        u = torch.rand(total, generator=gen, device="cuda", dtype=torch.float64)
        st["parents"] = ((u * own_index).floor().to(torch.int32)).where(own_index > 0, -1).to(torch.int32)
    return st


# ------------------------------------------------------------- plain forms
def _turn(x, cos, sin, interleaved):
    """The first 2 * cos.shape[-1] values of each row of x rotated, the others as they are."""
    r = cos.shape[-1]
    if interleaved:
        a, b = x[..., :2 * r:2], x[..., 1:2 * r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r], x[..., r:2 * r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., 2 * r:]], -1)


def _normed(x, w, t):
    x = x.to(t)
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.to(t)


def _rope_plain(st, t):
    """q, k, v after the norm and the rotation, in type t."""
    case = st["case"]
    pos = st["positions"].view(case["axes"], -1)
    axis = torch.repeat_interleave(torch.arange(case["axes"]), torch.tensor(st["sections"])).to(pos.device)
    angle = pos[axis].t().double() * st["inv_freq"].double()
    cos, sin = angle.cos().to(t)[:, None], angle.sin().to(t)[:, None]
    q = _turn(_normed(st["q"], st["qw"], t), cos, sin, case["interleaved"])
    k = _turn(_normed(st["k"], st["kw"], t), cos, sin, case["interleaved"])
    return q, k, st["v"].to(t)


def _ancestors(st):
    """[B][n][n]: whether draft j is i or an ancestor of i (products of the one-step matrix)."""
    b, n = st["ctx"].shape[0], st["max_new"]
    total = st["q"].shape[0]
    row = torch.arange(total, device="cuda")
    seq = torch.searchsorted(st["start"][1:].long(), row, right=True)
    i = row - st["start"].long()[seq]
    # parent -1 goes to a column that is cut off again
    step = torch.zeros(b, n, n + 1, device="cuda")
    step[seq, i, st["parents"].long()] = 1.0
    step = step[..., :n] + torch.eye(n, device="cuda")
    return torch.matrix_power(step, n) > 0


def _keys(st, cache, scales, t):
    """[B][Hkv][max_ctx][D] through the block tables."""
    pos = torch.arange(st["max_ctx"], device="cuda")
    bs = st["case"]["block_size"]
    blk = st["tables"].long().clamp(min=0)[:, pos // bs]
    x = (cache.view(torch.uint8) if scales is not None else cache)[blk, :, pos % bs]
    x = (x.view(torch.float8_e4m3fn).to(t) * scales.to(t).view(1, 1, -1, 1)) if scales is not None else x.to(t)
    return x.transpose(1, 2)


def _attend_plain(st, t):
    case = st["case"]
    h, g, d, n = case["heads"], case["kv_heads"], case["head_dim"], st["max_new"]
    b, total = st["ctx"].shape[0], st["q"].shape[0]
    start, ctx = st["start"].long(), st["ctx"].long()
    new = start[1:] - start[:-1]
    i, j = torch.arange(n, device="cuda"), torch.arange(st["max_ctx"], device="cuda")
    q = st["q"][(start[:-1, None] + i).clamp(max=total - 1)].to(t) * st["scale"]  # [B][n][H][D]
    q = q.view(b, n, g, h // g, d).permute(0, 2, 3, 1, 4).reshape(b, g, h // g * n, d)
    s = (q @ _keys(st, st["k_cache"], st["k_scales"], t).transpose(2, 3)).view(b, g, h // g, n, -1)
    first = (ctx - new)[:, None, None]
    if case["op"] == "prefill":
        seen = j <= first + i[:, None]
    else:
        draft = (j - first).expand(b, n, -1)
        seen = (draft < 0) | (_ancestors(st).gather(2, draft.clamp(0, n - 1)) & (draft < new[:, None, None]))
    s.masked_fill_(~seen[:, None, None], -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True)).exp_()
    s /= s.sum(-1, keepdim=True)
    o = s.view(b, g, h // g * n, -1) @ _keys(st, st["v_cache"], st["v_scales"], t)
    o = o.view(b, g, h // g, n, d).permute(0, 3, 1, 2, 4).reshape(b, n, h, d)
    row = torch.arange(total, device="cuda")
    seq = torch.searchsorted(start[1:], row, right=True)
    return o[seq, row - start[seq]]


def _codes(x, scales):
    return (x / scales.to(x.dtype).view(1, -1, 1)).clamp(-448, 448)


def run(state):
    st = state
    case = st["case"]
    if own:
        from paged_kv_cache_323_b200 import pagedkv as pk

        fp8 = (st["k_scales"], st["v_scales"]) if case["dtype"] == "fp8" else ()
        if case["op"] == "rope":
            call = pk.qk_norm_rope_append_fp8 if fp8 else pk.qk_norm_rope_append
            call(st["q_out"], st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], *fp8, st["slots"],
                 st["positions"], st["inv_freq"], q_weight=st["qw"], k_weight=st["kw"], eps=1e-6,
                 sections=st["sections"], interleaved=case["interleaved"])
            return {"q": st["q_out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
        if case["op"] == "prefill":
            call = pk.paged_attention_prefill_fp8 if fp8 else pk.paged_attention_prefill
            call(st["out"], st["q"], st["k_cache"], st["v_cache"], *fp8, st["tables"], st["ctx"], st["start"],
                 st["scale"])
        else:
            call = pk.paged_attention_tree_fp8 if fp8 else pk.paged_attention_tree
            call(st["out"], st["q"], st["k_cache"], st["v_cache"], *fp8, st["tables"], st["ctx"], st["start"],
                 st["parents"], st["scale"])
        return {"out": st["out"]}
    if case["op"] == "rope":
        q, k, v = _rope_plain(st, torch.float32)
        kc, vc = st["k_cache"], st["v_cache"]
        at, bs = st["slots"][:case["tokens"]], case["block_size"]
        k, v = k[:case["tokens"]], v[:case["tokens"]]
        if case["dtype"] == "fp8":
            k, v = (_codes(x, s).to(torch.float8_e4m3fn).view(torch.uint8)
                    for x, s in ((k, st["k_scales"]), (v, st["v_scales"])))
            kc, vc = kc.view(torch.uint8), vc.view(torch.uint8)
        kc[at // bs, :, at % bs] = k.to(kc.dtype)
        vc[at // bs, :, at % bs] = v.to(vc.dtype)
        return {"q": q.to(st["q"].dtype), "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    return {"out": _attend_plain(st, torch.float32).to(st["q"].dtype)}


# ---------------------------------------------------- definition, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    h, g, d, bs = case["heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    if case["op"] == "rope":
        pos = st["positions"].double().view(case["axes"], -1)
        bounds = np.concatenate([[0], np.cumsum(st["sections"])])
        out = []
        for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
            x = x.double()
            if w is not None:
                x = x / (x.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * w.double()
            y = x.clone()
            for a in range(case["axes"]):
                for i in range(int(bounds[a]), int(bounds[a + 1])):
                    p, r = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + case["rotary"] // 2)
                    z = (pos[a] * st["inv_freq"][i].double())[:, None]
                    y[..., p] = x[..., p] * z.cos() - x[..., r] * z.sin()
                    y[..., r] = x[..., p] * z.sin() + x[..., r] * z.cos()
            out.append(y)
        at = st["slots"][:case["tokens"]]
        pools = []
        for cache, x, s in ((st["k_cache"], out[1], st["k_scales"]), (st["v_cache"], st["v"].double(), st["v_scales"])):
            pool = cache.double()
            if s is not None:
                x = (x / s.double()[:, None]).clamp(-448, 448)
            pool[at // bs, :, at % bs] = x[:case["tokens"]]
            pools.append(pool)
        return {"q": out[0], "k_cache": pools[0], "v_cache": pools[1]}
    start, ctx = st["start"].tolist(), st["ctx"].tolist()
    res = torch.zeros(start[-1], h, d, dtype=torch.float64, device="cuda")
    for s in range(case["seqs"]):
        c, n = ctx[s], start[s + 1] - start[s]
        blk = st["tables"][s, :-(-c // bs)].long()
        anc = None
        if case["op"] == "tree":
            par = st["parents"][start[s]:start[s + 1]].tolist()
            anc = torch.zeros(n, n, dtype=torch.bool)
            for i in range(n):
                j = i
                while j >= 0:
                    anc[i, j] = True
                    j = par[j]
            anc = anc.cuda()
        for u in range(g):
            k, v = (cache[blk, u].to(torch.float64).reshape(-1, d)[:c] for cache in (st["k_cache"], st["v_cache"]))
            if case["dtype"] == "fp8":
                k, v = k * st["k_scales"][u].double(), v * st["v_scales"][u].double()
            for x in range(u * (h // g), (u + 1) * (h // g)):
                for i0 in range(0, n, 4096):
                    i1 = min(n, i0 + 4096)
                    p = (st["q"][start[s] + i0:start[s] + i1, x].double() @ k.t()) * st["scale"]
                    if anc is None:
                        at = torch.arange(c, device="cuda")
                        p[at > (c - n + torch.arange(i0, i1, device="cuda"))[:, None]] = -math.inf
                    else:
                        p[:, c - n:][~anc[i0:i1]] = -math.inf
                    p = torch.softmax(p, -1)
                    res[start[s] + i0:start[s] + i1, x] = p @ v
    return {"out": res}
