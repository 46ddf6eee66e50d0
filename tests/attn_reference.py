"""Plain 64-bit forms of the operators around the paged cache (prompt
attention, drafted-tree attention, q/k norm and rotation), with the bounds
their rounding steps allow.  Elementary torch operations only."""
import math

import torch

F8_MAX = 448.0
ACT = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.bfloat16}
POOL = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}


def scales(kv_heads, device="cuda"):
    g = torch.arange(kv_heads, device=device, dtype=torch.float32)
    return (1.0 + 0.37 * g) / 32.0, (1.0 + 0.21 * g) / 24.0


class Batch:
    """Paged pools, tables and packed queries of sequences (queries, context)."""

    def __init__(self, seqs, *, dtype="bf16", heads=4, kv_heads=2, head_dim=128, block_size=16, seed=0,
                 spare=3, pad_rows=0, max_blocks=None, amp=1.0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.dtype, self.H, self.G, self.D, self.bs = dtype, heads, kv_heads, head_dim, block_size
        self.seqs = seqs
        need = [-(-c // block_size) for _, c in seqs]
        blocks = sum(need) + spare
        shape = (blocks, kv_heads, block_size, head_dim)
        ks, vs = scales(kv_heads)
        self.ks, self.vs = (ks, vs) if dtype == "fp8" else (None, None)
        self.kc, self.vc = (torch.randn(shape, generator=gen, device="cuda") * amp for _ in range(2))
        if dtype == "fp8":
            self.kc, self.vc = self.kc / ks.view(1, -1, 1, 1), self.vc / vs.view(1, -1, 1, 1)
        self.kc, self.vc = self.kc.to(POOL[dtype]), self.vc.to(POOL[dtype])
        order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
        self.tables = torch.full((len(seqs), max_blocks or max(need + [1])), -7, dtype=torch.int32, device="cuda")
        at = 0
        for s, k in enumerate(need):
            self.tables[s, :k] = order[at:at + k]
            at += k
        self.ctx = torch.tensor([c for _, c in seqs], dtype=torch.int32, device="cuda")
        start = [0]
        for n, _ in seqs:
            start.append(start[-1] + n)
        self.start_host = start
        self.start = torch.tensor(start, dtype=torch.int32, device="cuda")
        self.T = start[-1] + pad_rows
        self.q = torch.randn(self.T, heads, head_dim, generator=gen, device="cuda").to(ACT[dtype])
        self.out = torch.full((self.T, heads, head_dim), -77.0, device="cuda", dtype=ACT[dtype])
        self.scale = 1 / math.sqrt(head_dim)
        u = torch.rand(self.T, generator=gen, device="cuda")
        self.parents = torch.full((self.T,), -1, dtype=torch.int32, device="cuda")
        for s, (n, _) in enumerate(seqs):
            i = torch.arange(n, device="cuda")
            up = (u[start[s]:start[s] + n] * (i + 1)).floor().to(torch.int32) - 1  # -1 .. i - 1
            self.parents[start[s]:start[s] + n] = up

    def poison(self):
        """NaN in every slot that holds no token of a sequence."""
        used = torch.zeros(self.kc.shape[0], self.bs, dtype=torch.bool, device="cuda")
        for s, (_, c) in enumerate(self.seqs):
            pos = torch.arange(c, device="cuda")
            used[self.tables[s].long()[pos // self.bs], pos % self.bs] = True
        for cache in (self.kc, self.vc):
            x = cache.view(torch.uint8) if self.dtype == "fp8" else cache
            x.masked_fill_(~used[:, None, :, None], 0x7F if self.dtype == "fp8" else math.nan)

    def call(self, pk, tree=False, **kw):
        fp8 = (self.ks, self.vs) if self.dtype == "fp8" else ()
        f = getattr(pk, ("paged_attention_tree" if tree else "paged_attention_prefill") + ("_fp8" if fp8 else ""))
        more = (self.parents,) if tree else ()
        f(self.out, self.q, self.kc, self.vc, *fp8, self.tables, self.ctx, self.start, *more, self.scale, **kw)
        return self.out


def ancestors(parents):
    """[n][n]: j is i or an ancestor of i."""
    n = len(parents)
    m = torch.zeros(n, n, dtype=torch.bool)
    for i in range(n):
        j = i
        while j >= 0:
            m[i, j] = True
            j = parents[j]
    return m


def attend(b: Batch, tree=False, lost=()):
    """(out, bound) in 64 bits of the rows of b's sequences; `lost`: physical
    blocks that take no part.

    Bound: half a step of the output's type; weights rounded to bf16 before
    the product with v (bf16 and fp8 caches); scores accumulated in fp32
    (head_dim additions of |q||k|, each within 2^-24) and moving every weight by
    that much; exponentials within 2^-12 relative where they are rounded to
    bf16 next, 2^-21 else; sums of n weights within n 2^-24 (pairwise and
    blocked ones are far below)."""
    H, G, D, bs = b.H, b.G, b.D, b.bs
    ref = torch.zeros(b.T, H, D, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(ref)
    u = 2.0 ** -24
    narrow = b.dtype != "f32"
    for s, (n, c) in enumerate(b.seqs):
        if n == 0:
            continue
        r0 = b.start_host[s]
        pos = torch.arange(c, device="cuda")
        blk = b.tables[s].long()[pos // bs]
        ok = (blk >= 0) & (blk < b.kc.shape[0])
        for x in lost:
            ok &= blk != x
        blk = blk.clamp(0, b.kc.shape[0] - 1)
        seen = pos[None] <= (c - n + torch.arange(n, device="cuda"))[:, None]
        if tree:
            seen = torch.ones(n, c, dtype=torch.bool, device="cuda")
            seen[:, c - n:] = ancestors(b.parents[r0:r0 + n].tolist()).cuda()
        seen &= ok
        for g in range(G):
            def rows(cache, sc):
                x = cache.view(torch.uint8)[blk, g, pos % bs].view(cache.dtype) if b.dtype == "fp8" \
                    else cache[blk, g, pos % bs]
                return x.double() * (sc[g].double() if sc is not None else 1.0)
            k, v = rows(b.kc, b.ks), rows(b.vc, b.vs)
            for h in range(g * (H // G), (g + 1) * (H // G)):
                q = b.q[r0:r0 + n, h].double()
                # unseen keys: neither their score nor their value may matter
                kk = torch.where(ok[:, None], k, 0.0)
                sc = torch.where(seen, (q @ kk.nan_to_num(0, 0, 0).t()) * b.scale, -math.inf)
                bad_k = (~torch.isfinite(kk)).any(1)
                if bad_k.any():  # a row that sees such a key: whatever it gives
                    sc = torch.where(seen & bad_k[None], math.nan, sc)
                mag = torch.where(seen, (q.abs() @ kk.nan_to_num(0, 0, 0).abs().t()) * abs(b.scale), 0.0).amax(1)
                m = sc.amax(1, keepdim=True)
                p = torch.where(seen, (sc - m).exp(), 0.0)
                l = p.sum(1, keepdim=True)
                p = torch.where(l == 0, 0.0, p / l)
                vz = torch.where(torch.isfinite(v), v, 0.0)
                o = p @ vz
                badv = ~torch.isfinite(v)
                if badv.any():
                    for j in badv.any(1).nonzero().flatten().tolist():
                        hit = seen[:, j]
                        o[hit] = o[hit] + p[hit, j:j + 1] * torch.where(badv[j], v[j], 0.0)
                a = p @ vz.abs()
                rel = 2 * (D * u * mag[:, None] + c * u + (2.0 ** -12 if narrow else 2.0 ** -21)) \
                    + (2.0 ** -8 if narrow else 0.0)
                ref[r0:r0 + n, h] = o
                bound[r0:r0 + n, h] = rel * a + (2.0 ** -8 if narrow else u) * (o.abs() + rel * a)
    return ref, bound + 1e-30


def close(got, ref, bound, what=""):
    got = got.double()
    nan = torch.isnan(ref)
    assert bool((torch.isnan(got) | torch.isinf(got))[nan].all()), f"{what}: finite where the formula is not"
    d = (got - ref).abs()
    over = ~nan & ~(d <= bound) & ~((got == ref) & torch.isinf(ref))
    if bool(over.any()):
        i = tuple(over.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} past the bound, first at {i}: "
                             f"{float(got[i])} against {float(ref[i])}, bound {float(bound[i])}")


def rope(x, pos, inv_freq, sections, w, eps, interleaved):
    """x [T][heads][D] after the norm and the rotation, 64 bits; pos [axes][T]."""
    x = x.double()
    D = x.shape[-1]
    if w is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    y = x.clone()
    half = len(inv_freq)
    i = 0
    for a, cnt in enumerate(sections):
        for _ in range(cnt):
            p, r = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            z = (pos[a].double() * inv_freq[i].double())[:, None]
            y[..., p] = x[..., p] * z.cos() - x[..., r] * z.sin()
            y[..., r] = x[..., r] * z.cos() + x[..., p] * z.sin()
            i += 1
    assert y.shape[-1] == D
    return y
