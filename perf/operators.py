"""The paged-cache operators of libkvq as measured cases: a plain torch form of each and the library's own call.

Operators (``op`` of a case):
  map      kvq_page_map: block tables, row offsets and slot maps of a ragged batch, from its lengths
  cache    kvq_encode_paged of a batch's new keys and values, and kvq_decode_paged of the same rows
  paged    kvq_attend_paged: attention of each sequence's new tokens over its pages of the compressed cache
  prompt   kvq_attend_prompt: causal attention over whole packed prompts, before anything is compressed
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the step of a decode loop: 64 sequences, one new token each; some of them start a page
        dict(name="map_decode_64", op="map", seqs=64, ctx_lo=1, ctx_hi=8192, new_lo=1, new_hi=1, page=64, lens=1),
        # 1000 requests admitted or continued at once, some of them idle this step
        dict(name="map_prompt_1000", op="map", seqs=1000, ctx_lo=0, ctx_hi=2000, new_lo=0, new_hi=517, page=16, lens=2),
        # one new token of 64 sequences, Llama-3-8B heads, 2-bit codes
        dict(name="cache_decode_64", op="cache", seqs=64, ctx_lo=0, ctx_hi=8191, new_lo=1, new_hi=1, page=64, heads=8,
             dim=128, bits=2, group=128, rope=1, sinks=4, perm=False, lens=3),
        # ragged prompts of 32768 tokens in all, with a channel permutation and 4-bit codes
        dict(name="cache_prompt_4bit", op="cache", seqs=29, ctx_lo=0, ctx_hi=900, new_lo=3, new_hi=2257, page=32, heads=8,
             dim=128, bits=4, group=64, rope=2, sinks=4, perm=True, lens=4),
        # decode step, ragged batch of 64 Llama-3-8B sequences up to 8192 tokens
        dict(name="paged_decode_64", op="paged", seqs=64, ctx_lo=40, ctx_hi=8191, new_lo=1, new_hi=1, page=64, q_heads=32,
             heads=8, dim=128, bits=2, group=128, rope=1, sinks=4, perm=False, lens=5),
        # decode step, four long contexts of 32768 tokens
        dict(name="paged_decode_long", op="paged", seqs=4, ctx_lo=32768, ctx_hi=32768, new_lo=1, new_hi=1, page=128,
             q_heads=32, heads=8, dim=128, bits=2, group=128, rope=1, sinks=4, perm=False, lens=6),
        # decode step at the Llama-2-7B shape: 32 KV heads, two groups a record, permutation
        dict(name="paged_decode_mha", op="paged", seqs=8, ctx_lo=3500, ctx_hi=4096, new_lo=1, new_hi=1, page=16,
             q_heads=32, heads=32, dim=128, bits=2, group=64, rope=1, sinks=4, perm=True, lens=7),
        # a chunk of 512 prompt tokens on 16384 cached ones
        dict(name="paged_chunk_512", op="paged", seqs=1, ctx_lo=16384, ctx_hi=16384, new_lo=512, new_hi=512, page=64,
             q_heads=32, heads=8, dim=128, bits=4, group=128, rope=1, sinks=4, perm=False, lens=8),
        # continuous batching: short chunks and single tokens side by side, 3-bit codes
        dict(name="paged_mixed_12", op="paged", seqs=12, ctx_lo=0, ctx_hi=8000, new_lo=1, new_hi=131, page=48, q_heads=32,
             heads=8, dim=128, bits=3, group=64, rope=2, sinks=0, perm=False, lens=9),
        # one short prompt: a question of 77 tokens
        dict(name="prompt_77", op="prompt", seqs=1, new_lo=77, new_hi=77, q_heads=32, heads=8, dim=128, bf16=False, lens=10),
        # packed ragged prompts, Llama-3-8B heads
        dict(name="prompt_packed_9", op="prompt", seqs=9, new_lo=5, new_hi=1300, q_heads=32, heads=8, dim=128, bf16=False,
             lens=11),
        # one long prompt on a quarter of the heads (the share of one of four GPUs), bf16
        dict(name="prompt_16384", op="prompt", seqs=1, new_lo=16384, new_hi=16384, q_heads=8, heads=2, dim=128, bf16=True,
             lens=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["map", "cache", "paged", "paged", "prompt", "prompt"])
    c = dict(op=op, lens=rng.randrange(1 << 20))
    if op == "map":
        c.update(seqs=_log(rng, 1, 1000), ctx_lo=0, ctx_hi=_log(rng, 1, 8192), new_lo=rng.choice([0, 1]), page=rng.choice([16, 32, 48, 64, 128]))
        c["new_hi"] = _log(rng, 1, 512)
        return c
    dim = rng.choice([128, 128, 128, 64])
    heads, g = rng.choice([(1, 8), (2, 4), (4, 4), (5, 3), (8, 4), (8, 8), (8, 1), (32, 1)])
    if op == "prompt":
        c.update(seqs=_log(rng, 1, 24), new_lo=1, q_heads=heads * g, heads=heads, dim=dim, bf16=rng.random() < 0.5)
        c["new_hi"] = _log(rng, 1, max(1, min(8192, int(9000 * math.sqrt(32 / max(32, heads * g))) // c["seqs"])))
        return c
    bits = rng.choice([2, 2, 3, 4])
    c.update(page=rng.choice([16, 32, 48, 64, 128]), heads=heads, dim=dim, bits=bits, group=rng.choice([g_ for g_ in (32, 64, 128) if g_ <= dim]),
             rope=rng.choice([1, 2]), sinks=rng.choice([0, 1, 4]), perm=rng.random() < 0.4)
    if op == "cache":
        c.update(seqs=_log(rng, 1, 64), ctx_lo=0, ctx_hi=_log(rng, 1, 8192), new_lo=rng.choice([0, 1]))
        c["new_hi"] = _log(rng, 1, max(1, 262144 // (c["seqs"] * heads)))
        return c
    c.update(q_heads=heads * g)
    c["seqs"] = _log(rng, 1, 64)
    c["ctx_lo"] = 0
    c["ctx_hi"] = _log(rng, 1, min(32768, (1 << 22) // (c["seqs"] * heads)))
    c["new_lo"] = 1
    c["new_hi"] = rng.choice([1, _log(rng, 1, max(1, min(512, (1 << 28) // (c["seqs"] * heads * g * max(64, c["ctx_hi"])))))])
    return c


def _lens(c):
    """(cached tokens, new tokens) of each sequence: a fixed ragged draw of the case."""
    r = random.Random(c["lens"])
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["seqs"])]
    ctx = [r.randint(c["ctx_lo"], c["ctx_hi"]) if "ctx_lo" in c else 0 for _ in range(c["seqs"])]
    return ctx, new


def _pages(c):
    ctx, new = _lens(c)
    before = [-(-a // c["page"]) for a in ctx]
    after = [-(-(a + b) // c["page"]) for a, b in zip(ctx, new)]
    return before, after


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- inputs
def _cache(c, pages, gen):
    """Pages of a cache in use: any codes, group ranges of a rotated head (about +-2 standard deviations)."""
    H, D, ps, bits, ng = c["heads"], c["dim"], c["page"], c["bits"], c["dim"] // c["group"]
    codes = torch.randint(0, 256, (pages, H, ps, D * bits // 8), dtype=torch.uint8, device=DEV, generator=gen)
    z = -(1.2 + 0.8 * torch.rand((pages, H, ps, ng), device=DEV, generator=gen))
    s = (0.95 + 0.1 * torch.rand((pages, H, ps, ng), device=DEV, generator=gen)) * (-2.0 * z / (2 ** bits - 1))
    sz = torch.stack([s.half().view(torch.int16), z.half().view(torch.int16)], dim=-1).contiguous()
    sink = torch.randn((c["seqs"], H, c["sinks"], D), device=DEV, generator=gen).half() if c["sinks"] else None
    return codes, sz, sink


def _batch(c, gen):
    """Lengths, a shuffled page table and the row maps of the batch, as after the step's page map."""
    ctx, new = _lens(c)
    before, after = _pages(c)
    pages, width = max(1, sum(after)), max(1, max(after))
    order = torch.randperm(pages, device=DEV, generator=gen).to(torch.int32)
    S = c["seqs"]
    st = dict(n_rows=max(1, sum(new)), pages=pages, width=width, ctx=_int(ctx), new=_int(new), order=order)
    table = torch.full((S, width), -1, dtype=torch.int32, device=DEV)
    n_after = _int(after)
    col = torch.arange(width, device=DEV)[None]
    first = torch.cumsum(n_after, 0)[:, None] - n_after[:, None]
    held = col < n_after[:, None]
    st["table"] = torch.where(held, order[(first + col).clamp(max=pages - 1)], table).contiguous()
    st["cu"] = torch.cat([torch.zeros(1, device=DEV), torch.cumsum(st["new"], 0)]).to(torch.int32)
    st["kv_len"] = (st["ctx"] + st["new"]).to(torch.int32)
    r = torch.arange(st["n_rows"], device=DEV)
    seq = torch.searchsorted(st["cu"][1:].contiguous(), r.to(torch.int32), right=True).clamp(max=S - 1)
    live = r < st["cu"][-1]
    pos = st["ctx"][seq] + r - st["cu"][seq]
    slot = st["table"][seq, (pos // c["page"]).clamp(max=width - 1)] * c["page"] + pos % c["page"]
    st["seq"], st["pos"], st["slot"] = (torch.where(live, t, torch.full_like(t, -1)).to(torch.int32).contiguous() for t in (seq, pos, slot))
    return st


def _rope_table(rows, dim):
    m = torch.arange(rows, dtype=torch.float64, device=DEV)[:, None]
    a = m * 10000.0 ** (-2.0 * torch.arange(dim // 2, dtype=torch.float64, device=DEV) / dim)
    return torch.stack([torch.cos(a), torch.sin(a)], dim=-1).float().contiguous()


def _perm(c, gen):
    return torch.rand((c["heads"], c["dim"]), device=DEV, generator=gen).argsort(dim=1).to(torch.int16) if c["perm"] else None


def _hadamard(dim, dtype):
    i = torch.arange(dim, device=DEV)
    ones = (i[:, None] & i[None, :])
    bits = sum((ones >> k) & 1 for k in range(8))
    return (1 - 2 * (bits & 1)).to(dtype)


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        st["calls"], st["written"] = _bound(st)
    return st


def _inputs(case, seed):
    c, gen = case, torch.Generator(device=DEV)
    gen.manual_seed(seed)
    S = c["seqs"]
    if c["op"] == "prompt":
        ctx, new = _lens(c)
        n, Hq, H, D = sum(new), c["q_heads"], c["heads"], c["dim"]
        t = torch.bfloat16 if c["bf16"] else torch.float16
        qkv = torch.randn((n, Hq + 2 * H, D), device=DEV, generator=gen)
        # channels of the keys that stand out, as they do in trained models
        qkv[:, Hq:Hq + H] *= 1.0 + 3.0 * (torch.rand((H, D), device=DEV, generator=gen) < 0.03)
        st = dict(case=c, qkv=qkv.to(t), cu=_int([sum(new[:i]) for i in range(S + 1)]), out=torch.zeros((n, Hq, D), dtype=t, device=DEV),
                  scale=D ** -0.5, max_rows=max(new))
        return st
    st = _batch(c, gen)
    st["case"] = c
    if c["op"] == "map":
        before, _ = _pages(c)
        cols = torch.arange(st["width"], device=DEV)[None]
        st["before"] = torch.where(cols < _int(before)[:, None], st["table"], torch.full_like(st["table"], -1)).contiguous()
        spare = torch.randperm(st["pages"] + 5, device=DEV, generator=gen).to(torch.int32)
        st["free"], st["used"] = spare, _int([5])
        if own:
            from kv_cache_rotation_b200 import torch_api as TA
            st["desc"] = TA.make_desc(batch=st["pages"] + 5, heads=1, tokens=0, t_cap=c["page"], bits=2)
            st["batch"] = TA.make_paged(S, st["n_rows"], st["width"], block_table=st["before"])
            st["report"] = torch.zeros(4, dtype=torch.int32, device=DEV)
        return st
    H, D = c["heads"], c["dim"]
    rows = int(max(a + b for a, b in zip(*_lens(c)))) + 1
    st["rope"] = _rope_table(rows, D)
    st["had"] = _hadamard(D, torch.float32)
    st["kperm"], st["vperm"] = _perm(c, gen), _perm(c, gen)
    st["k"], st["v"] = _cache(c, st["pages"], gen), _cache(c, st["pages"], gen)
    if c["op"] == "cache":
        x = torch.randn((st["n_rows"], 2 * H, D), device=DEV, generator=gen)
        x *= 1.0 + 19.0 * (torch.rand((2 * H, D), device=DEV, generator=gen) < 0.02)
        st["kv"] = x.half()
        st["back"] = torch.zeros((2, st["n_rows"], H, D), dtype=torch.float16, device=DEV)
    else:
        st["q"] = torch.randn((st["n_rows"], c["q_heads"], D), device=DEV, generator=gen).half()
        st["out"] = torch.zeros_like(st["q"])
        st["scale"] = D ** -0.5
    if own:
        from kv_cache_rotation_b200 import torch_api as TA
        common = dict(batch=st["pages"], heads=H, head_dim=D, tokens=0, t_cap=c["page"], bits=c["bits"], group=c["group"],
                      n_sink=c["sinks"], rot="fwht_head")
        st["dk"], st["dv"] = TA.make_desc(rope=c["rope"], **common), TA.make_desc(rope=0, **common)
        st["tk"], st["tv"] = TA.make_tables(perm=st["kperm"], rope_cs=st["rope"]), TA.make_tables(perm=st["vperm"])
        st["kc"], st["vc"] = (TA.Packed(t[0], t[1], t[2], None) for t in (st["k"], st["v"]))
        st["batch"] = TA.Paged(cu_rows=st["cu"], kv_len=st["kv_len"], block_table=st["table"], seq=st["seq"], pos=st["pos"],
                               slot=st["slot"])
        if c["op"] == "paged":
            ctx, new = _lens(c)
            st["max_rows"], st["max_kv"] = max(new), max(a + b for a, b in zip(ctx, new))
            st["ws"] = TA.attend_paged_workspace(st["dk"], st["dv"], c["q_heads"], st["batch"], st["max_rows"], st["max_kv"])
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    if own:
        for call in st["calls"]:
            call()
        return st["written"]
    return _PLAIN[st["case"]["op"]](st)


def _bound(st):
    """The prepared calls that a serving loop keeps beside its buffers, and what they write."""
    from kv_cache_rotation_b200 import torch_api as TA
    c = st["case"]
    if c["op"] == "prompt":
        Hq, H, x = c["q_heads"], c["heads"], st["qkv"]
        call = TA.bind_attend_prompt(x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:], st["cu"], st["max_rows"], st["scale"], st["out"])
        return [call], st["out"]
    b = st["batch"]
    if c["op"] == "map":
        call = TA.bind_page_map(st["desc"], b, st["ctx"], st["new"], st["free"], st["used"], st["report"])
        return [call], dict(cu=b.cu_rows, kv_len=b.kv_len, table=b.block_table, seq=b.seq, pos=b.pos, slot=b.slot, report=st["report"])
    if c["op"] == "cache":
        H, kv, (k, v) = c["heads"], st["kv"], st["back"]
        return [TA.bind_encode_paged(st["dk"], kv[:, :H], b, st["tk"], st["kc"]),
                TA.bind_encode_paged(st["dv"], kv[:, H:], b, st["tv"], st["vc"]),
                TA.bind_decode_paged(st["dk"], st["kc"], b, st["tk"], k),
                TA.bind_decode_paged(st["dv"], st["vc"], b, st["tv"], v)], dict(k=k, v=v)
    call = TA.bind_attend_paged(st["dk"], st["dv"], st["q"], st["kc"], st["tk"], st["vc"], st["tv"], b, st["max_rows"], st["max_kv"],
                                st["scale"], st["out"], st["ws"])
    return [call], st["out"]


# ---------------------------------------------------------------- plain forms
def _plain_map(st):
    ps, S, width = st["case"]["page"], st["case"]["seqs"], st["width"]
    ctx, new, used, free = (st[k].long() for k in ("ctx", "new", "used", "free"))
    cu = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    k0, k1 = (ctx + ps - 1) // ps, torch.minimum((ctx + new + ps - 1) // ps, torch.tensor(width, device=DEV))
    need = (k1 - k0).clamp(min=0)
    first = torch.cumsum(need, 0) - need
    col = torch.arange(width, device=DEV)[None]
    at = used + first[:, None] + col - k0[:, None]
    page = torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], torch.full_like(at, -1))
    table = torch.where((col >= k0[:, None]) & (col < k1[:, None]), page, st["before"].long())
    r = torch.arange(st["n_rows"], device=DEV)
    live = r < cu[-1]
    seq = torch.searchsorted(cu[1:].contiguous(), r, right=True).clamp(max=S - 1)
    pos = ctx[seq] + r - cu[seq]
    held = table[seq, (pos // ps).clamp(max=width - 1)]
    slot = torch.where((pos // ps < width) & (held >= 0), held * ps + pos % ps, torch.full_like(pos, -1))
    none = torch.full_like(r, -1)
    seq, pos, slot = (torch.where(live, t, none) for t in (seq, pos, slot))
    total = used[0] + need.sum()
    report = torch.stack([cu[-1], total.clamp(max=free.numel()), (live & (slot < 0)).sum(), (total - free.numel()).clamp(min=0)])
    return {k: t.to(torch.int32) for k, t in dict(cu=cu, kv_len=ctx + new, table=table, seq=seq, pos=pos, slot=slot, report=report).items()}


def _pairs(x, cs, mode, inverse=False, wide=False):
    """RoPE of x [..., D] by the (cos, sin) rows cs [..., D/2, 2]; `wide`: the sum formed before it is rounded to 32 bits."""
    D = x.shape[-1]
    a, b = (x[..., 0::2], x[..., 1::2]) if mode == 1 else (x[..., :D // 2], x[..., D // 2:])
    c, s = cs[..., 0], cs[..., 1]
    if inverse:
        s = -s
    if wide:
        p = (a.double() * c.double() - (b * s).double()).float()
        q = (a.double() * s.double() + (b * c).double()).float()
    else:
        p, q = a * c - b * s, a * s + b * c
    return torch.stack([p, q], dim=-1).flatten(-2) if mode == 1 else torch.cat([p, q], dim=-1)


def _round_half(x, up):
    """x in 32 bits to the next half at or below it (at or above it if `up`)."""
    h = x.half()
    f, bits = h.float(), h.view(torch.int16).int()
    off = (f < x) if up else (f > x)
    toward = torch.where(f == 0, torch.full_like(bits, 1 if up else -32767), torch.where((f > 0) == up, bits + 1, bits - 1))
    return torch.where(off, toward, bits).to(torch.int16).view(torch.float16)


def _quantized(x, st, c, perm, rope):
    """The decoded rows of x [rows, H, D] after one trip through the quantizer, in the rotated basis: (scale, zero, codes)."""
    D, G, levels = c["dim"], c["group"], 2 ** c["bits"] - 1
    y = x.float()
    if rope:
        y = _pairs(y, st["rope"][st["pos"].long().clamp(min=0)][:, None], rope, wide=True)
    if perm is not None:
        y = torch.gather(y, -1, perm.long()[None].expand_as(y))
    # values next to a border between two codes: the transform's sums in the order of its stages
    for h in (1 << k for k in range(D.bit_length() - 1)):
        y = y.unflatten(-1, (D // (2 * h), 2, h))
        y = torch.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], dim=-2).flatten(-3)
    y = (y * torch.tensor(1.0 / math.sqrt(D), dtype=torch.float32, device=DEV)).unflatten(-1, (D // G, G))
    lo, hi = y.amin(-1, keepdim=True) + 0.0, y.amax(-1, keepdim=True) + 0.0
    z = _round_half(lo, False).float()
    s = _round_half((hi - z) / levels, True).float()
    inv = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    code = torch.round((y - z).double() * inv.double()).float()
    return s, z, code


def _restored(y, st, c, perm, rope):
    """Rotated rows y [rows, H, D] back in the basis of the inputs."""
    y = (y @ st["had"].to(y.dtype)) / math.sqrt(c["dim"])
    if perm is not None:
        y = torch.zeros_like(y).scatter(-1, perm.long()[None].expand_as(y), y)
    if rope:
        y = _pairs(y, st["rope"].to(y.dtype)[st["pos"].long().clamp(min=0)][:, None], rope, inverse=True)
    return y


def _plain_cache(st):
    c, H = st["case"], st["case"]["heads"]

    def trip(x, perm, rope):
        s, z, code = _quantized(x, st, c, perm, rope)
        y = _restored((z + code * s).flatten(-2), st, c, perm, rope).half()
        y = torch.where((st["pos"] < c["sinks"])[:, None, None], x, y)
        return torch.where((st["slot"] >= 0)[:, None, None], y, torch.zeros_like(y))

    return dict(k=trip(st["kv"][:, :H], st["kperm"], c["rope"]), v=trip(st["kv"][:, H:], st["vperm"], 0))


def _unpacked(codes, bits, D):
    at = torch.arange(D, device=DEV) * bits
    pad = torch.cat([codes, torch.zeros_like(codes[..., :1])], dim=-1)
    two = pad[..., at // 8].int() | (pad[..., at // 8 + 1].int() << 8)
    return (two >> (at % 8)) & (2 ** bits - 1)


def _rows_of(st, c, cache, perm, rope, table, n, dtype):
    """Keys or values [S, n, H, D] in attention space, read through `table` [S, width]."""
    codes, sz, sink = cache
    D, G, ps = c["dim"], c["group"], c["page"]
    at = torch.arange(n, device=DEV)
    page = table[:, at // ps].long().clamp(min=0)
    code = _unpacked(codes[page, :, at % ps], c["bits"], D).to(dtype).unflatten(-1, (D // G, G))
    s, z = (t.to(dtype)[..., None] for t in sz[page, :, at % ps].view(torch.float16).unbind(-1))
    y = ((z + code * s).flatten(-2) @ st["had"].to(dtype)) / math.sqrt(D)
    if perm is not None:
        y = torch.zeros_like(y).scatter(-1, perm.long()[None, None].expand_as(y), y)
    m = min(c["sinks"], n)
    if m:
        first = sink[:, :, :m].to(dtype).transpose(1, 2)
        y[:, :m] = _pairs(first, st["rope"].to(dtype)[:m][:, None], rope) if rope else first
    return y


def _softmax(s, mask):
    """Weights of the scores s where mask allows them; zeros in a row that it leaves empty."""
    s = s.masked_fill(~mask, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_paged(st):
    c = st["case"]
    S, Hq, H, D = c["seqs"], c["q_heads"], c["heads"], c["dim"]
    ctx, new = _lens(c)
    n, m = max(a + b for a, b in zip(ctx, new)), max(new)
    k = _rows_of(st, c, st["k"], st["kperm"], c["rope"], st["table"], n, torch.float32)
    v = _rows_of(st, c, st["v"], st["vperm"], 0, st["table"], n, torch.float32)
    seq = st["seq"].long()
    live = seq >= 0
    seq = seq.clamp(min=0)
    row = (torch.arange(st["n_rows"], device=DEV) - st["cu"][seq]).clamp(max=m - 1)
    q = torch.zeros((S, m, Hq, D), device=DEV)
    q[seq[live], row[live]] = st["q"].float()[live]
    q = q.view(S, m, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(S, H, -1, D)
    s = (q @ k.permute(0, 2, 3, 1)).unflatten(2, (Hq // H, m)) * st["scale"]
    last = (st["kv_len"] - st["new"])[:, None] + torch.arange(m, device=DEV)
    mask = torch.arange(n, device=DEV) <= last[..., None]
    p = _softmax(s, mask[:, None, None])
    o = (p.flatten(2, 3) @ v.transpose(1, 2)).unflatten(2, (Hq // H, m)).permute(0, 3, 1, 2, 4).reshape(S, m, Hq, D)
    return torch.where(live[:, None, None], o[seq, row], torch.zeros((), device=DEV)).half()


def _plain_prompt(st):
    c = st["case"]
    Hq, H = c["q_heads"], c["heads"]
    x = st["qkv"].float()
    n = x.shape[0]
    q, k, v = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    r = torch.arange(n, device=DEV)
    seq = torch.searchsorted(st["cu"][1:].contiguous(), r.to(torch.int32), right=True)
    mask = (seq[:, None] == seq[None]) & (r[:, None] >= r[None])
    s = q.view(n, H, Hq // H, -1).permute(1, 2, 0, 3).flatten(1, 2) @ k.permute(1, 2, 0)
    p = _softmax((s * st["scale"]).unflatten(1, (Hq // H, n)), mask)
    o = (p.flatten(1, 2) @ v.transpose(0, 1)).unflatten(1, (Hq // H, n))
    return o.permute(2, 0, 1, 3).reshape(n, Hq, -1).to(st["qkv"].dtype)


_PLAIN = dict(map=_plain_map, cache=_plain_cache, paged=_plain_paged, prompt=_plain_prompt)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    ctx, new = _lens(c)
    rows = max(1, sum(new))
    if c["op"] == "map":
        before, after = _pages(c)
        taken = sum(after) - sum(before)
        # lengths in; offsets, lengths, the pages taken (read from the free list, written to the table), three words a row out
        return {"bytes": 4 * (4 * c["seqs"] + 1 + 2 * taken + c["seqs"] + 3 * rows), "flops": 0}
    Hq, H, D = c.get("q_heads", 0), c["heads"], c["dim"]
    if c["op"] == "prompt":
        pairs = sum(b * (b + 1) // 2 for b in new)
        return {"bytes": 2 * rows * D * (2 * Hq + 2 * H), "flops": 4 * D * Hq * pairs}
    record = D * c["bits"] // 8 + 4 * (D // c["group"])
    if c["op"] == "cache":
        turn = D // 2 * 6
        butterfly = D * (D.bit_length() - 1)
        return {"bytes": 2 * rows * H * (2 * 2 * D + 2 * record) + rows * 2 * D * 4, "flops": 2 * rows * H * 2 * (butterfly + 3 * D) + 2 * rows * H * turn}
    pairs = sum(b * a + b * (b + 1) // 2 for a, b in zip(ctx, new))
    cached = sum(a + b for a, b in zip(ctx, new) if b)
    return {"bytes": 2 * cached * H * record + 4 * rows * Hq * D, "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = _inputs(case, seed)
    c = case
    if c["op"] == "map":
        return None
    S, H, D = c["seqs"], c["heads"], c["dim"]
    ctx, new = _lens(c)
    if c["op"] == "prompt":
        Hq = c["q_heads"]
        out = torch.zeros((sum(new), Hq, D), dtype=torch.float64, device=DEV)
        a = 0
        for n in new:
            for h in range(Hq):
                q, k, v = (st["qkv"][a:a + n, i].double() for i in (h, Hq + h // (Hq // H), Hq + H + h // (Hq // H)))
                for b in range(0, n, 4096):
                    e = min(n, b + 4096)
                    s = (q[b:e] @ k[:e].T) * st["scale"]
                    s.masked_fill_(torch.arange(b, e, device=DEV)[:, None] < torch.arange(e, device=DEV)[None], -math.inf)
                    out[a + b:a + e, h] = torch.softmax(s, -1) @ v[:e]
            a += n
        return out
    had = _hadamard(D, torch.float64) / math.sqrt(D)
    rope = st["rope"].double()
    rope = torch.complex(rope[..., 0], rope[..., 1])

    def turned(x, w):  # pair i of each row turned by the angle of w
        a, b = (x[..., 0::2], x[..., 1::2]) if c["rope"] == 1 else (x[..., :D // 2], x[..., D // 2:])
        t = torch.view_as_real(torch.complex(a, b) * w)
        return t.flatten(-2) if c["rope"] == 1 else torch.cat([t[..., 0], t[..., 1]], -1)

    def basis(perm):  # rotated row = row @ basis[h]
        eye = torch.eye(D, dtype=torch.float64, device=DEV)
        return torch.stack([(eye if perm is None else eye[:, perm[h].long()]) @ had for h in range(H)])

    if c["op"] == "cache":
        levels, G = 2 ** c["bits"] - 1, c["group"]

        def trip(x, perm, keys):
            w = rope[st["pos"].long().clamp(min=0)][:, None]
            y = turned(x.double(), w) if keys else x.double()
            m = basis(perm)
            y = torch.einsum("rhd,hde->rhe", y, m).unflatten(-1, (-1, G))
            lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
            z = lo.half()
            z = torch.where(z.double() > lo, torch.nextafter(z.cpu(), torch.tensor(-math.inf).half()).to(DEV), z).double()
            s0 = (hi - z) / levels
            s = s0.half()
            s = torch.where(s.double() < s0, torch.nextafter(s.cpu(), torch.tensor(math.inf).half()).to(DEV), s).double()
            y = z + torch.round((y - z) / torch.where(s > 0, s, torch.ones_like(s))) * s
            y = torch.einsum("rhe,hde->rhd", y.flatten(-2), m)
            y = turned(y, w.conj()) if keys else y
            y = torch.where((st["pos"] < c["sinks"])[:, None, None], x.double(), y)
            return torch.where((st["slot"] >= 0)[:, None, None], y, torch.zeros_like(y))

        return dict(k=trip(st["kv"][:, :H], st["kperm"], True), v=trip(st["kv"][:, H:], st["vperm"], False))
    Hq, ps = c["q_heads"], c["page"]
    out = torch.zeros((st["n_rows"], Hq, D), dtype=torch.float64, device=DEV)
    mk, mv = basis(st["kperm"]), basis(st["vperm"])
    table = st["table"].tolist()
    a = 0
    for i in range(S):
        n, m = ctx[i] + new[i], new[i]
        if not m:
            continue
        mine = torch.tensor(table[i][: -(-n // ps)], device=DEV)

        def held(cache, mat):
            codes, sz, sink = cache
            raw = codes[mine].transpose(1, 2).reshape(-1, H, codes.shape[-1])[:n]
            bit = (raw[..., None].int() >> torch.arange(8, device=DEV)) & 1
            code = (bit.flatten(-2).unflatten(-1, (D, c["bits"])) * (1 << torch.arange(c["bits"], device=DEV))).sum(-1).double()
            both = sz[mine].transpose(1, 2).reshape(-1, H, D // c["group"], 2)[:n].view(torch.float16).double()
            y = both[..., 1:] + code.unflatten(-1, (-1, c["group"])) * both[..., :1]
            return torch.einsum("rhe,hde->rhd", y.flatten(-2), mat)

        k, v = held(st["k"], mk), held(st["v"], mv)
        e = min(n, c["sinks"])
        if e:
            k[:e] = turned(st["k"][2][i, :, :e].double().transpose(0, 1), rope[:e][:, None])
            v[:e] = st["v"][2][i, :, :e].double().transpose(0, 1)
        for h in range(Hq):
            s = (st["q"][a:a + m, h].double() @ k[:, h // (Hq // H)].T) * st["scale"]
            s.masked_fill_(torch.arange(n, device=DEV)[None] > ctx[i] + torch.arange(m, device=DEV)[:, None], -math.inf)
            out[a:a + m, h] = torch.softmax(s, -1) @ v[:, h // (Hq // H)]
        a += m
    return out
