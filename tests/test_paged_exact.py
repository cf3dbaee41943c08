"""Attention over pages within what its roundings allow: every kernel, keys cut into several stretches, many
sequences; and that mistakes do not pass the bound."""
import numpy as np
import pytest

import paged_bounds as B
import paged_ref as R

torch = pytest.importorskip("torch")
import kv_cache_rotation_b200 as K  # noqa: E402
from kv_cache_rotation_b200 import torch_api as TA  # noqa: E402

gpu = pytest.mark.gpu


# ---------------------------------------------------------------- the bound catches mistakes (no GPU)
def _random_head(rng, n, D, bits, few):
    z = -(1.2 + 0.8 * rng.random((2, n, 1)))
    s = ((0.9 + 0.2 * rng.random(z.shape)) * (-2 * z / (2 ** bits - 1))).astype(np.float16).astype(float)
    z = z.astype(np.float16).astype(float)
    c = rng.integers(0, 2 ** bits, (2, n, D))
    y, mag = z + c * s, np.abs(z) + c * np.abs(s)
    none = np.zeros((0, D))
    return B.Head(none, none, y[0], y[1], mag[0], mag[1], None, True, few)


@pytest.mark.parametrize("few", [True, False], ids=["few", "tiles"])
@pytest.mark.parametrize("n,m,bits,D", [(60, 9, 2, 128), (300, 1, 2, 128), (300, 40, 4, 128), (1500, 1, 2, 128), (5000, 1, 2, 128), (2600, 20, 3, 64)])
def test_mistakes_do_not_pass_the_bound(n, m, bits, D, few):
    rng = np.random.default_rng(n + m)
    h = _random_head(rng, n, D, bits, few)
    q = rng.standard_normal((m, D)).astype(np.float16)
    qr = B.query_rows(q, None, True, few)
    q = q.astype(float)
    scale = D ** -0.5
    last = n - m + np.arange(m)
    seen = np.arange(n)[None] <= last[:, None]
    o, tol = h.attend(q, qr, seen, scale)

    def worst(got):
        return (np.linalg.norm(got - o, axis=1) / tol).min()
    assert worst(o) == 0
    assert worst(np.zeros_like(o)) > 10
    mean = np.where(seen, 1.0, 0.0)
    assert worst(B.back_turned((mean / mean.sum(-1, keepdims=True)) @ h.y_v, None, True)) > 10
    # a tile of keys, in the front, at the end, or half a stretch; then one block of 16 of a few thousand
    for lost, times in ((slice(0, 128), 3), (slice(max(n - m - 127, 1), n - m + 1), 3), (slice(n // 2, n // 2 + 256), 3), *([(slice(32, 48), 1)] if n < 5000 else [])):
        cut = seen.copy()
        cut[:, lost] = False
        assert worst(h.attend(q, qr, cut, scale)[0]) > times, lost
    assert worst(h.attend(q, qr, seen, scale * 1.05)[0]) > 1
    if n <= 60:  # one key: rows that miss their own, or see the next row's (half of them: a weight can be small)
        cut = seen.copy()
        cut[np.arange(m), last] = False
        assert np.median(np.linalg.norm(h.attend(q, qr, cut, scale)[0] - o, axis=1) / tol) > 2
        more = np.arange(n)[None] <= np.minimum(last + 1, n - 1)[:, None]
        assert ((np.linalg.norm(h.attend(q, qr, more, scale)[0] - o, axis=1) / tol)[:-1] > 2).mean() >= 0.5


def test_the_turn_of_a_query_row_is_the_hadamard_product():
    x = np.random.default_rng(0).standard_normal((5, 128)).astype(np.float16)
    want = x.astype(float) @ R.hadamard(128)
    assert np.abs(B.turned_fp32(x) - want).max() <= 8 * 2.0 ** -24 * np.linalg.norm(x.astype(float), axis=1).max()
    perm = np.random.default_rng(1).permutation(128)
    y = np.random.default_rng(2).standard_normal((5, 128))
    got = B.back_turned(y, perm, True)
    assert np.allclose((got * x).sum(-1), (y * (x.astype(float)[:, perm] @ R.hadamard(128))).sum(-1))


# ---------------------------------------------------------------- the kernels
def _rotated(t, which):
    """Per sequence: records (y, magnitudes) [n, H, D] of keys or values."""
    d, p = (t.dv, t.packs[1]) if which else (t.dk, t.packs[0])
    b, D = t.b, t.D
    codes, sz = p.codes.cpu().numpy(), p.scale_zero.cpu().numpy()
    out = []
    for s in range(len(b.ctx)):
        n = b.ctx[s] + b.new[s]
        pages = np.array(b.m["block_table"][s][:-(-n // b.ps)], dtype=int)
        c = codes[pages].transpose(0, 2, 1, 3).reshape(-1, t.H, D * d.bits // 8)[:n]
        f = sz[pages].transpose(0, 2, 1, 3, 4).reshape(-1, t.H, D // d.group, 2)[:n].view(np.float16).astype(float)
        cs = R.unpack(c, D, d.bits).reshape(n, t.H, D // d.group, d.group) * f[..., :1]
        out.append(((cs + f[..., 1:]).reshape(n, t.H, D), (np.abs(cs) + np.abs(f[..., 1:])).reshape(n, t.H, D)))
    return out


def _check(t, few, max_rows=1 << 30):
    """The kernel's output against its bound; returns the worst share of it."""
    got = t.out.double().cpu().numpy()
    q16 = t.q.cpu().numpy()
    keys, values = _rotated(t, 0), _rotated(t, 1)
    g, a, worst, rot = t.Hq // t.H, 0, 0.0, t.rot == "fwht_head"
    perm = [None if tb.perm is None else tb.perm.cpu().numpy().astype(int) for tb in (t.tk, t.tv)]
    for s in range(len(t.b.ctx)):
        ctx, m = t.b.ctx[s], t.b.new[s]
        n, e = ctx + m, min(m, max_rows)
        if e:
            k = min(n, t.n_sink)
            rows = [np.zeros((0, t.H, t.D))] * 2
            if k:
                rows = [p.sink.double().cpu().numpy()[(s + 1) % p.sink.shape[0], :, :k].transpose(1, 0, 2) for p in t.packs]
                if t.rope:
                    cs = t.tk.rope_cs.cpu().numpy()
                    rows[0] = np.stack([R.rope(rows[0][i], i, t.rope, cs) for i in range(k)])
            seen = np.arange(n)[None] <= ctx + np.arange(e)[:, None]
            for h in range(t.Hq):
                j = h // g
                pk, pv = (None if x is None else x[j] for x in perm)
                head = B.Head(rows[0][:, j], rows[1][:, j], keys[s][0][k:, j], values[s][0][k:, j], keys[s][1][k:, j],
                              values[s][1][k:, j], pv, rot, few)
                q = q16[a:a + e, h]
                o, tol = head.attend(q.astype(float), B.query_rows(q, pk, rot, few), seen, t.scale)
                err = np.linalg.norm(got[a:a + e, h] - o, axis=1)
                assert np.isfinite(err).all(), f"sequence {s}, head {h}: not finite"
                worst = max(worst, (err / tol).max())
            assert (got[a + e:a + m] == 7.0).all()
        a += m
    assert (got[a:] == 7.0).all()
    assert worst <= 1.0, f"error is {worst} of its bound"
    return worst


def _parts(t, max_rows, max_kv):
    """Partial results a row, from the size of the workspace: 4 D + 8 bytes each, of every row and query head."""
    nb = TA.attend_paged_workspace(t.dk, t.dv, t.Hq, t.b.p, max_rows, max_kv).numel()
    return nb // (t.b.n * t.Hq * (4 * t.D + 8))


FEW = dict(g128=(2, 128), g64=(2, 64), g32=(2, 32), b4=(4, 128), b4_g64=(4, 64), b4_g32=(4, 32))


@gpu
@pytest.mark.parametrize("name", FEW)
@pytest.mark.parametrize("ctx,new,Hq,rope,perm,n_sink,rot,ps,parts", [
    ([0, 1, 15, 16, 17, 200], [1] * 6, 4, 1, False, 4, "fwht_head", 16, 4),      # one column tile, one stretch
    ([700, 3, 513], [2, 1, 2], 4, 2, True, 1, "fwht_head", 48, 8),              # two rows each, two stretches
    ([300, 900], [4, 3], 4, 1, True, 2, "fwht_head", 7, 8),                     # 5 to 8 rows: two column tiles
    ([2900], [1], 16, 1, True, 4, "fwht_head", 64, 20),                         # eight rows of one token, many stretches
    ([5000, 4000], [1, 1], 8, 0, False, 0, "none", 128, 36),                    # the join of many parts
], ids=["one", "two_rows", "two_tiles", "eight_rows", "many_parts"])
def test_few_rows(name, ctx, new, Hq, rope, perm, n_sink, rot, ps, parts):
    from test_paged import Attend
    t = Attend(ctx, new, Hq, 2, 128, *FEW[name], rope, perm, n_sink, rot, ps, 2, seed=len(name))
    mk = max(c + n for c, n in zip(ctx, new))
    assert max(new) * Hq // 2 <= 8 and _parts(t, max(new), mk) >= parts
    t.call()()
    assert K.kvq_check(0) == K.KVQ_OK
    _check(t, True)


TILES = [
    # name, ctx, new, Hq, H, D, bits, group, rope, perm, sinks, rot, page, extra, partial results at least
    ("one_slot_bits3", [0, 1, 127, 128, 300], [1, 1, 2, 1, 3], 8, 2, 128, 3, 32, 1, False, 4, "fwht_head", 16, 1, 2),
    ("one_slot_d64", [700, 30], [1, 8], 8, 2, 64, 2, 64, 2, True, 3, "fwht_head", 48, 0, 4),
    ("one_slot_wide_join", [3000], [20], 4, 1, 128, 4, 128, 1, True, 2, "fwht_head", 64, 3, 10),
    ("one_slot_ragged", [2600, 0, 40], [9, 17, 1], 4, 1, 128, 2, 32, 1, False, 0, "none", 24, 2, 10),
    ("two_slots", [200, 0], [100, 64], 8, 2, 128, 2, 128, 1, False, 4, "fwht_head", 64, 0, 1),
    ("two_slots_stretches", [1900], [90], 4, 1, 128, 4, 64, 2, True, 4, "fwht_head", 48, 1, 3),
    ("two_slots_wide_join", [4800], [33], 4, 1, 128, 2, 128, 1, False, 2, "fwht_head", 16, 0, 9),
    ("two_slots_d64", [1300], [70], 4, 1, 64, 3, 32, 1, True, 0, "fwht_head", 7, 2, 3),
    ("two_slots_mha", [1500], [300], 1, 1, 128, 4, 128, 0, False, 0, "none", 128, 0, 3),
    ("tokens_beside_a_chunk", [0, 900, 33, 1400, 7, 100], [1, 1, 60, 1, 1, 2], 8, 2, 128, 2, 128, 1, False, 4, "fwht_head", 32, 4, 2),
    ("forty_sequences", [(37 * i) % 211 for i in range(40)], [1 + (5 * i) % 7 for i in range(40)], 4, 1, 128, 3, 64, 1, True, 4, "fwht_head", 16, 5, 2),
    ("forty_with_chunks", [(53 * i) % 190 for i in range(40)], [(11 * i) % 45 for i in range(40)], 8, 2, 64, 4, 32, 2, False, 1, "fwht_head", 16, 0, 1),
]


@gpu
@pytest.mark.parametrize("case", TILES, ids=[c[0] for c in TILES])
def test_tiles(case):
    from test_paged import Attend
    t = Attend(*case[1:14], seed=len(case[0]))
    ctx, new, g, T = case[1], case[2], case[3] // case[4], 128 // (case[3] // case[4])
    mk = max(c + n for c, n in zip(ctx, new))
    assert max(new) * g > 8 or case[6] == 3 or case[5] == 64
    assert (max(new) > T) == ("one_slot" not in case[0] and "forty_sequences" != case[0])
    assert _parts(t, max(new), mk) >= case[14]
    t.call()()
    assert K.kvq_check(0) == K.KVQ_OK
    _check(t, False)
    first = t.out.clone()
    t.out.fill_(7.0)
    t.call()()
    assert torch.equal(t.out, first)


@gpu
@pytest.mark.parametrize("few", [True, False], ids=["few", "tiles"])
def test_bounds_of_the_lengths_that_are_too_small(few):
    """The last stretch takes all that the bound left out."""
    from test_paged import Attend
    for max_kv in (0, 1, 600, 1 << 20):
        t = Attend([2000, 30], [2, 1] if few else [50, 3], 4, 1, 128, 2, 128, 1, False, 4, "fwht_head", 16, seed=3)
        t.call(max_kv=max_kv)()
        assert K.kvq_check(0) == K.KVQ_OK
        _check(t, few)


@gpu
def test_rows_beyond_max_rows():
    from test_paged import Attend
    t = Attend([1200, 0], [60, 9], 8, 2, 128, 2, 128, 1, False, 4, "fwht_head", 16)
    t.call(max_rows=33)()
    _check(t, False, max_rows=33)
    u = Attend([1200, 0], [6, 9], 8, 2, 128, 2, 128, 1, False, 4, "fwht_head", 16)
    u.call(max_rows=2)()
    _check(u, True, max_rows=2)


# ---------------------------------------------------------------- together
@gpu
@pytest.mark.parametrize("bits,group,n_sink,perm", [(2, 128, 4, True), (4, 64, 0, False), (3, 32, 1, True)])
def test_a_serving_run_within_its_roundings(bits, group, n_sink, perm):
    """Prompts, chunks, single tokens beside a chunk, idle steps: pages by kvq_page_map, records by kvq_encode_paged, and
    each step's attention against the records that are in the pool."""
    from types import SimpleNamespace

    from test_paged import _poison, _tables
    Hq, H, D, ps, S, P = 8, 2, 128, 16, 3, 60
    common = dict(batch=P, heads=H, head_dim=D, tokens=0, t_cap=ps, bits=bits, group=group, n_sink=n_sink, rot="fwht_head")
    dk, dv = TA.make_desc(rope=1, **common), TA.make_desc(rope=0, **common)
    tk, tv = _tables(D, H, 1, perm, 512, 5), _tables(D, H, 0, perm, 512, 6)
    kc, vc = TA.alloc_paged(dk, S + 2), TA.alloc_paged(dv, S + 2)
    _poison(kc), _poison(vc)
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    free, used = torch.randperm(P, device="cuda", generator=g).to(torch.int32), torch.zeros(1, **i32)
    table, ctx, sinks = torch.full((S, 24), -1, **i32), [0] * S, torch.tensor([1, 2, 3], **i32)
    shares = []
    for new in ([50, 33, 0], [1, 1, 120], [20, 1, 1], [1, 1, 1], [0, 0, 0], [1, 0, 2], [2, 70, 1], [1, 1, 1]):
        n = sum(new)
        b = TA.make_paged(S, n + 2, 24, block_table=table, sink_slot=sinks)
        rep = TA.page_map(dk, b, torch.tensor(ctx, **i32), torch.tensor(new, **i32), free, used)
        x = torch.randn(n + 2, Hq + 2 * H, D, device="cuda", generator=g).half()
        q, k, v = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
        TA.encode_paged(dk, k, b, tk, kc)
        TA.encode_paged(dv, v, b, tv, vc)
        out = torch.full((n + 2, Hq, D), 7.0, dtype=torch.float16, device="cuda")
        mr, mk = max(new), max(c + m for c, m in zip(ctx, new))
        TA.attend_paged(dk, dv, q, kc, tk, vc, tv, b, mr, mk, D ** -0.5, out, TA.attend_paged_workspace(dk, dv, Hq, b, mr, mk))
        assert K.kvq_check(0) == K.KVQ_OK and rep.tolist()[0] == n and rep.tolist()[2:] == [0, 0]
        t = SimpleNamespace(Hq=Hq, H=H, D=D, n_sink=n_sink, rope=1, rot="fwht_head", dk=dk, dv=dv, tk=tk, tv=tv, packs=[kc, vc], q=q,
                            out=out, scale=D ** -0.5, b=SimpleNamespace(ctx=ctx, new=new, ps=ps, m=dict(block_table=table.tolist())))
        shares.append(_check(t, mr * Hq // H <= 8 and bits != 3))
        ctx, used = [c + m for c, m in zip(ctx, new)], rep[1:2].clone()
    assert max(shares) <= 1.0
    held = table[table >= 0].tolist()
    assert len(set(held)) == len(held) == sum(-(-c // ps) for c in ctx)


# ---------------------------------------------------------------- records and queries of other sizes
def _flat(sz, r):
    sz[..., 0] = 0.0


def _some_flat(sz, r):
    sz[..., 0] *= (r < 0.5)


def _some_zero(sz, r):
    sz *= (r < 0.5)[..., None]


def _wide(sz, r):
    sz *= (2.0 ** torch.floor(r * 16 - 8))[..., None]


KINDS = dict(flat=_flat, some_flat=_some_flat, some_zero=_some_zero, wide=_wide, peaked=None, tiny_queries=None, large_queries=None)


@gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new,bits,group,few", [([1, 2], 2, 128, True), ([2, 2], 4, 32, True), ([17, 1], 3, 64, False), ([70, 3], 2, 64, False)],
                         ids=["few", "few_g32", "one_slot", "two_slots"])
def test_records_and_queries_of_all_sizes(new, bits, group, few, kind):
    """Groups without a range (a token of zeros, of equal values), ranges from 2^-8 to 2^7 of the usual, scores far apart,
    queries near fp16's ends: in keys, values and both."""
    from test_paged import Attend
    for which in ((0,), (1,), (0, 1)) if KINDS[kind] else ((),):
        t = Attend([900, 60], new, 4, 1, 128, bits, group, 1, True, 2, "fwht_head", 16, 1, seed=len(kind))
        g = torch.Generator(device="cuda").manual_seed(4)
        for i in which:
            sz = t.packs[i].scale_zero.view(torch.float16)
            x = sz.float()
            KINDS[kind](x, torch.rand(x.shape[:-1], device="cuda", generator=g))
            sz.copy_(torch.where(torch.isnan(sz), sz, x.half()))
        if not which:
            t.q.mul_({"peaked": 20.0, "tiny_queries": 2.0 ** -14, "large_queries": 2000.0}[kind])
            t.scale *= {"peaked": 1.0, "tiny_queries": 2.0 ** 14, "large_queries": 0.001}[kind]
        t.call()()
        assert K.kvq_check(0) == K.KVQ_OK
        _check(t, few)


@gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("new,Hq,bits,n_sink", [([1, 3], 2, 2, 4), ([4, 1], 4, 4, 0), ([20, 9], 8, 3, 1), ([200, 70], 8, 2, 4)],
                         ids=["few", "few_two", "one_slot", "two_slots"])
def test_a_query_row_that_is_not_finite_touches_no_other(new, Hq, bits, n_sink, bad):
    from test_paged import Attend
    t = Attend([300, 40], new, Hq, 2, 128, bits, 128, 1, False, n_sink, "fwht_head", 16)
    t.call()()
    clean = t.out.clone()
    row, head = new[0] - 1, Hq - 1
    t.q[row, head, 5] = bad
    t.out.fill_(7.0)
    t.call()()
    assert K.kvq_check(0) == K.KVQ_OK
    assert not torch.isfinite(t.out[row, head]).any()
    clean[row, head] = 0.0
    t.out[row, head] = 0.0
    assert torch.equal(t.out, clean)


# ---------------------------------------------------------------- shapes between the listed ones
@gpu
@pytest.mark.parametrize("Hq,H,new,ps,bits,group", [
    (3, 1, [1, 2, 1], 100, 2, 128), (9, 3, [2, 0, 1], 16, 4, 64), (10, 2, [1, 1, 0], 5, 2, 32), (7, 1, [1, 1, 1], 33, 4, 128),
    (6, 6, [8, 3, 5], 64, 2, 64), (5, 5, [7, 0, 1], 1, 4, 32), (12, 2, [1, 1, 1], 512, 2, 128)])
def test_few_rows_of_odd_groups_and_pages(Hq, H, new, ps, bits, group):
    from test_paged import Attend
    t = Attend([333, 0, 1100], new, Hq, H, 128, bits, group, 1, True, 3, "fwht_head", ps, 1, seed=Hq)
    t.call()()
    assert K.kvq_check(0) == K.KVQ_OK
    _check(t, True)


@gpu
def test_few_rows_of_many_sequences():
    from test_paged import Attend
    ctx = [(71 * i) % 400 for i in range(300)]
    t = Attend(ctx, [(i % 7 != 3) * 1 for i in range(300)], 4, 1, 128, 2, 128, 1, False, 2, "fwht_head", 16, 3)
    t.call()()
    assert K.kvq_check(0) == K.KVQ_OK
    _check(t, True)


@gpu
@pytest.mark.parametrize("Hq,H,new,ps", [(3, 1, [50, 9], 100), (10, 2, [13, 40], 33), (5, 1, [26, 1], 7), (11, 1, [12, 30], 512)])
def test_tiles_of_odd_groups_and_pages(Hq, H, new, ps):
    from test_paged import Attend
    for bits, group, D in ((4, 64, 128), (3, 32, 64)):
        t = Attend([333, 1100], new, Hq, H, D, bits, group, 2, True, 3, "fwht_head", ps, 1, seed=Hq)
        t.call()()
        assert K.kvq_check(0) == K.KVQ_OK
        _check(t, False)
