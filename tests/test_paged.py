"""The paged cache: page map, encode and decode of packed rows, attention of
new rows over pages, a run of them together, and their refusals."""
import math
import random

import numpy as np
import pytest

import paged_ref as R

torch = pytest.importorskip("torch")
import kv_cache_rotation_b200 as K  # noqa: E402
from kv_cache_rotation_b200 import torch_api as TA  # noqa: E402

gpu = pytest.mark.gpu
INV, UNS, ALI, OK = K.KVQ_ERR_INVALID, K.KVQ_ERR_UNSUPPORTED, K.KVQ_ERR_ALIGN, K.KVQ_OK


# ---------------------------------------------------------------- refusals (no GPU)
def _d(**kw):
    a = dict(batch=16, heads=2, head_dim=128, tokens=0, t_cap=32, bits=2, group=128, rope=0, n_sink=0)
    a.update(kw)
    return TA.make_desc(**a)


def _pg(**kw):
    p = K.kvq_paged()
    a = dict(n_seqs=2, n_rows=8, max_pages=4, sink_rows=0, cu_rows=4096, kv_len=4096, block_table=4096, seq=4096,
             pos=4096, slot=4096, sink_slot=None)
    a.update(kw)
    for n, v in a.items():
        setattr(p, n, v)
    return p


def _pk(**kw):
    p = K.kvq_packed()
    p.codes = p.scale_zero = 4096
    for n, v in kw.items():
        setattr(p, n, v)
    return p


def _tb(**kw):
    t = K.kvq_tables()
    for n, v in kw.items():
        setattr(t, n, v)
    return t


@pytest.mark.parametrize("d,pg,kw,status", [
    ({}, dict(n_rows=-1), {}, INV), ({}, dict(n_seqs=-1), {}, INV), ({}, dict(max_pages=0), {}, INV),
    (dict(batch=0), {}, {}, INV), (dict(rot="iso", quant="codebook"), {}, {}, UNS),
    (dict(rot="fwht_group", group_heads=2), {}, {}, UNS), (dict(batch=1 << 20, t_cap=1 << 11, heads=1), {}, {}, UNS),
    ({}, dict(n_seqs=16385), {}, UNS), ({}, dict(cu_rows=None), {}, INV), ({}, dict(kv_len=None), {}, INV),
    ({}, dict(block_table=None), {}, INV), ({}, dict(seq=None), {}, INV), ({}, dict(slot=4100), {}, ALI),
    ({}, dict(pos=4104), {}, ALI), ({}, dict(kv_len=4097), {}, ALI), ({}, {}, dict(ctx=None), INV), ({}, {}, dict(new=None), INV),
    ({}, {}, dict(free=None), INV), ({}, {}, dict(n_free=-1), INV), ({}, {}, dict(used=None), INV),
    ({}, {}, dict(report=None), INV), ({}, {}, dict(report=8192), INV), ({}, {}, dict(report=4098), ALI),
])
def test_page_map_refusals(d, pg, kw, status):
    a = dict(ctx=4096, new=4096, free=4096, n_free=8, used=8192, report=4096)
    a.update(kw)
    assert K.kvq_page_map(_d(**d), _pg(**pg), *a.values()) == status


@pytest.mark.parametrize("d,pg,pk,tb,kw,status", [
    (dict(batch=0), {}, {}, {}, {}, INV), (dict(rot="iso", quant="codebook"), {}, {}, {}, {}, UNS),
    ({}, dict(n_rows=-1), {}, {}, {}, INV), ({}, dict(n_rows=1 << 30), {}, {}, {}, UNS),
    ({}, dict(pos=None), {}, {}, {}, INV), ({}, dict(slot=None), {}, {}, {}, INV), ({}, dict(slot=4104), {}, {}, {}, ALI),
    ({}, {}, dict(codes=None), {}, {}, INV), ({}, {}, dict(codes=4104), {}, {}, ALI), ({}, {}, dict(scale_zero=None), {}, {}, INV),
    ({}, {}, {}, {}, dict(x=None), INV), ({}, {}, {}, {}, dict(x=4104), ALI), ({}, {}, {}, {}, dict(stride=248), INV),
    ({}, {}, {}, {}, dict(stride=260), ALI), (dict(rope=1), {}, {}, {}, {}, INV),
    (dict(rope=1), {}, {}, dict(rope_cs=4100, rope_rows=8), {}, ALI), ({}, {}, {}, dict(perm=4104), {}, ALI),
    (dict(n_sink=4), {}, dict(sink=4096), {}, {}, INV),                       # no sequence has a sink row
    (dict(n_sink=4), dict(sink_rows=2), {}, {}, {}, INV),                     # sinks need a buffer
    (dict(n_sink=4), dict(sink_rows=2, seq=None), dict(sink=4096), {}, {}, INV),
    (dict(n_sink=4), dict(sink_rows=2), dict(sink=4096), dict(sink_pos=4096), {}, UNS),
    (dict(n_sink=4), dict(sink_rows=2, sink_slot=4098), dict(sink=4096), {}, {}, ALI),
    ({}, dict(n_rows=0), {}, {}, {}, OK),
])
def test_encode_decode_paged_refusals(d, pg, pk, tb, kw, status):
    a = dict(x=4096, stride=256)
    a.update(kw)
    dd, p, c, t = _d(**d), _pg(**pg), _pk(**pk), _tb(**tb)
    assert K.kvq_encode_paged(dd, a["x"], a["stride"], p, t, c) == status
    assert K.kvq_decode_paged(dd, c, p, t, a["x"], a["stride"], 0) == status
    assert K.kvq_decode_paged(_d(), _pk(), _pg(), _tb(), 4096, 256, 2) == INV


@pytest.mark.parametrize("dk,dv,pg,kw,status", [
    (dict(batch=0), {}, {}, {}, INV), ({}, dict(rope=1), {}, {}, UNS), ({}, dict(bits=4), {}, {}, INV),
    ({}, dict(batch=8), {}, {}, INV), ({}, dict(t_cap=16), {}, {}, INV), ({}, dict(group=64), {}, {}, INV),
    ({}, dict(n_sink=2), {}, {}, INV), (dict(rot="iso", quant="codebook"), {}, {}, {}, UNS),
    ({}, {}, dict(n_rows=-1), {}, INV), ({}, {}, dict(kv_len=None), {}, INV), ({}, {}, dict(cu_rows=None), {}, INV),
    ({}, {}, dict(block_table=None), {}, INV), ({}, {}, dict(cu_rows=4098), {}, ALI),
    ({}, {}, {}, dict(hq=0), INV), ({}, {}, {}, dict(hq=7), INV), ({}, {}, {}, dict(hq=258, qs=258 * 128, os=258 * 128), UNS),
    ({}, {}, {}, dict(q=None), INV), ({}, {}, {}, dict(out=None), INV), ({}, {}, {}, dict(ws=None), INV),
    ({}, {}, {}, dict(q=4104), ALI), ({}, {}, {}, dict(out=4098), ALI), ({}, {}, {}, dict(ws=4160), ALI),
    ({}, {}, {}, dict(qs=1016), INV), ({}, {}, {}, dict(os=1016), INV), ({}, {}, {}, dict(qs=1028), ALI),
    ({}, {}, {}, dict(mr=-1), INV), ({}, {}, {}, dict(mk=-1), INV), ({}, {}, {}, dict(wb=0), INV),
    ({}, {}, {}, dict(scale=0.0), INV), ({}, {}, {}, dict(scale=math.inf), INV), ({}, {}, {}, dict(scale=math.nan), INV),
    ({}, {}, dict(n_rows=0), {}, OK), ({}, {}, dict(n_seqs=0), {}, OK), ({}, {}, {}, dict(mr=0), OK),
])
def test_attend_paged_refusals(dk, dv, pg, kw, status):
    a = dict(q=4096, qs=1024, hq=8, mr=8, mk=100, scale=0.1, out=4096, os=1024, ws=4096, wb=1 << 40)
    a.update(kw)
    assert K.kvq_attend_paged(_d(**dk), _d(**{**dk, **dv}), a["q"], a["qs"], a["hq"], _pk(), _tb(), _pk(), _tb(),
                              _pg(**pg), a["mr"], a["mk"], a["scale"], a["out"], a["os"], a["ws"], a["wb"]) == status


def test_attend_paged_workspace_is_enough_only_whole():
    d, p = _d(), _pg(n_seqs=64, n_rows=64)
    n = K.kvq_attend_paged_workspace_bytes(d, d, 8, p, 1, 5000)
    assert n > 0
    assert K.kvq_attend_paged(d, d, 4096, 1024, 8, _pk(), _tb(), _pk(), _tb(), p, 1, 5000, 0.1, 4096, 1024, 4096,
                              n - 1) == INV
    assert K.kvq_attend_paged_workspace_bytes(d, d, 7, p, 1, 5000) == 0
    assert K.kvq_attend_paged_workspace_bytes(d, _d(rope=1), 8, p, 1, 5000) == 0


def test_paged_struct_refuses_arrays_that_do_not_fit():
    with pytest.raises(ValueError):  # on the host
        TA.Paged(kv_len=torch.zeros(3, dtype=torch.int32)).struct()


# ---------------------------------------------------------------- page map
@gpu
@pytest.mark.parametrize("S,ps,width,lo,hi,nlo,nhi,pool,used,extra", [
    (1, 16, 4, 0, 0, 1, 1, 1, 0, 0), (5, 16, 12, 0, 90, 0, 60, 40, 3, 7), (64, 64, 40, 0, 2000, 1, 1, 200, 0, 0),
    (64, 1, 90, 0, 50, 0, 30, 3000, 5, 3), (700, 48, 20, 0, 700, -3, 90, 4000, 0, -100),
    (9, 16, 12, 0, 90, 0, 60, 5, 2, 1),          # the pool runs out
    (9, 16, 3, 0, 90, 0, 60, 90, 0, 2),          # the table is too short
    (3, 16, 8, 0, 90, 0, 20, 0, 0, 2),           # an empty pool
    (1000, 128, 2, 0, 0, 0, 3, 2000, 0, 40), (1030, 16, 4, -5, 30, 0, 1, 2000, 9, 5)])
def test_page_map(S, ps, width, lo, hi, nlo, nhi, pool, used, extra):
    r = random.Random(S * 7919 + ps)
    ctx, new = [r.randint(lo, hi) for _ in range(S)], [r.randint(nlo, nhi) for _ in range(S)]
    n_pages = pool + 6000
    pages = r.sample(range(n_pages), n_pages)
    free, other = pages[:pool], pages[pool:]
    table = [[-7] * width for _ in range(S)]
    for s in range(S):
        for k in range(min(width, -(-max(0, ctx[s]) // ps))):
            table[s][k] = other.pop() if other else 0
    n_rows = max(0, sum(max(0, n) for n in new) + extra)
    want = R.page_map(S, n_rows, width, ps, n_pages, ctx, new, table, free, used)
    i32 = dict(dtype=torch.int32, device="cuda")
    b = TA.make_paged(S, n_rows, width, block_table=torch.tensor(table, **i32))
    rep = TA.page_map(_d(batch=n_pages, t_cap=ps), b, torch.tensor(ctx, **i32), torch.tensor(new, **i32),
                      torch.tensor(free, **i32), torch.tensor([used], **i32))
    assert K.kvq_check(0) == OK
    for name in ("cu_rows", "kv_len", "block_table", "seq", "pos", "slot"):
        assert getattr(b, name).tolist() == want[name], name
    assert rep.tolist() == want["report"]


@gpu
def test_page_map_no_sequences_and_far_lengths():
    i32 = dict(dtype=torch.int32, device="cuda")
    b = TA.make_paged(0, 5, 1)
    rep = TA.page_map(_d(), b, torch.empty(0, **i32), torch.empty(0, **i32), torch.arange(3, **i32),
                      torch.tensor([1], **i32))
    assert rep.tolist() == [0, 1, 0, 0] and b.cu_rows.tolist() == [0] and b.slot.tolist() == [-1] * 5
    top = (1 << 31) - 1
    b = TA.make_paged(3, 8, 2)
    rep = TA.page_map(_d(), b, torch.tensor([top, 0, -9], **i32), torch.tensor([top, top, top], **i32),
                      torch.arange(3, **i32), torch.tensor([0], **i32))
    assert K.kvq_check(0) == OK
    assert b.cu_rows.tolist() == [0, top, top, top] and b.kv_len.tolist() == [top] * 3
    assert b.slot.tolist() == [-1] * 8
    # sequence 1 lacks 2 pages of its table, sequence 2 as many: 3 are there
    assert rep.tolist()[:2] == [top, 3] and rep.tolist()[3] == 1


# ---------------------------------------------------------------- encode / decode
ROWS = [
    # name, D, bits, group, rope, perm, n_sink, rot, H, page size
    ("g128", 128, 2, 128, 1, False, 0, "fwht_head", 2, 16), ("g64_perm_sinks", 128, 2, 64, 1, True, 4, "fwht_head", 3, 48),
    ("g32_bits3", 128, 3, 32, 2, True, 1, "fwht_head", 2, 1), ("bits3_g128", 128, 3, 128, 0, False, 0, "fwht_head", 1, 7),
    ("bits4", 128, 4, 128, 2, False, 5, "fwht_head", 4, 64), ("bits4_g32", 128, 4, 32, 0, True, 0, "fwht_head", 2, 16),
    ("none", 128, 4, 64, 1, False, 2, "none", 2, 16), ("d64", 64, 2, 64, 1, True, 3, "fwht_head", 5, 16),
    ("d64_bits3", 64, 3, 32, 2, False, 0, "fwht_head", 8, 32), ("d64_bits4", 64, 4, 32, 2, True, 1, "fwht_head", 1, 16),
]
LENS = ([0, 3, 40, 17, 2], [5, 0, 33, 64, 1])  # cached and new tokens


class Batch:
    """Sequences over a shuffled pool, their maps by the plain form, on the device."""

    def __init__(self, ctx, new, ps, extra=0, seed=0, spare=3, width=None):
        r = random.Random(seed)
        S = len(ctx)
        need = [-(-(c + n) // ps) for c, n in zip(ctx, new)]
        self.pages = sum(need) + spare
        self.width = width or max(need + [1])
        pool = r.sample(range(self.pages), self.pages)
        table = [[-1] * self.width for _ in range(S)]
        for s in range(S):
            for k in range(-(-ctx[s] // ps)):
                table[s][k] = pool.pop()
        self.ctx, self.new, self.ps = ctx, new, ps
        self.n = sum(new) + extra
        self.m = R.page_map(S, self.n, self.width, ps, self.pages, ctx, new, table, pool, 0)
        t = {k: torch.tensor(v, dtype=torch.int32, device="cuda").reshape(S, -1) if k == "block_table" else
             torch.tensor(v, dtype=torch.int32, device="cuda") for k, v in self.m.items() if k != "report"}
        self.p = TA.Paged(**t)


def _tables(D, H, rope, perm, rows, seed):
    g = torch.Generator().manual_seed(seed)
    t = TA.make_tables()
    if rope:
        t.rope_cs = TA.rope_table(rows, D)
    if perm:
        t.perm = torch.stack([torch.randperm(D, generator=g) for _ in range(H)]).to(torch.int16).cuda()
    return t


def _poison(pk):
    """A pool whose unwritten records are codes of ones and NaN scales."""
    pk.codes.fill_(0xff)
    pk.scale_zero.fill_(0x7e01)
    if pk.sink is not None:
        pk.sink.fill_(math.nan)


@gpu
@pytest.mark.parametrize("name,D,bits,group,rope,perm,n_sink,rot,H,ps", ROWS, ids=[c[0] for c in ROWS])
def test_encode_and_decode_paged_match_the_dense_cache(name, D, bits, group, rope, perm, n_sink, rot, H, ps):
    ctx, new = LENS
    b = Batch(ctx, new, ps, extra=4)
    g = torch.Generator().manual_seed(11)
    wide = torch.randn(b.n, 2 * H, D, generator=g)
    wide[:, :, ::17] *= 20.0
    wide = wide.half().cuda()
    x = wide[:, H // 2:H // 2 + H]  # rows of a wider projection
    d = _d(batch=b.pages, heads=H, head_dim=D, t_cap=ps, bits=bits, group=group, rope=rope, n_sink=n_sink, rot=rot)
    tb = _tables(D, H, rope, perm, 200, 3)
    S = len(ctx)
    b.p.sink_slot = torch.tensor([(s + 2) % (S + 1) for s in range(S)], dtype=torch.int32, device="cuda")
    pk = TA.alloc_paged(d, sink_rows=S + 1)
    _poison(pk)
    before = [t.clone() for t in (pk.codes, pk.scale_zero)]
    TA.encode_paged(d, x, b.p, tb, pk)
    out = torch.full((b.n, H, D), 7.0, dtype=torch.float32, device="cuda")
    half = torch.full((b.n, H + 1, D), 7.0, dtype=torch.float16, device="cuda")
    TA.decode_paged(d, pk, b.p, tb, out)
    TA.decode_paged(d, pk, b.p, tb, half[:, :H])
    assert K.kvq_check(0) == OK
    flat_c, flat_z = pk.codes.transpose(1, 2).flatten(0, 1), pk.scale_zero.transpose(1, 2).flatten(0, 1)
    written = torch.zeros(b.pages * ps, dtype=torch.bool, device="cuda")
    for s in range(S):
        a, e = b.m["cu_rows"][s], b.m["cu_rows"][s + 1]
        if a == e:
            continue
        slots = torch.tensor(b.m["slot"][a:e], device="cuda")
        written[slots] = True
        dd = TA.make_desc(batch=1, heads=H, head_dim=D, tokens=e - a, t0=ctx[s], t_cap=ctx[s] + e - a, bits=bits,
                          group=group, rope=rope, n_sink=n_sink, rot=rot)
        ref = TA.alloc_packed(dd)
        TA.encode(dd, x[a:e].transpose(0, 1).unsqueeze(0).contiguous(), tb, ref)
        assert torch.equal(flat_c[slots], ref.codes[0, :, ctx[s]:].transpose(0, 1))
        assert torch.equal(flat_z[slots], ref.scale_zero[0, :, ctx[s]:].transpose(0, 1))
        back = torch.empty(1, H, e - a, D, dtype=torch.float32, device="cuda")
        TA.decode(dd, ref, tb, back)
        back = back[0].transpose(0, 1)
        # both undo the transform in fp32: log2(D) sums, a product and a turn, each 2^-24 of the row's 2-norm
        tol = 16 * 2.0 ** -24 * back.norm(dim=-1, keepdim=True) + 2.0 ** -24
        assert ((out[a:e] - back).abs() <= tol).all()
        assert ((half[a:e, :H].float() - back).abs() <= tol + back.abs() * R.U16).all()
        m = min(n_sink, ctx[s] + e - a)
        if m > ctx[s]:
            assert torch.equal(pk.sink[(s + 2) % (S + 1), :, ctx[s]:m], ref.sink[0, :, ctx[s]:m])
            assert torch.equal(half[a:a + m - ctx[s], :H], x[a:a + m - ctx[s]])
    total = b.m["cu_rows"][-1]
    assert (out[total:] == 7.0).all() and (half[total:] == 7.0).all() and (half[:, H] == 7.0).all()
    keep_c, keep_z = (t.transpose(1, 2).flatten(0, 1)[~written] for t in before)
    assert torch.equal(flat_c[~written], keep_c) and torch.equal(flat_z[~written], keep_z)


@gpu
def test_rows_that_have_no_place_are_skipped():
    b = Batch([0], [8], 4)
    d = _d(batch=b.pages, heads=2, t_cap=4, rope=1, n_sink=2)
    tb = _tables(128, 2, 1, False, 6, 0)  # positions 6 and 7 have no RoPE row
    x = torch.randn(8, 2, 128, device="cuda").half()
    b.p.slot[3], b.p.slot[4], b.p.pos[5] = b.pages * 4, -5, -1
    b.p.seq[0] = 9  # a sink position of a sequence that is not there
    pk = TA.alloc_paged(d, sink_rows=1)
    TA.encode_paged(d, x, b.p, tb, pk)
    out = torch.full((8, 2, 128), 7.0, dtype=torch.float16, device="cuda")
    TA.decode_paged(d, pk, b.p, tb, out)
    assert K.kvq_check(0) == OK
    kept = [r for r in range(8) if (out[r] == 7.0).all()]
    assert kept == [0, 3, 4, 5, 6, 7]
    assert torch.equal(out[1], x[1])


# ---------------------------------------------------------------- attention over pages
ATT = [
    # name, ctx, new, Hq, H, D, bits, group, rope, perm, n_sink, rot, page size, extra rows
    ("decode", [0, 1, 127, 128, 300], [1] * 5, 8, 2, 128, 2, 128, 1, False, 4, "fwht_head", 16, 0),
    ("decode_mha_g64", [50, 700], [1, 1], 3, 3, 128, 2, 64, 1, True, 4, "fwht_head", 48, 2),
    ("decode_bits3", [5, 260, 513], [1, 1, 1], 8, 1, 128, 3, 32, 2, True, 0, "fwht_head", 7, 0),
    ("decode_bits4", [64, 129], [1, 1], 8, 2, 128, 4, 128, 1, False, 1, "fwht_head", 64, 0),
    ("decode_none", [33, 257], [1, 1], 4, 2, 128, 4, 64, 1, False, 2, "none", 32, 0),
    ("decode_d64", [33, 257], [1, 1], 10, 2, 64, 2, 64, 1, True, 3, "fwht_head", 16, 0),
    ("page_of_one", [20, 140], [1, 2], 4, 2, 128, 2, 128, 1, False, 2, "fwht_head", 1, 0),
    ("wide_group", [100], [1], 65, 1, 128, 2, 128, 1, False, 4, "fwht_head", 16, 0),
    ("group_of_128", [130], [2], 128, 1, 64, 4, 32, 1, False, 0, "fwht_head", 16, 0),
    ("chunk", [200], [100], 8, 2, 128, 2, 128, 1, False, 4, "fwht_head", 64, 0),
    ("chunk_from_zero", [0, 0], [130, 33], 8, 2, 128, 4, 64, 2, True, 4, "fwht_head", 16, 3),
    ("chunk_mha", [31], [300], 2, 2, 128, 3, 128, 1, False, 0, "fwht_head", 48, 0),
    ("chunk_d64", [90, 0], [70, 129], 6, 2, 64, 3, 32, 1, True, 2, "fwht_head", 24, 1),
    ("chunk_d64_g64", [400], [65], 2, 2, 64, 4, 64, 0, False, 0, "none", 16, 0),
    ("mixed", [0, 500, 3, 80, 0], [1, 1, 90, 0, 37], 8, 2, 128, 2, 64, 1, False, 4, "fwht_head", 32, 5),
    ("all_sinks", [0, 2], [3, 1], 4, 2, 128, 2, 128, 1, False, 8, "fwht_head", 16, 0),
    ("many_sinks", [0, 200], [40, 1], 4, 2, 128, 2, 128, 2, False, 40, "fwht_head", 16, 0),
    ("long_split", [5000], [1], 4, 1, 128, 2, 128, 1, False, 4, "fwht_head", 64, 0),
]


class Attend:
    """A pool in use: the batch's cached and new records are random, everything else is poison."""

    def __init__(self, ctx, new, Hq, H, D, bits, group, rope, perm, n_sink, rot, ps, extra=0, seed=0):
        self.b = b = Batch(ctx, new, ps, extra, seed)
        S = len(ctx)
        self.Hq, self.H, self.D, self.n_sink, self.rope, self.rot = Hq, H, D, n_sink, rope, rot
        common = dict(batch=b.pages, heads=H, head_dim=D, t_cap=ps, bits=bits, group=group, n_sink=n_sink, rot=rot)
        self.dk, self.dv = _d(rope=rope, **common), _d(rope=0, **common)
        self.tk, self.tv = _tables(D, H, rope, perm, max(n_sink, 1), seed), _tables(D, H, 0, perm, 0, seed + 1)
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.rand(s, device="cuda", generator=g)  # noqa: E731
        self.packs = []
        for d in (self.dk, self.dv):
            p = TA.alloc_paged(d, sink_rows=S + 2)
            _poison(p)
            z = -(1.2 + 0.8 * rnd(*p.scale_zero.shape[:-1]))
            s = (0.9 + 0.2 * rnd(*z.shape)) * (-2 * z / (2 ** bits - 1))
            sz = torch.stack([s.half().view(torch.int16), z.half().view(torch.int16)], -1)
            codes = torch.randint(0, 256, p.codes.shape, device="cuda", generator=g, dtype=torch.uint8)
            live = torch.zeros(b.pages, ps, dtype=torch.bool, device="cuda")
            for q in range(S):
                n = ctx[q] + new[q]
                for k in range(-(-n // ps)):
                    live[b.m["block_table"][q][k], :n - k * ps] = True
                if n_sink:
                    p.sink[(q + 1) % (S + 2), :, :n] = torch.randn(H, min(n, n_sink), D, device="cuda", generator=g).half()
            at = live[:, None].expand(-1, H, -1)
            p.codes[at], p.scale_zero[at] = codes[at], sz[at]
            self.packs.append(p)
        b.p.sink_slot = torch.tensor([(q + 1) % (S + 2) for q in range(S)], dtype=torch.int32, device="cuda")
        self.q = torch.randn(b.n, Hq, D, device="cuda", generator=g).half()
        self.out = torch.full_like(self.q, 7.0)
        self.scale = D ** -0.5

    def call(self, max_rows=None, max_kv=None, ws=None):
        mr = max(self.b.new) if max_rows is None else max_rows
        mk = max(c + n for c, n in zip(self.b.ctx, self.b.new)) if max_kv is None else max_kv
        if ws is None:
            ws = TA.attend_paged_workspace(self.dk, self.dv, self.Hq, self.b.p, mr, mk)
            ws.fill_(0xff)
        return TA.bind_attend_paged(self.dk, self.dv, self.q, self.packs[0], self.tk, self.packs[1], self.tv, self.b.p,
                                    mr, mk, self.scale, self.out, ws)

    def keys(self, s, which):
        """(rows in their own basis, rows as the products take them) [n, H, D] of sequence s."""
        b, p, d = self.b, self.packs[which], self.dv if which else self.dk
        tb = self.tv if which else self.tk
        n, ps, D = b.ctx[s] + b.new[s], b.ps, self.D
        pages = np.array(b.m["block_table"][s][:-(-n // ps)], dtype=int)
        codes = p.codes.cpu().numpy()[pages].transpose(0, 2, 1, 3).reshape(-1, self.H, D * d.bits // 8)[:n]
        sz = p.scale_zero.cpu().numpy()[pages].transpose(0, 2, 1, 3, 4).reshape(-1, self.H, D // d.group, 2)[:n]
        y = R.dequantized(codes, sz, D, d.bits, d.group)
        own = y @ R.hadamard(D) if self.rot == "fwht_head" else y.copy()
        if tb.perm is not None:
            perm = tb.perm.cpu().numpy().astype(int)
            for h in range(self.H):
                back = np.empty_like(own[:, h])
                back[:, perm[h]] = own[:, h]
                own[:, h] = back
        m = min(n, self.n_sink)
        if m:
            rows = p.sink.double().cpu().numpy()[(s + 1) % p.sink.shape[0], :, :m].transpose(1, 0, 2)
            if not which and self.rope:
                cs = tb.rope_cs.cpu().numpy()
                rows = np.stack([R.rope(rows[i], i, self.rope, cs) for i in range(m)])
            own[:m] = rows
        return own

    def check(self, out=None, max_rows=1 << 30, lost=None):
        """lost(s, n): whether key n of sequence s has no page."""
        out = (self.out if out is None else out).double().cpu().numpy()
        q = self.q.double().cpu().numpy()
        g, a, worst = self.Hq // self.H, 0, 0.0
        for s in range(len(self.b.ctx)):
            n, m = self.b.ctx[s] + self.b.new[s], self.b.new[s]
            if m:
                k, v = self.keys(s, 0), self.keys(s, 1)
                seen = np.arange(n)[None] <= self.b.ctx[s] + np.arange(m)[:, None]
                if lost is not None:
                    seen &= ~np.array([lost(s, i) for i in range(n)])[None]
                e = min(m, max_rows)
                for h in range(self.Hq):
                    qq, kk, vv = q[a:a + m, h], k[:, h // g], v[:, h // g]
                    p = R.softmax_rows(self.scale * (qq @ kk.T), seen)
                    o = p @ vv
                    # magnitudes in the basis of the products: an orthonormal turn keeps 2-norms, so
                    # sum |q'||y| <= |q||y|; values enter by their largest channel in any basis
                    qn, kn = np.linalg.norm(qq, axis=1)[:, None], np.linalg.norm(kk, axis=1)[None]
                    e_s = (self.scale * qn * kn * ((1 + R.U16) ** 2 - 1 + self.D * 2.0 ** -22)).max(-1, where=p > 0, initial=0.0)
                    rel = np.expm1(2 * e_s) + 2.0 ** -20 + 2 * R.U16 + n * 2.0 ** -22
                    err = (p @ np.linalg.norm(vv, axis=1)) * rel
                    tol = err[:, None] + R.U16 * np.abs(o) + 2.0 ** -24
                    d = np.abs(out[a:a + e, h] - o[:e])
                    assert np.all(np.isfinite(d)), f"sequence {s}, head {h}: not finite"
                    worst = max(worst, (d / tol[:e]).max(initial=0.0))
                assert (out[a + e:a + m] == 7.0).all()
            a += m
        assert (out[a:] == 7.0).all()  # rows behind the last sequence
        assert worst <= 1.0, f"error is {worst} of its bound"
        return worst


@gpu
@pytest.mark.parametrize("case", ATT, ids=[c[0] for c in ATT])
def test_attend_paged(case):
    t = Attend(*case[1:])
    t.call()()
    assert K.kvq_check(0) == OK
    t.check()
    first = t.out.clone()
    t.out.fill_(7.0)
    t.call()()
    assert torch.equal(t.out, first)  # the same bytes again


@gpu
@pytest.mark.parametrize("case", [ATT[0], ATT[9], ATT[14], ATT[17]], ids=lambda c: c[0])
@pytest.mark.parametrize("max_kv", [0, 1, 100, 1 << 20])
def test_attend_paged_any_bound_of_the_lengths(case, max_kv):
    t = Attend(*case[1:])
    t.call(max_kv=max_kv)()
    assert K.kvq_check(0) == OK
    t.check()


@gpu
def test_attend_paged_rows_beyond_max_rows_stay():
    t = Attend([40, 0], [60, 9], 8, 2, 128, 2, 128, 1, False, 4, "fwht_head", 16)
    t.call(max_rows=33)()
    t.check(max_rows=33)


@gpu
@pytest.mark.parametrize("new", [[1, 1], [50, 70]])
def test_attend_paged_missing_pages_are_left_out(new):
    t = Attend([200, 300], new, 8, 2, 128, 2, 128, 1, False, 0, "fwht_head", 16)
    t.b.p.block_table[0, 3] = -1
    t.b.p.block_table[1, 0] = t.b.pages
    t.b.p.block_table[1, 9] = 1 << 30
    t.call()()
    assert K.kvq_check(0) == OK
    t.check(lost=lambda s, n: n // 16 == 3 if s == 0 else n // 16 in (0, 9))


@gpu
def test_attend_paged_rows_that_see_nothing():
    """More new rows than cached tokens say: the first of them are before position 0."""
    t = Attend([0, 30], [20, 1], 8, 2, 128, 2, 128, 1, False, 0, "fwht_head", 16)
    t.b.p.kv_len[0] = 5
    t.call()()
    got = t.out[:20].clone()
    assert (got[:15] == 0).all() and torch.isfinite(got).all() and (got[15:] != 0).any(-1).all()
    u = Attend([0, 30], [20, 1], 8, 2, 128, 2, 128, 1, False, 0, "fwht_head", 16)
    u.b.p.block_table.fill_(-1)  # no key at all
    u.call()()
    assert (u.out == 0).all()
    u.b.p.kv_len.fill_(0)
    u.out.fill_(7.0)
    u.call()()
    assert K.kvq_check(0) == OK and (u.out == 0).all()


@gpu
@pytest.mark.parametrize("which", [0, 1], ids=["keys", "values"])
@pytest.mark.parametrize("S,Z", [(0x7c00, 0x3c00), (0x3c00, 0xfc00), (0x7e00, 0x7e00), (0x7bff, 0x7bff)],
                         ids=["scale inf", "zero -inf", "nan", "sum too large"])
@pytest.mark.parametrize("new,at,Hq,bits,group", [
    ([3, 2], 1, 2, 2, 128), ([4, 4], 3, 4, 4, 32), ([3, 1], 2, 4, 2, 64),   # few rows: one tile and two
    ([20, 4], 11, 8, 2, 128), ([32, 1], 31, 8, 3, 32),                      # one slot of rows
    ([200, 70], 130, 8, 4, 64), ([300, 9], 40, 4, 2, 128),                  # two, and more than one tile of rows
])
def test_attend_paged_later_records_that_are_not_finite(new, at, Hq, bits, group, S, Z, which):
    """A later token's record has no effect on a row, whatever it holds."""
    t = Attend([100, 60], new, Hq, 2, 128, bits, group, 0, False, 0, "fwht_head", 16, extra=2)
    t.call()()
    clean = t.out.clone()
    pos = 100 + at
    sz = t.packs[which].scale_zero
    sz[t.b.m["block_table"][0][pos // 16], :, pos % 16] = torch.tensor([S, Z], dtype=torch.int32).to(torch.int16).cuda()
    t.out.fill_(7.0)
    t.call()()
    assert K.kvq_check(0) == OK
    assert torch.equal(t.out[:at], clean[:at]) and torch.equal(t.out[new[0]:], clean[new[0]:])
    # an infinite key may have the score -inf and so no weight; a large finite scale is a value in fp32
    if S == 0x7e00 or (which == 1 and S != 0x7bff):
        assert not torch.isfinite(t.out[at:new[0]]).all(-1).any()


@gpu
def test_attend_paged_bad_lengths_stay_in_bounds():
    t = Attend([40, 60], [8, 1], 8, 2, 128, 2, 128, 1, False, 4, "fwht_head", 16)
    for cu, kv in (([0, 1 << 30, 9], [48, 61]), ([-4, 8, 9], [48, 61]), ([9, 8, 0], [48, 61]),
                   ([0, 8, 9], [1 << 30, -5])):
        t.b.p.cu_rows.copy_(torch.tensor(cu, dtype=torch.int32))
        t.b.p.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        t.call()()
        assert K.kvq_check(0) == OK
        torch.cuda.synchronize()


@gpu
def test_attend_paged_captured_on_another_stream_and_two_at_once():
    t = Attend([300, 20], [1, 1], 8, 2, 128, 2, 128, 1, False, 4, "fwht_head", 16)
    u = Attend([90, 200], [40, 3], 8, 2, 128, 4, 64, 1, False, 4, "fwht_head", 16, seed=5)
    one, two = t.call(), u.call()
    one(), two()
    torch.cuda.synchronize()
    t.out.fill_(7.0), u.out.fill_(7.0)
    torch.cuda.synchronize()
    sides = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(sides[0]):
            one()
        with torch.cuda.stream(sides[1]):
            two()
    torch.cuda.synchronize()
    t.check(), u.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(), two()
    t.q.normal_()
    t.out.fill_(7.0), u.out.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert K.kvq_check(0) == OK
    t.check(), u.check()


# ---------------------------------------------------------------- together
@gpu
@pytest.mark.parametrize("bits,group,n_sink", [(2, 128, 4), (4, 64, 0)])
def test_a_serving_run(bits, group, n_sink):
    """Two prompts, a prefill by kvq_attend_prompt, its keys and values into pages, a second chunk over
    them and single tokens after it, pages taken by kvq_page_map all along; each step's attention
    against kvq_attend over the same records in a dense cache (which keeps more bits), and the first
    against the prompt's own."""
    Hq, H, D, ps, S = 8, 2, 128, 16, 2
    common = dict(heads=H, head_dim=D, bits=bits, group=group, n_sink=n_sink, rot="fwht_head")
    d = {r: TA.make_desc(batch=40, tokens=0, t_cap=ps, rope=r, **common) for r in (0, 1)}
    tk, tv = _tables(D, H, 1, True, 256, 5), _tables(D, H, 0, True, 256, 6)
    kc, vc = TA.alloc_paged(d[1], S), TA.alloc_paged(d[0], S)
    _poison(kc), _poison(vc)
    i32 = dict(dtype=torch.int32, device="cuda")
    free, used = torch.randperm(40, device="cuda").to(torch.int32), torch.zeros(1, **i32)
    table, ctx = torch.full((S, 16), -1, **i32), torch.zeros(S, **i32)
    g = torch.Generator(device="cuda").manual_seed(1)
    hist = [[], []]
    for new in ([50, 33], [20, 1], [1, 1], [1, 0], [0, 17], [1, 1]):
        n = sum(new)
        b = TA.make_paged(S, n, 16, block_table=table)
        rep = TA.page_map(d[1], b, ctx, torch.tensor(new, **i32), free, used)
        x = torch.randn(n, Hq + 2 * H, D, device="cuda", generator=g).half()
        q, k, v = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
        TA.encode_paged(d[1], k, b, tk, kc)
        TA.encode_paged(d[0], v, b, tv, vc)
        out = torch.full((n, Hq, D), 7.0, dtype=torch.float16, device="cuda")
        mk = int((ctx + torch.tensor(new, **i32)).max())
        ws = TA.attend_paged_workspace(d[1], d[0], Hq, b, max(new), mk)
        TA.attend_paged(d[1], d[0], q, kc, tk, vc, tv, b, max(new), mk, D ** -0.5, out, ws)
        assert K.kvq_check(0) == OK and rep.tolist()[2:] == [0, 0]
        a = 0
        for s in range(S):
            for r in range(a, a + new[s]):
                hist[s].append((k[r], v[r]))
                T = len(hist[s])
                dd = {r_: TA.make_desc(batch=1, tokens=T, t_cap=T, rope=r_, **common) for r_ in (0, 1)}
                pk = []
                for r_, i, tb in ((1, 0, tk), (0, 1, tv)):
                    p = TA.alloc_packed(dd[r_])
                    TA.encode(dd[r_], torch.stack([e[i] for e in hist[s]], 1).unsqueeze(0).contiguous(), tb, p)
                    pk.append(p)
                ref = torch.empty(1, Hq, D, dtype=torch.float32, device="cuda")
                qr = q[r].unsqueeze(0).contiguous()
                TA.attend(dd[1], dd[0], qr, pk[0], tk, pk[1], tv, T, D ** -0.5, ref,
                          TA.attend_workspace(dd[1], dd[0], Hq, T))
                # roundings to fp16 of q and k (2 U16 of |q||k| scale in a score), p, v and the result
                kn = torch.stack([e[0].float().norm(dim=-1) for e in hist[s]]).max()
                vn = torch.stack([e[1].float().norm(dim=-1) for e in hist[s]]).max()
                e_s = D ** -0.5 * float(q[r].float().norm(dim=-1).max() * kn) * 1.5 * (2 * R.U16 + 2.0 ** -14)
                tol = float(vn) * 1.5 * (math.expm1(2 * e_s) + 3 * R.U16)
                assert (out[r].float() - ref[0]).abs().max() <= tol
            a += new[s]
        ctx, used = b.kv_len, rep[1:2].clone()
    assert len(set(table[table >= 0].tolist())) == int((table >= 0).sum())  # no page twice
