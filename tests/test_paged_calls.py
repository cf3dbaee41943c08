"""The calls of the paged cache that its other tests do not make: limits, empty steps, shared buffers, other
threads, devices and streams."""
import random
import threading

import pytest

import paged_ref as R

torch = pytest.importorskip("torch")
import kv_cache_rotation_b200 as K  # noqa: E402
from kv_cache_rotation_b200 import torch_api as TA  # noqa: E402

gpu = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- page map
def _map_call(S, seed=0, ps=16, width=3):
    """(call, check) of a page map of S sequences."""
    r = random.Random(S + seed)
    ctx, new = [r.randint(0, 20) for _ in range(S)], [r.randint(0, 2) for _ in range(S)]
    pool = list(range(2 * S + 8))
    r.shuffle(pool)
    table = [[-1] * width for _ in range(S)]
    for s in range(S):
        for k in range(-(-ctx[s] // ps)):
            table[s][k] = pool.pop()
    n = sum(new)
    want = R.page_map(S, n, width, ps, 2 * S + 8, ctx, new, table, pool, 0)
    b = TA.make_paged(S, n, width, block_table=_i32(table))
    report = torch.zeros(4, dtype=torch.int32, device="cuda")
    d = TA.make_desc(batch=2 * S + 8, heads=1, tokens=0, t_cap=ps, bits=2)
    call = TA.bind_page_map(d, b, _i32(ctx), _i32(new), _i32(pool), _i32([0]), report)

    def check():
        for name in ("cu_rows", "kv_len", "block_table", "seq", "pos", "slot"):
            assert getattr(b, name).tolist() == want[name], name
        assert report.tolist() == want["report"]
    return call, check


@gpu
@pytest.mark.parametrize("S", [6095, 6096, 6143, 6144, 16384])
def test_page_map_of_many_sequences(S):
    """Its shared memory passes what a block has without leave at 6096 sequences, static arrays included. Each size in a
    thread of its own, so that none counts on what another asked for."""
    got = []

    def one():
        try:
            call, check = _map_call(S)
            call()
            torch.cuda.synchronize()
            check()
            got.append(K.kvq_check(0))
        except Exception as e:  # noqa: BLE001
            got.append(e)
    t = threading.Thread(target=one)
    t.start()
    t.join()
    assert got == [K.KVQ_OK]


@gpu
def test_page_map_of_two_threads_with_different_sizes():
    """A thread's smaller call takes nothing away from another thread's larger one."""
    big, check_big = _map_call(16384, 1)
    big()
    torch.cuda.synchronize()
    got = []

    def other():
        try:
            small, check_small = _map_call(7000, 2)
            small()
            torch.cuda.synchronize()
            check_small()
            got.append(K.KVQ_OK)
        except Exception as e:  # noqa: BLE001
            got.append(e)
    t = threading.Thread(target=other)
    t.start()
    t.join()
    assert got == [K.KVQ_OK]
    big()
    torch.cuda.synchronize()
    check_big()
    assert K.kvq_check(0) == K.KVQ_OK


@gpu
def test_page_map_reports_rows_of_a_page_that_an_earlier_call_did_not_get():
    """The pool runs out in the middle of a prompt; the caller goes on. No later row of that page has a slot, and
    every report says so until the rows reach a page that could be taken."""
    d = TA.make_desc(batch=8, heads=1, tokens=0, t_cap=16, bits=2)
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    ctx, used = [0, 0], _i32([0])
    free = _i32([5, 3, 6])
    got = []
    for new, pool in (([16, 40], free), ([1, 1], free), ([2, 6], free), ([0, 0], free), ([14, 3], _i32([5, 3, 6, 0, 7]))):
        b = TA.make_paged(2, sum(new), 4, block_table=table)
        rep = TA.page_map(d, b, _i32(ctx), _i32(new), pool, used).tolist()
        assert K.kvq_check(0) == K.KVQ_OK
        assert rep[0] == sum(new) and rep[2] == b.slot.tolist().count(-1)
        got.append(rep[1:])
        used = _i32([rep[1]])
        ctx = [c + n for c, n in zip(ctx, new)]
    # call 1: sequence 0 takes a page, sequence 1 lacks its third (positions 32 .. 39). 2: sequence 0 lacks its second,
    # sequence 1 goes on in the lost page, position 40. 3: positions 17, 18 and 41 .. 46, all lost. 5: positions 19 .. 31
    # of sequence 0 are lost, 32 starts a page that is there; 47 of sequence 1 is lost, 48 and 49 have one.
    assert got == [[3, 8, 1], [3, 2, 1], [3, 8, 0], [3, 0, 0], [5, 14, 0]]


# ---------------------------------------------------------------- steps without rows
def test_calls_without_rows_take_null_tensors():
    """An empty tensor's address is null."""
    d = TA.make_desc(batch=16, heads=2, head_dim=128, tokens=0, t_cap=32, bits=2)
    pg = K.kvq_paged()
    pg.n_seqs, pg.n_rows, pg.max_pages = 2, 0, 4
    pg.cu_rows = pg.kv_len = pg.block_table = 4096
    pk, tb = K.kvq_packed(), K.kvq_tables()
    pk.codes = pk.scale_zero = 4096
    assert K.kvq_encode_paged(d, None, 256, pg, tb, pk) == K.KVQ_OK
    assert K.kvq_decode_paged(d, pk, pg, tb, None, 256, 0) == K.KVQ_OK
    n = K.kvq_attend_paged_workspace_bytes(d, d, 8, pg, 0, 100)
    assert n > 0
    assert K.kvq_attend_paged(d, d, None, 1024, 8, pk, tb, pk, tb, pg, 0, 100, 0.1, None, 1024, 4096, n) == K.KVQ_OK
    assert K.kvq_attend_prompt(None, 1024, None, 256, None, 256, 2, 0, 8, 2, 128, 0, 4096, 0, 0.1, None, 1024) == K.KVQ_OK
    pg.n_rows = 1  # with a row they are refused as ever
    assert K.kvq_encode_paged(d, None, 256, pg, tb, pk) == K.KVQ_ERR_INVALID
    assert K.kvq_encode_paged(d, 4096, 256, pg, tb, pk) == K.KVQ_ERR_INVALID
    assert K.kvq_decode_paged(d, pk, pg, tb, None, 256, 0) == K.KVQ_ERR_INVALID
    assert K.kvq_attend_paged(d, d, None, 1024, 8, pk, tb, pk, tb, pg, 1, 100, 0.1, None, 1024, 4096, 1 << 30) == K.KVQ_ERR_INVALID
    assert K.kvq_attend_prompt(None, 1024, None, 256, None, 256, 2, 1, 8, 2, 128, 0, 4096, 1, 0.1, None, 1024) == K.KVQ_ERR_INVALID


@gpu
@pytest.mark.parametrize("n_sink", [0, 4])
def test_a_step_in_which_no_sequence_has_a_new_token(n_sink):
    Hq, H, D, ps, S = 8, 2, 128, 16, 3
    common = dict(batch=12, heads=H, head_dim=D, tokens=0, t_cap=ps, bits=2, n_sink=n_sink)
    dk, dv = TA.make_desc(rope=1, **common), TA.make_desc(rope=0, **common)
    tk, tv = TA.make_tables(rope_cs=TA.rope_table(64, D)), TA.make_tables()
    kc, vc = TA.alloc_paged(dk, S), TA.alloc_paged(dv, S)
    table = torch.full((S, 4), -1, dtype=torch.int32, device="cuda")
    free, used, ctx = _i32(list(range(12))), _i32([0]), _i32([0] * S)
    for new in ([20, 3, 0], [0, 0, 0], [1, 0, 2], [0, 0, 0]):
        n = sum(new)
        b = TA.make_paged(S, n, 4, block_table=table)
        before, codes = table.clone(), kc.codes.clone()
        rep = TA.page_map(dk, b, ctx, _i32(new), free, used)
        x = torch.randn(n, Hq + 2 * H, D, device="cuda").half()
        TA.encode_paged(dk, x[:, Hq:Hq + H], b, tk, kc)
        TA.encode_paged(dv, x[:, Hq + H:], b, tv, vc)
        back = torch.empty(n, H, D, dtype=torch.float16, device="cuda")
        TA.decode_paged(dk, kc, b, tk, back)
        out = torch.empty(n, Hq, D, dtype=torch.float16, device="cuda")
        ws = TA.attend_paged_workspace(dk, dv, Hq, b, max(new), 64)
        TA.attend_paged(dk, dv, x[:, :Hq], kc, tk, vc, tv, b, max(new), 64, D ** -0.5, out, ws)
        empty = TA.attend_prompt(x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:], b.cu_rows, max(new), 0.1)
        assert K.kvq_check(0) == K.KVQ_OK and empty.shape == out.shape
        assert rep.tolist()[0] == n and rep.tolist()[2:] == [0, 0]
        assert b.kv_len.tolist() == (ctx + _i32(new)).tolist()
        if n == 0:
            assert torch.equal(table, before) and torch.equal(kc.codes, codes)
        else:
            assert torch.isfinite(out).all() and torch.isfinite(back).all()
        ctx, used = b.kv_len, rep[1:2].clone()


# ---------------------------------------------------------------- arrays that overlap
MAP = dict(cu_rows=3, kv_len=2, block_table=8, seq=8, pos=8, slot=8, report=4, ctx_len=2, new_len=2, free_pages=9, free_used=1)
WRITTEN = list(MAP)[:7]


@pytest.mark.parametrize("one,other", [(a, b) for i, a in enumerate(WRITTEN) for b in list(MAP)[i + 1:]])
def test_page_map_refuses_arrays_that_overlap(one, other):
    """Blocks read lengths while others write: kv_len as the next step's ctx_len would race. Addresses that
    nothing follows: without a device a call that is not refused ends there."""
    if torch.cuda.is_available():
        pytest.skip("made-up addresses")
    at = {n: 1 << 20 | i << 12 for i, n in enumerate(MAP)}

    def call():
        pg = K.kvq_paged()
        pg.n_seqs, pg.n_rows, pg.max_pages = 2, 8, 4
        for n in ("cu_rows", "kv_len", "block_table", "seq", "pos", "slot"):
            setattr(pg, n, at[n])
        d = TA.make_desc(batch=16, heads=1, tokens=0, t_cap=16, bits=2)
        return K.kvq_page_map(d, pg, at["ctx_len"], at["new_len"], at["free_pages"], 9, at["free_used"], at["report"])
    assert call() == K.KVQ_ERR_CUDA
    last = at[one] + 4 * (MAP[one] - 1)
    if other in ("seq", "pos", "slot"):  # on their own alignment
        last &= ~15
    at[other] = last  # its first word on the other's last
    assert call() == K.KVQ_ERR_INVALID


@gpu
def test_page_map_binding_refuses_its_own_lengths_and_takes_copies():
    d = TA.make_desc(batch=8, heads=1, tokens=0, t_cap=16, bits=2)
    b = TA.make_paged(2, 3, 4)
    free, new, report = _i32(list(range(8))), _i32([2, 1]), torch.zeros(4, dtype=torch.int32, device="cuda")
    TA.page_map(d, b, _i32([0, 0]), new, free, _i32([0]), report)
    with pytest.raises(ValueError, match="kv_len"):
        TA.page_map(d, b, b.kv_len, new, free, _i32([2]))
    with pytest.raises(ValueError, match="report"):
        TA.page_map(d, b, _i32([2, 1]), new, free, report[1:2], report)
    with pytest.raises(ValueError, match="seq"):
        TA.page_map(d, TA.Paged(b.cu_rows, b.kv_len, b.block_table, b.seq, b.seq, b.slot), _i32([2, 1]), new, free, _i32([2]))
    for _ in range(3):  # one batch for all steps
        rep = TA.page_map(d, b, b.kv_len.clone(), new, free, report[1:2].clone(), report)
    assert b.kv_len.tolist() == [8, 4] and rep.tolist() == [3, 2, 0, 0] and b.pos.tolist() == [6, 7, 3]


# ---------------------------------------------------------------- records that are not finite
@gpu
@pytest.mark.parametrize("S,Z", [(0x7c00, 0x3c00), (0xfc00, 0x3c00), (0x3c00, 0xfc00), (0x3c00, 0x7c00), (0x7e00, 0x7e00)],
                         ids=["scale inf", "scale -inf", "zero -inf", "zero inf", "nan"])
@pytest.mark.parametrize("new,Hq,bits,group,ctx", [
    ([1, 1], 4, 2, 128, 100), ([1, 1], 8, 4, 64, 1500), ([2, 1], 4, 2, 32, 100),  # few rows: one column tile, two
    ([20, 1], 8, 3, 32, 100), ([200, 3], 8, 4, 64, 600)])                         # one slot of rows, two
@pytest.mark.parametrize("which", [1, 0], ids=["value", "key"])
def test_a_cached_record_that_is_not_finite_shows_in_every_row_that_sees_it(which, new, Hq, bits, group, ctx, S, Z):
    """sum_n p_n v_n has no finite value then; it must not pass as the sum over the other keys. A key's channels are
    infinities of both signs (or NaN), and so is its score."""
    from test_paged import Attend
    t = Attend([ctx, ctx], new, Hq, 2, 128, bits, group, 0, False, 0, "fwht_head", 16, extra=1)
    t.call()()
    clean = t.out.clone()
    sz = t.packs[which].scale_zero
    sz[t.b.m["block_table"][0][37 // 16], :, 37 % 16] = torch.tensor([S, Z], dtype=torch.int32).to(torch.int16).cuda()
    t.out.fill_(7.0)
    t.call()()
    assert K.kvq_check(0) == K.KVQ_OK
    assert not torch.isfinite(t.out[:new[0]]).all(-1).any()
    assert torch.equal(t.out[new[0]:], clean[new[0]:])


# ---------------------------------------------------------------- a slot of two rows
@gpu
@pytest.mark.parametrize("D,bits,group", [(128, 2, 128), (128, 3, 32), (64, 4, 32)])
def test_a_slot_given_twice_holds_pieces_of_both_rows_and_nothing_else_changes(D, bits, group):
    H, ps, n = 3, 16, 400
    d = TA.make_desc(batch=(n + 15) // 16, heads=H, head_dim=D, tokens=0, t_cap=ps, bits=bits, group=group)
    x = torch.randn(n, H, D, device="cuda").half()
    slots = torch.randperm(n, device="cuda").to(torch.int32)
    tb, pos = TA.make_tables(), torch.arange(n, dtype=torch.int32, device="cuda")

    def records(rows, at):
        pk = TA.alloc_paged(d)
        TA.encode_paged(d, x[rows], TA.Paged(pos=pos[rows].contiguous(), slot=at), tb, pk)
        return pk.codes.transpose(1, 2).flatten(0, 1), pk.scale_zero.transpose(1, 2).flatten(0, 1)
    first, second = torch.arange(0, n - 100, device="cuda"), torch.arange(100, n, device="cuda")
    own = slots[:n - 100].contiguous()
    (c1, z1), (c2, z2) = records(first, own), records(second, own)  # rows 0 .. 299, rows 100 .. 399, on the same slots
    both = torch.cat([first, second])
    twice = torch.cat([own, own]).contiguous()
    one = torch.isin(torch.arange(c1.shape[0], device="cuda"), own[50:].long())  # slots that two rows have
    twice[n - 100:n - 50] = -1  # the second rows of the first fifty slots have none
    c, z = records(both, twice)
    assert K.kvq_check(0) == K.KVQ_OK
    assert torch.equal(c[~one], c1[~one]) and torch.equal(z[~one], z1[~one])
    assert ((c == c1) | (c == c2)).all()
    assert ((z == z1).all(-1) | (z == z2).all(-1)).all()  # (scale, zero) of a group is one word


# ---------------------------------------------------------------- what the binding checks
class Small:
    """A small cache and its calls, to be made wrong one argument at a time."""

    def __init__(self, n_sink=4):
        S, n, H, D, ps, pages = 2, 3, 2, 128, 16, 6
        common = dict(batch=pages, heads=H, head_dim=D, tokens=0, t_cap=ps, bits=2, n_sink=n_sink)
        self.dk, self.dv = TA.make_desc(rope=1, **common), TA.make_desc(rope=0, **common)
        perm = torch.arange(D, device="cuda").flip(0).to(torch.int16).repeat(H, 1)
        self.tk, self.tv = TA.make_tables(perm=perm, rope_cs=TA.rope_table(64, D)), TA.make_tables(perm=perm.clone())
        self.k, self.v = TA.alloc_paged(self.dk, S), TA.alloc_paged(self.dv, S)
        self.batch = TA.make_paged(S, n, 3, sink_slot=_i32([1, 0]))
        self.free, self.used, self.ctx, self.new = _i32(list(range(pages))), _i32([0]), _i32([0, 0]), _i32([2, 1])
        self.report = torch.zeros(4, dtype=torch.int32, device="cuda")
        self.x = torch.randn(n, H, D, device="cuda").half()
        self.q = torch.randn(n, 4, D, device="cuda").half()
        self.out, self.back = torch.empty_like(self.q), torch.empty_like(self.x)
        self.ws = TA.attend_paged_workspace(self.dk, self.dv, 4, self.batch, 2, 16)

    def calls(self):
        return dict(page_map=lambda: TA.bind_page_map(self.dk, self.batch, self.ctx, self.new, self.free, self.used, self.report),
                    encode=lambda: TA.bind_encode_paged(self.dk, self.x, self.batch, self.tk, self.k),
                    decode=lambda: TA.bind_decode_paged(self.dk, self.k, self.batch, self.tk, self.back),
                    attend=lambda: TA.bind_attend_paged(self.dk, self.dv, self.q, self.k, self.tk, self.v, self.tv, self.batch, 2,
                                                        16, 0.1, self.out, self.ws))


@gpu
@pytest.mark.parametrize("what,error", [
    (lambda t: setattr(t.k, "codes", t.k.codes[:5]), ValueError), (lambda t: setattr(t.k, "codes", t.k.codes[:, :1]), ValueError),
    (lambda t: setattr(t.k, "codes", t.k.codes.transpose(1, 2)), ValueError),
    (lambda t: setattr(t.k, "scale_zero", t.k.scale_zero[:5]), ValueError),
    (lambda t: setattr(t.k, "scale_zero", t.k.scale_zero.cpu()), ValueError),
    (lambda t: setattr(t.k, "sink", t.k.sink[:, :1]), ValueError), (lambda t: setattr(t.k, "sink", t.k.sink[:, :, :3].contiguous()), ValueError),
    (lambda t: setattr(t.k, "sink", t.k.sink[..., :64].contiguous()), ValueError), (lambda t: setattr(t.k, "sink", t.k.sink.float()), TypeError),
    (lambda t: setattr(t.tk, "perm", t.tk.perm[:1].contiguous()), ValueError), (lambda t: setattr(t.tk, "perm", t.tk.perm.int()), TypeError),
    (lambda t: setattr(t.tk, "rope_cs", t.tk.rope_cs[:, :32].contiguous()), ValueError),
    (lambda t: setattr(t.tk, "rope_cs", t.tk.rope_cs.half()), TypeError), (lambda t: setattr(t.tk, "rope_cs", t.tk.rope_cs.cpu()), ValueError),
], ids=["few pages", "few heads", "strides", "few scales", "host scales", "sink heads", "sink tokens", "sink width", "sink type",
        "perm heads", "perm type", "rope width", "rope type", "host rope"])
def test_binding_refuses_buffers_that_do_not_fit_the_descriptor(what, error):
    t = Small()
    what(t)
    for name in ("encode", "decode", "attend"):
        if name == "attend" and t.k.sink.shape != t.v.sink.shape:
            t.v.sink = t.k.sink  # so that it is not refused for the two caches' sinks
        with pytest.raises(error):
            t.calls()[name]()


@gpu
def test_binding_looks_at_the_device_of_every_tensor(monkeypatch):
    t = Small()
    for name, bind in t.calls().items():
        bind()()
    monkeypatch.setattr(TA.torch.cuda, "current_device", lambda: 1)
    for name, bind in t.calls().items():
        with pytest.raises(ValueError, match="current device"):
            bind()
    monkeypatch.undo()
    assert {id(x) for x in TA._tensors(t.batch, t.k, t.tk, t.q)} == {
        id(x) for x in (*vars(t.batch).values(), t.k.codes, t.k.scale_zero, t.k.sink, t.tk.perm, t.tk.rope_cs, t.q)}


@gpu
def test_a_bound_call_is_made_on_its_device(monkeypatch):
    """On another current device the library would launch there, on this one's addresses."""
    t = Small()
    monkeypatch.setattr(TA.torch.cuda, "device_count", lambda: 2)
    calls = {name: bind() for name, bind in t.calls().items()}
    x = torch.randn(3, 4, 128, device="cuda").half()
    calls["prompt"] = TA.bind_attend_prompt(x[:, :2], x[:, 2:3], x[:, 3:], _i32([0, 3]), 3, 0.1, torch.empty(3, 2, 128, device="cuda").half())
    with monkeypatch.context() as m:
        m.setattr(TA.torch.cuda, "current_device", lambda: 1)
        for call in calls.values():
            with pytest.raises(ValueError, match="cuda:1"):
                call()
    for call in calls.values():
        call()
    assert K.kvq_check(0) == K.KVQ_OK


@gpu
def test_a_bound_call_keeps_the_tensors_it_was_bound_to():
    """It holds their addresses; a batch, cache or table whose field gets another tensor must not free them."""
    import gc
    import weakref
    t = Small()
    calls = {name: bind() for name, bind in t.calls().items()}
    held = [(obj, f) for obj in (t.batch, t.k, t.v, t.tk, t.tv) for f, v in vars(obj).items() if v is not None]
    refs = []
    for obj, f in held:
        refs.append(weakref.ref(getattr(obj, f)))
        setattr(obj, f, getattr(obj, f).clone())
    gc.collect()
    assert all(r() is not None for r in refs)
    del calls
    gc.collect()
    assert all(r() is None for r in refs)


@gpu
@pytest.mark.parametrize("as_int", [False, True])
def test_outputs_that_a_call_makes_belong_to_its_stream(as_int):
    """Else the call could write memory that work of the current stream still uses."""
    side = torch.cuda.Stream()
    stream = side.cuda_stream if as_int else side

    def owner(t):
        for seg in torch.cuda.memory_snapshot():
            if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
                return seg["stream"]
    t, x = Small(), torch.randn(3, 4, 128, device="cuda").half()
    side.wait_stream(torch.cuda.current_stream())
    rep = TA.page_map(t.dk, t.batch, t.ctx, t.new, t.free, t.used, stream=stream)
    out = TA.attend_prompt(x[:, :2], x[:, 2:3], x[:, 3:], t.batch.cu_rows, 2, 0.1, stream=stream)
    side.synchronize()
    assert owner(rep) == owner(out) == side.cuda_stream
    assert owner(TA.attend_prompt(x[:, :2], x[:, 2:3], x[:, 3:], t.batch.cu_rows, 2, 0.1)) == torch.cuda.current_stream().cuda_stream
    assert rep.tolist() == [3, 2, 0, 0] and torch.isfinite(out).all()


def test_alloc_paged_leaves_the_descriptor_alone(monkeypatch):
    """Another thread may be using it."""
    d = TA.make_desc(batch=3, heads=2, tokens=0, t_cap=16, bits=2, n_sink=4)
    seen, plain = [], TA.alloc_packed
    monkeypatch.setattr(TA, "alloc_packed", lambda *a: (seen.append(d.n_sink), plain(*a))[1])
    p = TA.alloc_paged(d, sink_rows=5, device="cpu")
    assert seen == [4] and d.n_sink == 4
    assert p.codes.shape == (3, 2, 16, 32) and p.sink.shape == (5, 2, 4, 128)
    assert TA.alloc_paged(TA.make_desc(batch=3, heads=2, tokens=0, t_cap=16, bits=2), device="cpu").sink is None


@pytest.mark.parametrize("bad", [1 << 31, 1 << 32, -(1 << 31) - 1])
def test_counts_that_do_not_fit_32_bits_are_refused(bad, monkeypatch):
    """Not cut to their low bits: max_rows = 2^32 would be 0, and every row left as it was."""
    monkeypatch.setattr(TA.torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(TA.torch.cuda, "device_count", lambda: 1)
    good = (4096, 1024, 4096, 256, 4096, 256, 0, 0, 8, 2, 128, 0, 4096, 0, 0.1, 4096, 1024)
    TA._call("kvq_attend_prompt", good, (), 0)()  # no row: nothing is launched
    for i in (6, 7, 8, 9, 10, 11, 13):
        with pytest.raises(ValueError, match="32 bits"):
            TA._call("kvq_attend_prompt", good[:i] + (bad,) + good[i + 1:], (), 0)


@gpu
def test_a_bound_call_is_made_with_the_descriptor_it_was_bound_with():
    """Buffers were checked against that one; a later change of it must not reach the kernels."""
    t = Small()
    calls = {name: bind() for name, bind in t.calls().items()}
    for call in calls.values():
        call()
    want = [x.clone() for x in (t.batch.block_table, t.k.codes, t.back, t.out)]
    # values that the library refuses, should they reach it
    t.dk.batch = t.dv.batch = 0
    for call in calls.values():
        call()
    assert K.kvq_check(0) == K.KVQ_OK
    assert all(torch.equal(a, b) for a, b in zip(want, (t.batch.block_table, t.k.codes, t.back, t.out)))


def test_shared_memory_of_rows_with_strides():
    """Against the addresses of the elements themselves."""
    buf = torch.zeros(4000, dtype=torch.int16)

    def at(t):
        return set((torch.arange(4000).as_strided(t.shape, t.stride(), t.storage_offset()) if t.numel() else torch.empty(0)).flatten().tolist())
    r = random.Random(3)
    both = 0
    for _ in range(4000):
        far = r.choice([40, 64])
        t = [buf.as_strided((r.randint(0, 5), r.choice([1, 2, 3]), 8), (far, 8, 1), r.randint(0, 90)) for _ in range(2)]
        meets = bool(at(t[0]) & at(t[1]))
        for a, b in (t, t[::-1]):
            if t[0].stride(0) == t[1].stride(0):
                assert TA._meet(a, b) == meets
            else:  # with different strides whatever lies between each other counts
                assert TA._meet(a, b) or not meets
        both += meets
    assert 500 < both < 3500
    x = buf[:3000].view(50, 6, 10)
    assert not TA._meet(x[:, :2], x[:, 2:4]) and TA._meet(x[:, :3], x[:, 2:4]) and TA._meet(x, x) and not TA._meet(x[:20], x[20:])
    flat = buf[:16].view(torch.int32)
    assert TA._meet(flat[:4], flat[3:]) and not TA._meet(flat[:4], flat[4:])


@gpu
@pytest.mark.parametrize("name,what", [
    ("encode", lambda t: setattr(t, "x", t.k.codes.view(-1)[:1536].view(torch.float16).view(3, 2, 128))),
    ("encode", lambda t: setattr(t.k, "sink", t.x[:2].unsqueeze(0).repeat(2, 1, 2, 1).contiguous()) or setattr(t, "x", t.k.sink.view(-1)[:768].view(3, 2, 128))),
    ("decode", lambda t: setattr(t, "back", t.k.codes.view(-1)[:1536].view(torch.float16).view(3, 2, 128))),
    ("decode", lambda t: setattr(t, "back", t.tk.rope_cs.view(-1)[:768].view(3, 2, 128))),
    ("attend", lambda t: setattr(t, "out", t.q)),
    ("attend", lambda t: setattr(t, "out", t.ws[:t.q.nbytes].view(torch.float16).view(3, 4, 128))),
    ("attend", lambda t: setattr(t, "ws", t.v.codes.view(-1))),
], ids=["rows in the codes", "rows in the sinks", "codes", "table", "queries", "workspace", "values"])
def test_outputs_that_overlap_are_refused(name, what):
    t = Small()
    what(t)
    with pytest.raises(ValueError, match="overlap"):
        t.calls()[name]()


@gpu
def test_prompt_outputs_beside_the_inputs_and_over_them():
    x = torch.randn(40, 4 + 2 * 2 + 4, 128, device="cuda").half()  # q, k, v and room for the output in one buffer
    q, k, v, room = x[:, :4], x[:, 4:6], x[:, 6:8], x[:, 8:]
    cu = _i32([0, 40])
    want = TA.attend_prompt(q.clone(), k.clone(), v.clone(), cu, 40, 0.1)
    for over in (q, x[:, 2:6], x[:, 4:8], x[:, 7:11]):
        with pytest.raises(ValueError, match="overlap"):
            TA.attend_prompt(q, k, v, cu, 40, 0.1, over)
    TA.attend_prompt(q, k, v, cu, 40, 0.1, room)
    assert K.kvq_check(0) == K.KVQ_OK
    assert torch.equal(room, want)


@gpu
def test_a_permutation_of_any_shape_is_taken():
    """The library reads H * head_dim numbers; a flat tensor of them is as good."""
    t = Small()
    flat = {name: bind for name, bind in t.calls().items()}
    t.tk.perm, t.tv.perm = t.tk.perm.view(-1), t.tv.perm.view(1, -1)
    for bind in flat.values():
        bind()()
    assert K.kvq_check(0) == K.KVQ_OK
    t.tk.perm = t.tk.perm[:-1].contiguous()
    with pytest.raises(ValueError, match="perm"):
        t.calls()["encode"]()


# ---------------------------------------------------------------- offsets beyond 32 bits
@gpu
@pytest.mark.parametrize("bits,new", [(4, [1, 2]), (2, [1, 1]), (3, [40, 3]), (4, [60, 1])], ids=["few", "few_2", "one_slot", "two_slots"])
def test_pages_whose_records_lie_beyond_4_gb(bits, new):
    """The same records in a small pool and at the far end of a large one: the same bytes out."""
    H, D, ps, Hq, S = 8, 128, 64, 32, 2
    far = ((1 << 32) + (1 << 28)) // (H * ps * D * bits // 8)  # pages
    n, ctx = sum(new), [100, 30]
    g = torch.Generator(device="cuda").manual_seed(bits)
    x = torch.randn(n + sum(ctx), Hq + 2 * H, D, device="cuda", generator=g).half()
    got = []
    for pages in (16, far):
        common = dict(batch=pages, heads=H, head_dim=D, tokens=0, t_cap=ps, bits=bits, n_sink=1)
        dk, dv = TA.make_desc(rope=1, **common), TA.make_desc(rope=0, **common)
        tk, tv = TA.make_tables(rope_cs=TA.rope_table(256, D)), TA.make_tables()
        kc, vc = TA.alloc_paged(dk, S, zero=False), TA.alloc_paged(dv, S, zero=False)
        free, used = _i32([pages - 1 - i for i in range(8)]), _i32([0])
        table, have, at = torch.full((S, 4), -1, dtype=torch.int32, device="cuda"), [0, 0], 0
        for step in (ctx, new):
            m = sum(step)
            b = TA.make_paged(S, m, 4, block_table=table)
            rep = TA.page_map(dk, b, _i32(have), _i32(step), free, used)
            rows = x[at:at + m]
            TA.encode_paged(dk, rows[:, Hq:Hq + H], b, tk, kc)
            TA.encode_paged(dv, rows[:, Hq + H:], b, tv, vc)
            at, used, have = at + m, rep[1:2].clone(), [h + s for h, s in zip(have, step)]
        assert int(b.slot.min()) * H * D * bits // 8 > (1 << 32) or pages == 16
        back = torch.empty(m, H, D, dtype=torch.float16, device="cuda")
        TA.decode_paged(dv, vc, b, tv, back)
        out = torch.empty(m, Hq, D, dtype=torch.float16, device="cuda")
        ws = TA.attend_paged_workspace(dk, dv, Hq, b, max(new), 256)
        TA.attend_paged(dk, dv, rows[:, :Hq], kc, tk, vc, tv, b, max(new), 256, D ** -0.5, out, ws)
        assert K.kvq_check(0) == K.KVQ_OK
        got.append((back, out))
    assert torch.isfinite(got[0][1]).all() and got[0][1].abs().max() > 0.1
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@gpu
def test_rows_whose_strides_pass_32_bits():
    """Row strides of 2^23 elements: row 300 begins beyond 4 GB."""
    n, Hq, H, D, far = 300, 4, 2, 128, 1 << 23
    buf = torch.empty(n * far, dtype=torch.float16, device="cuda")

    def rows(at, heads):
        return buf.as_strided((n, heads, D), (far, D, 1), at)
    q, k, v, out, back = rows(0, Hq), rows(1024, H), rows(2048, H), rows(4096, Hq), rows(8192, H)
    g = torch.Generator(device="cuda").manual_seed(2)
    for t in (q, k, v):
        t.copy_(torch.randn(t.shape, device="cuda", generator=g))
    out.fill_(7.0), back.fill_(7.0)
    cu = _i32([0, 20, n])
    TA.attend_prompt(q, k, v, cu, n, 0.1, out)
    assert torch.equal(out, TA.attend_prompt(q.contiguous(), k.contiguous(), v.contiguous(), cu, n, 0.1))
    common = dict(batch=24, heads=H, head_dim=D, tokens=0, t_cap=16, bits=4)
    dk, dv = TA.make_desc(rope=1, **common), TA.make_desc(rope=0, **common)
    tk, tv = TA.make_tables(rope_cs=TA.rope_table(300, D)), TA.make_tables()
    b = TA.make_paged(2, n, 18)
    TA.page_map(dk, b, _i32([0, 0]), _i32([20, n - 20]), _i32(list(range(24))), _i32([0]))
    got = []
    for near in (False, True):
        kc, vc = TA.alloc_paged(dk), TA.alloc_paged(dv)
        x = [t.contiguous() if near else t for t in (q, k, v)]
        o, r = (torch.empty(n, Hq, D, dtype=torch.float16, device="cuda"), torch.empty(n, H, D, dtype=torch.float16, device="cuda")) if near else (out, back)
        TA.encode_paged(dk, x[1], b, tk, kc), TA.encode_paged(dv, x[2], b, tv, vc)
        TA.decode_paged(dk, kc, b, tk, r)
        TA.attend_paged(dk, dv, x[0], kc, tk, vc, tv, b, 280, 280, 0.1, o, TA.attend_paged_workspace(dk, dv, Hq, b, 280, 280))
        got.append([t.clone() for t in (kc.codes, vc.codes, r, o)])
    assert K.kvq_check(0) == K.KVQ_OK
    assert all(torch.equal(a, c) for a, c in zip(*got))
