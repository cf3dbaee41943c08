"""kvq_attend_prompt where a call has more tiles than the GPU has SMs: two slots of query rows a block, several tiles of
keys, both types, both head sizes; bounds and reference as in test_prompt."""
import math

import pytest

torch = pytest.importorskip("torch")
import kv_cache_rotation_b200 as K  # noqa: E402
from test_prompt import _check, _inputs, _run  # noqa: E402

gpu = pytest.mark.gpu


def _two_slots(lens, Hq, H, extra=0, max_rows=None):
    """Whether a call takes two slots: more row tiles of 2 (128 / group) tokens, at most, than SMs."""
    tt = 2 * (128 // (Hq // H))
    n, mr = sum(lens) + extra, max(lens) if max_rows is None else max_rows
    tiles = min(n // tt + len(lens), len(lens) * -(-mr // tt))
    return tiles * H > torch.cuda.get_device_properties(0).multi_processor_count


CASES = [
    # name, lens, Hq, H, D, dtype, extra rows
    ("edges_of_tiles", [127, 128, 129, 255, 256, 257, 383, 385], 32, 32, 128, "f16", 0),
    ("edges_d64_bf16", [127, 128, 129, 255, 256, 257, 383, 385, 1], 32, 32, 64, "bf16", 3),
    ("ring_wraps", [1200], 32, 32, 128, "f16", 0),
    ("ring_wraps_bf16", [1190], 32, 32, 128, "bf16", 7),
    ("ring_wraps_d64", [1270], 32, 32, 64, "f16", 0),
    ("two_per_head", [300, 1, 513, 64], 32, 16, 128, "bf16", 1),
    ("three_per_head", [150, 43, 85, 1, 168, 252], 48, 16, 128, "f16", 2),
    ("four_per_head", [700, 65, 64, 0, 63], 64, 16, 128, "f16", 5),
    ("four_per_head_bf16", [700, 65, 64, 0, 63], 64, 16, 128, "bf16", 0),
    ("four_per_head_d64", [333, 700, 2], 64, 16, 64, "f16", 1),
    ("seven_per_head", [333, 77, 5], 112, 16, 128, "bf16", 0),
    ("many_per_head", [170, 3], 130, 2, 128, "f16", 4),
    ("forty_sequences", [(17 * i) % 150 + 1 for i in range(40)], 32, 8, 128, "f16", 3),
    ("forty_d64", [(29 * i) % 190 for i in range(40)], 24, 8, 64, "bf16", 0),
]


@gpu
@pytest.mark.parametrize("name,lens,Hq,H,D,dtype,extra", CASES, ids=[c[0] for c in CASES])
def test_two_slots(name, lens, Hq, H, D, dtype, extra):
    assert _two_slots(lens, Hq, H, extra)
    x, cu = _inputs(lens, Hq, H, D, dtype, extra, seed=len(name))
    out = _run(x, cu, Hq, H, max(lens), D ** -0.5)
    assert K.kvq_check(0) == K.KVQ_OK
    _check(x, lens, Hq, H, out, D ** -0.5, max(lens))
    assert torch.equal(_run(x, cu, Hq, H, max(lens), D ** -0.5), out)  # the same bytes again


@gpu
@pytest.mark.parametrize("D,dtype", [(128, "f16"), (64, "bf16")])
def test_two_slots_peaked_scores(D, dtype):
    """Scores of hundreds, later keys weigh more: the references rise and the sums are rescaled, slot by slot."""
    lens, Hq, H = [1100, 200], 32, 16
    x, cu = _inputs(lens, Hq, H, D, dtype, 0, seed=3, big=5.0)
    x[:, Hq:Hq + H] *= torch.linspace(0.2, 2.0, 1300)[:, None, None].to(x.dtype)
    assert _two_slots(lens, Hq, H)
    out = _run(x, cu, Hq, H, 1100, D ** -0.5)
    _check(x, lens, Hq, H, out, D ** -0.5, 1100)


@gpu
def test_two_slots_rows_beyond_max_rows_stay():
    lens, Hq, H = [400, 30, 171, 200, 190, 300], 32, 32
    x, cu = _inputs(lens, Hq, H, 128, "f16", 0, seed=4)
    assert _two_slots(lens, Hq, H, max_rows=170)
    out = _run(x, cu, Hq, H, 170, 0.1)
    _check(x, lens, Hq, H, out, 0.1, 170)


@gpu
@pytest.mark.parametrize("Hq,H", [(32, 32), (48, 16)], ids=["one_per_head", "three_per_head"])
@pytest.mark.parametrize("D,dtype", [(128, "f16"), (128, "bf16"), (64, "f16")])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_two_slots_masked_places_have_no_effect(bad, D, dtype, Hq, H):
    """Infinities and NaN in later rows of either slot's tiles, in other sequences and behind the last one."""
    lens = [90, 500, 3]
    assert _two_slots(lens, Hq, H, 40)
    x, cu = _inputs(lens, Hq, H, D, dtype, 40, seed=5)
    clean = _run(x, cu, Hq, H, 500, 0.1)
    for at in (93, 90 + 127, 90 + 128, 90 + 200, 90 + 384, 90 + 499):  # from this row on, and the last sequence
        y = x.clone()
        y[at:] = bad
        got = _run(y, cu, Hq, H, 500, 0.1)
        assert K.kvq_check(0) == K.KVQ_OK
        assert torch.equal(got[:at], clean[:at])
        assert torch.isnan(got[at:593]).all()
        w = x.clone()
        w[at, Hq + H:] = bad  # the values of this row alone
        got = _run(w, cu, Hq, H, 500, 0.1)
        assert torch.equal(got[:at], clean[:at]) and torch.equal(got[590:], clean[590:])
        want = torch.full_like(got[at:590], bad)  # a weight above zero times an infinity is that infinity
        assert torch.equal(torch.nan_to_num(got[at:590], 5.0, 6.0, -6.0), torch.nan_to_num(want, 5.0, 6.0, -6.0))
    z = x.clone()
    z[593:] = bad
    assert torch.equal(_run(z, cu, Hq, H, 500, 0.1), clean)


@gpu
def test_two_slots_captured_and_two_at_once():
    from kv_cache_rotation_b200 import torch_api as TA
    lens, Hq, H = [600, 64, 70], 32, 32
    assert _two_slots(lens, Hq, H, 2)
    x, cu = _inputs(lens, Hq, H, 128, "f16", 2, seed=7)
    xs, cc = [x.cuda(), _inputs(lens, Hq, H, 128, "f16", 2, seed=9)[0].cuda()], cu.cuda()
    outs = [torch.full((736, Hq, 128), 7.0, dtype=torch.float16, device="cuda") for _ in xs]
    calls = [TA.bind_attend_prompt(a[:, :Hq], a[:, Hq:Hq + H], a[:, Hq + H:], cc, 600, 0.1, o) for a, o in zip(xs, outs)]
    calls[0](), calls[1]()
    torch.cuda.synchronize()
    sides = torch.cuda.Stream(), torch.cuda.Stream()
    for o in outs:
        o.fill_(7.0)
    torch.cuda.synchronize()
    for _ in range(5):
        for side, call in zip(sides, calls):
            with torch.cuda.stream(side):
                call()
    torch.cuda.synchronize()
    for a, o in zip(xs, outs):
        _check(a.cpu(), lens, Hq, H, o, 0.1, 600)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls[0](), calls[1]()
    y = _inputs(lens, Hq, H, 128, "f16", 2, seed=8)[0]
    xs[0].copy_(y)
    for o in outs:
        o.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert K.kvq_check(0) == K.KVQ_OK
    _check(y, lens, Hq, H, outs[0], 0.1, 600)
    _check(xs[1].cpu(), lens, Hq, H, outs[1], 0.1, 600)


@gpu
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("lens,Hq,H", [([70, 300], 8, 2), ([70, 300, 700], 64, 16)], ids=["one_slot", "two_slots"])
def test_a_query_row_that_is_not_finite_touches_no_other(lens, Hq, H, bad):
    x, cu = _inputs(lens, Hq, H, 128, "f16", 0, seed=5)
    assert _two_slots(lens, Hq, H) == (H == 16)
    clean = _run(x, cu, Hq, H, max(lens), 0.1)
    x[200, Hq - 1, 5] = bad
    got = _run(x, cu, Hq, H, max(lens), 0.1)
    assert K.kvq_check(0) == K.KVQ_OK
    assert not torch.isfinite(got[200, Hq - 1]).any()
    got[200, Hq - 1] = clean[200, Hq - 1] = 0.0
    assert torch.equal(got, clean)
