"""kvq_attend_prompt against attention in 64 bits, and its refusals."""
import ctypes
import math

import numpy as np
import pytest

import paged_ref as R

torch = pytest.importorskip("torch")
import kv_cache_rotation_b200 as K  # noqa: E402
from kv_cache_rotation_b200 import torch_api as TA  # noqa: E402

gpu = pytest.mark.gpu


# ---------------------------------------------------------------- refusals (no GPU)
def _args(**kw):
    a = dict(q=4096, qs=1024, k=4096, ks=256, v=4096, vs=256, S=1, n=8, hq=8, h=2, d=128, t=0, cu=4096, mr=8,
             scale=0.1, out=4096, os=1024)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), K.KVQ_ERR_INVALID), (dict(n=-1), K.KVQ_ERR_INVALID), (dict(mr=-1), K.KVQ_ERR_INVALID),
    (dict(hq=0), K.KVQ_ERR_INVALID), (dict(h=0), K.KVQ_ERR_INVALID), (dict(hq=9), K.KVQ_ERR_INVALID),
    (dict(t=2), K.KVQ_ERR_INVALID), (dict(d=96), K.KVQ_ERR_UNSUPPORTED),
    (dict(hq=258, h=2, qs=258 * 128, os=258 * 128), K.KVQ_ERR_UNSUPPORTED),
    (dict(q=None), K.KVQ_ERR_INVALID), (dict(cu=None), K.KVQ_ERR_INVALID), (dict(out=None), K.KVQ_ERR_INVALID),
    (dict(q=4104), K.KVQ_ERR_ALIGN), (dict(v=4098), K.KVQ_ERR_ALIGN), (dict(cu=4098), K.KVQ_ERR_ALIGN),
    (dict(qs=1016), K.KVQ_ERR_INVALID), (dict(ks=128), K.KVQ_ERR_INVALID), (dict(os=1000), K.KVQ_ERR_INVALID),
    (dict(qs=1028), K.KVQ_ERR_ALIGN), (dict(vs=260), K.KVQ_ERR_ALIGN),
    (dict(scale=0.0), K.KVQ_ERR_INVALID), (dict(scale=-1.0), K.KVQ_ERR_INVALID),
    (dict(scale=math.nan), K.KVQ_ERR_INVALID), (dict(scale=math.inf), K.KVQ_ERR_INVALID),
    (dict(n=(1 << 31) - 1), K.KVQ_ERR_UNSUPPORTED), (dict(ks=1 << 40), K.KVQ_ERR_UNSUPPORTED),
    (dict(n=0), K.KVQ_OK), (dict(S=0), K.KVQ_OK), (dict(mr=0), K.KVQ_OK),
])
def test_prompt_refusals(kw, status):
    assert K.kvq_attend_prompt(*_args(**kw)) == status


def test_prompt_python_refusals():
    x = torch.zeros(4, 8, 128, dtype=torch.float16)
    with pytest.raises(ValueError):  # not on the GPU
        TA.attend_prompt(x, x, x, torch.zeros(2, dtype=torch.int32), 4, 1.0)
    with pytest.raises(TypeError):
        TA.attend_prompt(np.zeros(4), x, x, torch.zeros(2, dtype=torch.int32), 4, 1.0)


# ---------------------------------------------------------------- numerics
def _reference(q, k, v, lens, scale, max_rows, u):
    """(out, bound) [n, Hq, D] in 64 bits; rows of no sequence are NaN."""
    n, Hq, D = q.shape
    g = Hq // k.shape[1]
    out, tol = np.full((n, Hq, D), np.nan), np.zeros((n, Hq, D))
    a = 0
    for m in lens:
        e = min(m, max_rows)
        for h in range(Hq):
            qq, kk, vv = q[a:a + e, h], k[a:a + e, h // g], v[a:a + e, h // g]
            p = R.softmax_rows(scale * (qq @ kk.T), np.tril(np.ones((e, e), bool)))
            o = p @ vv
            out[a:a + e, h] = o
            # q, k and v enter as they are; the products run in the channels' own basis
            mag = scale * (np.abs(qq) @ np.abs(kk).T)
            err = (mag * D * 2.0 ** -23).max(-1, where=p > 0, initial=0.0)[:, None]
            rel = np.expm1(2 * err) + 2.0 ** -20 + u + e * 2.0 ** -22
            tol[a:a + e, h] = (p @ np.abs(vv)) * rel + u * np.abs(o) + 2.0 ** -24
        a += m
    return out, tol


CASES = [
    # lens, Hq, H, D, dtype, extra rows behind the last sequence
    ("one_token", [1], 4, 1, 128, "f16", 0),
    ("two_tokens", [2], 4, 4, 128, "f16", 0),
    ("gqa_ragged", [5, 0, 1, 63, 64, 65, 130], 8, 2, 128, "f16", 3),
    ("mha_edges", [127, 128, 129, 255, 256, 257], 2, 2, 128, "f16", 0),
    ("bf16", [300, 7, 77], 8, 2, 128, "bf16", 5),
    ("d64", [200, 1, 129], 8, 4, 64, "f16", 2),
    ("d64_bf16_mha", [385], 3, 3, 64, "bf16", 0),
    ("three_per_head", [150, 43, 44], 6, 2, 128, "f16", 1),
    ("many_per_head", [70, 3], 65, 1, 128, "f16", 0),
    ("all_of_a_tile", [40], 128, 1, 64, "f16", 0),
    ("seven_per_head", [333], 7, 1, 128, "bf16", 9),
    ("many_short", [1, 2, 3] * 40, 8, 2, 128, "f16", 0),
    ("long", [1200], 4, 1, 128, "f16", 0),
]


def _inputs(lens, Hq, H, D, dtype, extra, seed=0, big=1.0):
    g = torch.Generator().manual_seed(seed)
    n = sum(lens) + extra
    t = torch.float16 if dtype == "f16" else torch.bfloat16
    x = (torch.randn(n, Hq + 2 * H, D, generator=g) * big).to(t)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    return x, cu


def _run(x, cu, Hq, H, max_rows, scale, out=None, stream=None):
    xc = x.cuda() if not x.is_cuda else x
    if out is None:
        out = torch.full((x.shape[0], Hq, x.shape[2]), 7.0, dtype=x.dtype, device="cuda")
    TA.attend_prompt(xc[:, :Hq], xc[:, Hq:Hq + H], xc[:, Hq + H:], cu.cuda(), max_rows, scale, out, stream)
    return out


def _check(x, lens, Hq, H, out, scale, max_rows):
    u = R.U16 if x.dtype == torch.float16 else R.UB16
    q, k, v = (t.double().numpy() for t in (x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]))
    ref, tol = _reference(q, k, v, lens, scale, max_rows, u)
    got = out.double().cpu().numpy()
    none = np.isnan(ref).all((1, 2))
    assert np.all(got[none] == 7.0)  # rows of no sequence are left as they were
    err = np.abs(got - ref)[~none]
    assert np.all(np.isfinite(err)), "not finite"
    over = err / tol[~none]
    assert over.max(initial=0.0) <= 1.0, f"error is {over.max()} of its bound"


@gpu
@pytest.mark.parametrize("name,lens,Hq,H,D,dtype,extra", CASES, ids=[c[0] for c in CASES])
def test_prompt(name, lens, Hq, H, D, dtype, extra):
    x, cu = _inputs(lens, Hq, H, D, dtype, extra)
    out = _run(x, cu, Hq, H, max(lens), D ** -0.5)
    assert K.kvq_check(0) == K.KVQ_OK
    _check(x, lens, Hq, H, out, D ** -0.5, max(lens))


@gpu
def test_prompt_peaked_scores():
    """Scores of a few hundred: the running maximum moves by far more than one step of it."""
    x, cu = _inputs([400], 4, 2, 128, "f16", 0, seed=3, big=5.0)
    x[:, 4:6] *= torch.linspace(0.2, 2.0, 400)[:, None, None].half()  # later keys weigh more
    out = _run(x, cu, 4, 2, 400, 128 ** -0.5)
    _check(x, [400], 4, 2, out, 128 ** -0.5, 400)


@gpu
def test_prompt_rows_beyond_max_rows_stay():
    x, cu = _inputs([100, 30], 8, 2, 128, "f16", 0, seed=4)
    out = _run(x, cu, 8, 2, 37, 0.1)
    _check(x, [100, 30], 8, 2, out, 0.1, 37)


@gpu
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_prompt_masked_places_have_no_effect(bad, D):
    """Infinities and NaN in later rows, in other sequences and behind the last one."""
    lens, Hq, H = [90, 200, 3], 8, 2
    x, cu = _inputs(lens, Hq, H, D, "f16", 40, seed=5)
    clean = _run(x, cu, Hq, H, 200, 0.1)
    y = x.clone()
    y[93:] = bad      # from row 3 of the second sequence on
    got = _run(y, cu, Hq, H, 200, 0.1)
    assert K.kvq_check(0) == K.KVQ_OK
    assert torch.equal(got[:93], clean[:93])
    assert torch.isnan(got[93:293]).all()
    z = x.clone()
    z[293:] = bad     # behind the last sequence
    assert torch.equal(_run(z, cu, Hq, H, 200, 0.1), clean)
    w = x.clone()
    w[150, Hq + H:] = bad  # values of one row inside the second sequence
    got = _run(w, cu, Hq, H, 200, 0.1)
    assert torch.equal(got[:150], clean[:150]) and torch.equal(got[290:], clean[290:])
    # a weight above zero times an infinity is that infinity
    want = torch.full_like(got[150:290], bad)
    assert torch.equal(torch.nan_to_num(got[150:290], 5.0, 6.0, -6.0), torch.nan_to_num(want, 5.0, 6.0, -6.0))


@gpu
def test_prompt_bad_offsets_stay_in_bounds():
    """Offsets that are not ascending or run past the rows are cut to them."""
    x, _ = _inputs([64], 8, 2, 128, "f16", 0, seed=6)
    for cu in ([0, 1 << 30], [-5, 64], [64, 0], [0, 40, 20, 64]):
        out = _run(x, torch.tensor(cu, dtype=torch.int32), 8, 2, 64, 0.1)
        assert K.kvq_check(0) == K.KVQ_OK
        assert torch.isfinite(out).all()


@gpu
def test_prompt_captured_and_on_another_stream():
    lens, Hq, H = [130, 64], 8, 2
    x, cu = _inputs(lens, Hq, H, 128, "f16", 2, seed=7)
    xc, cc = x.cuda(), cu.cuda()
    out = torch.full((196, Hq, 128), 7.0, dtype=torch.float16, device="cuda")
    call = TA.bind_attend_prompt(xc[:, :Hq], xc[:, Hq:Hq + H], xc[:, Hq + H:], cc, 130, 0.1, out)
    call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out.fill_(7.0)
        call()
    side.synchronize()
    _check(x, lens, Hq, H, out, 0.1, 130)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    y = _inputs(lens, Hq, H, 128, "f16", 2, seed=8)[0]
    xc.copy_(y)
    out.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert K.kvq_check(0) == K.KVQ_OK
    _check(y, lens, Hq, H, out, 0.1, 130)


@gpu
def test_prompt_same_bytes_twice():
    x, cu = _inputs([700, 33], 8, 2, 128, "bf16", 0, seed=9)
    assert torch.equal(_run(x, cu, 8, 2, 700, 0.1), _run(x, cu, 8, 2, 700, 0.1))
