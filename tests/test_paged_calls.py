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
