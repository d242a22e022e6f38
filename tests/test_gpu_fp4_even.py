"""Decode over 4-bit caches with the slabs dealt out evenly: windows, first tokens, the step's append, and bad data, at
sizes that take the workspace (needs a GB300).  Bounds: those of test_gpu_fp4.py."""
import numpy as np
import pytest

import oracle as O
import workloads as W
from fp4_ref import K_UNIT, V_UNIT
from harness import out_f64
from test_gpu_fp4 import BIG, SENTINEL, Step, case, check, within_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def pa():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_32_gb300 as pa
    pa.build()
    return pa


def even_case(pa, rows, lens, hq, hkv, block_size, window, sinks, table_tokens, **kw):
    """A step whose table holds table_tokens, for which the call uses a workspace."""
    slack = table_tokens // block_size - -(-max(lens) // block_size)
    w = case(rows, lens, [1] * len(lens), hq, hkv, block_size, window, sinks, slack_blocks=slack, **kw)
    desc = pa.pa_cache_desc(w.num_blocks, block_size, hkv, 128, pa.PA_FP4_E2M1)
    assert pa.pa_decode_fp4_workspace_size(len(lens), hq, w.width, desc, window=window, num_sinks=sinks) > 0
    return w


def append_slots(w):
    at = [w.table[i, (L - 1) // w.B] * w.B + (L - 1) % w.B if L else -1 for i, L in enumerate(w.lens)]
    return np.array(at, np.int64)


def check_step(pa, w):
    """A step against 64 bits, its bits again, and, with an append, the caches' bytes."""
    import torch
    s, t = Step(w), Step(w)
    ref = w.reference()
    s.decode()
    check(s, ref, "even")
    if w.new_key is None:
        assert torch.equal(s.out, t.decode())
        return
    pa.pa_reshape_and_cache_fp4(t.k, t.v, t.nk, t.nv, torch.from_numpy(append_slots(w)).cuda(), K_UNIT, V_UNIT,
                                err_flag=t.err)
    assert torch.equal(s.k, t.k) and torch.equal(s.v, t.v)
    t.nk = t.nv = None
    assert torch.equal(s.out, t.decode())  # over the written caches: the same bits


LONG = [0, 40000, 1, 33, 33500, 700, 0, 32]


@pytest.mark.parametrize("rows,hq,hkv,block_size", [("f16", 8, 2, 16), ("bf16", 24, 2, 32), ("bf16", 32, 2, 48),
                                                    ("f16", 3, 3, 64), ("bf16", 17, 1, 256)])
@pytest.mark.parametrize("window,sinks", [(32768, 100), (33000, 0), (20000, 13017), (BIG, 5)])
@pytest.mark.parametrize("append", [False, True])
def test_long_contexts(pa, rows, hq, hkv, block_size, window, sinks, append):
    """Windows that cut long contexts, first tokens whose slabs are shared out too, groups of more than eight heads (two
    CTAs at one tile, one of which stores the new token)."""
    w = even_case(pa, rows, LONG, hq, hkv, block_size, window, sinks, 65536 // 768 * 768, seed=hq + sinks, append=append)
    check_step(pa, w)


@pytest.mark.parametrize("rows,hq,hkv,block_size", [("bf16", 16, 8, 16), ("f16", 40, 4, 48)])
@pytest.mark.parametrize("window,sinks,append", [(2100, 40, True), (2600, 0, False), (1000, 1500, True), (BIG, 0, True)])
def test_many_contexts(pa, rows, hq, hkv, block_size, window, sinks, append):
    """More items than fill the table's shares evenly, empty sequences among them."""
    rng = np.random.default_rng(hkv)
    lens = [int(x) for x in rng.integers(1, 4000, 32)] + [0, 1, 4031]
    check_step(pa, even_case(pa, rows, lens, hq, hkv, block_size, window, sinks, 4224, seed=window or 1, append=append))


@pytest.mark.parametrize("rows", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [-0.09, 0.0, 1e-36])
def test_any_scale(pa, rows, scale):
    w = even_case(pa, rows, [3000, 77, 5, 0, 900], 8, 2, 16, BIG, 0, 40000, seed=3)
    w.scale = scale
    check_step(pa, w)


@pytest.mark.parametrize("power", [-120, 100])
def test_queries_of_any_size(pa, power):
    w = even_case(pa, "bf16", [3000, 77], 8, 2, 16, BIG, 0, 40000, seed=3)
    ref = w.reference()
    w.q = W.to_storage(O.to_f64(w.q, "bf16") * 2.0 ** power, "bf16")
    w.scale *= 2.0 ** -power
    s = Step(w)
    s.decode()
    check(s, ref, "scaled queries")


@pytest.mark.parametrize("append", [False, True])
def test_bad_block(pa, append):
    """A block outside the pool is reported; the other sequences are right, those that share a CTA with it too.  With the
    new token's own block outside, nothing is written for that sequence."""
    import torch
    lens = [500, 40000, 31, 6000]
    w = even_case(pa, "bf16", lens, 24, 2, 32, BIG, 0, 65536, seed=4, append=append)
    ref = w.reference()
    for s_bad, at in ((1, 20000 // 32), (1, 0), (3, 5999 // 32)):
        s, t = Step(w), Step(w)
        s.table[s_bad, at] = w.num_blocks
        s.decode()
        assert int(s.err.item()) == 1
        keep = [i for i in range(4) if i != s_bad]
        ok, err, _ = within_bound(out_f64(s.out)[keep], ref[keep], "bf16")
        assert ok, err
        if append:
            slots = append_slots(w)
            if at == (lens[s_bad] - 1) // 32:
                slots[s_bad] = -1
            pa.pa_reshape_and_cache_fp4(t.k, t.v, t.nk, t.nv, torch.from_numpy(slots).cuda(), K_UNIT, V_UNIT)
            assert torch.equal(s.k, t.k) and torch.equal(s.v, t.v)


@pytest.mark.parametrize("bad", [40033, -3, 2 ** 31 - 1, -2 ** 31])
def test_length_outside_the_table(pa, bad):
    w = even_case(pa, "f16", [300, 50, 4000], 8, 2, 16, BIG, 0, 40032, seed=6)
    s = Step(w)
    s.lens[1] = bad
    s.decode()
    got, ref = out_f64(s.out), w.reference()
    assert int(s.err.item()) == 5 and np.all(got[1] == SENTINEL)
    assert within_bound(got[[0, 2]], ref[[0, 2]], "f16")[0]


@pytest.mark.parametrize("rows", ["f16", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nan_query_is_a_nan_row(pa, rows, value):
    """Through the join (an item of many CTAs) and without it; no other row.  (An infinity meets keys of both signs.)"""
    w = even_case(pa, rows, [9000, 400, 20], 12, 1, 16, BIG, 0, 40000, seed=5)
    s, ref = Step(w), w.reference()
    hit = [(0, 3), (0, 11), (1, 0), (2, 9)]
    for at in hit:
        s.q[at[0], at[1], 7] = value
    s.decode()
    assert int(s.err.item()) == 0
    got = out_f64(s.out)
    for at in hit:
        assert np.isnan(got[at]).all()
        got[at] = ref[at]
    assert within_bound(got, ref, rows)[0]


def test_only_empty_sequences(pa):
    w = even_case(pa, "f16", [0, 0, 0], 8, 2, 16, BIG, 0, 40000, seed=7)
    s = Step(w)
    s.decode()
    assert int(s.err.item()) == 0 and np.all(out_f64(s.out) == 0)
