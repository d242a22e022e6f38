"""Caches held in 4 bits: calls and values at the edges of what they take (needs a GB300)."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def pa():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_32_gb300 as pa
    pa.build()
    return pa


def test_copy_blocks_without_a_descriptor(pa):
    """Whole blocks, codes and scales, and no other byte."""
    import torch
    k, v = (torch.randint(0, 256, (6, 3, 3, 1152), dtype=torch.uint8, device="cuda") for _ in range(2))
    want = k.clone(), v.clone()
    for t in want:
        t[4], t[1] = t[0], t[5]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_copy_blocks(k, v, torch.tensor([[0, 4], [5, 1]], dtype=torch.int32, device="cuda"), err_flag=err)
    assert int(err.item()) == 0 and torch.equal(k, want[0]) and torch.equal(v, want[1])


def lagging_cache(pa, length, low, unit):
    """One sequence's blocks of 16 in bf16: keys +-6 (the first `low` tokens the negative ones), every value the largest
    number that a cache of this unit holds.  The scores of queries of ones rise by 7.9 binary orders behind the low tokens,
    which the running maximum of what starts at the low ones does not follow."""
    import torch
    key = torch.full((length, 1, 128), 6.0, dtype=torch.bfloat16, device="cuda")
    key[:low] = -6.0
    value = torch.full_like(key, 2688.0 * unit)
    k, v = (pa.fp4_cache(length // 16, 1, 16) for _ in range(2))
    pa.pa_reshape_and_cache_fp4(k, v, key, value, torch.arange(length, device="cuda"), 1.0, unit)
    return k, v, 7.9 / (2 * 128 * 6 * 1.4426950408889634)


@pytest.mark.parametrize("power", [100, -100])
@pytest.mark.parametrize("form,length", [("clusters", 4000), ("even", 40000), ("tiles", 4096)])
def test_value_unit_at_its_ends(pa, form, length, power):
    """Values that the rows' type holds come out as they are, however large or small the unit and whatever a row has added
    up before the division: every value is the same number, a weighted mean of it within 2^-11 for the rounding of the
    weights, and half a step of bf16."""
    import torch
    unit, seqs = 2.0 ** power, 160
    k, v, scale = lagging_cache(pa, length, 192, unit)
    table = torch.arange(length // 16, dtype=torch.int32, device="cuda").repeat(seqs, 1)
    lens = torch.full((seqs,), length, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if form == "tiles":
        q = torch.ones(300, 8, 128, dtype=torch.bfloat16, device="cuda")
        out = torch.zeros_like(q)
        start = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
        pa.pa_prefill_fp4(out, q, k, v, table[:1].contiguous(), lens[:1], start, 300, scale, 1.0, unit, err_flag=err)
    else:
        q = torch.ones(seqs, 8, 128, dtype=torch.bfloat16, device="cuda")
        out = torch.zeros_like(q)
        need = pa.pa_decode_fp4_workspace_size(seqs, 8, length // 16, pa.fp4_cache_desc(k))
        assert need > 0
        kw = dict(alibi_slopes=torch.zeros(8, device="cuda")) if form == "clusters" else {}  # (ALiBi: always in clusters)
        pa.pa_decode_fp4(out, q, k, v, table, lens, scale, 1.0, unit, err_flag=err, **kw)
    assert int(err.item()) == 0
    want = 2688.0 * unit
    far = (out.double() / want - 1).abs().max().item()
    assert far <= 2.0 ** -11 + 2.0 ** -8, far


@pytest.mark.parametrize("rows", ["f16", "bf16"])
@pytest.mark.parametrize("form", ["clusters", "even", "tiles", "split tiles"])
def test_many_small_weights_beside_a_large_one(pa, rows, form):
    """The first token takes nearly everything, and 2^20 others of 2^-25.5 each have a share of 2 % between them: their
    values are 1, the first one's 0.  Off by at most 2^-11 for the weights' rounding, half a step of the rows' type, and
    what fp32 sums lose: 16 weights of 2^-25.5 at a time against a sum of 1 to 2^-23 of it lose up to 0.36 of their share
    of the sum (0.36 * 2 % of the result), and against their own sum, of values times weights, up to 2^-7 of it."""
    import torch
    t = torch.float16 if rows == "f16" else torch.bfloat16
    length, unit = 1 << 20, 1.0 / 6
    # block 0 holds the first token and 15 others, block 1 others only; a sequence is block 0, then block 1 over and over
    key = torch.full((32, 1, 128), -6.0, dtype=t, device="cuda")
    value = torch.ones_like(key)
    key[0], value[0] = 6.0, 0.0
    k, v = (pa.fp4_cache(2, 1, 16) for _ in range(2))
    pa.pa_reshape_and_cache_fp4(k, v, key, value, torch.arange(32, device="cuda"), 1.0, unit)
    scale = 25.5 / (2 * 128 * 6 * 1.4426950408889634)
    seqs = 160 if form in ("clusters", "even") else 1
    table = torch.ones(seqs, length // 16, dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    lens = torch.full((seqs,), length, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if seqs > 1:
        q = torch.ones(seqs, 8, 128, dtype=t, device="cuda")
        out, seen = torch.zeros_like(q), torch.full((seqs,), float(length), dtype=torch.float64)
        kw = dict(alibi_slopes=torch.zeros(8, device="cuda")) if form == "clusters" else {}  # (ALiBi: always in clusters)
        pa.pa_decode_fp4(out, q, k, v, table, lens, scale, 1.0, unit, err_flag=err, **kw)
    else:
        n = 1200 if form == "split tiles" else 1200 * 16
        q = torch.ones(n, 8, 128, dtype=t, device="cuda")
        out, seen = torch.zeros_like(q), torch.arange(length - n + 1, length + 1, dtype=torch.float64)
        start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        pa.pa_prefill_fp4(out, q, k, v, table, lens, start, n, scale, 1.0, unit, err_flag=err)
    assert int(err.item()) == 0
    w = (seen - 1) * 2.0 ** -25.5
    want = (w / (1 + w))[:, None, None]
    far = ((out.cpu().double() - want).abs() / (2.0 ** -11 * 1.25 + want * (2.0 ** -8 + 2.0 ** -6))).max().item()
    assert far <= 1, far
