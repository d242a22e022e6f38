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
