"""Block tables on the GPU: batches without a request (needs a GB300)."""
import numpy as np
import pytest

from test_gpu_tables import Device, Model

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def pa():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_32_gb300 as pa
    pa.build()
    return pa


@pytest.mark.parametrize("rows", [0, 3])
def test_no_requests(pa, rows):
    """query_start is the one sum there is, 0, whatever it held; the stack stays."""
    d = Device(Model(0, 4, 16, 8, np.random.default_rng(0)), rows)
    free = d.free.clone()
    for _ in range(2):
        d.extend(pa, [])
        assert d.error() == 0 and d.start.tolist() == [0] and d.slots.tolist() == [-1] * rows
        d.start.fill_(77)
        d.trim(pa, [])
    assert d.top.tolist() == [8] and d.free.tolist() == free.tolist()
