"""What the paged cache promises at its limits: calls whose two forms share shared memory, values that are
not finite or near the end of their type, waits that give up, long lists of pages."""

import numpy as np
import pytest
import torch

from exact_io_aware_91_b200 import api
from test_gpu_paged import BF16, F16, Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)
    yield
    assert api.fa_last_device_status() == api.FA_OK


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


@pytest.mark.parametrize("d,prefix", [(128, 3100), (256, 3100)])
def test_short_rows_then_a_dense_prefix_on_the_same_shared_memory(d, prefix):
    # own keys in the few-rows form, the prefix in the dense one: half of the CTAs go from the first to the
    # second, whose ring holds what the first one's row sums were in
    rng = np.random.default_rng(d)
    c = Cache([int(x) for x in rng.integers(1, 300, 100)], prefix, 4, d, 32, BF16, seed=d)
    q = c.queries(16, 1)
    table, lens, pre = i32(c.table), i32(c.lens), i32(c.prefix)
    run = lambda: api.fa_paged_attn(q, c.k, c.v, table, lens, pre, prefix)  # noqa: E731
    want = run()
    c.check(q, want)
    for got in [run() for _ in range(50)]:
        assert all(torch.equal(a, b) for a, b in zip(want, got))
