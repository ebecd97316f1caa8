"""What the paged cache promises at its limits: calls whose two forms share shared memory, values that are
not finite or near the end of their type, waits that give up, long lists of pages."""

import time

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


# few: own keys in the few-rows form, alone, with a prefix in the same form, or in the dense one; dense: T = 40
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,prefix", [(1, 0), (1, 200), (1, 6100), (40, 0), (40, 500)])
@pytest.mark.parametrize("segment", [1, 2, 4])
def test_waits_that_give_up_end_the_call(d, T, prefix, segment):
    rng = np.random.default_rng(d + T + prefix)
    lens = [int(x) for x in rng.integers(1, 300, 200)] + [-1, 3000, 0, 7]  # five items per CTA and more
    c = Cache(lens, prefix, 4, d, 32, BF16, seed=d)
    q = c.queries(16, T)
    table, n, pre = i32(c.table), i32(lens), i32(c.prefix) if prefix else None
    want = api.fa_paged_attn(q, c.k, c.v, table, n, pre, prefix)
    ws = torch.empty(api.fa_paged_attn_workspace_size(api.paged_problem(q, c.k, c.v, table, prefix)),
                     dtype=torch.uint8, device="cuda")
    o, lse = torch.full_like(q, 3.0), torch.full(q.shape[:3], 5.0, device="cuda")
    assert api.fa_last_device_status() == api.FA_OK
    stream = torch.cuda.current_stream()
    for fill in (0, 0x7F, 0xFF):  # what the notes that nobody writes hold
        ws.fill_(fill)
        api.fa_selftest_paged_give_up(q, c.k, c.v, table, n, pre, prefix, o, lse, ws, segment)
        t0 = time.time()
        while not stream.query():
            assert time.time() - t0 < 30.0, "the call did not end"
        assert api.fa_last_device_status() == api.FA_ERR_TIMEOUT
        dead = lens.index(-1)
        assert bool((o[dead] == 3.0).all()) and bool((lse[dead] == 5.0).all())
    got = api.fa_paged_attn(q, c.k, c.v, table, n, pre, prefix, workspace=ws)
    live = n >= 0  # the others hold whatever new memory held
    assert all(torch.equal(a[live], b[live]) for a, b in zip(want, got))


def test_giving_up_at_a_part_that_no_cta_has_changes_nothing():
    c = Cache([100, 7, 3000], 50, 2, 64, 16, BF16)
    q = c.queries(8, 1)
    table, n, pre = i32(c.table), i32(c.lens), i32(c.prefix)
    want = api.fa_paged_attn(q, c.k, c.v, table, n, pre, 50)
    o, lse = torch.zeros_like(q), torch.zeros_like(want[1])
    ws = torch.empty(api.fa_paged_attn_workspace_size(api.paged_problem(q, c.k, c.v, table, 50)), dtype=torch.uint8,
                     device="cuda")
    api.fa_selftest_paged_give_up(q, c.k, c.v, table, n, pre, 50, o, lse, ws, 1 << 30)
    assert api.fa_last_device_status() == api.FA_OK
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
