"""The page operations (fa_pages_*) on the GPU against their plain definitions: tables, lengths and
counts are whole numbers and contents are copied, so everything has to be equal."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import PageTable
from exact_io_aware_91_b200 import api

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


class Both:
    """The same cache twice: on the GPU (two planes of `page` elements each) and as the oracle's table."""

    def __init__(self, rows, width, pages, ps=8, page=(2, 3, 8), wide=0, stacked=True, planes=2, dtype=torch.bfloat16):
        self.ps = ps
        whole = torch.full((rows, width + wide), -1, dtype=torch.int32, device="cuda")
        self.table = whole[:, :width]
        self.lens = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        label = torch.arange(pages, device="cuda").view(1, -1, *[1] * len(page))
        # page p of plane i holds 3 p + i (mod 251) everywhere: exact in every type
        self.pool = ((3 * label + torch.arange(planes, device="cuda").view(-1, 1, *[1] * len(page))) % 251).expand(
            planes, pages, *page).to(dtype).contiguous()
        self.start = self.pool.clone()
        self.planes = self.pool if stacked else [self.pool[i] for i in range(planes)]
        self.o = PageTable(ps, self.table.tolist(), self.lens.tolist(), self.refs.tolist())

    def args(self):
        return self.ps, self.table, self.lens, self.refs

    def check(self):
        assert self.lens.tolist() == self.o.lens
        assert self.refs.tolist() == self.o.refs
        assert self.table.tolist() == self.o.table
        assert torch.equal(self.pool, self.start[:, self.o.content])
        assert api.fa_last_device_status() == api.FA_OK

    def reserve(self, new, status=api.FA_OK):
        api.fa_pages_reserve(*self.args(), i32(new))
        refused = self.o.reserve(new)
        assert api.fa_last_device_status() == (api.FA_ERR_NO_PAGES if refused else status)
        self.check()

    def fork(self, parents, children):
        api.fa_pages_fork(self.planes, *self.args(), i32(parents), i32(children))
        refused = self.o.fork(parents, children)
        assert api.fa_last_device_status() == (api.FA_ERR_NO_PAGES if refused else api.FA_OK)
        self.check()

    def free(self, rows):
        api.fa_pages_free(*self.args(), i32(rows))
        self.o.free([r for r in rows if r >= 0])
        self.check()

    def compact(self, in_place):
        out = (self.table, self.refs) if in_place else (None, None)
        t, r, m = api.fa_pages_compact(self.planes, *self.args(), block_table_out=out[0], ref_counts_out=out[1])
        assert m.tolist() == self.o.compact()
        self.table, self.refs = t, r
        self.check()


@pytest.mark.parametrize("stacked,wide,ps,planes", [(True, 0, 8, 2), (False, 3, 16, 5), (False, 0, 64, 300)])
def test_a_long_run_of_operations(stacked, wide, ps, planes):
    rng = np.random.default_rng(ps)
    rows, width, pages = 40, 9, 200
    c = Both(rows, width, pages, ps, wide=wide, stacked=stacked, planes=planes)
    for step in range(60):
        what = step % 4 if step < 8 else rng.integers(0, 4)
        if what == 0:
            c.reserve([int(x) if rng.random() < 0.3 else -1 for x in rng.integers(0, ps * width + 1, rows)])
        elif what == 1:
            live = [b for b in range(rows) if c.o.lens[b] >= 0]
            empty = [b for b in range(rows) if c.o.lens[b] < 0]
            if live and empty:
                kids = [int(b) for b in rng.permutation(empty)[:11]]
                c.fork([int(rng.choice(live)) for _ in kids], kids)
        elif what == 2:
            rows_out = [int(b) for b in rng.permutation(rows)[:9]]
            c.free(rows_out + [-1, rows_out[0], rows_out[3]])  # padding and second mentions
        else:
            c.compact(in_place=bool(step & 1))


def test_large_tables():
    # more pages than the deciding block scans in one step, more rows than its threads
    c = Both(1500, 12, 9001, 16, page=(8,), planes=1)
    rng = np.random.default_rng(1)
    c.reserve([int(x) for x in rng.integers(0, 16 * 12 + 1, 1500)])
    c.free([int(b) for b in rng.permutation(1500)[:700]])
    c.compact(in_place=False)
    empty = [b for b in range(1500) if c.o.lens[b] < 0]
    live = [b for b in range(1500) if c.o.lens[b] > 0]
    c.fork([int(x) for x in rng.choice(live, len(empty))], empty)
    c.free(live)
    c.compact(in_place=True)


def test_rows_are_served_in_order_until_pages_run_out():
    c = Both(5, 4, 7, 8)
    c.reserve([9, 24, 32, 0, 1])  # 2 + 3 fit, 4 do not, and what comes after does not either
    assert c.lens.tolist() == [9, 24, -1, -1, -1]
    c.reserve([16, 24, 3, -1, 9])  # no new page for row 0, one for row 2, then too few
    assert c.lens.tolist() == [16, 24, 3, -1, -1]
    c.free([0])
    c.fork([1, 1, 2], [0, 3, 4])  # full pages shared, one copied
    assert c.refs.tolist().count(3) == 3
    c.free([0, 1, 2, 3, 4])
    assert not c.refs.any()


def test_a_length_beyond_the_table_is_reported():
    c = Both(3, 2, 10, 8)
    api.fa_pages_reserve(*c.args(), i32([17, 16, 2 ** 31 - 1]))
    assert api.fa_last_device_status() == api.FA_ERR_INDEX
    c.o.reserve([-1, 16, -1])
    c.check()


def test_bad_rows_and_forks_are_left_out_and_reported():
    c = Both(6, 3, 20, 8)
    c.reserve([10, 20, 5, -1, -1, -1])
    for rows in ([6], [2 ** 31 - 1]):
        api.fa_pages_free(*c.args(), i32(rows))
        assert api.fa_last_device_status() == api.FA_ERR_INDEX
        c.check()
    for par, chi in (([0], [0]), ([0], [6]), ([7], [3]), ([3], [4]), ([0], [1]), ([0, 4], [4, 5]), ([4, 0], [3, 4])):
        api.fa_pages_fork(c.planes, *c.args(), i32(par), i32(chi))
        assert api.fa_last_device_status() == api.FA_ERR_INDEX, (par, chi)
        c.check()
    api.fa_pages_fork(c.planes, *c.args(), i32([0, 1, -1, 1]), i32([3, 3, 4, -1]))  # the first of two counts
    assert api.fa_last_device_status() == api.FA_ERR_INDEX
    c.o.fork([0], [3])
    c.check()
    # an entry that nobody counted: its count stays 0
    c.refs[c.table[2, 0].item()] = 0
    api.fa_pages_free(*c.args(), i32([2]))
    assert api.fa_last_device_status() == api.FA_ERR_INDEX
    assert (c.refs >= 0).all() and c.lens[2] == -1
    # an entry that names no page
    c.table[1, 1] = 99
    api.fa_pages_free(*c.args(), i32([1]))
    assert api.fa_last_device_status() == api.FA_ERR_INDEX
    assert (c.refs >= 0).all()


@pytest.mark.parametrize("page,dtype", [((8,), torch.bfloat16), ((2, 16, 64), torch.float16), ((3, 8, 128), torch.float32),
                                        ((16, 33), torch.uint8), ((1, 1024, 17), torch.bfloat16)])
@pytest.mark.parametrize("n", [1, 13, 40])
def test_copy(page, dtype, n):
    c = Both(1, 1, 90, page=page, dtype=dtype, planes=3)
    order = np.random.default_rng(n).permutation(90)
    src, dst = order[:n].copy(), order[n:2 * n].copy()
    if n > 2:
        src[1], dst[2] = src[0], -1  # one source twice, one pair skipped
    api.fa_pages_copy(c.planes, i32(src), i32(dst))
    want = c.start.clone()
    for s, d in zip(src, dst):
        if d >= 0:
            want[:, d] = c.start[:, s]
    assert torch.equal(c.pool, want)


def test_conflicting_copies_are_left_out_and_reported():
    for src, dst, done in (([1, 2], [5, 5], [(1, 5)]),        # the first of two with one dst
                           ([1, 5], [5, 6], [(5, 6)]),        # dst 5 is read by another pair
                           ([1, 2], [2, 1], []),              # a swap
                           ([1, 20, 3], [5, 6, 20], []),      # 20 pages: 0..19 (and 1 -> 5 below)
                           ([4, 4, -1], [4, 9, 9], [(4, 9)])):  # a page onto itself is no copy
        c = Both(1, 1, 20, page=(40,))
        api.fa_pages_copy(c.planes, i32(src), i32(dst))
        bad = (src, dst) != ([4, 4, -1], [4, 9, 9])
        assert api.fa_last_device_status() == (api.FA_ERR_INDEX if bad else api.FA_OK)
        if src == [1, 20, 3]:
            done = [(1, 5)]
        want = c.start.clone()
        for s, d in done:
            want[:, d] = c.start[:, s]
        assert torch.equal(c.pool, want), (src, dst)


def test_pages_with_space_between_them():
    whole = torch.arange(2 * 10 * 64, device="cuda").view(2, 10, 64).to(torch.int32)
    want = whole.clone()
    api.fa_pages_copy([whole[0, :, :32], whole[1, :, :32]], i32([1, 2]), i32([7, 8]))
    want[:, 7, :32], want[:, 8, :32] = whole[:, 1, :32], whole[:, 2, :32]
    assert torch.equal(whole, want)


@pytest.mark.parametrize("d,ps,T,dtype", [(64, 8, 1, torch.bfloat16), (128, 16, 5, torch.float16), (256, 32, 40, torch.bfloat16)])
@pytest.mark.parametrize("order", ["head", "token"])
def test_write(d, ps, T, dtype, order):
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    lens = [T, 3 * ps + 1, 0, -1, 1, ps * 4]
    pages, hkv = 40, 3
    shape = (2, pages, hkv, ps, d) if order == "head" else (2, pages, ps, hkv, d)
    pool = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
    pool = pool if order == "head" else pool.transpose(2, 3)
    table = torch.randperm(pages, generator=g, device="cuda").int()[:6 * 6].view(6, 6)
    lens = [x if -(-x // ps) <= 6 else 6 * ps for x in lens]
    k, v = (torch.randn(6, hkv, T, d, generator=g, device="cuda", dtype=dtype) for _ in range(2))
    want = pool.clone()
    for b, n in enumerate(lens):
        for t in range(T):
            pos = n - T + t
            if n >= 0 and pos >= 0:
                want[0, table[b, pos // ps], :, pos % ps] = k[b, :, t]
                want[1, table[b, pos // ps], :, pos % ps] = v[b, :, t]
    api.fa_pages_write(k, v, pool[0], pool[1], table, i32(lens))
    assert torch.equal(pool, want)
    # entries and lengths out of range write nothing and are reported
    table = table.clone()
    table[0] = -5
    table[1] = pages
    lens = [1, 1, 6 * ps + 1, -1, -1, -1]
    api.fa_pages_write(k[:, :, :1].contiguous(), v[:, :, :1].contiguous(), pool[0], pool[1], table, i32(lens))
    assert api.fa_last_device_status() == api.FA_ERR_INDEX
    assert torch.equal(pool, want)


def test_captured_and_on_another_stream():
    c = Both(8, 5, 60, 8)
    ws = torch.empty(api.fa_pages_workspace_size(8, 60), dtype=torch.uint8, device="cuda")
    new, rows = i32([9, -1, 30, -1, 12, -1, -1, 40]), i32([0, 7])
    par, chi = i32([2, 2, 4]), i32([1, 3, 5])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        api.fa_pages_reserve(*c.args(), new, workspace=ws)
        api.fa_pages_fork(c.planes, *c.args(), par, chi, workspace=ws)
        api.fa_pages_free(*c.args(), rows)
        api.fa_pages_compact(c.planes, *c.args(), block_table_out=c.table, ref_counts_out=c.refs,
                             page_map=torch.empty(60, dtype=torch.int32, device="cuda"), workspace=ws)
    c.check()  # capturing ran nothing
    graph.replay()
    torch.cuda.synchronize()
    c.o.reserve([9, -1, 30, -1, 12, -1, -1, 40])
    c.o.fork([2, 2, 4], [1, 3, 5])
    c.o.free([0, 7])
    c.o.compact()
    c.check()
    api.fa_pages_free(*c.args(), i32([1, 2, 3]), stream=side)
    api.fa_pages_reserve(*c.args(), i32([5] * 8), stream=side)
    side.synchronize()
    c.o.free([1, 2, 3])
    c.o.reserve([5] * 8)
    c.check()


def test_the_binding_refuses_what_does_not_fit():
    c = Both(4, 3, 20)
    one = i32([1])
    with pytest.raises(ValueError):
        api.fa_pages_copy(c.pool[0, 0, 0], one, one)  # two dimensions: no planes
    with pytest.raises(ValueError):
        api.fa_pages_copy([c.pool[0], c.pool[1].float()], one, one)
    with pytest.raises(ValueError):
        api.fa_pages_copy([c.pool[0].transpose(1, 2)], one, one)
    with pytest.raises(ValueError):
        api.fa_pages_copy(c.pool, one, i32([1, 2]))
    with pytest.raises(ValueError):
        api.fa_pages_reserve(*c.args(), one)
    with pytest.raises(ValueError):
        api.fa_pages_free(8, c.table.long(), c.lens, c.refs, one)
    with pytest.raises(ValueError):
        api.fa_pages_free(8, c.table, c.lens[:2], c.refs, one)
    with pytest.raises(ValueError):
        api.fa_pages_compact(c.planes, *c.args(), page_map=one)
    with pytest.raises(ValueError):
        api.fa_pages_compact(c.planes, *c.args(), block_table_out=c.table[:2])
    with pytest.raises(api.FAError):
        api.fa_pages_fork(c.planes, *c.args(), i32([0] * 5), i32([1] * 5))
    with pytest.raises(api.FAError):
        api.fa_pages_compact(c.pool[:, :10], *c.args())
    with pytest.raises(api.FAError):
        api.fa_pages_free(12, *c.args()[1:], one)


@pytest.mark.parametrize("n_planes,page_bytes", [(0, 0), (0, 96), (2, 0)])
def test_tables_alone(n_planes, page_bytes):
    """No planes, or pages without bytes: tables and counts change as ever, and lists are checked."""
    c = Both(4, 6, 20)
    lib, stream = api.library(), torch.cuda.current_stream().cuda_stream
    ptrs = (ctypes.c_void_p * 2)(c.pool.data_ptr(), c.pool.data_ptr())
    pl = api.FaPagePlanes(ctypes.cast(ptrs, ctypes.POINTER(ctypes.c_void_p)), n_planes, 20, page_bytes, page_bytes)
    t = api.FaPageTable(4, 6, c.table.stride(0), c.ps, 20, c.table.data_ptr(), c.lens.data_ptr(), c.refs.data_ptr())
    ws = torch.empty(api.fa_pages_workspace_size(4, 20), dtype=torch.uint8, device="cuda")
    pl, t = ctypes.byref(pl), ctypes.byref(t)
    c.reserve([20, -1, -1, 8])
    par, chi, old, new = i32([0, 3]), i32([1, 2]), i32([0, 25]), i32([7, 3])
    assert lib.fa_pages_fork(pl, t, par.data_ptr(), chi.data_ptr(), 2, ws.data_ptr(), ws.numel(), stream) == api.FA_OK
    c.o.fork([0, 3], [1, 2])
    c.o.content = list(range(20))  # nothing is copied
    c.check()
    c.free([0])
    out = torch.empty(20, dtype=torch.int32, device="cuda")
    assert lib.fa_pages_compact(pl, t, c.table.data_ptr(), c.refs.data_ptr(), out.data_ptr(), ws.data_ptr(),
                                ws.numel(), stream) == api.FA_OK
    assert out.tolist() == c.o.compact()
    c.o.content = list(range(20))
    c.check()
    assert lib.fa_pages_copy(pl, old.data_ptr(), new.data_ptr(), 2, stream) == api.FA_OK
    assert api.fa_last_device_status() == api.FA_ERR_INDEX
    c.check()


def test_pages_without_elements_and_pools_without_pages():
    c = Both(4, 6, 20)
    empty = torch.empty(2, 20, 0, dtype=torch.bfloat16, device="cuda")
    c.reserve([20, -1, -1, 8])
    api.fa_pages_fork(empty, *c.args(), i32([0, 3]), i32([1, 2]))
    c.o.fork([0, 3], [1, 2])
    c.o.content = list(range(20))
    c.check()
    api.fa_pages_copy(empty, i32([0, 1]), i32([7, 8]))
    c.check()
    api.fa_pages_copy(c.pool[:, :0], i32([-1, 2]), i32([3, 2]))  # skipped, both of them
    assert api.fa_last_device_status() == api.FA_OK
    api.fa_pages_copy(c.pool[:, :0], i32([1]), i32([0]))
    assert api.fa_last_device_status() == api.FA_ERR_INDEX
    Both(3, 2, 0).reserve([4, -1, 0])  # nobody is served
