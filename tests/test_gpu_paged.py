"""Attention over the paged cache (fa_paged_attn) on the GPU against the float64 definition.

Tolerances.  u is half a step of the tensors' type (torch.finfo(type).eps / 2).  A score is a sum
of d products accumulated in fp32, each addition off by at most 2^-23 of the running sum of
magnitudes (the tensor core may truncate), so it is off by at most d 2^-23 max_j scale sum_i
|q_i k_ji|; as an exponent that, the fp32 arithmetic of the softmax (a few 2^-22) and the sums over
n keys (n 2^-23) make up the relative error `delta` of every weight.  The weights are rounded to
the type once (u) for the product with V, not for the row sum, hence
    |o - exact| <= u |o| + (u + 2 delta) sum_j p_j |v_j|    (+ fp16: 2^-25 sum_j |v_j| for weights
    below fp16's normal range; the row sum is at least 1)
    |lse - exact| <= 2 delta + 2^-22 |lse|.
"""

import numpy as np
import pytest
import torch

from oracle import paged_attention
from exact_io_aware_91_b200 import api

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)
    yield
    assert api.fa_last_device_status() == api.FA_OK


class Cache:
    """A pool of pages with the tokens of sequences and of a prefix in scattered pages; every slot
    that no sequence uses holds NaN."""

    def __init__(self, lens, prefix_len, hkv, d, ps, dtype, seed=0, order="head", spiky=0.0, spare=3):
        g = np.random.default_rng(seed)
        per = [-(-max(0, x) // ps) for x in lens]
        n_pre = -(-prefix_len // ps)
        pages = sum(per) + n_pre + spare
        ids = g.permutation(pages)
        width = max(1, max(per, default=1)) + 1
        self.table = np.full((len(lens), width), -7, np.int32)  # entries nobody owns are never followed
        self.prefix = ids[:n_pre].astype(np.int32)
        at = n_pre
        pools = np.full((2, pages, hkv, ps, d), np.nan, np.float32)
        for tab, n in [(self.prefix, prefix_len)] + [(self.table[b], lens[b]) for b in range(len(lens))]:
            if tab is not self.prefix:
                k = -(-max(0, n) // ps)
                tab[:k] = ids[at:at + k]
                at += k
            for e in range(-(-max(0, n) // ps)):
                m = min(ps, n - e * ps)
                pools[:, tab[e], :, :m] = g.standard_normal((2, hkv, m, d))
                if spiky:
                    loud = g.random((hkv, m, 1)) < spiky
                    pools[0, tab[e], :, :m] *= np.where(loud, 8.0, 1.0)
        t = torch.from_numpy(pools).to(dtype).cuda()
        if order == "token":  # (num_pages, page_size, H_kv, d) in memory
            t = t.transpose(2, 3).contiguous().transpose(2, 3)
        elif order == "mixed":  # K and V of a page side by side, rows padded
            wide = torch.full((pages, 2, hkv, ps, d + 8), float("nan"), dtype=dtype, device="cuda")
            wide[..., :d] = t.transpose(0, 1)
            t = wide[..., :d].transpose(0, 1)
        self.k, self.v = t[0], t[1]
        self.lens, self.prefix_len, self.d, self.dtype = list(lens), prefix_len, d, dtype
        self.g = g

    def run(self, q, causal=True, scale=None, **kw):
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
        return api.fa_paged_attn(q, self.k, self.v, dev(self.table), dev(self.lens),
                                 prefix_table=dev(self.prefix) if self.prefix_len else None,
                                 prefix_len=self.prefix_len, causal=causal, scale=scale, **kw)

    def check(self, q, got, causal=True, scale=None):
        o, lse = (x.double().cpu().numpy() for x in got)
        scale = self.d ** -0.5 if scale is None else scale
        O, L, mean_abs, sum_abs, big, n = paged_attention(q, self.k, self.v, self.table, self.lens, self.prefix,
                                                          self.prefix_len, scale, causal)
        u = torch.finfo(self.dtype).eps / 2
        delta = 2.0 ** -23 * (self.d * big + n + 8)
        tol = u * np.abs(O) + (u + 2 * delta[..., None]) * mean_abs
        if self.dtype == F16:
            tol = tol + 2.0 ** -25 * sum_abs
        live = np.array(self.lens) >= 0
        assert np.isfinite(o[live]).all()
        over = (np.abs(o - O) / (tol * 1.001 + 1e-30))[live]
        assert over.size == 0 or over.max() <= 1, f"o is {over.max():.3f} of its tolerance off"
        none = (n == 0) & live[:, None, None]
        assert (lse[none] == -np.inf).all() and (o[none] == 0).all()
        some = (n > 0) & live[:, None, None]
        err = np.abs(lse[some] - L[some]) / (2 * delta + 2.0 ** -22 * np.abs(L))[some]
        assert err.size == 0 or err.max() <= 1, f"lse is {err.max():.3f} of its tolerance off"

    def queries(self, H, T):
        return torch.from_numpy(self.g.standard_normal((len(self.lens), H, T, self.d))).to(self.dtype).cuda()


def case(lens, prefix, H, hkv, T, d, ps, dtype=BF16, causal=True, order="head", spiky=0.0):
    c = Cache(lens, prefix, hkv, d, ps, dtype, seed=len(lens) * 1000 + prefix + d + ps, order=order, spiky=spiky)
    q = c.queries(H, T)
    c.check(q, c.run(q, causal), causal)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("ps", [8, 16, 64, 256])
def test_types_head_dims_and_page_sizes(d, dtype, ps):
    case([1, 300, 129, 0, 17], 200, 8, 2, 1, d, ps, dtype)


@pytest.mark.parametrize("lens", [[1], [0], [127], [128], [129], [63, 64, 65], [1000, 1, 511], [2, 0, 0, 3]])
@pytest.mark.parametrize("prefix", [0, 1, 128, 391])
def test_lengths(lens, prefix):
    case(lens, prefix, 4, 2, 1, 128, 16)


@pytest.mark.parametrize("H,hkv", [(1, 1), (5, 5), (6, 1), (12, 4), (24, 2), (64, 1), (130, 1)])
@pytest.mark.parametrize("d", [64, 256])
def test_head_groups(H, hkv, d):
    case([70, 3, 260], 140, H, hkv, 1, d, 32)


@pytest.mark.parametrize("T", [2, 3, 5, 16, 33, 150])
@pytest.mark.parametrize("causal", [True, False])
def test_several_tokens(T, causal):
    case([T, T + 200, 1, 0, T - 1, 2 * T], 77, 6, 2, T, 64, 16, BF16, causal)
    case([T, 400], 0, 4, 4, T, 128, 8, F16, causal)


def test_a_prompt_of_many_tokens():
    case([600, 641], 90, 2, 1, 600, 128, 64)
    case([300], 0, 2, 1, 300, 256, 16, F16)


@pytest.mark.parametrize("order", ["token", "mixed"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_strides(order, d):
    case([100, 5, 333], 50, 6, 3, 2, d, 16, BF16, order=order)


def test_many_sequences_share_the_prefix():
    rng = np.random.default_rng(0)
    case(list(rng.integers(0, 40, 150)), 333, 4, 1, 1, 64, 16)  # 600 rows against the prefix
    case(list(rng.integers(0, 20, 45)), 700, 14, 2, 1, 128, 8)  # groups of 7 rows: 18 sequences to 126 rows
    case(list(rng.integers(0, 9, 7)), 260, 33, 1, 2, 128, 32)   # 66 rows each


@pytest.mark.parametrize("d,prefix", [(64, 6100), (128, 3100), (256, 3100)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_a_long_prefix_for_many_sequences(d, prefix, dtype):
    # enough (rows, key tile) pairs that the prefix takes the 128-row products, the sequences' own keys do not
    rng = np.random.default_rng(d)
    case([int(x) for x in rng.integers(-1, 40, 100)], prefix, 16, 4, 1, d, 32, dtype)


def test_sharp_rows():
    case([900, 40, 1500], 800, 8, 2, 1, 128, 16, BF16, spiky=0.01)
    case([900, 40, 1500], 800, 8, 2, 1, 128, 16, F16, spiky=0.01)
    case([900, 40], 300, 4, 2, 3, 256, 16, BF16, spiky=0.02)


def test_a_long_sequence_beside_short_ones():
    case([9000, 1, 30, 4000], 0, 4, 1, 1, 64, 64)


@pytest.mark.parametrize("d,ps", [(64, 16), (128, 32), (256, 64)])
@pytest.mark.parametrize("group,T", [(1, 1), (4, 1), (4, 3), (4, 5), (4, 10), (4, 40)])
def test_many_tiles_for_every_multiprocessor(d, ps, group, T):
    # some 900 (item, key tile) pairs: every multiprocessor walks over several items, some of many tiles
    rng = np.random.default_rng(d + T)
    lens = [int(x) for x in rng.integers(0, 1500, 12)] + [1, 3000]
    case(lens, 1100, 8 * group, 8, T, d, ps)
    case(lens, 0, 8 * group, 8, T, d, ps, F16)


def test_a_large_scale_and_equal_scores():
    c = Cache([200, 3], 100, 2, 64, 16, BF16, seed=4)
    q = c.queries(4, 1)
    c.check(q, c.run(q, scale=3.0), scale=3.0)
    q.zero_()  # every score is 0: o is the mean of V
    c.check(q, c.run(q))


def test_rows_without_a_sequence_are_left_as_they_were():
    c = Cache([5, -1, 30, -3], 20, 2, 64, 16, BF16, seed=1)
    q = c.queries(4, 2)
    o = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:3], 9.0, device="cuda")
    got = c.run(q, o=o, lse=lse)
    assert got[0] is o and got[1] is lse
    c.check(q, got)
    assert (o[[1, 3]] == 7).all() and (lse[[1, 3]] == 9).all()


def test_repeated_calls_are_identical_and_need_nothing_of_the_workspace():
    c = Cache([700, 31, 1200], 900, 4, 128, 16, BF16, seed=2)
    q = c.queries(16, 1)
    pr = api.paged_problem(q, c.k, c.v, torch.from_numpy(c.table).cuda(), 900)
    ws = torch.empty(api.fa_paged_attn_workspace_size(pr), dtype=torch.uint8, device="cuda")
    ref = None
    for fill in (0, 255, 77):
        ws.fill_(fill)
        got = c.run(q, workspace=ws)
        if ref is None:
            ref = [x.clone() for x in got]
            c.check(q, got)
        assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_every_block_of_a_sequence_is_read_beyond_32_bit_offsets():
    # a pool of more than 2^32 bytes (and elements) of which the sequences use the far end
    ps, hkv, d, pages = 64, 8, 128, 40000
    pool = torch.zeros(2, pages, hkv, ps, d, dtype=BF16, device="cuda")
    assert pool[0].numel() > 2 ** 31 and pool[0].numel() * 2 > 2 ** 32
    c = Cache([150, 70], 60, hkv, d, ps, BF16, seed=3)
    n = c.k.shape[0]
    far = np.array([pages - 1 - 4321 * i for i in range(n)], np.int32)
    pool[0][torch.from_numpy(far).long().cuda()] = c.k
    pool[1][torch.from_numpy(far).long().cuda()] = c.v
    q = c.queries(16, 1)
    want = c.run(q)
    c.table = np.where(c.table >= 0, far[np.maximum(c.table, 0)], c.table)
    c.prefix = far[c.prefix]
    c.k, c.v = pool[0], pool[1]
    got = c.run(q)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_bad_pages_are_left_out_and_reported():
    for entry in (-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1):
        c = Cache([100, 40], 30, 2, 64, 16, BF16, seed=5)
        q = c.queries(4, 1)
        api.fa_last_device_status()
        good = c.run(q)
        assert api.fa_last_device_status() == api.FA_OK
        c.table[0, 2] = entry
        got = c.run(q)
        assert api.fa_last_device_status() == api.FA_ERR_INDEX
        assert torch.equal(got[0][1], good[0][1])  # the other sequence has its values
        assert torch.isfinite(got[0]).all()
    c = Cache([100, 40], 30, 2, 64, 16, BF16, seed=5)
    c.lens[1] = 10 ** 7  # more than the table's row holds
    c.table[1, 3:] = 0
    c.run(c.queries(4, 1))
    assert api.fa_last_device_status() == api.FA_ERR_INDEX
    c = Cache([100, 40], 30, 2, 64, 16, BF16, seed=5)
    c.prefix[1] = -1
    c.run(c.queries(4, 1))
    assert api.fa_last_device_status() == api.FA_ERR_INDEX


def test_another_stream_and_a_captured_graph():
    c = Cache([400, 33, 1000], 500, 2, 128, 16, BF16, seed=6)
    q = c.queries(8, 1)
    want = [x.clone() for x in c.run(q)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.run(q, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    got = c.run(q, stream=side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    table, lens = (torch.from_numpy(np.asarray(x, np.int32)).cuda() for x in (c.table, c.lens))
    prefix = torch.from_numpy(c.prefix).cuda()
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")
    pr = api.paged_problem(q, c.k, c.v, table, 500)
    ws = torch.empty(api.fa_paged_attn_workspace_size(pr), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.fa_paged_attn(q, c.k, c.v, table, lens, prefix, 500, o=o, lse=lse, workspace=ws)
    for shrink in (0, 30, 100):  # the lengths are read when the graph runs
        c.lens = [400 - shrink, 33 - shrink // 4, 1000 - shrink]
        lens.copy_(torch.tensor(c.lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        c.check(q, (o, lse))


def test_no_lse_and_empty_batches():
    c = Cache([50], 0, 2, 64, 16, BF16)
    q = c.queries(4, 1)
    o, lse = c.run(q)
    lib = api.library()
    import ctypes
    table, lens = (torch.from_numpy(np.asarray(x, np.int32)).cuda() for x in (c.table, c.lens))
    pr = api.paged_problem(q, c.k, c.v, table)
    ws = torch.empty(api.fa_paged_attn_workspace_size(pr), dtype=torch.uint8, device="cuda")
    o2 = torch.zeros_like(o)
    st = lib.fa_paged_attn(ctypes.byref(pr), q.data_ptr(), c.k.data_ptr(), c.v.data_ptr(), table.data_ptr(),
                           lens.data_ptr(), None, o2.data_ptr(), None, ws.data_ptr(), ws.numel(),
                           torch.cuda.current_stream().cuda_stream)
    assert st == api.FA_OK and torch.equal(o, o2)
    got = api.fa_paged_attn(q[:0], c.k, c.v, table[:0], lens[:0])
    assert got[0].shape == (0, 4, 1, 64)
    got = api.fa_paged_attn(q[:, :, :0].contiguous(), c.k, c.v, table, lens)
    assert got[0].shape == (1, 4, 0, 64)


def test_the_binding_refuses_what_does_not_fit():
    c = Cache([50, 20], 10, 2, 64, 16, BF16)
    q = c.queries(4, 1)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    table, lens, prefix = dev(c.table), dev(c.lens), dev(c.prefix)
    good = dict(q=q, k_pages=c.k, v_pages=c.v, block_table=table, seq_lens=lens, prefix_table=prefix, prefix_len=10)
    api.fa_paged_attn(**good)
    for change in (dict(q=q.float()), dict(q=q.half()), dict(q=q.transpose(1, 2)), dict(q=q[:, :, 0]),
                   dict(k_pages=c.k.half()), dict(k_pages=c.k[:, :1]), dict(v_pages=c.v[:-1]),
                   dict(k_pages=c.k[..., :32]), dict(block_table=table.long()), dict(block_table=table[:1]),
                   dict(block_table=table.t().contiguous().t()), dict(seq_lens=lens.long()), dict(seq_lens=lens[:1]),
                   dict(seq_lens=lens.cpu()), dict(prefix_table=None), dict(prefix_len=17), dict(o=q[:1]),
                   dict(lse=torch.zeros(2, 4, device="cuda")), dict(o=q.half())):
        with pytest.raises(ValueError):
            api.fa_paged_attn(**{**good, **change})
    for change in (dict(prefix_len=-1), dict(scale=0.0), dict(workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(api.FAError):
            api.fa_paged_attn(**{**good, **change})


def test_a_batch_without_sequences_ends_before_what_follows_it():
    """Nobody wants the results, but the prefix parts of such a call are written: the next call on its
    workspace, or a write to the pages, must not meet them."""
    c = Cache([40, 9, 130, 64] * 8, 6000, 2, 128, 16, BF16)
    q = c.queries(8, 1)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
    table, lens, prefix, dead = dev(c.table), dev(c.lens), dev(c.prefix), dev([-1] * 32)
    ws = torch.empty(api.fa_paged_attn_workspace_size(api.paged_problem(q, c.k, c.v, table, 6000)),
                     dtype=torch.uint8, device="cuda")
    args = dict(block_table=table, prefix_table=prefix, prefix_len=6000)
    want, want_lse = api.fa_paged_attn(q, c.k, c.v, seq_lens=lens, **args)
    other, rest = torch.full_like(q, 3.0), torch.full_like(want, 7.0)
    rest_lse = torch.full_like(want_lse, 7.0)
    got = []
    for _ in range(20):
        api.fa_paged_attn(other, c.k, c.v, seq_lens=dead, workspace=ws, o=rest, lse=rest_lse, **args)
        got.append(api.fa_paged_attn(q, c.k, c.v, seq_lens=lens, workspace=ws, **args))
    for o, lse in got:
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
    assert bool((rest == 7.0).all()) and bool((rest_lse == 7.0).all())
