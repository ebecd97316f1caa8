"""The paged cache as a serving loop uses it: one cache of several layers, prompts admitted, a shared
system prompt, decode steps, sequences forked, freed and compacted -- against a plain record of
every sequence's keys and values, attended densely in float64."""

import numpy as np
import pytest
import torch

import oracle
from exact_io_aware_91_b200 import api

pytestmark = pytest.mark.gpu
PS, HKV, H, D, LAYERS = 16, 2, 8, 64, 2


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)
    yield
    assert api.fa_last_device_status() == api.FA_OK


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


class Server:
    """Row 0 of the table holds the system prompt; the other rows are sequences.  `seen` records what
    each row was given: (K, V) per layer as float64 arrays (H_kv, n, d)."""

    def __init__(self, rows, pages, seed, dtype=torch.bfloat16, width=20):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.dtype = dtype
        self.pool = torch.full((2 * LAYERS, pages, HKV, PS, D), float("nan"), dtype=dtype, device="cuda")
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.seen = [None] * rows
        self.rows = rows

    def state(self):
        return PS, self.table, self.lens, self.refs

    def feed(self, new):
        """new: tokens to add per row (0: none).  One reserve, then one write per layer."""
        T = max(new)
        want = [self.len_of(b) + n if n else -1 for b, n in enumerate(new)]
        api.fa_pages_reserve(*self.state(), i32(want))
        some = [b for b, n in enumerate(new) if n]
        lens = self.lens.clone()
        lens[[b for b in range(self.rows) if b not in some]] = -1  # the others are not written to
        for layer in range(LAYERS):
            k, v = (torch.randn(self.rows, HKV, T, D, generator=self.g, device="cuda", dtype=self.dtype)
                    for _ in range(2))
            # a row with fewer tokens has them at the end: the ones in front belong to positions it
            # already has, so they are the old ones again
            for b in some:
                for x, which in ((k, 0), (v, 1)):
                    old = T - new[b]
                    have = self.len_of(b)
                    if old and have:
                        m = min(old, have)
                        past = torch.from_numpy(self.seen[b][layer][which][:, have - m:have]).cuda()
                        x[b, :, old - m:old] = past.to(self.dtype)
            api.fa_pages_write(k, v, self.pool[2 * layer], self.pool[2 * layer + 1], self.table, lens)
            for b in some:
                add = [x[b, :, T - new[b]:].double().cpu().numpy() for x in (k, v)]
                if self.seen[b] is None:
                    self.seen[b] = [None] * LAYERS
                self.seen[b][layer] = add if self.seen[b][layer] is None else [
                    np.concatenate([p, a], axis=1) for p, a in zip(self.seen[b][layer], add)]

    def len_of(self, b):
        return 0 if self.seen[b] is None or self.seen[b][-1] is None else self.seen[b][-1][0].shape[1]

    def free(self, rows):
        api.fa_pages_free(*self.state(), i32(rows))
        for b in rows:
            self.seen[b] = None

    def fork(self, parents, children):
        api.fa_pages_fork(self.pool, *self.state(), i32(parents), i32(children))
        for p, c in zip(parents, children):
            self.seen[c] = [[x.copy() for x in kv] for kv in self.seen[p]]

    def compact(self):
        api.fa_pages_compact(self.pool, *self.state(), block_table_out=self.table, ref_counts_out=self.refs)
        n = int((self.refs > 0).sum())
        assert (self.refs[:n] > 0).all() and not self.refs[n:].any()

    def attend(self, T):
        """Attention of the newest T tokens of every sequence, all layers, behind the system prompt."""
        assert api.fa_last_device_status() == api.FA_OK
        P = self.len_of(0)
        for layer in range(LAYERS):
            q = torch.randn(self.rows - 1, H, T, D, generator=self.g, device="cuda", dtype=self.dtype)
            o, lse = api.fa_paged_attn(q, self.pool[2 * layer], self.pool[2 * layer + 1], self.table[1:], self.lens[1:],
                                       prefix_table=self.table[0], prefix_len=P, causal=True)
            for b in range(1, self.rows):
                if self.seen[b] is None:
                    continue
                k, v = (np.concatenate([self.seen[0][layer][i], self.seen[b][layer][i]], axis=1) for i in range(2))
                n, m = k.shape[1], self.len_of(b)
                live = min(T, m)  # queries in front of the sequence see the prefix only
                full = np.zeros((1, H, n, D))
                full[0, :, n - live:] = q[b - 1, :, T - live:].double().cpu().numpy()
                O, L = oracle.attention_forward_gqa(full, k[None], v[None], D ** -0.5, True)
                # |V| is below 5 and a weight is off by half a step: two half steps of 5 bound o's error
                tol = 2 * 5 * torch.finfo(self.dtype).eps / 2
                np.testing.assert_allclose(o[b - 1, :, T - live:].double().cpu().numpy(), O[0, :, n - live:], atol=tol)
                np.testing.assert_allclose(lse[b - 1, :, T - live:].double().cpu().numpy(), L[0, :, n - live:],
                                           atol=1e-4, rtol=0)
        assert api.fa_last_device_status() == api.FA_OK


@pytest.mark.parametrize("dtype,system", [(torch.bfloat16, 37), (torch.float16, 160), (torch.bfloat16, 1)])
def test_a_serving_run(dtype, system):
    s = Server(rows=9, pages=70, seed=system, dtype=dtype)
    s.feed([system] + [0] * 8)
    s.feed([0, 21, 40, 5, 0, 0, 0, 0, 0])      # prompts of different lengths
    s.attend(3)
    for _ in range(4):                          # decode
        s.feed([0, 1, 1, 1, 0, 0, 0, 0, 0])
        s.attend(1)
    s.fork([1, 1, 2, 3], [4, 5, 6, 7])          # samples of the answers so far
    s.attend(1)
    for _ in range(9):                          # they go apart, over page borders
        s.feed([0, 1, 1, 1, 1, 1, 1, 1, 0])
    s.attend(4)
    s.free([1, 6, 3])
    s.compact()
    s.attend(2)
    s.feed([0, 30, 2, 0, 1, 3, 17, 1, 50])      # freed rows taken by new prompts beside running ones
    s.attend(5)
    s.free([6])
    s.fork([8, 1], [3, 6])
    s.compact()
    s.feed([0, 1, 1, 1, 1, 1, 1, 1, 1])
    s.attend(1)
    s.free(list(range(9)))
    assert not s.refs.any() and (s.lens == -1).all()


def test_a_decode_step_replayed_as_a_graph():
    # reserve, write and attention captured once; lengths, tables and tokens change between replays
    s = Server(rows=5, pages=60, seed=9)
    s.feed([40, 10, 31, 16, 0])
    k, v, want = (torch.zeros(4, HKV, 1, D, dtype=s.dtype, device="cuda") for _ in range(3))
    want = torch.full((5,), -1, dtype=torch.int32, device="cuda")
    q, o = (torch.zeros(4, H, 1, D, dtype=s.dtype, device="cuda") for _ in range(2))
    lse = torch.zeros(4, H, 1, device="cuda")
    pr = api.paged_problem(q, s.pool[0], s.pool[1], s.table[1:], 40)
    ws = torch.empty(api.fa_paged_attn_workspace_size(pr), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(api.fa_pages_workspace_size(5, 60), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.fa_pages_reserve(*s.state(), want, workspace=ws2)
        api.fa_pages_write(k, v, s.pool[0], s.pool[1], s.table[1:], s.lens[1:])
        api.fa_paged_attn(q, s.pool[0], s.pool[1], s.table[1:], s.lens[1:], s.table[0], 40, o=o, lse=lse, workspace=ws)
    for step in range(20):
        if step == 7:
            s.free([2])
        live = [b for b in range(1, 5) if s.seen[b] is not None]
        for x in (k, v, q):
            x.normal_(generator=s.g)
        want.copy_(i32([-1] + [s.len_of(b) + 1 if b in live else -1 for b in range(1, 5)]))
        o.fill_(3.0)
        graph.replay()
        for b in live:
            s.seen[b][0] = [np.concatenate([a, x[b - 1].double().cpu().numpy()], axis=1)
                            for a, x in zip(s.seen[b][0], (k, v))]
            s.seen[b][1] = s.seen[b][0]
            kk, vv = (np.concatenate([s.seen[0][0][i], s.seen[b][0][i]], axis=1) for i in range(2))
            full = np.zeros((1, H, kk.shape[1], D))
            full[0, :, -1:] = q[b - 1].double().cpu().numpy()
            O, L = oracle.attention_forward_gqa(full, kk[None], vv[None], D ** -0.5, True)
            np.testing.assert_allclose(o[b - 1].double().cpu().numpy(), O[0, :, -1:], atol=2 * 5 * 2.0 ** -8)
            np.testing.assert_allclose(lse[b - 1].double().cpu().numpy(), L[0, :, -1:], atol=1e-4, rtol=0)
        for b in range(1, 5):
            if b not in live:
                assert (o[b - 1] == 3).all()
    assert api.fa_last_device_status() == api.FA_OK


def test_two_calls_at_a_time_on_their_own_streams_and_workspaces():
    s = Server(rows=6, pages=80, seed=3)
    s.feed([90, 100, 3, 150, 60, 17])
    qs = [torch.randn(5, H, t, D, generator=s.g, device="cuda", dtype=s.dtype) for t in (1, 6)]
    run = lambda q, stream=None: api.fa_paged_attn(q, s.pool[0], s.pool[1], s.table[1:], s.lens[1:], s.table[0], 90,  # noqa: E731
                                                   stream=stream)
    want = [[x.clone() for x in run(q)] for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [run(q, st) for q, st in zip(qs, streams)]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert all(torch.equal(a, b) for a, b in zip(w, g))


def test_compacting_a_cache_without_pages_passes_the_table_on():
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    lens = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    out, refs, page_map = api.fa_pages_compact(torch.zeros(1, 0, 8, device="cuda"), 8, table, lens, none)
    assert torch.equal(out, table) and refs.numel() == page_map.numel() == 0
