"""What the paged cache promises at its limits: calls whose two forms share shared memory, values that are
not finite or near the end of their type, waits that give up, long lists of pages."""

import time

import numpy as np
import pytest
import torch

from oracle import paged_attention
from exact_io_aware_91_b200 import api
from test_gpu_paged import BF16, F16, Cache
from test_gpu_pages import Both

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


def legal(parents, children, lens):
    """The forks that their description lets happen, each held against all others."""
    keep = []
    pairs = list(zip(parents, children))
    for i, (p, c) in enumerate(pairs):
        if p < 0 or c < 0:
            continue
        others = [x for j, x in enumerate(pairs) if j != i and min(x) >= 0]
        bad = p >= len(lens) or c >= len(lens) or p == c
        bad = bad or lens[p] < 0 or lens[c] > 0
        bad = bad or any(x[1] == p or x[0] == c for x in others) or any(x[1] == c for x in pairs[:i] if min(x) >= 0)
        if not bad:
            keep.append(i)
    return keep


@pytest.mark.parametrize("seed", range(12))
def test_forks_that_exclude_one_another(seed):
    rng = np.random.default_rng(seed)
    c = Both(30, 3, 200, 8)
    c.reserve([int(x) if x else -1 for x in rng.integers(0, 24, 30)])
    n = int(rng.integers(1, 31))
    ids = lambda k: [int(x) for x in rng.integers(-2, 33, k)]  # noqa: E731
    live, empty = ([b for b in range(30) if (c.o.lens[b] >= 0) == yes] for yes in (True, False))
    par = [int(rng.choice(live)) if live and rng.random() < 0.8 else x for x in ids(n)]
    chi = [int(rng.choice(empty)) if empty and rng.random() < 0.8 else x for x in ids(n)]
    keep = legal(par, chi, c.o.lens)
    bad = len(keep) < sum(1 for p, x in zip(par, chi) if p >= 0 and x >= 0)
    api.fa_pages_fork(c.planes, *c.args(), i32(par), i32(chi))
    assert api.fa_last_device_status() == (api.FA_ERR_INDEX if bad else api.FA_OK)
    c.o.fork([par[i] for i in keep], [chi[i] for i in keep])
    c.check()


def test_a_quarter_of_a_million_forks():
    n = 1 << 18
    c = Both(2 * n, 1, 2 * n, 8, page=(8,), planes=1)
    c.reserve([1 + b % 8 if b < n else -1 for b in range(2 * n)])  # one in eight has a full page
    order = np.random.default_rng(0).permutation(n)
    par, chi = i32(order), i32(np.arange(n, 2 * n))
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    api.fa_pages_fork(c.planes, *c.args(), par, chi)
    b.record()
    assert not c.o.fork([int(x) for x in order], list(range(n, 2 * n)))
    c.check()
    assert a.elapsed_time(b) < 60  # ms; each fork against every other one is some hundreds


def copied(src, dst, pages):
    """The pairs that the description of fa_pages_copy lets happen, and whether any is left out."""
    pairs = [(int(s), int(d)) for s, d in zip(src, dst)]
    used = [(s, d) for s, d in pairs if s >= 0 and d >= 0 and s != d]
    good = [(s, d) for s, d in used if s < pages and d < pages]
    sources, seen, done = {s for s, _ in good}, set(), []
    for s, d in good:
        if d not in sources and d not in seen:
            done.append((s, d))
        seen.add(d)
    return done, len(done) < len(used)


@pytest.mark.parametrize("n,clean", [(3000, True), (32767, True), (32768, True), (49999, True), (3000, False),
                                     (32767, False), (32768, False), (49999, False), (1 << 21, False)])
def test_long_lists_of_copies(n, clean):
    rng = np.random.default_rng(n)
    pages = 100000
    c = Both(1, 1, pages, page=(8,), planes=2)
    if clean:
        order = rng.permutation(pages)
        src, dst = order[:n].copy(), order[n:2 * n].copy()
        src[7:n // 2] = src[:n // 2 - 7]  # sources more than once
    else:  # destinations twice, near and far apart, sources that are destinations, ids out of range
        src, dst = rng.integers(-3, pages // 2, n), rng.integers(-3, pages + 3, n)
        src[rng.random(n) < 1e-4] = pages
        dst[n // 2:n // 2 + 50] = dst[:50]
        dst[101:160] = dst[100:159]
        src[n - 40:] = dst[n // 3:n // 3 + 40]
        src[200:220] = dst[200:220]
    done, bad = copied(src, dst, pages)
    api.fa_pages_copy(c.planes, i32(src), i32(dst))
    assert api.fa_last_device_status() == (api.FA_ERR_INDEX if bad else api.FA_OK)
    assert bad != clean
    want = c.start.clone()
    s, d = (torch.tensor(x, device="cuda") for x in zip(*done))
    want[:, d] = c.start[:, s]
    assert torch.equal(c.pool, want)


def test_half_a_million_copies():
    n = 1 << 19
    c = Both(1, 1, 2 * n, page=(8,), planes=1)
    order = torch.randperm(2 * n, device="cuda").int()
    src, dst = order[:n].contiguous(), order[n:].contiguous()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    api.fa_pages_copy(c.planes, src, dst)
    b.record()
    want = c.start.clone()
    want[:, dst.long()] = c.start[:, src.long()]
    assert torch.equal(c.pool, want)
    assert a.elapsed_time(b) < 60  # ms; a look through the list for each pair reads 2 TB


# (H, T, prefix) with two key/value heads: few rows written at once / joined; 160 rows written at once / behind
# the prefix; 80 rows joined with a prefix in tiles of its own
FORMS = [(8, 1, 0), (8, 3, 200), (8, 40, 0), (8, 40, 200), (8, 20, 200)]


def place(c, b, token):
    """Page and slot of a sequence's own token (b >= 0) or of a prefix token (b < 0)."""
    ps = c.k.shape[2]
    table = c.prefix if b < 0 else c.table[b]
    return int(table[token // ps]), token % ps


def status_of(c, q, want, **kw):
    got = c.run(q, **kw)
    assert api.fa_last_device_status() == want
    return got


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("H,T,prefix", FORMS)
def test_values_that_are_not_finite_are_reported(d, dtype, H, T, prefix):
    c = Cache([300, 50, 44, 400], prefix, 2, d, 16, dtype, seed=d + T)
    q = c.queries(H, T)
    clean = status_of(c, q, api.FA_OK)
    c.check(q, clean)
    for pool, bad in ((c.v, np.inf), (c.v, -np.inf), (c.v, np.nan), (c.k, np.nan), (c.k, np.inf)):
        page, slot = place(c, 0, 10)
        keep = pool[page, 1, slot, 3].item()
        pool[page, 1, slot, 3] = bad
        got = status_of(c, q, api.FA_ERR_RANGE)
        for x, y in zip(got, clean):  # the other sequences, and the heads that do not read it
            assert torch.equal(x[1:], y[1:]) and torch.equal(x[0, :H // 2], y[0, :H // 2])
        pool[page, 1, slot, 3] = keep
        if prefix:
            page, slot = place(c, -1, 5)
            keep = pool[page, 1, slot, 3].item()
            pool[page, 1, slot, 3] = bad
            got = status_of(c, q, api.FA_ERR_RANGE)
            for x, y in zip(got, clean):
                assert torch.equal(x[:, :H // 2], y[:, :H // 2])
            pool[page, 1, slot, 3] = keep
    for bad in (np.inf, -np.inf, np.nan):
        odd = q.clone()
        odd[2, 1, T - 1, 7] = bad
        got = status_of(c, odd, api.FA_ERR_RANGE)
        for x, y in zip(got, clean):
            same = torch.ones(x.shape[:3], dtype=torch.bool, device="cuda")
            same[2, 1, T - 1] = False
            assert torch.equal(x[same], y[same])
    # nobody sees what a row without a sequence holds
    c.lens[2] = -1
    q[2] = float("nan")
    got = status_of(c, q, api.FA_OK)
    assert torch.equal(got[0][[0, 1, 3]], clean[0][[0, 1, 3]])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,T,prefix", FORMS)
def test_scores_and_sums_beyond_fp32(d, H, T, prefix):
    c = Cache([300, 50], prefix, 2, d, 16, BF16, seed=d + T + 1)
    q = c.queries(H, T).abs() + 0.5
    pages = [int(x) for x in c.table[0][:19]] + [int(x) for x in c.prefix]
    # one score of -inf: the weight is 0, as it is for a score of -1000 and less
    page, slot = place(c, 0, 10)
    c.k[page, :, slot] = -1000.0
    want = status_of(c, q, api.FA_OK)
    c.k[page, :, slot] = -3e38
    got = status_of(c, q, api.FA_OK)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    # every score of a row is -inf: not a row without keys
    k = c.k.clone()
    c.k[pages] = -3e38
    o, lse = status_of(c, q, api.FA_ERR_RANGE)
    assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all()
    c.k.copy_(k)
    # finite products, and a scale that takes them out of range
    o, lse = status_of(c, q, api.FA_ERR_RANGE, scale=2e38)
    assert torch.isnan(o).any()
    # large values: up to 2^119 / keys they are handled, sums beyond fp32 are reported
    zero = torch.zeros_like(q)
    n = 300 + prefix
    c.v[pages] = 2.0 ** (118 - int(np.log2(n)))
    o, _ = status_of(c, zero, api.FA_OK)
    visible = o[0, :, -1]  # the last query sees every key
    assert torch.equal(visible, torch.full_like(visible, 2.0 ** (118 - int(np.log2(n)))))
    c.v[pages] = 2.0 ** 127
    status_of(c, zero, api.FA_ERR_RANGE)


def test_rows_that_see_nothing_are_no_error():
    for H, T, prefix in FORMS:
        c = Cache([0, 300, 2], 0, 2, 64, 16, BF16, seed=T)
        q = c.queries(H, T)
        c.check(q, status_of(c, q, api.FA_OK))
        c.check(q, status_of(c, q, api.FA_OK, causal=False), causal=False)


def check_small_weights(c, q, got, scale):
    """As Cache.check, for fp16 weights that are multiplied by 2^7 before they are rounded: what is off by half
    of fp16's smallest step (2^-25) is 2^-32 of a row's weight."""
    o, lse = (x.double().cpu().numpy() for x in got)
    O, L, mean_abs, sum_abs, big, n = paged_attention(q, c.k, c.v, c.table, c.lens, c.prefix, c.prefix_len, scale, True)
    u = torch.finfo(c.dtype).eps / 2
    delta = 2.0 ** -23 * (c.d * big + n + 8)
    tol = u * np.abs(O) + (u + 2 * delta[..., None]) * mean_abs + 2.0 ** -32 * sum_abs + 2.0 ** -25
    some = n > 0
    assert (np.abs(o - O)[some] <= 1.001 * tol[some]).all(), (np.abs(o - O) / tol)[some].max()
    assert (np.abs(lse[some] - L[some]) <= 2 * delta[some] + 2.0 ** -22 * np.abs(L[some])).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,T,prefix", FORMS)
def test_small_weights_of_many_keys_count_in_fp16(d, H, T, prefix):
    # one key with nearly all the weight and V = 0, 10^5 with weights of 2^-25.2 and V = 1, and so many sequences
    # (of the same pages) that each one's keys lie in two or three parts
    n = 150
    c = Cache([100000], prefix, 2, d, 64, F16, seed=3)
    c.k.zero_()
    c.v.fill_(1.0)
    page, slot = place(c, 0, 1234)
    c.k[page, :, slot, 0] = 17.47
    c.v[page, :, slot] = 0.0
    q = torch.zeros(n, H, T, d, dtype=F16, device="cuda")
    q[..., 0] = 1.0
    one, table = q[:1], c.table
    c.table, c.lens = np.repeat(table, n, axis=0), [100000] * n
    o, lse = status_of(c, q, api.FA_OK, scale=1.0)
    c.table, c.lens = table, [100000]
    for b in (0, n - 1):
        check_small_weights(c, one, (o[b:b + 1], lse[b:b + 1]), 1.0)
    # the others have the same inputs: within the same bound of the first
    assert (o.double() - o[:1].double()).abs().max() <= 2 * (2.0 ** -32 * 1e5 + 0.004 * 0.03)
    assert (o[:, :, -1] > 0.0025).all()  # 10^5 2^-25.2 = 0.00259 in all


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,T,prefix", FORMS)
@pytest.mark.parametrize("scale", [0.125, 1.0])
def test_fp16_weights_of_random_keys(d, H, T, prefix, scale):
    c = Cache([700, 33, 1500], prefix, 2, d, 16, F16, seed=d + T)
    q = c.queries(H, T)
    check_small_weights(c, q, status_of(c, q, api.FA_OK, scale=scale), scale)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,T,prefix", FORMS)
def test_large_scores_stay_finite_in_fp16(d, H, T, prefix):
    # scores up to some 2^26 in base 2, whose differences fp32 rounds to multiples of 4: one key takes each row,
    # or several of one score, so an element of o is at most the largest of V
    c = Cache([700, 33, 1500], prefix, 2, d, 16, F16, seed=d)
    q = c.queries(H, T)
    o, _ = status_of(c, q, api.FA_OK, scale=4e7 / d ** 0.5 / 6)
    top = max(c.v[place(c, b, t)[0], :, place(c, b, t)[1]].abs().max().item()
              for b, n in [(-1, prefix)] + list(enumerate(c.lens)) for t in range(n))
    assert o.abs().max() <= top * (1 + 2.0 ** -10)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,T,prefix", FORMS)
def test_a_mean_of_fp16s_largest_values_is_finite(d, H, T, prefix):
    # one key of weight 1, the others of weights that fp16 rounds up by nearly 2^-11: off by that, the mean of
    # V = 65504 would pass 65520, from which on fp16 rounds to infinity
    c = Cache([2000, 40], prefix, 2, d, 16, F16, seed=d)
    steps = np.arange(1, 300) / 64.0  # differences of scores
    w = 2.0 ** 7 * np.exp(-steps)
    up = steps[np.argmax(w.astype(np.float16).astype(np.float64) / w)]
    c.k.zero_()
    c.v.fill_(65504.0)
    for b in ((-1, 0) if prefix else (0,)):  # a key of weight 1 in every other tile at least
        for t in range(0, [2000, 40, prefix][b], 64):
            page, slot = place(c, b, t)
            c.k[page, :, slot, 0] = up
    q = torch.zeros(2, H, T, d, dtype=F16, device="cuda")
    q[..., 0] = 1.0
    for sign in (1.0, -1.0):
        o, _ = status_of(c, q, api.FA_OK, scale=1.0)
        assert (o[0, :, -1] * sign >= 65504 * (1 - 2.0 ** -10)).all() and torch.isfinite(o).all()
        c.v.neg_()
