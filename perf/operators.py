"""Cases and plain forms of the paged key/value cache: attention over its pages (with a
prefix shared by the whole batch) and the operations on the pages themselves.

``run`` computes an operator in elementary torch operations, or with ``own`` set through
``exact_io_aware_91_b200.api``.  The operators:

  attn     ``fa_paged_attn``: T new tokens per sequence against shared prefix + own tokens
  write    ``fa_pages_write``: new K, V tokens into their pages; with ``admit`` the slot of a
           finished sequence is handed to a prompt (free, reserve, write)
  copy     ``fa_pages_copy``: whole pages, in every plane (K and V of each layer)
  fork     ``fa_pages_free`` + ``fa_pages_fork``: sequences replaced by copies of others that
           share their full pages (one step of a beam search or of parallel sampling)
  compact  ``fa_pages_compact``: live pages moved to the front of the pool
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
DEV = "cuda"


def _api():
    from exact_io_aware_91_b200 import api

    return api


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a couple of chat turns after a short system prompt: latency counts
        dict(name="attn_small", op="attn", B=2, H=8, Hkv=2, T=1, d=128, ps=16, prefix=100, lo=1, hi=40, dtype="bf16",
             causal=True),
        # ordinary decoding, ragged batch, nothing shared: the bytes of the cache count
        dict(name="attn_ragged", op="attn", B=37, H=32, Hkv=8, T=1, d=128, ps=64, prefix=0, lo=1, hi=16384,
             dtype="bf16", causal=True),
        # many questions to one long document: its products are dense and shared
        dict(name="attn_prefix", op="attn", B=128, H=32, Hkv=8, T=1, d=128, ps=32, prefix=32785, lo=1, hi=512,
             dtype="bf16", causal=True),
        # draft tokens verified five at a time, plain multi-head attention, head dim 64
        dict(name="attn_draft", op="attn", B=24, H=16, Hkv=16, T=5, d=64, ps=16, prefix=2000, lo=5, hi=4096,
             dtype="f16", causal=True),
        # one token of every sequence of a decode step: latency counts
        dict(name="write_token", op="write", B=64, Hkv=8, T=1, d=128, ps=16, lo=1, hi=4096, dtype="bf16",
             admit=False),
        # prompts enter the slots of finished sequences
        dict(name="write_prompt", op="write", B=16, Hkv=8, T=4096, d=128, ps=64, lo=1, hi=2048, dtype="bf16",
             admit=True),
        # a few pages of two layers (K and V each)
        dict(name="copy_few", op="copy", planes=4, pages=512, n=7, ps=16, Hkv=8, d=128, dtype="bf16"),
        # many pages of eight layers: the bytes count
        dict(name="copy_many", op="copy", planes=16, pages=2048, n=701, ps=16, Hkv=8, d=128, dtype="bf16"),
        # four samples of one answer branch off
        dict(name="fork_samples", op="fork", B=8, keep=1, planes=4, pages=1024, ps=16, Hkv=8, d=128, lo=200, hi=900,
             dtype="bf16"),
        # a beam step of many long sequences over sixteen layers
        dict(name="fork_beams", op="fork", B=96, keep=24, planes=32, pages=4096, ps=32, Hkv=4, d=64, lo=100, hi=4000,
             dtype="f16"),
        # a small pool after a few sequences ended
        dict(name="compact_small", op="compact", B=8, live=0.6, planes=4, pages=500, ps=16, Hkv=8, d=128,
             dtype="bf16"),
        # a large, scattered pool
        dict(name="compact_large", op="compact", B=64, live=0.5, planes=16, pages=4096, ps=16, Hkv=8, d=128,
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "write", "copy", "fork", "compact"])
    limit = {o: max(_cost(c) for c in listed() if c["op"] == o) for o in ("attn", "write", "copy", "fork", "compact")}
    while True:
        dt = rng.choice(["bf16", "f16"])
        if op == "attn":
            hkv = rng.choice([1, 2, 4, 8, 16])
            t = rng.choice([1, 1, 1, 2, 3, 5, 8, 17])
            hi = _log_int(rng, t, 131072)
            case = dict(op=op, B=_log_int(rng, 1, 128), H=hkv * rng.choice([1, 2, 3, 4, 8]), Hkv=hkv, T=t,
                        d=rng.choice([64, 128, 128, 256]), ps=rng.choice([8, 16, 32, 64, 128, 256]),
                        prefix=rng.choice([0, 1]) * _log_int(rng, 1, 40000), lo=min(t, hi), hi=hi, dtype=dt,
                        causal=rng.random() < 0.8)
        elif op == "write":
            admit = rng.random() < 0.5
            case = dict(op=op, B=_log_int(rng, 1, 64), Hkv=rng.choice([1, 2, 3, 8]),
                        T=_log_int(rng, 1, 4096) if admit else rng.choice([1, 1, 2, 5]), d=rng.choice([64, 128, 256]),
                        ps=rng.choice([8, 16, 64, 128]), lo=1, hi=_log_int(rng, 1, 4096), dtype=dt, admit=admit)
        elif op == "copy":
            pages = _log_int(rng, 16, 2048)
            case = dict(op=op, planes=_log_int(rng, 1, 32), pages=pages, n=_log_int(rng, 1, pages // 2),
                        ps=rng.choice([8, 16, 32]), Hkv=rng.choice([1, 2, 8]), d=rng.choice([64, 128, 256]), dtype=dt)
        elif op == "fork":
            b = rng.randint(2, 96)
            lo = _log_int(rng, 1, 1000)
            case = dict(op=op, B=b, keep=rng.randint(1, b - 1), planes=_log_int(rng, 1, 32),
                        pages=_log_int(rng, 1024, 4096), ps=rng.choice([8, 16, 32]), Hkv=rng.choice([1, 2, 4]),
                        d=rng.choice([64, 128]), lo=lo, hi=_log_int(rng, lo, 4000), dtype=dt)
        else:
            case = dict(op=op, B=rng.randint(1, 64), live=round(rng.uniform(0.05, 0.95), 3),
                        planes=_log_int(rng, 1, 16), pages=_log_int(rng, 64, 4096), ps=rng.choice([8, 16, 32]),
                        Hkv=rng.choice([1, 2, 8]), d=rng.choice([64, 128, 256]), dtype=dt)
        if _cost(case) <= limit[op] and _held(case) <= 6e9:
            return case


def _lens(case):
    """Lengths spread evenly over lo .. hi; their order depends on the seed, their sum does not."""
    b = case["B"]
    if b == 1:
        return [case["hi"]]
    return [case["lo"] + (case["hi"] - case["lo"]) * i // (b - 1) for i in range(b)]


def _visible(case):
    """(query, own key) pairs of all sequences."""
    t = case["T"]
    n = 0
    for length in _lens(case):
        n += sum(max(0, min(length, length - t + i + 1)) for i in range(t)) if case["causal"] else t * length
    return n


def _page_bytes(case):
    return case["ps"] * case["Hkv"] * case["d"] * 2


def _moved_pages(case):
    """Whole pages that an operation on pages moves."""
    if case["op"] == "copy":
        return case["n"]
    if case["op"] == "fork":
        lens = _fork_lens(case)
        return sum(1 for i in range(case["B"] - case["keep"]) if lens[i % case["keep"]] % case["ps"])
    live = int(round(case["live"] * case["pages"]))
    return int(round(live * (1.0 - live / case["pages"])))  # expected: live pages beyond the first `live` ids


def _fork_lens(case):
    """Lengths of the kept sequences of a fork; all their pages, and the copies, fit the pool."""
    k = case["keep"]
    ps, room = case["ps"], case["pages"] - case["B"]
    lens = [case["lo"] + (case["hi"] - case["lo"]) * i // max(1, k - 1) for i in range(k)]
    cap = max(1, room // k - 1) * ps
    return [min(x, cap) for x in lens]


def work(case):
    if case["op"] == "attn":
        b, h, hkv, t, d, p = (case[x] for x in ("B", "H", "Hkv", "T", "d", "prefix"))
        own_len = sum(_lens(case))
        by = 2 * 2 * hkv * d * (p + own_len) + 2 * 2 * b * h * t * d + 4 * b * h * t + 4 * b
        by += 4 * (-(-p // case["ps"]) + sum(-(-x // case["ps"]) for x in _lens(case)))
        return {"bytes": by, "flops": 4 * d * h * (b * t * p + _visible(case))}
    if case["op"] == "write":
        by = 2 * 2 * (2 * case["B"] * case["Hkv"] * case["T"] * case["d"])
        if case["admit"]:  # old entries and new ones, and their counts read and written
            old = sum(-(-x // case["ps"]) for x in _lens(case))
            new = case["B"] * -(-case["T"] // case["ps"])
            by += 12 * (old + new)
        return {"bytes": by + 8 * case["B"], "flops": 0}
    by = 2 * _moved_pages(case) * _page_bytes(case) * case["planes"]
    if case["op"] == "copy":
        by += 8 * case["n"]
    elif case["op"] == "fork":
        lens = _fork_lens(case)
        entries = sum(-(-lens[i % case["keep"]] // case["ps"]) for i in range(case["B"] - case["keep"]))
        by += 4 * 7 * entries  # freed entries and counts, parents' entries read, children's written, counts raised
    else:
        by += 4 * (4 * case["pages"])  # entries read and written, counts read, page map written
    return {"bytes": by, "flops": 0}


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.5e12 + w["flops"] / 1.4e15


def _held(case):
    if case["op"] == "attn":
        return 4 * case["Hkv"] * case["d"] * (case["prefix"] + sum(_lens(case)))
    if case["op"] == "write":
        return 4 * case["B"] * case["Hkv"] * case["d"] * (2 * case["T"] + case["hi"])
    return case["planes"] * case["pages"] * _page_bytes(case)


# ------------------------------------------------------------------------------ the inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _tables(np_rng, lens, ps, pages, max_pages):
    """A table of distinct, scattered pages; entries behind a sequence's end are -1."""
    order = np_rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), max_pages), -1, np.int32)
    at = 0
    for b, length in enumerate(lens):
        k = -(-length // ps)
        table[b, :k] = order[at:at + k]
        at += k
    return table, order[at:]


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


def prepare(case, seed):
    g, nr = _gen(seed), np.random.default_rng(seed)
    dt = DTYPES[case["dtype"]]
    op, ps = case["op"], case["ps"]
    st = dict(case=case)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=dt)  # noqa: E731
    if op == "attn":
        lens = nr.permutation(_lens(case))
        used = sum(-(-int(x) // ps) for x in lens)
        n_prefix = -(-case["prefix"] // ps)
        pages = used + n_prefix + 3
        table, rest = _tables(nr, lens, ps, pages, max(1, -(-case["hi"] // ps)))
        st["k_pages"], st["v_pages"] = (rand(pages, case["Hkv"], ps, case["d"]) for _ in range(2))
        # one key in a hundred is larger: rows with a sharp softmax beside flat ones
        loud = torch.rand(pages, case["Hkv"], ps, 1, generator=g, device=DEV) < 0.01
        st["k_pages"] *= torch.where(loud, 4.0, 1.0).to(dt)
        st["q"] = rand(case["B"], case["H"], case["T"], case["d"])
        st["table"], st["lens"] = _i32(table), _i32(lens)
        st["prefix_table"] = _i32(rest[:n_prefix]) if n_prefix else None
        st["o"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros(case["B"], case["H"], case["T"], device=DEV)
        if own:
            api = _api()
            pr = api.paged_problem(st["q"], st["k_pages"], st["v_pages"], st["table"], case["prefix"],
                                   causal=case["causal"])
            st["ws"] = torch.empty(max(1, api.fa_paged_attn_workspace_size(pr)), dtype=torch.uint8, device=DEV)
        return st
    if op == "write":
        old = nr.permutation(_lens(case))
        lens = old if case["admit"] else old - 1 + case["T"]
        per_row = -(-max(case["T"], int(lens.max())) // ps)
        pages = case["B"] * per_row + 3
        table, _ = _tables(nr, lens, ps, pages, per_row)
        refs = np.zeros(pages, np.int32)
        refs[table[table >= 0]] = 1
        st["k_pages"], st["v_pages"] = (rand(pages, case["Hkv"], ps, case["d"]) for _ in range(2))
        st["k"], st["v"] = (rand(case["B"], case["Hkv"], case["T"], case["d"]) for _ in range(2))
        st["table"], st["lens"], st["refs"] = _i32(table), _i32(lens), _i32(refs)
        st["rows"] = _i32(np.arange(case["B"]))
        st["new_lens"] = _i32(np.full(case["B"], case["T"]))
        if own:
            st["ws"] = torch.empty(_api().fa_pages_workspace_size(case["B"], pages), dtype=torch.uint8, device=DEV)
        return st
    pages, planes = case["pages"], case["planes"]
    st["pool"] = rand(planes, pages, case["Hkv"], ps, case["d"])  # K and V of every layer
    if op == "copy":
        order = nr.permutation(pages)
        st["src"], st["dst"] = _i32(order[:case["n"]]), _i32(order[case["n"]:2 * case["n"]])
        return st
    if op == "fork":
        kept = _fork_lens(case)
        lens = np.full(case["B"], -1, np.int64)
        slots = nr.permutation(case["B"])
        parents, children = slots[:case["keep"]], slots[case["keep"]:]
        lens[parents] = kept
        table, _ = _tables(nr, np.maximum(lens, 0), ps, pages, -(-int(lens.max()) // ps))
        refs = np.zeros(pages, np.int32)
        refs[table[table >= 0]] = 1
        st["children"] = _i32(children)
        st["parents"] = _i32(parents[np.arange(len(children)) % case["keep"]])
        n_rows = case["B"]
    else:
        live = int(round(case["live"] * pages))
        n_rows = case["B"]
        cuts = np.sort(nr.integers(0, live + 1, n_rows - 1)) if n_rows > 1 else np.zeros(0, np.int64)
        owned = np.diff(np.concatenate([[0], cuts, [live]]))
        lens = np.maximum(0, owned * ps - nr.integers(0, ps, n_rows) * (owned > 0))
        table, _ = _tables(nr, lens, ps, pages, max(1, live))  # one sequence may own every live page
        refs = np.zeros(pages, np.int32)
        refs[table[table >= 0]] = 1
    st["table"], st["lens"], st["refs"] = _i32(table), _i32(lens), _i32(refs)
    if op == "compact":
        st["table_out"], st["refs_out"] = torch.empty_like(st["table"]), torch.empty_like(st["refs"])
        st["map"] = torch.empty_like(st["refs"])
    if own:
        st["ws"] = torch.empty(_api().fa_pages_workspace_size(n_rows, pages), dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------------- one pass through
def run(st):
    return (_OWN if own else _PLAIN)[st["case"]["op"]](st)


def _own_attn(st):
    c = st["case"]
    return _api().fa_paged_attn(st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens"],
                                prefix_table=st["prefix_table"], prefix_len=c["prefix"], causal=c["causal"],
                                o=st["o"], lse=st["lse"], workspace=st["ws"])


def _own_write(st):
    api, ps = _api(), st["case"]["ps"]
    if st["case"]["admit"]:
        api.fa_pages_free(ps, st["table"], st["lens"], st["refs"], st["rows"])
        api.fa_pages_reserve(ps, st["table"], st["lens"], st["refs"], st["new_lens"], workspace=st["ws"])
    api.fa_pages_write(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["lens"])
    return st["k_pages"], st["v_pages"], st["table"], st["lens"], st["refs"]


def _own_copy(st):
    _api().fa_pages_copy(st["pool"], st["src"], st["dst"])
    return st["pool"]


def _own_fork(st):
    api, ps = _api(), st["case"]["ps"]
    api.fa_pages_free(ps, st["table"], st["lens"], st["refs"], st["children"])
    api.fa_pages_fork(st["pool"], ps, st["table"], st["lens"], st["refs"], st["parents"], st["children"],
                      workspace=st["ws"])
    return [st["pool"], st["table"], st["lens"], st["refs"]]


def _own_compact(st):
    _api().fa_pages_compact(st["pool"], st["case"]["ps"], st["table"], st["lens"], st["refs"],
                            block_table_out=st["table_out"], ref_counts_out=st["refs_out"], page_map=st["map"],
                            workspace=st["ws"])
    return [st["pool"], st["table_out"], st["refs_out"], st["map"]]


_OWN = {"attn": _own_attn, "write": _own_write, "copy": _own_copy, "fork": _own_fork, "compact": _own_compact}


def _rows_of(pages, table, n_tok, ps):
    """The first n_tok tokens that each row of `table` names, (rows, H_kv, n_tok, d) in fp32."""
    x = pages[table[:, :-(-n_tok // ps)].clamp(min=0).long()].float()
    rows, k, hkv, _, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(rows, hkv, k * ps, d)[:, :, :n_tok]


def _plain_attn(st):
    c = st["case"]
    b, h, hkv, t, d, p, ps = (c[x] for x in ("B", "H", "Hkv", "T", "d", "prefix", "ps"))
    q = st["q"].float().view(b, hkv, h // hkv * t, d) / math.sqrt(d)
    n = c["hi"]
    lens = st["lens"].long()
    v_own = _rows_of(st["v_pages"], st["table"], n, ps)
    s = q @ _rows_of(st["k_pages"], st["table"], n, ps).transpose(2, 3)
    last = lens[:, None] - t + torch.arange(t, device=DEV) if c["causal"] else (lens[:, None] - 1).expand(b, t)
    seen = torch.arange(n, device=DEV) <= last[:, :, None]  # (B, T, n)
    s = s.view(b, hkv, h // hkv, t, n).masked_fill(~seen[:, None, None], -math.inf).view(b, hkv, -1, n)
    m = s.amax(-1, keepdim=True)
    if p:
        k_p, v_p = (_rows_of(x, st["prefix_table"][None], p, ps)[0] for x in (st["k_pages"], st["v_pages"]))
        rows = q.transpose(0, 1).reshape(hkv, -1, d)  # the same prefix for the rows of every sequence
        s_p = rows @ k_p.transpose(1, 2)
        m_p = s_p.amax(-1).view(hkv, b, -1, 1).transpose(0, 1)
        m = torch.maximum(m, m_p)
    safe = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(s - safe)
    total, o = e.sum(-1, keepdim=True), e @ v_own
    if p:
        e_p = torch.exp(s_p - safe.transpose(0, 1).reshape(hkv, -1, 1))
        back = lambda x: x.view(hkv, b, -1, x.shape[-1]).transpose(0, 1)  # noqa: E731
        total, o = total + back(e_p.sum(-1, keepdim=True)), o + back(e_p @ v_p)
    o = torch.where(total > 0, o / total, 0.0).view(b, h, t, d).to(st["q"].dtype)
    return o, (m + torch.log(total)).view(b, h, t)


def _owned(st, lens):
    """Which entries of the table belong to their rows."""
    n = -(-lens.clamp(min=0).long() // st["case"]["ps"])
    return torch.arange(st["table"].shape[1], device=DEV) < n[:, None]


def _plain_free(st, rows):
    rows = rows.long()
    mine = _owned(st, st["lens"])[rows]
    entries = st["table"][rows]
    st["refs"].index_add_(0, entries.clamp(min=0).long().flatten(), -mine.int().flatten())
    st["table"][rows] = torch.where(mine, -1, entries)
    st["lens"][rows] = -1


def _free_pages(st):
    """Page ids, the free ones first and in order, and how many are free."""
    used = (st["refs"] > 0).int()
    return torch.sort(used, stable=True).indices, (used == 0).sum()


def _plain_write(st):
    c = st["case"]
    ps, t = c["ps"], c["T"]
    if c["admit"]:
        _plain_free(st, st["rows"])
        have = -(-st["lens"].clamp(min=0).long() // ps)
        want = -(-st["new_lens"].long() // ps)
        need = (want - have).clamp(min=0)
        upto = need.cumsum(0)
        order, n_free = _free_pages(st)
        granted = (need == 0) | (upto <= n_free)
        e = torch.arange(st["table"].shape[1], device=DEV)
        taken = (e >= have[:, None]) & (e < want[:, None]) & granted[:, None]
        rank = (upto - need)[:, None] + e - have[:, None]
        page = order[rank.clamp(0, order.numel() - 1)]
        st["refs"].index_add_(0, page.flatten(), taken.int().flatten())
        st["table"].copy_(torch.where(taken, page.int(), st["table"]))
        grows = granted & (st["new_lens"] > st["lens"].clamp(min=0))
        st["lens"].copy_(torch.where(grows, st["new_lens"], st["lens"]))
    pos = st["lens"].long()[:, None] - t + torch.arange(t, device=DEV)
    page = st["table"].long().gather(1, pos // ps)
    for pool, x in ((st["k_pages"], st["k"]), (st["v_pages"], st["v"])):
        pool[page, :, pos % ps] = x.transpose(1, 2)
    return st["k_pages"], st["v_pages"], st["table"], st["lens"], st["refs"]


def _plain_copy(st):
    src, dst = st["src"].long(), st["dst"].long()
    st["pool"][:, dst] = st["pool"][:, src]
    return st["pool"]


def _plain_fork(st):
    ps = st["case"]["ps"]
    _plain_free(st, st["children"])
    par, chi = st["parents"].long(), st["children"].long()
    lens = st["lens"][par].long()
    full, need = lens // ps, (lens % ps > 0).long()
    upto = need.cumsum(0)
    order, n_free = _free_pages(st)
    granted = (need == 0) | (upto <= n_free)
    e = torch.arange(st["table"].shape[1], device=DEV)
    shared = (e < full[:, None]) & granted[:, None]
    tail = (e == full[:, None]) & (need > 0)[:, None] & granted[:, None]
    fresh = order[(upto - need).clamp(0, order.numel() - 1)]
    old = st["table"][par]
    st["refs"].index_add_(0, old.clamp(min=0).long().flatten(), shared.int().flatten())
    st["refs"].index_add_(0, fresh, tail.sum(1).int())
    st["table"][chi] = torch.where(shared, old, torch.where(tail, fresh[:, None].int(), st["table"][chi]))
    st["lens"][chi] = torch.where(granted, st["lens"][par], st["lens"][chi])
    some = tail.any(1)
    src = old.long().gather(1, full.clamp(max=old.shape[1] - 1)[:, None])[:, 0]
    src, dst = src[some], fresh[some]
    st["pool"][:, dst] = st["pool"][:, src]
    return [st["pool"], st["table"], st["lens"], st["refs"]]


def _plain_compact(st):
    live = st["refs"] > 0
    ids = torch.arange(live.numel(), device=DEV)
    n = live.sum()
    src, dst = ids[live & (ids >= n)], ids[~live & (ids < n)]
    where_to = torch.where(live, ids, -1)
    where_to[src] = dst
    st["map"].copy_(where_to)
    st["refs_out"].copy_(torch.where(live, st["refs"], 0))
    st["refs_out"][dst] = st["refs"][src]
    st["refs_out"][src] = 0
    mine = _owned(st, st["lens"])
    st["table_out"].copy_(torch.where(mine, st["map"][st["table"].clamp(min=0).long()], st["table"]))
    st["pool"][:, dst] = st["pool"][:, src]
    return [st["pool"], st["table_out"], st["refs_out"], st["map"]]


_PLAIN = {"attn": _plain_attn, "write": _plain_write, "copy": _plain_copy, "fork": _plain_fork,
          "compact": _plain_compact}


# --------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The attention of each sequence by its definition; the other operators move values only."""
    if case["op"] != "attn":
        return None
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    b, h, hkv, t, d, p, ps = (case[x] for x in ("B", "H", "Hkv", "T", "d", "prefix", "ps"))
    lens, table = st["lens"].tolist(), st["table"].tolist()
    prefix = st["prefix_table"].tolist() if p else []
    out = torch.zeros(b, h, t, d, dtype=torch.float64, device=DEV)
    lse = torch.full((b, h, t), -math.inf, dtype=torch.float64, device=DEV)

    def tokens(pool, pages, n):  # (H_kv, n, d)
        idx = torch.tensor(pages[:-(-n // ps)], dtype=torch.long, device=DEV)
        return torch.cat(list(pool[idx].double()), dim=1)[:, :n] if n else pool[:0].double().reshape(hkv, 0, d)

    k_pre, v_pre = tokens(st["k_pages"], prefix, p), tokens(st["v_pages"], prefix, p)
    for i in range(b):
        n = lens[i]
        keys = torch.cat([k_pre, tokens(st["k_pages"], table[i], n)], dim=1)
        vals = torch.cat([v_pre, tokens(st["v_pages"], table[i], n)], dim=1)
        for g in range(hkv):
            heads = slice(g * (h // hkv), (g + 1) * (h // hkv))
            scores = torch.einsum("htd,nd->htn", st["q"][i, heads].double(), keys[g]) * (d ** -0.5)
            for j in range(t):
                stop = p + (max(0, n - t + j + 1) if case["causal"] else n)
                if stop > 0:
                    row = scores[:, j, :stop]
                    lse[i, heads, j] = torch.logsumexp(row, dim=-1)
                    out[i, heads, j] = torch.softmax(row, dim=-1) @ vals[g, :stop]
    return out, lse
