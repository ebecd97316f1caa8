"""Plain definitions of the paged cache: attention over pages in float64, and the page
operations one entry at a time on Python integers.

``paged_attention`` gathers each sequence's keys and values by its table and applies the
attention formula row by row; ``PageTable`` states what each operation does in the order
its description gives.  Both are written for reading, not for speed.
"""

import numpy as np


def _f64(x) -> np.ndarray:
    if hasattr(x, "detach"):
        x = x.detach().double().cpu().numpy()
    return np.asarray(x, dtype=np.float64)


def gather(pages: np.ndarray, table, n: int) -> np.ndarray:
    """The first n tokens that `table` names, (H_kv, n, d)."""
    _, h, ps, d = pages.shape
    out = np.zeros((h, n, d))
    for j in range(0, n, ps):
        m = min(ps, n - j)
        out[:, j:j + m] = pages[table[j // ps], :, :m]
    return out


def paged_attention(q, k_pages, v_pages, block_table, seq_lens, prefix_table, prefix_len, scale, causal):
    """Returns o, lse and, for error bounds, per element sum_j p_j |v_j|, sum_j |v_j| and per row
    max_j scale sum_i |q_i k_ji| and the number of keys.  Rows of negative length are NaN in o, lse."""
    q, kp, vp = _f64(q), _f64(k_pages), _f64(v_pages)
    table, lens = np.asarray(block_table), [int(x) for x in seq_lens]
    B, H, T, d = q.shape
    group = H // kp.shape[1]
    o, lse = np.full(q.shape, np.nan), np.full(q.shape[:3], np.nan)
    mean_abs, sum_abs = np.zeros(q.shape), np.zeros(q.shape)
    big, count = np.zeros(q.shape[:3]), np.zeros(q.shape[:3])
    pre_k, pre_v = (gather(x, prefix_table, prefix_len) for x in (kp, vp))
    for b in range(B):
        if lens[b] < 0:
            continue
        ks = np.concatenate([pre_k, gather(kp, table[b], lens[b])], axis=1)
        vs = np.concatenate([pre_v, gather(vp, table[b], lens[b])], axis=1)
        own = np.array([max(0, lens[b] - T + t + 1) if causal else lens[b] for t in range(T)])
        n = prefix_len + own  # keys that each query sees: the first n
        count[b] = n
        seen = np.arange(ks.shape[1]) < n[:, None]
        some = n > 0
        o[b][:, ~some], lse[b][:, ~some] = 0.0, -np.inf
        for h in range(H if some.any() else 0):
            k, v = ks[h // group], vs[h // group]
            s = np.where(seen, scale * (q[b, h] @ k.T), -np.inf)[some]
            m = s.max(axis=1, keepdims=True)
            e = np.exp(s - m)
            total = e.sum(axis=1, keepdims=True)
            o[b, h, some] = (e @ v) / total
            lse[b, h, some] = (m + np.log(total))[:, 0]
            mean_abs[b, h, some] = (e @ np.abs(v)) / total
            sum_abs[b, h, some] = seen[some] @ np.abs(v)
            big[b, h, some] = (scale * (np.abs(q[b, h]) @ np.abs(k).T) * seen).max(axis=1)[some]
    return o, lse, mean_abs, sum_abs, big, count


class PageTable:
    """block_table (lists), seq_lens, ref_counts, and the pages' contents as one label per page."""

    def __init__(self, page_size, block_table, seq_lens, ref_counts, content=None):
        self.ps = page_size
        self.table = [[int(x) for x in row] for row in block_table]
        self.lens = [int(x) for x in seq_lens]
        self.refs = [int(x) for x in ref_counts]
        self.content = list(range(len(self.refs))) if content is None else list(content)

    def owned(self, b):
        return -(-max(self.lens[b], 0) // self.ps)

    def free_pages(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def reserve(self, new_lens):
        pool = self.free_pages()
        asked, refused = 0, []
        for b, new in enumerate(int(x) for x in new_lens):
            if new <= max(self.lens[b], 0):
                continue
            have = self.owned(b)
            need = -(-new // self.ps) - have
            asked += need
            if need > 0 and asked > len(pool):
                refused.append(b)
                continue
            for i in range(need):
                page = pool[asked - need + i]
                self.table[b][have + i] = page
                self.refs[page] = 1
            self.lens[b] = new
        return refused

    def fork(self, parents, children):
        pool = self.free_pages()
        asked, refused = 0, []
        for i, (p, c) in enumerate(zip(parents, children)):
            length = self.lens[p]
            full, tail = divmod(length, self.ps)
            asked += tail > 0
            if tail and asked > len(pool):
                refused.append(i)
                continue
            for e in range(full):
                self.table[c][e] = self.table[p][e]
                self.refs[self.table[p][e]] += 1
            if tail:
                page = pool[asked - 1]
                self.table[c][full] = page
                self.refs[page] = 1
                self.content[page] = self.content[self.table[p][full]]
            self.lens[c] = length
        return refused

    def free(self, rows):
        for b in rows:
            for e in range(self.owned(b)):
                self.refs[self.table[b][e]] -= 1
                self.table[b][e] = -1
            self.lens[b] = -1

    def compact(self):
        """Returns the page map."""
        live = [p for p, r in enumerate(self.refs) if r > 0]
        n = len(live)
        page_map = [p if r > 0 else -1 for p, r in enumerate(self.refs)]
        holes = [p for p in range(n) if self.refs[p] == 0]
        for src, dst in zip([p for p in live if p >= n], holes):
            page_map[src] = dst
            self.refs[dst], self.refs[src] = self.refs[src], 0
            self.content[dst] = self.content[src]
        for b, row in enumerate(self.table):
            for e in range(self.owned(b)):
                row[e] = page_map[row[e]]
        return page_map
