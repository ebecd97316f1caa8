"""Host-only checks of the paged cache's entry points: every refusal comes before the GPU is
touched, and empty problems are no-ops."""

import ctypes

import pytest
import torch

from exact_io_aware_91_b200 import api
from exact_io_aware_91_b200 import build as fa_build

A = 0x10000  # fake device address, never dereferenced: 256-byte aligned
ST = (8 * 16 * 64, 16 * 64, 64)


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return api.library()


def problem(B=2, H=8, H_kv=2, T=1, d=64, dtype=api.FA_BF16, page_size=16, num_pages=10, max_pages=4, table_stride=4,
            prefix_len=0, causal=1, scale=0.125, ks=ST, vs=ST):
    ll3 = ctypes.c_longlong * 3
    return api.FaPagedProblem(B, H, H_kv, T, d, dtype, page_size, num_pages, max_pages, table_stride, prefix_len,
                              causal, scale, ll3(*ks), ll3(*vs))


def attn(lib, p, q=A, k=A, v=A, table=A, lens=A, prefix=A, o=A, lse=A, ws=A, ws_bytes=1 << 40):
    return lib.fa_paged_attn(None if p is None else ctypes.byref(p), q, k, v, table, lens, prefix, o, lse, ws, ws_bytes,
                             None)


def write(lib, p, k=A, v=A, kp=A, vp=A, table=A, lens=A):
    return lib.fa_pages_write(None if p is None else ctypes.byref(p), k, v, kp, vp, table, lens, None)


BAD = [
    (dict(B=-1), "INVALID_ARG"), (dict(T=-1), "INVALID_ARG"), (dict(H_kv=0), "INVALID_ARG"),
    (dict(dtype=2), "INVALID_ARG"), (dict(num_pages=-1), "INVALID_ARG"), (dict(max_pages=-1), "INVALID_ARG"),
    (dict(table_stride=3), "INVALID_ARG"), (dict(ks=(8 * 16 * 64, 16 * 64, 60)), "INVALID_ARG"),
    (dict(vs=(8 * 16 * 64, 16 * 64 + 4, 64)), "INVALID_ARG"), (dict(ks=(0, 16 * 64, 64)), "INVALID_ARG"),
    (dict(d=96), "UNSUPPORTED"), (dict(d=512), "UNSUPPORTED"), (dict(page_size=4), "UNSUPPORTED"),
    (dict(page_size=24), "UNSUPPORTED"), (dict(page_size=2048), "UNSUPPORTED"),
    (dict(num_pages=(1 << 20) + 1), "UNSUPPORTED"), (dict(B=1 << 25), "UNSUPPORTED"),
    (dict(T=1 << 27), "UNSUPPORTED"), (dict(max_pages=1 << 27, table_stride=1 << 27), "UNSUPPORTED"),
]
BAD_ATTN = [
    (dict(H=7), "INVALID_ARG"), (dict(H=0), "INVALID_ARG"), (dict(prefix_len=-1), "INVALID_ARG"),
    (dict(causal=2), "INVALID_ARG"), (dict(scale=0.0), "INVALID_ARG"), (dict(scale=float("nan")), "INVALID_ARG"),
    (dict(scale=float("inf")), "INVALID_ARG"), (dict(prefix_len=(1 << 30) + 1), "UNSUPPORTED"),
    (dict(B=1 << 20, max_pages=1 << 16, table_stride=1 << 16), "UNSUPPORTED"),  # 2^31 units and more
]


@pytest.mark.parametrize("change,status", BAD + BAD_ATTN)
def test_attention_refuses_bad_problems(lib, change, status):
    p = problem(**change)
    assert attn(lib, p) == getattr(api, "FA_ERR_" + status)
    assert api.fa_paged_attn_workspace_size(p) == 0


@pytest.mark.parametrize("change,status", BAD)
def test_write_refuses_bad_problems(lib, change, status):
    assert write(lib, problem(**change)) == getattr(api, "FA_ERR_" + status)


def test_pointers_are_checked(lib):
    p = problem(prefix_len=5)
    assert attn(lib, None) == api.FA_ERR_INVALID_ARG and write(lib, None) == api.FA_ERR_INVALID_ARG
    for name in ("q", "k", "v", "table", "lens", "prefix", "o", "ws"):
        assert attn(lib, p, **{name: None}) == api.FA_ERR_INVALID_ARG, name
    for name in ("q", "k", "v", "o", "ws"):
        assert attn(lib, p, **{name: A + 8}) == api.FA_ERR_MISALIGNED, name
    for name in ("table", "lens", "prefix", "lse"):
        assert attn(lib, p, **{name: A + 2}) == api.FA_ERR_MISALIGNED, name
    assert attn(lib, p, ws_bytes=api.fa_paged_attn_workspace_size(p) - 1) == api.FA_ERR_INVALID_ARG
    for name in ("k", "v", "kp", "vp", "table", "lens"):
        assert write(lib, p, **{name: None}) == api.FA_ERR_INVALID_ARG, name
    for name in ("k", "v", "kp", "vp"):
        assert write(lib, p, **{name: A + 8}) == api.FA_ERR_MISALIGNED, name


def test_empty_problems_are_no_ops(lib):
    nothing = dict(q=None, k=None, v=None, table=None, lens=None, prefix=None, o=None, lse=None, ws=None)
    for change in (dict(B=0), dict(T=0)):
        assert attn(lib, problem(**change), **nothing) == api.FA_OK
        assert api.fa_paged_attn_workspace_size(problem(**change)) == 0
    assert write(lib, problem(T=0), k=None, v=None, kp=None, vp=None, table=None, lens=None) == api.FA_OK


def table(rows=4, max_pages=4, table_stride=4, page_size=16, num_pages=10, block_table=A, seq_lens=A, ref_counts=A):
    return api.FaPageTable(rows, max_pages, table_stride, page_size, num_pages, block_table, seq_lens, ref_counts)


def planes(ptrs=(A, A), num_pages=10, page_bytes=4096, page_stride=4096):
    a = (ctypes.c_void_p * max(1, len(ptrs)))(*ptrs)
    return api.FaPagePlanes(ctypes.cast(a, ctypes.POINTER(ctypes.c_void_p)), len(ptrs), num_pages, page_bytes,
                            page_stride)


def calls(lib, t=None, pl=None, ws=A, ws_bytes=1 << 40, lists=A, n=2, out=A):
    t, pl = ctypes.byref(t or table()), ctypes.byref(pl or planes())
    return {
        "copy": lib.fa_pages_copy(pl, lists, lists, n, None),
        "reserve": lib.fa_pages_reserve(t, lists, ws, ws_bytes, None),
        "fork": lib.fa_pages_fork(pl, t, lists, lists, n, ws, ws_bytes, None),
        "free": lib.fa_pages_free(t, lists, n, None),
        "compact": lib.fa_pages_compact(pl, t, out, out, out, ws, ws_bytes, None),
    }


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), "INVALID_ARG"), (dict(max_pages=-1), "INVALID_ARG"), (dict(num_pages=-1), "INVALID_ARG"),
    (dict(table_stride=3), "INVALID_ARG"), (dict(block_table=None), "INVALID_ARG"), (dict(seq_lens=None), "INVALID_ARG"),
    (dict(ref_counts=None), "INVALID_ARG"), (dict(page_size=12), "UNSUPPORTED"), (dict(page_size=4096), "UNSUPPORTED"),
    (dict(num_pages=(1 << 20) + 1), "UNSUPPORTED"), (dict(rows=(1 << 24) + 1), "UNSUPPORTED"),
    (dict(block_table=A + 2), "MISALIGNED"), (dict(seq_lens=A + 1), "MISALIGNED"), (dict(ref_counts=A + 2), "MISALIGNED"),
])
def test_page_tables_are_checked(lib, change, status):
    t = table(**change)
    got = calls(lib, t=t, pl=planes(num_pages=t.num_pages) if 0 <= t.num_pages <= 1 << 20 else None)
    for name in ("reserve", "fork", "free", "compact"):
        assert got[name] == getattr(api, "FA_ERR_" + status), name


@pytest.mark.parametrize("change,status", [
    (dict(ptrs=(A, None)), "INVALID_ARG"), (dict(num_pages=-1), "INVALID_ARG"), (dict(page_bytes=-16), "INVALID_ARG"),
    (dict(page_stride=4080), "INVALID_ARG"), (dict(ptrs=(A,) * 1025), "UNSUPPORTED"),
    (dict(ptrs=(A, A + 8)), "MISALIGNED"), (dict(page_bytes=4088), "MISALIGNED"), (dict(page_stride=4104), "MISALIGNED"),
])
def test_planes_are_checked(lib, change, status):
    got = calls(lib, pl=planes(**change))
    for name in ("copy", "fork", "compact"):
        assert got[name] == getattr(api, "FA_ERR_" + status), name


def test_lists_workspaces_and_counts_are_checked(lib):
    got = calls(lib, lists=None)
    assert all(got[x] == api.FA_ERR_INVALID_ARG for x in ("copy", "reserve", "fork", "free"))
    got = calls(lib, lists=A + 2)
    assert all(got[x] == api.FA_ERR_MISALIGNED for x in ("copy", "reserve", "fork", "free"))
    got = calls(lib, n=-1)
    assert all(got[x] == api.FA_ERR_INVALID_ARG for x in ("copy", "fork", "free"))
    assert calls(lib, n=5)["fork"] == api.FA_ERR_INVALID_ARG  # more forks than rows
    need = api.fa_pages_workspace_size(4, 10)
    for bad in (dict(ws=None), dict(ws_bytes=need - 1)):
        got = calls(lib, **bad)
        assert all(got[x] == api.FA_ERR_INVALID_ARG for x in ("reserve", "fork", "compact"))
    got = calls(lib, ws=A + 64)
    assert all(got[x] == api.FA_ERR_MISALIGNED for x in ("reserve", "fork", "compact"))
    assert calls(lib, out=None)["compact"] == api.FA_ERR_INVALID_ARG
    assert calls(lib, out=A + 2)["compact"] == api.FA_ERR_MISALIGNED
    got = calls(lib, pl=planes(num_pages=11))  # another pool than the table's
    assert got["fork"] == got["compact"] == api.FA_ERR_INVALID_ARG
    got = calls(lib, n=0)
    assert got["copy"] == got["fork"] == got["free"] == api.FA_OK
    got = calls(lib, t=table(rows=0, block_table=None, seq_lens=None), n=0)
    assert got["reserve"] == got["free"] == api.FA_OK
    assert api.fa_pages_workspace_size(-1, 4) == 0 and api.fa_pages_workspace_size(4, -1) == 0


def test_new_status_names(lib):
    assert api.status_str(api.FA_ERR_INDEX) == "FA_ERR_INDEX"
    assert api.status_str(api.FA_ERR_NO_PAGES) == "FA_ERR_NO_PAGES"


def test_the_binding_refuses_tensors_off_the_gpu():
    t = torch.zeros(2, 4, dtype=torch.int32)
    v = torch.zeros(2, dtype=torch.int32)
    q, pool = torch.zeros(2, 2, 1, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    for call in (lambda: api.fa_paged_attn(q, pool, pool, t, v), lambda: api.fa_pages_write(q, q, pool, pool, t, v),
                 lambda: api.fa_pages_free(16, t, v, v, v), lambda: api.fa_pages_copy([pool], v, v),
                 lambda: api.fa_pages_reserve(16, t, v, v, v), lambda: api.fa_pages_copy([], v, v),
                 lambda: api.fa_pages_compact([pool], 16, t, v, v), lambda: api.fa_pages_fork([pool], 16, t, v, v, v, v)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_valid_calls_without_a_gpu_fail_loudly(lib):
    assert attn(lib, problem()) == api.FA_ERR_CUDA
    assert write(lib, problem()) == api.FA_ERR_CUDA
    assert set(calls(lib).values()) == {api.FA_ERR_CUDA}
