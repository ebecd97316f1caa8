"""Host-only checks of the paged cache's self-test and limits: every refusal comes before the GPU is touched."""

import ctypes


from exact_io_aware_91_b200 import api
from test_paged_abi import A, calls, lib, problem  # noqa: F401


def give_up(lib, segment, ws_bytes=1 << 40, q=A, **change):  # noqa: F811
    p = problem(**change)
    return lib.fa_selftest_paged_give_up(ctypes.byref(p), q, A, A, A, A, A, A, A, A, ws_bytes, segment, None)


def test_the_self_test_refuses_what_the_call_refuses(lib):  # noqa: F811
    for segment in (0, -1, -2 ** 31):
        assert give_up(lib, segment) == api.FA_ERR_INVALID_ARG
    assert give_up(lib, 1, d=96) == api.FA_ERR_UNSUPPORTED
    assert give_up(lib, 1, q=A + 8) == api.FA_ERR_MISALIGNED
    assert give_up(lib, 1, ws_bytes=0) == api.FA_ERR_INVALID_ARG
    assert give_up(lib, 1, B=0) == api.FA_OK


def test_a_list_of_pairs_has_a_limit(lib):  # noqa: F811
    assert calls(lib, n=(1 << 24) + 1)["copy"] == api.FA_ERR_UNSUPPORTED
