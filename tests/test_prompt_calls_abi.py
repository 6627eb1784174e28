"""The prompt chunks' self-test switch and calls without rows through the C ABI.  No GPU: nothing is launched."""
from test_paged_abi import OK, SHAPE
from test_prompt_abi import lib, prefill  # noqa: F401


def test_selftest_limits(lib):  # noqa: F811
    for bad in (-1, 2001, -2 ** 31, 2 ** 31 - 1):
        assert lib.gdn_selftest_paged_prefill_wait(bad) == SHAPE
    assert lib.gdn_selftest_paged_prefill_wait(2000) == OK and lib.gdn_selftest_paged_prefill_wait(0) == OK


def test_calls_without_rows_take_any_workspace(lib):  # noqa: F811
    for ws, nbytes in ((None, 0), (None, 1 << 20), (64, 1 << 20), (1 << 20, 0), (1 << 20, 3)):
        assert prefill(lib, n=0, ws=ws, nbytes=nbytes) == OK and prefill(lib, B=0, ws=ws, nbytes=nbytes) == OK
