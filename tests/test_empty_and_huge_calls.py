"""Calls at the ends of what the arguments allow, as far as they go without a GPU: an
accepted call is refused for its output, which these place over q, or for q itself."""
import ctypes

import pytest

import paged_kv_decode_15_gb300 as pkd
from tests.test_serving_boundary import FAKE, attend, prefix


@pytest.fixture(scope="module")
def lib():
    pkd.build()
    return pkd.load_library()


def error(lib):
    return lib.pkd_last_error().decode()


def test_a_table_without_columns_may_be_null(lib):
    assert attend(lib, table=None, stride=0, max_kv=0) == pkd.EINVAL and "overlaps" in error(lib)
    assert prefix(lib, table=None, stride=0, max_kv=0) == pkd.EINVAL and "overlaps" in error(lib)
    assert prefix(lib, ptable=None, pstride=0, max_prefix=0) == pkd.EINVAL and "overlaps" in error(lib)
    for call, name in ((attend, "table"), (prefix, "table"), (prefix, "ptable")):
        assert call(lib, **{name: None}) == pkd.EINVAL and "null" in error(lib)
    assert prefix(lib, ptable=None, pstride=0, max_prefix=0, plens=None) == pkd.EINVAL and "null" in error(lib)


def test_the_most_that_no_requests_bring_is_nothing(lib):
    """An empty batch whose caller takes the largest of no lengths."""
    assert attend(lib, T=0, max_q=0) == pkd.OK and attend(lib, B=0, T=0, max_q=0) == pkd.OK
    assert lib.pkd_paged_attention_workspace_size(0, 0, 0, 4, 2, 128, 16, 100, pkd.BF16, None) > 0
    assert attend(lib, T=1, max_q=0) == pkd.EINVAL and "max_query_len" in error(lib)
    assert attend(lib, T=0, max_q=-1) == pkd.EINVAL and "max_query_len" in error(lib)
