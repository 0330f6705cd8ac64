"""Calls at the ends of what the arguments allow, as far as they go without a GPU: an
accepted call is refused for its output, which these place over q, or for q itself."""
import pytest

import paged_kv_decode_15_gb300 as pkd
from tests.test_serving_boundary import attend, prefix, rope


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


def test_products_of_sizes_that_wrap_around_64_bits(lib):
    """Each product is 2^63 or 2^64: as a 64-bit number negative, or 0."""
    big = dict(Hq=1 << 22, Hkv=1 << 15, q_stride=1 << 30)
    for T in (1 << 41, 1 << 42):
        assert attend(lib, T=T, max_q=1 << 20, **big) == pkd.EUNSUPPORTED and "2^31" in error(lib)
    # pages * heads * page size, within the bounds of each alone
    for pages, P in ((1 << 22, 1 << 30), (1 << 23, 1 << 30)):
        many = dict(Hq=1 << 11, Hkv=1 << 11, q_stride=1 << 18, num_pages=pages, P=P)
        assert attend(lib, **many) == pkd.EUNSUPPORTED and "cache too large" in error(lib)
        assert prefix(lib, Hq=1 << 11, Hkv=1 << 11, num_pages=pages, P=P) == pkd.EUNSUPPORTED and "cache too large" in error(lib)
    assert attend(lib, q_stride=1 << 61) == pkd.EUNSUPPORTED and "q_stride" in error(lib)
    for pages in (1 << 59, (1 << 60) + 1):
        assert rope(lib, num_pages=pages) == pkd.EUNSUPPORTED and "cache too large" in error(lib)
