"""Sizes at which the paged cache's calls stop, on the host."""
import pytest

from tests.test_cache_host import _attend, _cache, _read, _write, kz  # noqa: F401


def test_a_cache_without_units_takes_rows_without_memory(kz):  # noqa: F811
    c = _cache(kz, units=0, page_table=None, lens=None)
    assert _write(kz, c, k=None, v=None) == kz.OK and _read(kz, c, k=None, v=None) == kz.OK
    assert _attend(kz, c, q=None, out=None) == kz.OK
    assert _write(kz, _cache(kz), k=None) == kz.ERR_INVALID_ARG


@pytest.mark.parametrize("page_rows", [16, 32, 64, 128])
def test_units_end_before_positions_do(kz, page_rows):  # noqa: F811
    """The attention kernels look up to a few tiles past a unit's last row with 32-bit
    positions, which must not pass 2^31."""
    most = (2 ** 31 - 1 - 4096) // page_rows
    c = _cache(kz, page_rows=page_rows, max_pages=most + 1)
    for call in (_write, _read, _attend):
        assert call(kz, c) == kz.ERR_UNSUPPORTED
    assert kz.cache_attention_workspace_size(c, 4, 8) == 0
    # the largest that is left: nothing to refuse (and nothing to do)
    c = _cache(kz, page_rows=page_rows, max_pages=most)
    assert _read(kz, c, n=0) == kz.OK and _attend(kz, c, n_q=0) == kz.OK
    assert kz.cache_attention_workspace_size(c, 4, 8) > 0
