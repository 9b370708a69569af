"""Calls that could only write one place twice, or read what they have overwritten, are
refused before the device is touched (no GPU needed)."""

import pytest

from exact_io_aware_69_b200 import build, fa

from test_paged_boundary import P, append, cache, rope, strides


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return fa.load_paged()


@pytest.mark.parametrize("kw", [
    dict(syq=strides(b=0)), dict(syq=strides(h=0)), dict(syq=strides(n=0)),
    dict(syk=strides(b=0)), dict(syk=strides(h=0)), dict(syk=strides(n=0)),
    dict(hq=0, syk=strides(n=0)),
])
def test_rotated_rows_that_share_memory(lib, kw):
    assert rope(lib, **kw) == fa.FA_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(yq=P, syq=strides(h=1024, n=128)), dict(yq=P, sq=strides(b=0)),
    dict(yk=P + 0x200000, sk=strides(h=0)), dict(yk=P + 0x200000, syk=strides(n=2048)),
])
def test_rotation_in_place_with_other_strides(lib, kw):
    assert rope(lib, **kw) == fa.FA_ERR_INVALID


@pytest.mark.parametrize("kw", [dict(k_page=0), dict(k_head=0), dict(k_row=0), dict(v_page=0),
                                dict(v_head=0), dict(v_row=0)])
def test_pages_that_share_memory(lib, kw):
    assert append(lib, cache(**kw)) == fa.FA_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,code", [
    (dict(syq=strides(h=0)), fa.FA_ERR_UNSUPPORTED), (dict(syq=strides(n=0)), fa.FA_ERR_UNSUPPORTED),
    (dict(yq=P + 0x700000, syq=strides(h=1024, n=128)), fa.FA_ERR_INVALID),
])
def test_appended_queries(lib, kw, code):
    assert append(lib, cache(), **kw) == code
