"""fa.device_status over the two libraries' error words, against stand-ins for both."""

import types

import pytest

from exact_io_aware_69_b200 import fa


class Word:
    """An error word as the libraries keep it: read and cleared at once."""

    def __init__(self, value):
        self.value = value

    def __call__(self, stream):
        value, self.value = self.value, fa.FA_OK
        return value


@pytest.mark.parametrize("first", [fa.FA_OK, fa.FA_ERR_TIMEOUT])
@pytest.mark.parametrize("second", [None, fa.FA_OK, fa.FA_ERR_INVALID])
def test_no_error_is_lost(monkeypatch, first, second):
    """Every word that holds an error is returned by one call, the first library's first;
    then all is well. (second None: the paged library has not been loaded.)"""
    words = Word(first), Word(second)
    monkeypatch.setattr(fa, "load", lambda: types.SimpleNamespace(fa_get_device_status=words[0]))
    monkeypatch.setattr(fa, "_paged_lib", None if second is None else
                        types.SimpleNamespace(fa_paged_device_status=words[1]))
    stream = types.SimpleNamespace(cuda_stream=0)
    errors = [e for e in (first, second) if e not in (None, fa.FA_OK)]
    assert [fa.device_status(stream) for _ in range(3)] == errors + [fa.FA_OK] * (3 - len(errors))
