"""What the workspace query refuses before it touches a device."""
import ctypes

import pytest

import compressed_decode_attention_fdms_b200 as fd


@pytest.fixture(scope="module")
def lib():
    from compressed_decode_attention_fdms_b200 import build
    build.build()
    return fd.load_library()


def test_workspace_of_a_null_cache(lib):
    n = ctypes.c_size_t(5)
    for uses in (0, 7, 8):
        assert lib.fdms_prefill_workspace_for(None, 1, 1, 1, uses, ctypes.byref(n)) == \
            fd.FDMS_ERR_INVALID_ARG
