"""Calls of the 8-bit operators that are refused before any device work."""
from test_quantized_checks import I, L, lib, read, refused  # noqa: F401


def test_read_into_one_buffer_is_refused(lib):  # noqa: F811
    refused(lib, read(lib, k=I, v=I), L.ERR_INVALID_ARG, "the same")
