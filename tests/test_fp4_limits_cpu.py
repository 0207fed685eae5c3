"""Sizes at the limits that include/mxfp4.h states, on a machine without a GPU: the
last that is taken gets past the checks of shapes (to a missing pointer), the
next is refused as a shape."""
import re

import pytest

from tests.test_fp4_library_cpu import HEADER, NULL, P, SHAPE, lib  # noqa: F401


def _doc(name):
    """The comment before a declaration."""
    text = open(HEADER).read()
    at = re.search(r"\b%s\(" % name, text).start()
    return " ".join(text[text.rindex("/*", 0, at):at].replace("*", " ").split())


@pytest.mark.parametrize("k", [32, 160, 480])
def test_columns_of_the_decode_forms(k, lib):  # noqa: F811
    most = (1 << 27) - 16
    for n, status in ((most, NULL), (most + 1, SHAPE), (1 << 27, SHAPE), ((1 << 31) - 1, SHAPE)):
        assert lib.mx_linear_decode(P, k, P, P, 1, 3, n, k, None, 0, None) == status, n
    most = min(most, ((1 << 36) - 1) // (2 * k))
    for n, status in ((most, NULL), (most + 1, SHAPE)):
        assert lib.mx_gated_ffn_decode(P, k, P, P, 1, 3, n, k, 0, None, None) == status, n
    assert "n <= 2^27 - 16" in _doc("mx_linear_decode") and "cols <= 2^27 - 16" in _doc("mx_gated_ffn_decode")


def test_what_the_decode_forms_do_past_the_range_is_said():
    assert "+-Inf" in _doc("mx_linear_decode")
