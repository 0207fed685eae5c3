"""Every function that the kernels' sources declare for each other is called:
nothing stays that no entry point reaches."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_precision_quantization_amd", "csrc")


def _code(path):
    return re.sub(r"//[^\n]*", "", open(path).read())


@pytest.mark.parametrize("header", sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*_launch.h"))))
def test_declared_functions_are_called(header):
    names = set(re.findall(r"^(?:hipError_t|int64_t|int32_t|size_t|bool)\s+(\w+)\(", _code(os.path.join(CSRC, header)), re.M))
    assert names
    rest = "".join(_code(p) for p in glob.glob(os.path.join(CSRC, "*")) if os.path.basename(p) != header)
    for name in names:
        # once where it is defined, and where it is called
        assert len(re.findall(r"\b%s\s*\(" % name, rest)) >= 2, name
