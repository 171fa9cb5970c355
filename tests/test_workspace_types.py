"""Workspace sizes are asked for with a type; one that the calls refuse is refused (no GPU needed)."""
import pytest
import torch

import gated_delta_rule_109_b200 as kda
from gated_delta_rule_109_b200 import build as kbuild


@pytest.fixture(scope="module", autouse=True)
def _built():
    kbuild.build()


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.int8, torch.float8_e4m3fn])
def test_types_that_the_calls_refuse(dtype):
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        kda.la_workspace_bytes(1, 65536, 4, 128, 128, dtype)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        kda.la_workspace_bytes(1, 65536, 4, 128, 128, dtype, backward=True)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        kda.paged_decode_workspace_bytes(32, 8, 128, dtype)


def test_types_that_they_take():
    sizes = [kda.la_workspace_bytes(1, 65536, 4, 128, 128, t) for t in (torch.bfloat16, torch.float32)]
    assert all(n > 0 for n in sizes) and sizes[0] != sizes[1]
    assert all(kda.paged_decode_workspace_bytes(32, 8, 128, t) > 0 for t in (torch.bfloat16, torch.float32))
