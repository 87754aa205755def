"""The binding's arguments that are not tensors (no GPU needed)."""
import pytest
import torch

import bit_quantized_gemv_amd as q
from test_ops_abi import tensors

from test_ops_abi import L  # noqa: F401  (builds the library if it is not there)


class Unsure:
    def __bool__(self):
        raise OverflowError("neither")


@pytest.mark.parametrize("op", ["moe", "route"])
def test_a_flag_that_raises(L, op):  # noqa: F811
    """The error of a truth value that cannot be told is raised as it is, before the call."""
    a = {**tensors("moe"), "renormalize": Unsure()}
    with pytest.raises(OverflowError, match="neither"):
        if op == "moe":
            q.moe(**a)
        else:
            q.route(a["x"], a["router"], top_k=2, renormalize=a["renormalize"])
    with pytest.raises(RuntimeError, match="ambiguous"):
        q.route(a["x"], a["router"], top_k=2, renormalize=torch.zeros(2))


@pytest.mark.parametrize("kw", [dict(bits="4"), dict(group_size=64.0), dict(bits=None)])
def test_numbers(L, kw):  # noqa: F811
    with pytest.raises(TypeError, match="must be an integer"):
        q.affine_lora(**{**tensors("lora"), **kw})
