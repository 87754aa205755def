"""The experts' outputs are rounded once, at the end: a bf16 output is the fp32 output of the same call, rounded."""
import pytest
import torch

from test_gpu_moe import call_experts, call_moe, problem, some_ids

pytestmark = pytest.mark.gpu


# one token and a few (whole tokens), pairs as they come, pairs sorted by expert, windows of scales
@pytest.mark.parametrize("bits,gs,T,E,k,D,F", [(4, 64, 1, 16, 4, 512, 256), (2, 64, 3, 5, 2, 320, 448), (4, 64, 12, 40, 9, 256, 320),
                                               (2, 64, 64, 16, 2, 1024, 512), (4, 64, 150, 3, 1, 512, 5760),
                                               (2, 128, 128, 8, 4, 768, 1920), (4, 128, 254, 6, 1, 1280, 1152), (2, 64, 40, 2, 2, 128, 81920)])
@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_experts_round_once(bits, gs, T, E, k, D, F, x):
    p = problem(T, E, k, D, F, bits, gs, x=x, seed=T)
    ids, weights = some_ids(T, E, k)
    ids[::5, 0] = -1
    wide = call_experts(p, weights, ids)
    assert torch.equal(call_experts(p, weights, ids, out_dtype=torch.bfloat16), wide.bfloat16())


@pytest.mark.parametrize("T", [1, 13, 70])
def test_moe_rounds_once(T):
    p = problem(T, 16, 4, 512, 256, seed=T)
    assert torch.equal(call_moe(p, out_dtype=torch.bfloat16)[0], call_moe(p)[0].bfloat16())
