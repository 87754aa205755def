"""Sizes outside the operators' limits are refused by name through the tensors' calls too
(the C ABI's refusals: test_ops_abi.py).  Nothing is launched."""
import pytest
import torch

import bit_quantized_gemv_amd as q
from ops_util import DEV

pytestmark = pytest.mark.gpu


def zeros(*shape, dt=torch.bfloat16):
    return torch.zeros(*shape, dtype=dt, device=DEV)


def codes(*shape):
    return zeros(*shape, dt=torch.int32)


def refused(status, f, *args, **kw):
    with pytest.raises(q.QmvError) as e:
        f(*args, **kw)
    assert e.value.status == status, str(e.value)


@pytest.mark.parametrize("M,N,L,R,status", [(3, 8, 2, 513, 11), (3, 8, 2, 0, 11), (3, 8, 0, 4, 11), (65537, 8, 2, 4, 5), (3, 0, 2, 4, 4),
                                            (3, 8, 65537, 1, 11)])
def test_lora(M, N, L, R, status):
    refused(status, q.affine_lora, codes(N, 8), zeros(N, 1), zeros(N, 1), zeros(M, 64), zeros(L, R, 64), zeros(L, N, R), codes(M),
            bits=4, group_size=64)


@pytest.mark.parametrize("T,E,k,D,status", [(3, 1025, 2, 64, 12), (3, 40, 33, 64, 12), (65537, 4, 2, 64, 5), (3, 4, 2, 12, 4)])
def test_route(T, E, k, D, status):
    refused(status, q.route, zeros(T, D), zeros(E, D), top_k=k)


def experts(E):
    return (codes(E, 128, 8), zeros(E, 128, 1), zeros(E, 128, 1)), (codes(E, 64, 8), zeros(E, 64, 1), zeros(E, 64, 1))


@pytest.mark.parametrize("T,E,k,status", [(3, 4, 0, 12), (3, 4, 33, 12), (3, 0, 2, 12), (3, 1025, 2, 12), (65537, 4, 2, 5)])
def test_experts(T, E, k, status):
    refused(status, q.experts, zeros(T, 64), zeros(T, k, dt=torch.float32), codes(T, k), *experts(E), bits=4, group_size=64)


@pytest.mark.parametrize("T,E,k,status", [(3, 40, 33, 12), (3, 1025, 2, 12), (65537, 4, 2, 5)])
def test_moe(T, E, k, status):
    refused(status, q.moe, zeros(T, 64), zeros(E, 64), *experts(E), top_k=k, bits=4, group_size=64)


@pytest.mark.parametrize("B,S,V,status", [(1, 256, 10, 14), (65536, 0, 1, 14), (2, 3, 0, 14)])
def test_verify(B, S, V, status):
    refused(status, q.verify, zeros(B, S + 1, V), codes(B, S), zeros(B, S + 1, dt=torch.float32))
