"""Sizes and uses of the layer operators that reach their further code paths:
large counts, other streams, graphs of bound calls, kernels chosen for many
tokens.  Bounds and helpers are those of test_gpu_layer."""

import numpy as np
import pytest
import torch

import workloads
from test_gpu_layer import Gated, normal

csf = pytest.importorskip("moe_weight_decode_amd")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch.device("cuda:0")


@pytest.mark.parametrize("S", [3_000_000, 4_194_304 + 37])
def test_millions_of_slots_of_one_expert(dev, S):
    # blocks of 16 slots times tiles passes 32 bits; every slot's result is its token's
    F, K, T = 16, 32, 1000
    c = Gated(1, F, K, [T], workloads.NVFP4, seed=21, T=T)
    token = torch.arange(T, dtype=torch.int32, device=dev)
    h, gu = csf.moe_gated(c.stack, c.tw, c.x, c.ta, c.te, token, save=True)
    dh = normal(np.random.default_rng(3), T, F, dtype=torch.bfloat16)
    dx, dgu = csf.moe_gated_backward(c.stack, c.dense(), c.tw, dh, gu, c.ta, c.te)
    rows = token.repeat((S + T - 1) // T)[:S].contiguous()
    es, at = torch.tensor([0, S], dtype=torch.int32, device=dev), rows.long()
    hs, gus = csf.moe_gated(c.stack, c.tw, c.x, c.ta, es, rows, save=True)
    assert torch.equal(hs, h[at]) and torch.equal(gus, gu[at])
    dxs, dgus = csf.moe_gated_backward(c.stack, c.dense(), c.tw, dh[at], gus, c.ta, es)
    assert torch.equal(dxs, dx[at]) and torch.equal(dgus, dgu[at])
