"""Calls of the operators that their documentation allows: the smallest tables, streams given explicitly, results
changed in place, gradients that arrive at any address, scoring without gradients."""
import pytest
import torch

import catalogue_cross_entropy_amd as rece

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 4096, 4097, 70000, 300000])
@pytest.mark.parametrize("C,d", [(1, 8), (2, 8), (1, 16), (3, 24)])
@pytest.mark.parametrize("bf16_grads", [False, True])
def test_embed_gradient_of_a_small_table_is_cleared(n, C, d, bf16_grads):
    """Every row of the gradient is written, however few there are and whatever lay there: ids that are all padding
    leave zeros, one id its row alone."""
    op = rece.ItemEmbedding(n, C, d, bf16_grads=bf16_grads)
    dout = torch.ones(n, d, dtype=torch.bfloat16, device="cuda")
    ids = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    gdt = torch.bfloat16 if bf16_grads else torch.float32
    print(f"[gpu] embed gradient n={n} C={C} d={d} bf16_grads={bf16_grads}", flush=True)
    got = op.backward(ids, dout, dtable=torch.full((C, d), float("nan"), dtype=gdt, device="cuda"))
    assert not bool(got.any())
    ids[n // 2] = C - 1
    got = op.backward(ids, dout, dtable=torch.full((C, d), float("nan"), dtype=gdt, device="cuda"))
    assert bool((got[C - 1] == 1).all()) and not bool(got[:C - 1].any())
