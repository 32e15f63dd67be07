"""How near the operators come to their 64-bit forms where float32 or bf16 intermediates would show."""
import pytest
import torch

import catalogue_cross_entropy_amd as rece
import ops_reference as R
import test_gpu_logprob as TL

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("s,C,d,entropy", [
    (8, 2000, 64, False), (8, 2000, 64, True), (70, 9, 32, False), (300, 12, 128, True), (300, 12, 256, False),
    (9, 700, 256, True), (70, 400, 128, False), (600, 40, 64, False), (40, 30000, 64, False),
])
def test_logprob_bf16_gradients_round_the_results_alone(s, C, d, entropy):
    """bf16 gradients are the float32 ones rounded, but for 2^-16 of each weight (two bf16 terms, each off by at most
    half a step: 2^-8 of 2^-8).  Few positions or few items: results much smaller than their terms, where weights
    rounded to bf16 would be off by up to 13 times the bound."""
    X, Y, ids, dlogp, dent, bad = TL._case(s, C, d, "bf16", seed=s + C + d, pad=0.1, peak=0.5)
    if not entropy:
        dent = None
    print(f"[gpu] logprob bf16 gradients s={s} C={C} d={d} entropy={entropy}", flush=True)
    _, _, dX, dY = TL._run(X, Y, ids, dlogp, dent, 0.9, entropy, True)
    w = R.logprob(X, Y, ids, 0.9, dlogp, dent)
    assert bool((dX[bad] == 0).all())
    for name, got in (("dX", dX), ("dY", dY)):
        assert got.dtype == torch.bfloat16
        bound = w["p_" + name] + 2.0 ** -8 * w["b_" + name]
        bound = bound + R.U[torch.bfloat16] * (w[name].abs() + bound) + 1e-30
        err = (got.double() - w[name]).abs()
        assert bool((err <= bound).all()), (name, float((err / bound).max()))
