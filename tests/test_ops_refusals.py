"""Further refusals of the operators, before anything is enqueued: no GPU is needed."""
import pytest

import catalogue_cross_entropy_amd as rece
from test_ops_abi import _lp_bwd, _lp_fwd


@pytest.mark.parametrize("T", [2.0 ** -20 * 0.99, 1e-8, 1e-30, 1e-44, 2.0 ** 64 * 1.01, 1e30, 3e38])
def test_logprob_temperatures_out_of_range(T):
    assert _lp_fwd(T=T) == 1 and "temperature" in rece.lib().rece_last_error().decode()
    assert _lp_bwd(T=T) == 1
    with pytest.raises(ValueError):
        rece.LogProb(10, 20, 64, temperature=T)


@pytest.mark.parametrize("T", [2.0 ** -20, 1e-6, 1e6, 2.0 ** 64])
def test_logprob_temperatures_in_range(T):
    assert rece.LogProb(10, 20, 64, temperature=T).temperature == T
