"""The smallest temperatures that the logits' calls take, without a GPU: what is
accepted has a finite 1 / T and a finite log2(e) / T, the two factors that the
kernels work with."""
import pytest

from float8_mixed_precision_gb300 import binding

INVALID, ALIGN = 1, 2
P = 1 << 40


@pytest.fixture(scope="module")
def L():
    from float8_mixed_precision_gb300 import build
    build.build()
    return binding.lib()


def test_factors_are_finite(L):
    # 1 / T is finite down to 2.94e-39, log2(e) / T down to 4.24e-39.  An
    # argument off its alignment is refused after the temperature.
    for T, want in ((2.5e-39, INVALID), (3.5e-39, INVALID), (4.2e-39, INVALID), (4.3e-39, ALIGN), (1.0, ALIGN)):
        assert L.f8_token_logprobs(P, 0, 4, 100, 104, P + 4, T, 5, P, P, P, P, P, None) == want, T
        assert L.f8_distill_fwd(P, 0, 4, 100, 104, P, P, 8, T, 1, P + 2, P, P, None) == want, T
        assert L.f8_token_logprobs_bwd(P, 0, 4, 100, 104, P + 4, P, P, P, P, T, 2 * P, 104, P, None) == want, T
