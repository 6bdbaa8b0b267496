"""The logits' gradient of the entropy at small temperatures, where |lse| is in
the tens of thousands and one step of a bf16 logit is hundreds of units of its
exponent: only the row's largest logits have a gradient, and tokens below them,
masked ones among them, none."""
import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def f8():
    import float8_mixed_precision_gb300 as m
    from float8_mixed_precision_gb300 import build
    build.build()
    m.lib()
    return m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("top,T", [(40.0, 5e-4), (500.0, 0.01), (1000.0, 0.01), (2000.0, 0.05),
                                   (3000.0, 0.02), (1.0, 1e-5), (-600.0, 0.01)])
def test_small_temperatures(f8, top, T, dtype):
    rows, vocab = 6, 4099
    g = torch.Generator(device=DEV).manual_seed(int(top))
    # bf16 values in both types: neighbouring ones are at least 100 exponent units apart
    z = top - abs(top) * (0.02 + 0.3 * torch.rand((rows, vocab), generator=g, device=DEV))
    z = z.to(torch.bfloat16)
    at = torch.rand((rows, vocab), generator=g, device=DEV).argsort(1)[:, :3]
    z.scatter_(1, at, top)                                       # three tokens share the mass
    z[1, 2::3] = float("-inf")
    z[2, 1::3] = torch.finfo(torch.bfloat16).min
    z[1:3].scatter_(1, at[1:3], top)
    z = z.to(dtype)
    tokens = at[:, 0].clone()
    tokens[3] = (z[3] < top).int().argmax()                     # one without mass
    a = torch.randn(rows, generator=g, device=DEV)
    h = torch.randn(rows, generator=g, device=DEV)
    _, ent, lse, _, _ = f8.f8_token_logprobs(z, tokens, temperature=T)
    assert lse.abs().max().item() < 2 ** 24
    for da, dh in ((a, h), (None, h)):
        d = f8.f8_token_logprobs_bwd(z, tokens, lse, ent, da, dh, temperature=T)
        r, b = ref.token_logprobs_bwd(z, tokens, lse, ent, da, dh, T)
        ref.check(d, r, b + ref.rounding(r, dtype) * (r != 0), f"top {top} T {T} {dtype}")
        rest = z < top
        rest[torch.arange(rows, device=DEV), tokens] = False
        assert not d[rest].any()
    assert f8.f8_last_device_status() == 0
