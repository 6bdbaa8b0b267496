"""One row of a padded head's logits, with the gradient in the logits' own
buffer, as for any other number of rows."""
import pytest
import torch

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
@pytest.mark.parametrize("vocab,pad", [(1, 7), (1001, 7), (50003, 13)])
def test_one_row_in_place(f8, vocab, pad, dtype):
    g = torch.Generator(device=DEV).manual_seed(vocab)
    full = torch.full((1, vocab + pad), float("nan"), dtype=dtype, device=DEV)
    full[:, :vocab] = (torch.randn((1, vocab), generator=g, device=DEV) * 2).to(dtype)
    two = torch.cat((full, full))
    tokens = torch.zeros(2, dtype=torch.int64, device=DEV)
    one = torch.ones(2, device=DEV)
    _, ent, lse, ids, top = f8.f8_token_logprobs(two[:, :vocab], tokens, top_k=1)
    top = top - 0.1
    _, dlse, rest = f8.f8_distill_fwd(two[:, :vocab], ids, top, tail=True)

    def calls(n):
        yield lambda z, buf: f8.f8_token_logprobs_bwd(z, tokens[:n], lse[:n], ent[:n], one[:n], one[:n], dlogits=buf)
        yield lambda z, buf: f8.f8_distill_bwd(z, ids[:n], top[:n], dlse[:n], rest[:n], one[:n], tail=True, dlogits=buf)
        yield lambda z, buf: f8.f8_distill_fwd_bwd(z, ids[:n], top[:n], one[:n], tail=True, dlogits=buf)[1]

    for of_two, of_one in zip(calls(2), calls(1)):
        want = of_two(two[:, :vocab], torch.full_like(two, 3.0))
        own = full.clone()
        got = of_one(own[:, :vocab], own)
        assert got is own and torch.equal(own, want[:1]) and not own[:, vocab:].any()
    assert f8.f8_last_device_status() == 0
