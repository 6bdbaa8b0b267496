"""The norm modules and the logits' functions of float8_mixed_precision_gb300.nn
without a GPU: which torch norms they take over (sharing their Parameters), and
that they refuse what libf8 cannot take instead of computing it in torch."""
import pytest
import torch

from float8_mixed_precision_gb300 import nn as f8nn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from float8_mixed_precision_gb300 import build
    build.build()


def test_norms_share_parameters():
    a = torch.nn.LayerNorm(48, eps=1e-3, dtype=torch.bfloat16)
    m = f8nn.LayerNorm.from_norm(a)
    assert m.weight is a.weight and m.bias is a.bias and m.eps == 1e-3 and m.dim == 48
    b = torch.nn.LayerNorm(48, bias=False)
    m = f8nn.LayerNorm.from_norm(b)
    assert m.weight is b.weight and m.bias is None
    c = torch.nn.RMSNorm(48, eps=1e-6)
    m = f8nn.RMSNorm.from_norm(c)
    assert m.weight is c.weight and m.bias is None and m.eps == 1e-6
    assert [n for n, _ in f8nn.LayerNorm(16).named_parameters()] == ["weight", "bias"]
    assert [n for n, _ in f8nn.RMSNorm(16).named_parameters()] == ["weight"]
    assert "eps=1e-06" in repr(m)


def test_norm_refusals():
    for bad in (torch.nn.LayerNorm((4, 8)), torch.nn.LayerNorm(8, elementwise_affine=False)):
        with pytest.raises(ValueError):
            f8nn.LayerNorm.from_norm(bad)
    for bad in (torch.nn.RMSNorm((4, 8), eps=1e-5), torch.nn.RMSNorm(8),
                torch.nn.RMSNorm(8, eps=1e-5, elementwise_affine=False)):
        with pytest.raises(ValueError):
            f8nn.RMSNorm.from_norm(bad)
    with pytest.raises(ValueError):
        f8nn.RMSNorm(0)
    m = f8nn.RMSNorm(8)
    with pytest.raises(ValueError, match="8 features"):
        m(torch.zeros((2, 9), dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        m(torch.zeros((2, 8), dtype=torch.float16))
    with pytest.raises(ValueError, match="device tensors"):
        m(torch.zeros((2, 8), dtype=torch.bfloat16))             # host tensors: no CPU path


def test_logit_refusals():
    z = torch.zeros((2, 3, 40))
    tokens = torch.zeros((2, 3), dtype=torch.int64)
    ids, values = torch.zeros((2, 3, 4), dtype=torch.int32), torch.zeros((2, 3, 4))
    with pytest.raises(ValueError, match="leading shape"):
        f8nn.token_logprobs(z, tokens[:, :2])
    with pytest.raises(ValueError, match="leading shape"):
        f8nn.distill_loss(z, ids[:, :2], values[:, :2])
    with pytest.raises(ValueError, match="leading shape"):
        f8nn.distill_loss(z, ids, values[..., :2])
    for vocab in (0, 41):
        with pytest.raises(ValueError, match="vocab"):
            f8nn.token_logprobs(z, tokens, vocab=vocab)
        with pytest.raises(ValueError, match="vocab"):
            f8nn.distill_loss(z, ids, values, vocab=vocab)
    with pytest.raises(ValueError, match="device tensors"):
        f8nn.token_logprobs(z, tokens)
    with pytest.raises(ValueError, match="device tensors"):
        f8nn.distill_loss(z, ids, values, vocab=33)


def test_example_imports():
    from float8_mixed_precision_gb300 import example_distill
    assert callable(example_distill.main) and callable(example_distill.student_step)
