"""What the torch forms and the C entry points of the language-model operators decide on the host: scalars that
change between calls, and refusals.  (Addresses below are never read.)"""
import pytest
import torch

from binarized_convolution_b200 import lm_ops


def test_a_scalar_given_as_a_tensor_is_read_at_every_call():
    def token(**kw):
        a = dict(rows=2, stride=8, vocab=8, dtype=torch.float32, top=0, temperature=1.0)
        return lm_ops._token_desc(*{**a, **kw}.values())[0]

    for scalar in (torch.tensor(0.5), torch.nn.Parameter(torch.tensor([0.5]))):
        assert token(temperature=scalar).temperature == 0.5
        with torch.no_grad():
            scalar.fill_(2.0)
        assert token(temperature=scalar).temperature == 2.0
    top = torch.tensor(3)
    assert token(top=top).top == 3
    top.fill_(5)
    assert token(top=top).top == 5
    assert token(temperature=2).temperature == 2.0
    for bad in (dict(temperature="1.0"), dict(temperature=None), dict(top=1.5)):
        with pytest.raises(TypeError):
            token(**bad)
