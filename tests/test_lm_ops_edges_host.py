"""What the torch forms and the C entry points of the language-model operators decide on the host: scalars that
change between calls, and refusals.  (Addresses below are never read.)"""
import pytest
import torch

import binarized_convolution_b200 as bc
from binarized_convolution_b200 import _native as nat
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


P, INVALID = 1 << 20, 1


def test_token_logprobs_refuses_operands_off_their_elements_boundary():
    lib = bc.load_library()
    desc = nat.bconv_token_desc_t(4, 100, 100, nat.DTYPE_BF16, 5, 1.0)
    calls = ((lib.bconv_token_logprobs_forward, 7, (), {1: 8}),        # logits, tokens, then floats and indexes
             (lib.bconv_token_logprobs_backward, 7, (100,), {1: 8, 6: 2}))  # d_logits last, of the logits' type
    for fn, count, rest, sizes in calls:
        for at in range(count):
            size = 2 if at == 0 else sizes.get(at, 4)
            ptrs = [P] * count
            ptrs[at] = P + size // 2
            assert fn(desc, *ptrs, *rest, None) == INVALID, (fn.__name__, at)


def test_token_logprobs_refuses_temperatures_whose_inverse_overflows():
    """Also where 1 / temperature is finite but log2(e) / temperature is not: from 2.94e-39 to 4.24e-39."""
    lib = bc.load_library()
    for temperature in (1e-45, 2.9e-39, 3e-39, 4.2e-39):
        desc = nat.bconv_token_desc_t(4, 100, 100, nat.DTYPE_BF16, 5, temperature)
        assert lib.bconv_token_logprobs_forward(desc, *[P] * 7, None) == INVALID, temperature
        assert lib.bconv_token_logprobs_backward(desc, *[P] * 7, 100, None) == INVALID, temperature
    desc = nat.bconv_token_desc_t(0, 100, 100, nat.DTYPE_BF16, 5, 4.3e-39)
    assert lib.bconv_token_logprobs_forward(desc, *[P] * 7, None) == 0


def test_block_norm_status_needs_a_device():
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    with pytest.raises(bc.BconvError):
        bc.bconv_block_norm_sync_status()


def test_a_quant_fc_has_no_methods_of_the_bit_packed_layers():
    for name in ("forward_io", "set_output_terms", "bits_shape", "forward_to_bits", "forward_from_bits"):
        assert not hasattr(bc.QuantFC, name), name
        assert hasattr(bc.BinaryConv2d, name) and hasattr(bc.BinaryFC, name), name
    for name in ("close", "__enter__", "__exit__", "sync_status", "forward_into"):
        assert hasattr(bc.QuantFC, name), name
