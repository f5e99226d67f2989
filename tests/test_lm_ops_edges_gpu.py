"""Edges of the language-model operators that the documentation names: rows that a mask leaves empty, operands
that change between calls, views, sizes on both sides of a choice of kernel."""
import pytest
import torch

import binarized_convolution_b200 as bc
from test_lm_ops_gpu import TYPES, norm_inputs, rnd

pytestmark = pytest.mark.gpu


def test_scalars_that_change_between_calls():
    x, tokens = rnd(1, 3, 500), torch.tensor([0, 7, 499], device="cuda")
    r, b, pre, post, _ = norm_inputs(2, 5, 64, 0, torch.float32)
    scalar = torch.nn.Parameter(torch.tensor(0.5, device="cuda"))

    def results(v):
        f = bc.token_logprobs(x, tokens, top=3, temperature=v)
        d = bc.token_logprobs_backward(x, tokens, f.lse, f.entropy, d_logprob=f.lse, temperature=v)
        out = bc.block_norm(r, b, pre_weight=pre, post_weight=post, residual_scale=v, eps=v)
        grad = bc.block_norm_backward(out[0], b, pre_weight=pre, post_weight=post, residual_scale=v, eps=v,
                                      d_residual_out=r, d_normed=b)
        return [t for t in (*f, d, *out, *grad) if t is not None]

    for value in (0.5, 2.0, 0.25):
        with torch.no_grad():
            scalar.fill_(value)
        assert all(torch.equal(p, q) for p, q in zip(results(scalar), results(value)))


@pytest.mark.parametrize("dtype", TYPES)
def test_no_gradient_reaches_a_row_of_minus_infinity_alone(dtype):
    """Its own token's entry included, wherever that lies: in whole 8-element steps or in front of and behind them."""
    vocab = 1501
    base = torch.full((3, vocab + 8), float("-inf"), dtype=dtype, device="cuda")
    base[2] = 0.0
    for first in (0, 3):
        logits = base[:, first:first + vocab]
        for token in (0, 1, 4, 700, vocab - 1):
            tokens = torch.tensor([token, -1, token], device="cuda")
            f = bc.token_logprobs(logits, tokens, temperature=0.5)
            assert (f.lse[:2] == float("-inf")).all()
            one = torch.ones(3, device="cuda")
            for kw in (dict(d_logprob=one), dict(d_entropy=one), dict(d_logprob=one, d_entropy=one)):
                d = bc.token_logprobs_backward(logits, tokens, f.lse, f.entropy, temperature=0.5, **kw)
                assert (d[:2] == 0).all()
                if "d_logprob" in kw:
                    assert d[2, token] > 0
