"""Edges of the language-model operators that the documentation names: rows that a mask leaves empty, operands
that change between calls, views, sizes on both sides of a choice of kernel."""
import pytest
import torch

import binarized_convolution_b200 as bc
from binarized_convolution_b200 import lm_ops
import test_lm_ops_gpu as gpu
from test_lm_ops_gpu import TYPES, U, norm_inputs, rnd

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


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", [(3001, 1003), (1302, 4003)])
def test_block_norm_first_and_last_row_of_unaligned_arrays_stay_in_their_rows(rows, width, dtype):
    """Rows off 16-byte boundaries are copied in 16-byte pieces, but for the edges of the first and the last row;
    later rows in the same place of shared memory must not see those edges."""
    r, b, pre, post, _ = norm_inputs(rows, rows, width, 0, dtype)
    do, dn = rnd(1, rows, width, dtype=dtype), rnd(2, rows, width, dtype=dtype)
    kw = dict(pre_weight=pre, post_weight=post)
    arrays = [torch.empty(rows * width + 1, dtype=dtype, device="cuda")[1:].view(rows, width) for _ in range(4)]
    results = []
    for edge in (1.0, 1000.0):
        for array, values in zip(arrays, (r, b, do, dn)):
            array.copy_(values)
            array[0].mul_(edge)
            array[-1].mul_(edge)
        r1, b1, do1, dn1 = arrays
        first = bc.block_norm(r1, b1, **kw)[:2] + bc.block_norm_backward(r1, b1, d_residual_out=do1, d_normed=dn1, **kw)[:2]
        for _ in range(5):
            again = bc.block_norm(r1, b1, **kw)[:2] + bc.block_norm_backward(r1, b1, d_residual_out=do1, d_normed=dn1, **kw)[:2]
            assert all(torch.equal(p, q) for p, q in zip(first, again))
        results.append(first)
    assert all(torch.equal(p[1:-1], q[1:-1]) for p, q in zip(*results))


@pytest.mark.parametrize("width", [1024, 1027])
def test_block_norm_status_of_the_waits(width):
    """Whether a kernel that requests rows ahead gave up a wait comes back from the status call, and a graph's
    replays report to the same place."""
    rows = 3000
    r, b, pre, post, _ = norm_inputs(3, rows, width, 0, torch.bfloat16)
    stream = torch.cuda.current_stream().cuda_stream
    out = bc.block_norm(r, b, pre_weight=pre, post_weight=post)
    bc.bconv_block_norm_sync_status(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = bc.block_norm(r, b, pre_weight=pre, post_weight=post)
        bc.block_norm_backward(r, b, pre_weight=pre, post_weight=post, d_normed=r)
    graph.replay()
    bc.bconv_block_norm_sync_status(stream)
    assert all(torch.equal(p, q) for p, q in zip(out, held))


def test_block_norm_gate_of_more_rows_than_there_are():
    """rows_per_gate up to the largest int64: one gate row for all rows."""
    rows, width = 2500, 96
    out, b, pre, post, _ = norm_inputs(5, rows, width, 0, torch.float32)
    g, d = rnd(6, 1, width), rnd(7, rows, width)

    def run(per):
        kw = dict(pre_weight=pre, post_weight=post, gate=g, rows_per_gate=per)
        return (*bc.block_norm(out, b, **kw), *bc.block_norm_backward(out, b, d_normed=d, **kw))

    want = run(rows)
    for per in (rows + 1, 1 << 62, (1 << 63) - rows, (1 << 63) - 1):
        # (what the allocator may hand out again)
        poison = [torch.full((1, width), float("nan"), device="cuda") for _ in range(64)]
        del poison
        assert all(torch.equal(p, q) for p, q in zip(run(per), want)), per


def test_block_norm_rows_per_gate_is_a_positive_number_read_at_every_call():
    r, b, _, _, g = norm_inputs(8, 6, 32, 1, torch.float32)
    for bad in (0, -2):
        with pytest.raises(ValueError):
            bc.block_norm(r, b, gate=g, rows_per_gate=bad)
    with pytest.raises(TypeError):
        bc.block_norm(r, b, gate=g, rows_per_gate=1.0)
    per = torch.tensor(1)
    for n in (1, 2, 3):
        per.fill_(n)
        got = bc.block_norm(r, b, gate=g[:6 // n], rows_per_gate=per).residual_out
        assert torch.equal(got, bc.block_norm(r, b, gate=g[:6 // n].repeat_interleave(n, 0)).residual_out)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [40, 5000, 60000])
def test_token_logprobs_of_nearly_certain_tokens(vocab, dtype):
    """One other entry of probability p from 2e-5 to 2e-7: the sum 1 + p is rounded to fp32 (half a step: U), and that
    is the only rounding of the log probability -log(1 + p) and of the entropy that p's size does not shrink."""
    rows = 64
    logits = torch.full((rows, vocab), float("-inf"), device="cuda")
    logits[:, 7] = 0.0
    logits[:, 11] = -11.0 - torch.arange(rows, device="cuda") / 16
    logits = logits.to(dtype)
    tokens = torch.full((rows,), 7, dtype=torch.int64, device="cuda")
    got = bc.token_logprobs(logits, tokens, top=2)
    gap = -logits[:, 11].double()
    p = (-gap).exp()
    log_sum = torch.log1p(p)
    # exp2 is off by 2^-22 and by its argument's rounding (22 U), the last logarithm by 2 steps of its own size
    slack = 64 * U * p * (1 + gap) + U
    assert ((got.logprob.double() + log_sum).abs() <= slack).all()
    assert ((got.lse.double() - log_sum).abs() <= slack).all()
    assert ((got.top_logprob[:, 0].double() + log_sum).abs() <= slack).all()
    assert ((got.entropy.double() - (log_sum + p * gap / (1 + p))).abs() <= slack + 2 * U * p * gap).all()


# widths at which the shared memory of the CTAs beside each other is nearly all of it, and where two stages of a row cease to fit
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width,per", [(20000, 384, 0), (9000, 800, 1000), (9001, 724, 0), (9000, 840, 500),
                                            (1200, 5496, 0), (1201, 5499, 300), (1200, 5504, 0),
                                            (1201, 5523, 300), (1100, 7000, 0)])
def test_block_norm_at_the_edges_of_the_ring(rows, width, per, dtype):
    gpu.test_block_norm(rows, width, per, dtype)
    gpu.test_block_norm_backward(rows, width, per, dtype)


# calls of 9 to 16 rows whose rows leave room for one CTA on an SM, and their neighbours that leave room for two
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,k,n,group", [(14, 3584, 5000, 128), (13, 3584, 5000, 128), (14, 3400, 20000, 64),
                                            (15, 3328, 700, 32), (10, 4992, 20000, 128), (9, 5504, 9000, 5504),
                                            (9, 5505, 300, 128), (12, 4096, 6000, 128)])
def test_quant_fc_where_one_cta_fits(rows, k, n, group, dtype):
    gpu.test_quant_fc(rows, k, n, group, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [37, 4999, 20001])
def test_token_logprobs_backward_of_views(vocab, dtype):
    """Gradients whose rows lie otherwise than the logits', from the torch form and with a row stride of their own:
    the values, and nothing written between the rows."""
    from binarized_convolution_b200 import _native as nat

    rows, temperature = 6, 0.7
    base = rnd(vocab, rows, vocab + 21, dtype=dtype, scale=3.0)
    tokens = torch.tensor([0, 1, -1, 11, vocab // 2, vocab - 1], device="cuda")
    g, ge = rnd(1, rows), rnd(2, rows)
    for first in (0, 5, 16):
        x = base[:, first:first + vocab]
        f = bc.token_logprobs(x, tokens, temperature=temperature)
        want, mag = gpu.token_grad_ref(x, tokens, g, ge, temperature)
        p = (x.double() / temperature).log_softmax(1).exp()
        # (as for contiguous rows)
        bound = U * (200 + vocab / 512) * (mag + want.abs()) + p * ge.double().abs()[:, None] / temperature * U * 200 * 12
        got = bc.token_logprobs_backward(x, tokens, f.lse, f.entropy, d_logprob=g, d_entropy=ge, temperature=temperature)
        gpu.close(got, want, bound)
        for shift, stride in ((0, vocab + 3), (1, vocab + 16), (8, vocab + 21), (first, vocab + 21)):
            wide = torch.full((rows * stride + 32,), 7.0, dtype=dtype, device="cuda")
            d = wide[shift:shift + rows * stride].view(rows, stride)
            desc = nat.bconv_token_desc_t(rows, x.stride(0), vocab, lm_ops._DTYPES[dtype], 0, temperature)
            bc.bconv_token_logprobs_backward(desc, x.data_ptr(), tokens.data_ptr(), f.lse.data_ptr(), f.entropy.data_ptr(),
                                             g.data_ptr(), ge.data_ptr(), d.data_ptr(), stride,
                                             torch.cuda.current_stream().cuda_stream)
            gpu.close(d[:, :vocab], want, bound)
            assert (d[:, vocab:] == 7).all() and (wide[:shift] == 7).all() and (wide[shift + rows * stride:] == 7).all()
