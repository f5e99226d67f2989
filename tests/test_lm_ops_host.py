"""Refusals of the language-model operators' C entry points and of their torch forms: everything
here is decided on the host, before any device work, so it runs without a GPU.  (Addresses
below are never read.)"""
import ctypes

import numpy as np
import pytest
import torch

import binarized_convolution_b200 as bc
from binarized_convolution_b200 import _native as nat

INVALID, UNSUPPORTED, NO_DEVICE = 1, 2, 6
P, ODD = 1 << 20, (1 << 20) + 1  # an aligned address and one that no element of 2 bytes has


def _quant_desc(**kw):
    d = dict(in_channels=64, out_channels=8, group_size=32, neuron=0, in_dtype=1, out_dtype=1)
    d.update(kw)
    return nat.bfc_quant_desc_t(**d)


def _quant_create(desc, codes=True, scale=True, bias=None):
    a = np.zeros(4096, np.float32)
    p = a.ctypes.data_as(ctypes.c_void_p)
    h = ctypes.c_void_p()
    st = bc.load_library().bfc_quant_create(ctypes.byref(desc) if desc else None, p if codes else None,
                                            p if scale else None, None, bias, ctypes.byref(h))
    assert h.value is None
    return st


@pytest.mark.parametrize("kw,expect", [
    (dict(in_channels=0), INVALID), (dict(out_channels=0), INVALID), (dict(group_size=0), INVALID),
    (dict(neuron=2), INVALID), (dict(in_dtype=3), INVALID), (dict(out_dtype=-1), INVALID),
    (dict(group_size=48), UNSUPPORTED), (dict(in_channels=1000, group_size=192), UNSUPPORTED),
    (dict(in_channels=(1 << 20) + 1), UNSUPPORTED), (dict(out_channels=(1 << 20) + 1), UNSUPPORTED),
])
def test_quant_create_refuses(kw, expect):
    assert _quant_create(_quant_desc(**kw)) == expect


def test_quant_create_refuses_missing_arrays_and_handles():
    lib = bc.load_library()
    assert _quant_create(None) == INVALID
    assert _quant_create(_quant_desc(), codes=False) == INVALID
    assert _quant_create(_quant_desc(), scale=False) == INVALID
    assert _quant_create(_quant_desc(), bias=ODD) == INVALID
    assert lib.bfc_quant_create(ctypes.byref(_quant_desc()), P, P, None, None, None) == INVALID
    junk = ctypes.cast((ctypes.c_uint32 * 64)(), ctypes.c_void_p)
    for h in (None, junk):
        assert lib.bfc_quant_forward(h, P, 64, 1, P, 8, None, None) == INVALID
        assert lib.bfc_quant_workspace_bytes(h, P, 64, 1) == -1
        assert lib.bfc_quant_input_feature_channels(h) == -1
        assert lib.bfc_quant_output_feature_channels(h) == -1
        assert lib.bfc_quant_sync_status(h, None) == INVALID
    assert lib.bfc_quant_destroy(None) == 0
    assert lib.bfc_quant_destroy(junk) == INVALID


def test_quant_create_without_a_device():
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    assert _quant_create(_quant_desc()) == NO_DEVICE


def _norm_desc(**kw):
    d = dict(rows=4, rows_per_gate=2, width=16, dtype=1, residual_scale=1.0, eps=1e-6)
    d.update(kw)
    return nat.bconv_block_norm_desc_t(**d)


NORM_FWD = dict(residual=P, block=P, gate=P, post=P, pre=P, out=P, normed=P)
NORM_BWD = dict(residual_out=P, block=P, gate=P, post=P, pre=P, d_out=P, d_normed=P, d_residual=P, d_block=P,
                d_pre=P, d_post=P, d_gate=P, ws=P)


def _norm(direction, desc_kw, ptr_kw):
    lib = bc.load_library()
    fn, ptrs = ((lib.bconv_block_norm_forward, NORM_FWD) if direction == "forward" else
                (lib.bconv_block_norm_backward, NORM_BWD))
    assert set(ptr_kw) <= set(ptrs)
    return fn(_norm_desc(**desc_kw), *{**ptrs, **ptr_kw}.values(), None)


@pytest.mark.parametrize("direction", ["forward", "backward"])
@pytest.mark.parametrize("kw,expect", [
    (dict(rows=-1), INVALID), (dict(width=0), INVALID), (dict(dtype=3), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(residual_scale=float("nan")), INVALID),
    (dict(rows_per_gate=0), INVALID), (dict(width=32769), UNSUPPORTED),
])
def test_block_norm_refuses_descriptors(direction, kw, expect):
    assert _norm(direction, kw, {}) == expect


@pytest.mark.parametrize("kw", [
    dict(residual=None), dict(residual=ODD), dict(block=ODD), dict(gate=ODD), dict(normed=ODD), dict(pre=P + 2),
    dict(block=None), dict(block=None, gate=None), dict(pre=None), dict(normed=None), dict(out=None),
    dict(block=None, gate=None, post=None, pre=None, normed=None, out=None),
])
def test_block_norm_forward_refuses_operands(kw):
    assert _norm("forward", {}, kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(residual_out=None), dict(ws=None), dict(ws=P + 16), dict(block=None), dict(gate=None), dict(post=None),
    dict(pre=None), dict(d_normed=ODD), dict(d_gate=P + 1), dict(block=None, gate=None, d_gate=None),
])
def test_block_norm_backward_refuses_operands(kw):
    assert _norm("backward", {}, kw) == INVALID


def test_null_descriptors_and_workspaces():
    lib = bc.load_library()
    assert lib.bconv_block_norm_forward(None, *[P] * 7, None) == INVALID
    assert lib.bconv_block_norm_backward(None, *[P] * 13, None) == INVALID
    assert lib.bconv_block_norm_workspace_bytes(None) == -1
    assert lib.bconv_block_norm_workspace_bytes(_norm_desc(width=-3)) == -1
    assert lib.bconv_block_norm_workspace_bytes(_norm_desc(rows=0)) == 0
    assert lib.bconv_block_norm_workspace_bytes(_norm_desc(rows=10 ** 6, width=4096)) > 0
    assert lib.bconv_token_logprobs_forward(None, *[P] * 7, None) == INVALID
    assert lib.bconv_token_logprobs_backward(None, *[P] * 7, 100, None) == INVALID


def _token_desc(**kw):
    d = dict(rows=4, stride=100, vocab=100, dtype=1, top=5, temperature=1.0)
    d.update(kw)
    return nat.bconv_token_desc_t(**d)


BAD_TOKEN_DESCS = [dict(rows=-1), dict(vocab=0), dict(stride=99), dict(dtype=5), dict(temperature=0.0),
                   dict(temperature=-1.0), dict(temperature=float("nan")), dict(temperature=float("inf")),
                   dict(temperature=1e-39), dict(vocab=(1 << 30) + 1, stride=1 << 31)]


@pytest.mark.parametrize("kw", BAD_TOKEN_DESCS + [dict(top=-1), dict(top=65), dict(vocab=4, top=5)])
def test_token_logprobs_forward_refuses_descriptors(kw):
    assert bc.load_library().bconv_token_logprobs_forward(_token_desc(**kw), *[P] * 7, None) == INVALID


@pytest.mark.parametrize("kw", BAD_TOKEN_DESCS)
def test_token_logprobs_backward_refuses_descriptors(kw):
    assert bc.load_library().bconv_token_logprobs_backward(_token_desc(**kw), *[P] * 7, 1 << 31, None) == INVALID


def test_token_logprobs_refuses_operands():
    fwd, bwd = bc.load_library().bconv_token_logprobs_forward, bc.load_library().bconv_token_logprobs_backward
    d = _token_desc()
    for at, value in ((0, None), (0, ODD), (1, None), (5, None), (6, None)):  # logits, tokens, the top pair
        ptrs = [P] * 7
        ptrs[at] = value
        assert fwd(d, *ptrs, None) == INVALID, at
    assert fwd(_token_desc(top=0), *[P] * 7, None) == INVALID  # top outputs without top
    for at, value in ((0, None), (0, ODD), (1, None), (2, None), (3, None), (6, None), (6, ODD)):
        ptrs = [P] * 7
        ptrs[at] = value
        assert bwd(d, *ptrs, 100, None) == INVALID, at
    assert bwd(d, *[P] * 6, P + 4096, 99, None) == INVALID    # d_stride below the vocabulary
    assert bwd(d, *[P] * 6, P, 128, None) == INVALID          # in place with another stride


def test_no_rows_is_no_work():
    lib = bc.load_library()
    assert lib.bconv_block_norm_forward(_norm_desc(rows=0), *[P] * 7, None) == 0
    assert lib.bconv_token_logprobs_forward(_token_desc(rows=0), *[P] * 7, None) == 0
    assert lib.bconv_token_logprobs_backward(_token_desc(rows=0), *[P] * 7, 100, None) == 0


def test_torch_forms_refuse_host_tensors_and_types():
    x = torch.zeros(2, 8)
    with pytest.raises(TypeError):
        bc.block_norm(x, x, pre_weight=torch.ones(8))
    with pytest.raises(TypeError):
        bc.block_norm_backward(x, x, pre_weight=torch.ones(8), d_normed=x)
    with pytest.raises(TypeError):
        bc.token_logprobs(x)
    with pytest.raises(TypeError):
        bc.token_logprobs_backward(x, None, x[:, 0], None)
    with pytest.raises(ValueError):
        bc.block_norm(x)
    codes, scale = torch.zeros(8, 64, dtype=torch.uint8), torch.ones(8, 2)
    for kw in (dict(codes=codes.int(), scale=scale), dict(codes=codes, scale=scale.int()),
               dict(codes=codes, scale=scale, dtype=torch.float64), dict(codes=codes, scale=scale, zero=scale)):
        with pytest.raises(TypeError):
            bc.QuantFC(64, 8, group_size=32, **kw)
    for kw in (dict(scale=scale), dict(codes=codes[:4], scale=scale), dict(codes=codes, scale=scale[:, :1]),
               dict(codes=codes, scale=scale, bias=torch.zeros(7)), dict(packed=codes, scale=scale)):
        with pytest.raises(ValueError):
            bc.QuantFC(64, 8, group_size=32, **kw)
    with pytest.raises(ValueError):
        bc.QuantFC(64, 8, codes=codes, scale=scale, group_size=0)
    with pytest.raises(bc.BconvError):
        bc.QuantFC(64, 8, codes=codes, scale=torch.ones(8, 2), group_size=48)


def test_pack_puts_even_channels_low():
    codes = torch.randint(0, 16, (3, 7), dtype=torch.uint8)
    packed = bc.QuantFC.pack(codes)
    assert packed.shape == (3, 4) and packed.dtype == torch.uint8
    for f in range(7):
        assert torch.equal((packed[:, f // 2] >> (4 * (f % 2))) & 15, codes[:, f])
    assert torch.equal(packed[:, 3] >> 4, torch.zeros(3, dtype=torch.uint8))
