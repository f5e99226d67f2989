"""The language-model operators against their definitions in 64 bits.

Tolerances count roundings.  U is the unit roundoff of fp32 (2^-24); an output of type t is
rounded once more, by at most finfo(t).eps / 2 of its value.  A sum of n terms in any order
is off by at most about n U times the sum of their magnitudes; the bounds below put in for n the
longest chain of additions of any kernel (for tensor-core sums, which may cut instead of
round, twice U).  exp2 and log2 are the hardware's approximations (2^-22 relative, respectively 2^-22
absolute), rsqrt has 2^-22.
"""
import numpy as np
import pytest
import torch

import binarized_convolution_b200 as bc

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def half_step(t):
    return torch.finfo(t).eps / 2


def rnd(seed, *shape, dtype=torch.float32, scale=1.0, device="cuda"):
    g = torch.Generator("cpu").manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(dtype).to(device)


def close(got, want, bound):
    """|got - want| <= bound + half a step of got's type (plus its smallest subnormal step)."""
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}[got.dtype]
    err = (got.double() - want).abs()
    limit = bound + half_step(got.dtype) * (want.abs() + bound) + tiny
    worst = (err - limit).max().item() if err.numel() else -1
    assert torch.isfinite(got).all()
    assert worst <= 0, f"off by {err.max().item():.3e}, {worst:.3e} over the bound"


# ---------------------------------------------------------------------------------- QuantFC


def quant_case(seed, k, n, group, zero, bias):
    g = torch.Generator("cpu").manual_seed(seed)
    groups = -(-k // group)
    codes = torch.randint(0, 16, (n, k), generator=g, dtype=torch.uint8)
    scale = 0.01 * (0.2 + torch.rand(n, groups, generator=g)) * torch.sign(torch.rand(n, groups, generator=g) - 0.2)
    z = torch.randint(0, 16, (n, groups), generator=g, dtype=torch.uint8) if zero else None
    b = torch.randn(n, generator=g) if bias else None
    column = torch.arange(k) // group
    w = (codes.double() - (8.0 if z is None else z.double()[:, column])) * scale.double()[:, column]
    return codes, scale, z, b, w.cuda()


def quant_check(got, x, w, b, group, relu=False):
    want = x.double() @ w.t()
    mag = x.double().abs() @ w.abs().t()
    if b is not None:
        want, mag = want + b.double().cuda(), mag + b.double().abs().cuda()
    # a group's (or 128 channels') sum, one addition a group or 128 channels, a few for splits and the bias
    steps = min(128, group) + -(-x.shape[-1] // min(group, 128)) + 16
    close(got, want.clamp_min(0) if relu else want, 2 * U * steps * mag)


QUANT_SHAPES = [
    # rows, k, n, group
    (1, 32, 1, 32), (1, 128, 128, 128), (1, 4096, 512, 128), (2, 200, 130, 32), (3, 129, 127, 64),
    (4, 1000, 257, 128), (7, 4096, 96, 256), (8, 512, 640, 64), (9, 640, 200, 128), (16, 2048, 384, 32),
    (17, 300, 33, 1000), (31, 1111, 129, 128), (33, 256, 256, 64), (64, 1024, 1024, 128), (65, 384, 640, 32),
    (100, 4096, 300, 128), (127, 520, 136, 64), (128, 768, 256, 256), (129, 1000, 384, 128), (255, 128, 128, 32),
    (256, 2048, 512, 128), (257, 136, 264, 64), (400, 1537, 1000, 128), (700, 640, 2000, 640), (1, 25088, 64, 128),
    (5, 12544, 256, 64), (40, 25088, 130, 128), (1, 1, 1, 32), (2, 31, 3, 32), (3, 33, 5, 32),
    # fp32: parts as rows of their own, up to 32 rows, with and without shared input channels
    (9, 25088, 512, 128), (32, 4096, 1000, 64), (31, 640, 18900, 128), (20, 300, 19000, 32), (33, 2048, 700, 128),
    # several tiles a CTA: few tokens and many
    (40, 256, 20000, 128), (33, 160, 25000, 32), (70, 384, 30000, 64), (96, 129, 19500, 128), (17, 900, 40000, 256),
    (1500, 130, 5000, 64), (900, 256, 9000, 32), (2100, 300, 3000, 128), (4000, 64, 640, 64), (200, 1000, 20000, 128),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,k,n,group", QUANT_SHAPES)
def test_quant_fc(rows, k, n, group, dtype):
    seed = rows * 7 + k + n
    zero, bias, relu = seed % 2 == 0, seed % 3 == 0, seed % 5 == 0
    out_dtype = torch.float32 if seed % 4 == 0 else dtype
    codes, scale, z, b, w = quant_case(seed, k, n, group, zero, bias)
    x = rnd(seed, rows, k, dtype=dtype)
    with bc.QuantFC(k, n, codes=codes, scale=scale, zero=z, bias=b, group_size=group, relu=relu, dtype=dtype,
                    out_dtype=out_dtype) as fc:
        y = fc(x)
        fc.sync_status()
        assert y.dtype == out_dtype and y.shape == (rows, n)
        quant_check(y, x, w, b, group, relu)
        assert torch.equal(y, fc(x))  # bit for bit


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 6, 20, 150])
def test_quant_fc_strided_and_unaligned_rows(rows, dtype):
    k, n, group = 384, 200, 128
    codes, scale, z, b, w = quant_case(rows, k, n, group, True, True)
    with bc.QuantFC(k, n, codes=codes.cuda(), scale=scale.cuda(), zero=z.cuda(), bias=b.cuda(), group_size=group,
                    dtype=dtype) as fc:
        base = rnd(rows, rows + 2, 2 * k + 3, dtype=dtype)
        for x in (base[:rows, :k], base[1:rows + 1, 3:k + 3], base[:rows, 8:8 + k].t().contiguous().t()):
            wide = torch.full((rows + 1, n + 5), 7.0, dtype=dtype, device="cuda")
            out = wide[:rows, 2:n + 2]
            fc.forward_into(x, out)
            quant_check(out, x, w, b, group)
            assert (wide[rows] == 7).all() and (wide[:, :2] == 7).all() and (wide[:, n + 2:] == 7).all()
        fc.sync_status()
        x = base[:rows, :k].contiguous().reshape(1, rows, k)
        assert torch.equal(fc(x)[0], fc(x[0]))


def test_quant_fc_what_lies_behind_the_rows_does_not_matter():
    k, n = 200, 140  # neither fills its tile
    codes, scale, z, b, w = quant_case(3, k, n, 64, True, False)
    for dtype in TYPES:
        with bc.QuantFC(k, n, codes=codes, scale=scale, zero=z, group_size=64, dtype=dtype) as fc:
            for rows in (1, 5, 30, 140):
                base = rnd(rows, rows + 1, k + 8, dtype=dtype)
                base[:, k:] = float("nan")
                base[rows:] = float("inf")
                quant_check(fc(base[:rows, :k]), base[:rows, :k], w, None, 64)


def test_quant_fc_non_finite_inputs_stay_in_their_rows():
    k, n = 512, 256
    codes, scale, z, b, w = quant_case(5, k, n, 128, False, False)
    for dtype in TYPES:
        with bc.QuantFC(k, n, codes=codes, scale=scale, group_size=128, dtype=dtype) as fc:
            for rows in (2, 40, 130):
                x = rnd(rows, rows, k, dtype=dtype)
                clean = fc(x).clone()
                x[1, 77] = float("nan")
                y = fc(x)
                keep = torch.arange(rows, device="cuda") != 1
                assert torch.equal(y[keep], clean[keep]) and y[1].isnan().all()


def test_quant_fc_large_and_small_values():
    k, n = 256, 128
    codes, scale, z, b, w = quant_case(6, k, n, 64, True, False)
    for dtype, s in ((torch.float32, 1e30), (torch.float32, 1e-30), (torch.bfloat16, 2.0 ** 100),
                     (torch.bfloat16, 2.0 ** -100), (torch.float16, 2.0 ** 5), (torch.float16, 2.0 ** -14)):
        for rows in (3, 50, 200):
            x = rnd(rows, rows, k, dtype=torch.float32, scale=s).to(dtype)
            with bc.QuantFC(k, n, codes=codes, scale=scale, zero=z, group_size=64, dtype=dtype,
                            out_dtype=torch.float32) as fc:
                quant_check(fc(x), x, w, None, 64)


def test_quant_fc_no_rows_and_refusals():
    codes, scale, z, b, w = quant_case(1, 64, 8, 32, False, False)
    fc = bc.QuantFC(64, 8, codes=codes, scale=scale, group_size=32)
    assert fc(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")).shape == (0, 8)
    assert (fc.input_feature_channels, fc.output_feature_channels) == (64, 8)
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(2, 8, dtype=torch.bfloat16, device="cuda")
    for bad, to, err in ((x.cpu(), out, TypeError), (x.float(), out, TypeError), (x[:, :32], out, ValueError),
                         (x, out.float(), TypeError), (x, out[:1], ValueError), (x, out.t().contiguous().t(), ValueError)):
        with pytest.raises(err):
            fc.forward_into(bad, to)
    h = fc.handle
    args = dict(in_ptr=x.data_ptr(), in_stride=64, rows=2, out_ptr=out.data_ptr(), out_stride=8)
    for kw in (dict(rows=-1), dict(rows=(1 << 24) + 1), dict(in_stride=63), dict(out_stride=7), dict(in_ptr=None),
               dict(out_ptr=None), dict(in_ptr=x.data_ptr() + 1), dict(workspace_ptr=x.data_ptr() + 16)):
        with pytest.raises(bc.BconvError):
            bc.bfc_quant_forward(h, **{**args, **kw})
    assert bc.bfc_quant_workspace_bytes(h, x.data_ptr(), 64, -1) == -1
    fc.close()
    with pytest.raises(ValueError):
        fc(x)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 24, 200])
def test_quant_fc_streams_and_graphs(rows, dtype):
    """One layer on two streams at once, and replayed from two graphs, on inputs that change."""
    k, n = 1000, 700  # (an odd width: rows are staged)
    codes, scale, z, b, w = quant_case(rows, k, n, 128, True, True)
    fc = bc.QuantFC(k, n, codes=codes, scale=scale, zero=z, bias=b, group_size=128, dtype=dtype)
    xs = [rnd(i, rows, k, dtype=dtype) for i in range(4)]
    want = [fc(x).clone() for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, fc(xs[i])))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i, y in got)
    graphs, ins, outs = [], [x.clone() for x in xs[:2]], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fc(ins[i]))
        graphs.append(g)
    for i in range(2):
        ins[i].copy_(xs[2 + i])
    torch.cuda.synchronize()
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                graphs[i].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(outs[i], want[2 + i]) for i in range(2))
    fc.sync_status()
    del graphs


@pytest.mark.parametrize("rows", [1, 7, 50, 300])
def test_quant_fc_layers_one_after_another(rows):
    """Layers that read what the layer before wrote, without waiting: a kernel may start, and read its codes, while
    the one before it still runs, but not its rows."""
    k = 512
    cases = [quant_case(i, k, k, 128, True, False) for i in range(4)]
    layers = [bc.QuantFC(k, k, codes=c[0], scale=c[1], zero=c[2], dtype="bf16") for c in cases]
    x = rnd(rows, rows, k, dtype=torch.bfloat16)
    torch.cuda.synchronize()
    want = []
    for _ in range(5):
        y = x
        for layer in layers:
            y = layer(y)
            torch.cuda.synchronize()
        want.append(y)
    a, b = torch.empty_like(x), torch.empty_like(x)  # two buffers in turn: written again while the next layer starts
    got = []
    for _ in range(20):
        a.copy_(x)
        for i, layer in enumerate(layers):
            layer.forward_into((a, b)[i % 2], (b, a)[i % 2])
        got.append(a.clone())
    assert all(torch.equal(y, want[0]) for y in want + got)


def test_quant_fc_past_two_gigabytes_of_offsets():
    """Input and output offsets beyond 2^31 elements (rows far apart)."""
    k, n, rows = 64, 32, 3
    codes, scale, z, b, w = quant_case(9, k, n, 32, True, False)
    stride = (1 << 30) + 24
    base = torch.empty(2 * stride + k, dtype=torch.bfloat16, device="cuda")
    x = base.as_strided((rows, k), (stride, 1))
    x.copy_(rnd(1, rows, k, dtype=torch.bfloat16))
    with bc.QuantFC(k, n, codes=codes, scale=scale, zero=z, group_size=32, dtype=torch.bfloat16) as fc:
        quant_check(fc(x), x, w, None, 32)
        out = torch.empty(2 * stride + n, dtype=torch.bfloat16, device="cuda").as_strided((rows, n), (stride, 1))
        fc.forward_into(x, out)
        quant_check(out, x, w, None, 32)


# ---------------------------------------------------------------------------------- block norm


def norm_ref(residual, block, pre, post, gate, per, alpha, eps):
    """(residual_out, normed) in the inputs' (64-bit) type."""
    def rms(v, w):
        return v / ((v * v).mean(-1, keepdim=True) + eps).sqrt() * w

    out = residual
    if block is not None:
        p = block if post is None else rms(block, post)
        if gate is not None:
            p = p * gate[torch.arange(p.shape[0], device=p.device) // per]
        out = residual + alpha * p
    return out, None if pre is None else rms(out, pre)


NORM_SHAPES = [  # rows, width, rows per gate (0: no gate)
    (1, 1, 1), (1, 8, 0), (1, 4096, 1), (2, 7, 1), (3, 64, 2), (5, 100, 0), (17, 256, 5), (64, 1001, 64),
    (33, 2048, 1), (300, 512, 7), (700, 264, 1000), (150, 2056, 40), (40, 4096, 0), (900, 1024, 450), (9, 8192, 4),
    (6, 8200, 3), (4, 12345, 2), (7, 16384, 3), (3, 32768, 2), (2, 32761, 1),
    (1200, 1032, 7), (700, 1500, 350), (900, 2047, 0), (640, 4096, 100), (500, 4099, 500), (400, 8192, 3), (310, 7001, 0),
    (299, 1025, 1),
]


def norm_inputs(seed, rows, width, per, dtype, post=True):
    gates = -(-rows // per) if per else 0
    r = rnd(seed, rows, width, dtype=dtype, scale=2.0)
    b = rnd(seed + 1, rows, width, dtype=dtype)
    g = rnd(seed + 2, gates, width, dtype=dtype) if per else None
    pre = 1 + 0.2 * rnd(seed + 3, width)
    pw = 1 + 0.2 * rnd(seed + 4, width) if post else None
    return r, b, pre, pw, g


def opt64(*ts):
    return [None if t is None else t.double() for t in ts]


# a thread adds up to 32 squares, then 5 + 32 partial sums: 70 U on the mean, half of it on the root,
# and a handful of roundings behind it
ROW = 80 * U


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width,per", NORM_SHAPES)
def test_block_norm(rows, width, per, dtype):
    post, alpha, eps = (rows + width) % 3 != 0, 0.5 + (rows % 3), 1e-5
    r, b, pre, pw, g = norm_inputs(rows + width, rows, width, per, dtype, post)
    out, normed = bc.block_norm(r, b, pre_weight=pre, post_weight=pw, gate=g, rows_per_gate=per or None,
                                residual_scale=alpha, eps=eps)
    r64, b64, pre64, pw64, g64 = opt64(r, b, pre, pw, g)
    want, want_n = norm_ref(r64, b64, pre64, pw64, g64, per, alpha, eps)
    mag = r64.abs() + (want - r64).abs()
    close(out, want, ROW * mag)
    rs = 1 / ((want * want).mean(1, keepdim=True) + eps).sqrt()
    close(normed, want_n, 2 * ROW * mag * rs * pre64.abs())


@pytest.mark.parametrize("dtype", TYPES)
def test_block_norm_parts(dtype):
    """Without a block, without the next norm, without the norm behind the block, strided inputs."""
    rows, width = 37, 520
    r, b, pre, pw, g = norm_inputs(1, rows, width, 0, dtype)
    r64, b64, pre64, pw64, _ = opt64(r, b, pre, pw, None)
    same, normed = bc.block_norm(r, pre_weight=pre)
    assert same is r
    want = norm_ref(r64, None, pre64, None, None, 0, 1.0, 1e-6)[1]
    close(normed, want, 2 * ROW * want.abs())
    out, none = bc.block_norm(r, b)
    assert none is None
    close(out, r64 + b64, 2 * U * (r64.abs() + b64.abs()))
    padded = torch.full((rows, 2 * width), float("nan"), dtype=dtype, device="cuda")
    padded[:, ::2] = r
    again = bc.block_norm(padded[:, ::2], b.t().contiguous().t(), pre_weight=pre, post_weight=pw)
    first = bc.block_norm(r, b, pre_weight=pre, post_weight=pw)
    assert all(torch.equal(x, y) for x, y in zip(again, first))
    shaped = bc.block_norm(r.reshape(1, rows, width), b.reshape(1, rows, width), pre_weight=pre, post_weight=pw)
    assert all(torch.equal(x[0], y) for x, y in zip(shaped, first))
    # unaligned rows: the same values within their roundings
    odd = torch.empty(rows * width + 1, dtype=dtype, device="cuda")[1:].view(rows, width)
    odd.copy_(r)
    for x, y in zip(bc.block_norm(odd, b, pre_weight=pre, post_weight=pw), first):
        close(x, y.double(), (half_step(dtype) + 2 * ROW) * y.double().abs() + 4 * ROW)


def test_block_norm_in_place_and_zero_rows():
    from binarized_convolution_b200 import _native as nat

    rows, width = 50, 1024
    r, b, pre, pw, g = norm_inputs(2, rows, width, 25, torch.bfloat16)
    want = bc.block_norm(r, b, pre_weight=pre, post_weight=pw, gate=g, rows_per_gate=25)
    desc = nat.bconv_block_norm_desc_t(rows, 25, width, nat.DTYPE_BF16, 1.0, 1e-6)
    s = torch.cuda.current_stream().cuda_stream
    r1, b1 = r.clone(), b.clone()
    bc.bconv_block_norm_forward(desc, r1.data_ptr(), b1.data_ptr(), g.data_ptr(), pw.data_ptr(), pre.data_ptr(),
                                r1.data_ptr(), b1.data_ptr(), s)
    assert torch.equal(r1, want[0]) and torch.equal(b1, want[1])
    zero = torch.zeros(3, 64, device="cuda")
    out, normed = bc.block_norm(zero, zero, pre_weight=pre[:64], post_weight=pw[:64])
    assert (out == 0).all() and (normed == 0).all()
    for x in bc.block_norm(zero[:0], zero[:0], pre_weight=pre[:64]):
        assert x.shape == (0, 64)
    grad = bc.block_norm_backward(zero[:0], zero[:0], pre_weight=pre[:64], post_weight=pw[:64], gate=zero[:0],
                                  d_normed=zero[:0])
    assert (grad.d_pre_weight == 0).all() and (grad.d_post_weight == 0).all() and grad.d_gate.shape == (0, 64)


def norm_grad_ref(out, block, pre, post, gate, per, alpha, eps, d_out, d_normed):
    """Gradients by the formulas, in 64 bits, and the sums of magnitudes their bounds go by."""
    rows = out.shape[0]
    ones = torch.ones(out.shape[1], dtype=torch.float64, device=out.device)
    dr, mag = (d_out, d_out.abs()) if d_out is not None else (torch.zeros_like(out), torch.zeros_like(out))
    grads, mags = {}, {}
    if d_normed is not None:
        rs = ((out * out).mean(1, keepdim=True) + eps).rsqrt()
        u = d_normed * pre
        dr = dr + rs * (u - out * rs ** 2 * (u * out).mean(1, keepdim=True))
        mag = mag + rs * (u.abs() + out.abs() * rs ** 2 * (u * out).abs().mean(1, keepdim=True))
        grads["d_pre_weight"], mags["d_pre_weight"] = (d_normed * out * rs).sum(0), (d_normed * out * rs).abs().sum(0)
    elif pre is not None:
        grads["d_pre_weight"] = mags["d_pre_weight"] = torch.zeros_like(ones)
    grads["d_residual"], mags["d_residual"] = dr, mag
    if block is not None:
        at = torch.arange(rows, device=out.device) // max(per, 1)
        g = gate[at] if gate is not None else 1.0
        bs = ((block * block).mean(1, keepdim=True) + eps).rsqrt() if post is not None else 1.0
        w = post if post is not None else ones
        q, qm = alpha * g * dr, (alpha * (g if gate is None else g.abs()) * mag)
        if gate is not None:
            d = alpha * dr * block * bs * w
            m = alpha * mag * (block * bs * w).abs()
            grads["d_gate"] = torch.zeros_like(gate).index_add_(0, at, d)
            mags["d_gate"] = torch.zeros_like(gate).index_add_(0, at, m)
        if post is not None:
            grads["d_post_weight"], mags["d_post_weight"] = (q * block * bs).sum(0), (qm * (block * bs).abs()).sum(0)
            v, vm = q * w, qm * w.abs()
            grads["d_block"] = bs * (v - block * bs ** 2 * (v * block).mean(1, keepdim=True))
            mags["d_block"] = bs * (vm + block.abs() * bs ** 2 * (vm * block.abs()).mean(1, keepdim=True))
        else:
            grads["d_block"], mags["d_block"] = q, qm
    return grads, mags


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width,per", NORM_SHAPES)
def test_block_norm_backward(rows, width, per, dtype):
    seed = rows + width
    post, alpha, eps = seed % 3 != 0, 0.5 + (rows % 3), 1e-5
    out, b, pre, pw, g = norm_inputs(seed, rows, width, per, dtype, post)
    d_out = rnd(seed + 7, rows, width, dtype=dtype) if seed % 5 else None
    d_normed = rnd(seed + 8, rows, width, dtype=dtype) if seed % 4 else None
    got = bc.block_norm_backward(out, b, pre_weight=pre, post_weight=pw, gate=g, rows_per_gate=per or None,
                                 residual_scale=alpha, eps=eps, d_residual_out=d_out, d_normed=d_normed)
    grads, mags = norm_grad_ref(*opt64(out, b, pre, pw, g), per, alpha, eps, *opt64(d_out, d_normed))
    for name, want in grads.items():
        x = getattr(got, name)
        assert x.shape == want.shape, name
        # a row's value carries three row sums (and the one behind them); the sums over rows add up to
        # rows / 296 (all of a CTA's rows) + 296 / 16 + 16 terms one after another
        chain = 4 * ROW + (U * (rows / 296 + 40) if name in ("d_pre_weight", "d_post_weight", "d_gate") else 0)
        close(x, want, chain * mags[name])
    for name in ("d_post_weight", "d_gate"):
        assert (getattr(got, name) is None) == (name not in grads)
    again = bc.block_norm_backward(out, b, pre_weight=pre, post_weight=pw, gate=g, rows_per_gate=per or None,
                                   residual_scale=alpha, eps=eps, d_residual_out=d_out, d_normed=d_normed)
    assert all((x is None and y is None) or torch.equal(x, y) for x, y in zip(got, again))


def test_block_norm_backward_parts():
    rows, width = 20, 136
    out, b, pre, pw, g = norm_inputs(3, rows, width, 0, torch.float32)
    d = rnd(9, rows, width)
    got = bc.block_norm_backward(out, pre_weight=pre, d_normed=d)
    want, mags = norm_grad_ref(*opt64(out, None, pre, None, None), 0, 1.0, 1e-6, None, d.double())
    close(got.d_residual, want["d_residual"], 4 * ROW * mags["d_residual"])
    assert got.d_block is None and got.d_gate is None and got.d_post_weight is None
    got = bc.block_norm_backward(out, b, pre_weight=pre, post_weight=pw)  # no gradient comes in
    for x in got:
        assert x is None or (x == 0).all()


@pytest.mark.parametrize("per", [0, 1, 7, 100])
def test_block_norm_gradient_against_differences(per):
    rows, width, alpha, eps = 15, 72, 0.8, 1e-5
    r, b, pre, pw, g = norm_inputs(4, rows, width, per, torch.float32)
    do, dn = rnd(5, rows, width), rnd(6, rows, width)
    at64 = opt64(r, b, pre, pw, g)

    def loss(*leaves):
        o, n = norm_ref(*leaves, max(per, 1), alpha, eps)
        return (o * do.double()).sum() + (n * dn.double()).sum()

    out = norm_ref(*at64, max(per, 1), alpha, eps)[0].float()
    got = bc.block_norm_backward(out, b, pre_weight=pre, post_weight=pw, gate=g, rows_per_gate=per or None,
                                 residual_scale=alpha, eps=eps, d_residual_out=do, d_normed=dn)
    h = 1e-5
    for i, grad in enumerate((got.d_residual, got.d_block, got.d_pre_weight, got.d_post_weight, got.d_gate)):
        if grad is None:
            continue
        v = rnd(10 + i, *at64[i].shape).double()
        up, down = list(at64), list(at64)
        up[i], down[i] = at64[i] + h * v, at64[i] - h * v
        slope = (loss(*up) - loss(*down)) / (2 * h)
        # differences: h^2 of the third derivative and 1e-16 / h of the loss; the sum over the gradient: its roundings
        assert abs((grad.double() * v).sum() - slope) <= 1e-6 * (grad.double() * v).abs().sum() + 1e-6


def test_block_norm_many_rows_share_gates():
    """More gate rows than CTAs, gates that CTAs cut anywhere, and one gate over all."""
    rows, width = 2500, 64
    out, b, pre, pw, _ = norm_inputs(11, rows, width, 0, torch.float32)
    d = rnd(12, rows, width)
    for per in (1, 2, 3, 8, 9, 100, 1249, 2500, 9999):
        g = rnd(per, -(-rows // per), width)
        got = bc.block_norm_backward(out, b, pre_weight=pre, post_weight=pw, gate=g, rows_per_gate=per, d_normed=d)
        want, mags = norm_grad_ref(*opt64(out, b, pre, pw, g), per, 1.0, 1e-6, None, d.double())
        close(got.d_gate, want["d_gate"], (4 * ROW + 60 * U) * mags["d_gate"])


@pytest.mark.parametrize("width", [1024, 1027])
@pytest.mark.parametrize("dtype", TYPES)
def test_block_norm_in_place_over_many_rows(width, dtype):
    """Outputs over their inputs, as the header allows it, where rows are requested ahead of their use."""
    from binarized_convolution_b200 import _native as nat

    rows, per = 2000, 64
    r, b, pre, pw, g = norm_inputs(21, rows, width, per, dtype)
    do, dn = rnd(22, rows, width, dtype=dtype), rnd(23, rows, width, dtype=dtype)
    kw = dict(pre_weight=pre, post_weight=pw, gate=g, rows_per_gate=per)
    code = {torch.float32: nat.DTYPE_F32, torch.bfloat16: nat.DTYPE_BF16, torch.float16: nat.DTYPE_F16}[dtype]
    desc = nat.bconv_block_norm_desc_t(rows, per, width, code, 1.0, 1e-6)
    s = torch.cuda.current_stream().cuda_stream
    out, normed = bc.block_norm(r, b, **kw)
    for first, second in ((0, 1), (1, None)):  # (residual_out over residual, normed over block); residual_out over block
        r1, b1, free = r.clone(), b.clone(), torch.empty_like(r)
        to = [r1, b1][first], b1 if second == 1 else free
        bc.bconv_block_norm_forward(desc, r1.data_ptr(), b1.data_ptr(), g.data_ptr(), pw.data_ptr(), pre.data_ptr(),
                                    to[0].data_ptr(), to[1].data_ptr(), s)
        assert torch.equal(to[0], out) and torch.equal(to[1], normed)
    want = bc.block_norm_backward(out, b, d_residual_out=do, d_normed=dn, **kw)
    ws = torch.empty(bc.bconv_block_norm_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
    for swap in (False, True):
        d1, d2 = do.clone(), dn.clone()
        to = (d2, d1) if swap else (d1, d2)
        sums = [torch.empty_like(x) for x in want[2:]]
        bc.bconv_block_norm_backward(desc, out.data_ptr(), b.data_ptr(), g.data_ptr(), pw.data_ptr(), pre.data_ptr(),
                                     d1.data_ptr(), d2.data_ptr(), to[0].data_ptr(), to[1].data_ptr(),
                                     *[x.data_ptr() for x in sums], ws.data_ptr(), s)
        assert all(torch.equal(x, y) for x, y in zip((*to, *sums), want))


# enough rows for the kernels that request rows ahead: whole and odd widths, gates cut anywhere
RING_SHAPES = [(1303, 4000, 500), (1300, 4001, 0), (1302, 4003, 7), (2500, 2001, 100), (2501, 2000, 1), (610, 8191, 610),
               (620, 8192, 0), (19000, 257, 0), (13003, 400, 77), (1303, 4104, 9), (1010, 6001, 0), (1013, 6144, 400)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width,per", RING_SHAPES)
def test_block_norm_many_rows(rows, width, per, dtype):
    test_block_norm(rows, width, per, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width,per", RING_SHAPES)
def test_block_norm_backward_many_rows(rows, width, per, dtype):
    test_block_norm_backward(rows, width, per, dtype)


@pytest.mark.parametrize("width", [1024, 1027])
@pytest.mark.parametrize("dtype", TYPES)
def test_block_norm_many_rows_parts(width, dtype):
    """Without a block, without the next norm, over the inputs: the same rows as a call of fewer rows gives."""
    from binarized_convolution_b200 import _native as nat

    rows, few = 5000, 200
    r, b, pre, pw, _ = norm_inputs(41, rows, width, 0, dtype)
    r64, b64, pre64, pw64 = opt64(r, b, pre, pw)
    same, normed = bc.block_norm(r, pre_weight=pre)
    assert torch.equal(same, r)
    want = norm_ref(r64, None, pre64, None, None, 0, 1.0, 1e-6)[1]
    close(normed, want, 2 * ROW * want.abs())
    out, none = bc.block_norm(r, b, post_weight=pw)
    assert none is None
    want = norm_ref(r64, b64, None, pw64, None, 0, 1.0, 1e-6)[0]
    close(out, want, ROW * (r64.abs() + (want - r64).abs()))
    out, normed = bc.block_norm(r, b, pre_weight=pre, post_weight=pw)
    code = {torch.float32: nat.DTYPE_F32, torch.bfloat16: nat.DTYPE_BF16, torch.float16: nat.DTYPE_F16}[dtype]
    desc = nat.bconv_block_norm_desc_t(rows, 0, width, code, 1.0, 1e-6)
    s = torch.cuda.current_stream().cuda_stream
    r1, b1 = r.clone(), b.clone()
    bc.bconv_block_norm_forward(desc, r1.data_ptr(), b1.data_ptr(), 0, pw.data_ptr(), pre.data_ptr(), b1.data_ptr(),
                                r1.data_ptr(), s)
    assert torch.equal(b1, out) and torch.equal(r1, normed)
    do, dn = rnd(42, rows, width, dtype=dtype), rnd(43, rows, width, dtype=dtype)
    got = bc.block_norm_backward(out, b, pre_weight=pre, post_weight=pw, d_residual_out=do, d_normed=dn)
    grads, mags = norm_grad_ref(*opt64(out[-few:], b[-few:], pre, pw, None), 0, 1.0, 1e-6, *opt64(do[-few:], dn[-few:]))
    for name in ("d_residual", "d_block"):  # (row by row)
        close(getattr(got, name)[-few:], grads[name], 4 * ROW * mags[name])
    ws = torch.empty(bc.bconv_block_norm_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
    d1, d2 = do.clone(), dn.clone()
    bc.bconv_block_norm_backward(desc, out.data_ptr(), b.data_ptr(), 0, pw.data_ptr(), pre.data_ptr(), d1.data_ptr(),
                                 d2.data_ptr(), d2.data_ptr(), d1.data_ptr(), 0, 0, 0, ws.data_ptr(), s)
    assert torch.equal(d2, got.d_residual) and torch.equal(d1, got.d_block)


def test_block_norm_backward_asked_for_parts():
    """Any of the results may be left out, and the workspace where no sum over rows is wanted."""
    from binarized_convolution_b200 import _native as nat

    for rows, width in ((20, 136), (700, 640)):
        out, b, pre, pw, g = norm_inputs(31, rows, width, 10, torch.float32)
        do, dn = rnd(32, rows, width), rnd(33, rows, width)
        want = bc.block_norm_backward(out, b, pre_weight=pre, post_weight=pw, gate=g, rows_per_gate=10,
                                      d_residual_out=do, d_normed=dn)
        desc = nat.bconv_block_norm_desc_t(rows, 10, width, nat.DTYPE_F32, 1.0, 1e-6)
        ws = torch.empty(bc.bconv_block_norm_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
        for keep in range(5):
            only = [torch.full_like(x, 7.0) if i == keep else None for i, x in enumerate(want)]
            bc.bconv_block_norm_backward(desc, out.data_ptr(), b.data_ptr(), g.data_ptr(), pw.data_ptr(), pre.data_ptr(),
                                         do.data_ptr(), dn.data_ptr(), *[None if x is None else x.data_ptr() for x in only],
                                         ws.data_ptr() if keep >= 2 else None, torch.cuda.current_stream().cuda_stream)
            assert torch.equal(only[keep], want[keep]), keep


def test_block_norm_refusals():
    x, w = torch.zeros(4, 16, device="cuda"), torch.ones(16, device="cuda")
    with pytest.raises(TypeError):
        bc.block_norm(x, x.half(), pre_weight=w)
    with pytest.raises(TypeError):
        bc.block_norm(x, x, pre_weight=w.half())
    with pytest.raises(TypeError):
        bc.block_norm(x, x.cpu(), pre_weight=w)
    for kw in (dict(pre_weight=w[:8]), dict(gate=x[:3], rows_per_gate=2), dict(gate=x[:, :8]),
               dict(gate=x, rows_per_gate=-1)):
        with pytest.raises(ValueError):
            bc.block_norm(x, x, **kw)
    with pytest.raises(ValueError):
        bc.block_norm(x, pre_weight=w, gate=x)
    with pytest.raises(ValueError):
        bc.block_norm_backward(x, x, d_normed=x)
    wide = torch.zeros(1, 32769, device="cuda")
    with pytest.raises(bc.BconvError):
        bc.block_norm(wide, wide)


def test_block_norm_graph_and_streams():
    rows, width = 600, 2048
    r, b, pre, pw, g = norm_inputs(13, rows, width, 200, torch.bfloat16)
    do, dn = rnd(14, rows, width, dtype=torch.bfloat16), rnd(15, rows, width, dtype=torch.bfloat16)
    kw = dict(pre_weight=pre, post_weight=pw, gate=g, rows_per_gate=200, residual_scale=0.3)

    def both():
        o, n = bc.block_norm(r, b, **kw)
        return (o, n, *bc.block_norm_backward(o, b, d_residual_out=do, d_normed=dn, **kw))

    graph = torch.cuda.CUDAGraph()
    both()
    with torch.cuda.graph(graph):
        held = both()
    r.copy_(rnd(16, rows, width, dtype=torch.bfloat16))
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = both()
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(held, other))


# ---------------------------------------------------------------------------------- token log probabilities


def token_ref(logits, tokens, top, temperature):
    """Definitions in 64 bits; rows of -inf alone as documented."""
    x = logits.double() / temperature
    m = x.amax(1, keepdim=True)
    empty = m[:, 0] == float("-inf")
    shifted = torch.where(empty[:, None], 0.0, x - torch.where(empty[:, None], 0.0, m))
    total = shifted.exp().sum(1, keepdim=True)
    logp = shifted - total.log()
    p = logp.exp()
    lse = torch.where(empty, float("-inf"), (m + total.log())[:, 0])
    entropy = torch.where(empty, 0.0, -torch.special.xlogy(p, p).sum(1))
    logp = torch.where(empty[:, None] | (x == float("-inf")), float("-inf"), logp)
    got = {"lse": lse, "entropy": entropy}
    if tokens is not None:
        got["logprob"] = logp.gather(1, tokens.clamp(0, x.shape[1] - 1)[:, None])[:, 0]
        got["logprob"] = torch.where(tokens < 0, 0.0, torch.where(tokens >= x.shape[1], float("nan"), got["logprob"]))
    if top:
        order = torch.sort(logits.double(), dim=1, descending=True, stable=True).indices[:, :top]
        got["top_index"], got["top_logprob"] = order, logp.gather(1, order)
    return got


def token_check(got, logits, tokens, top, temperature):
    want = token_ref(logits, tokens, top, temperature)
    vocab = logits.shape[1]
    # a thread adds vocab / 512 terms, then 9 + 16 + 8 partial ones; exp2 is off by 2^-22 and by the roundings of its argument (up to 30, below which terms do not count)
    chain = U * (vocab / 512 + 40 + 64)
    inv = 1 / temperature

    def check(name, scale):
        x, y = getattr(got, name), want[name]
        finite = torch.isfinite(y)
        assert torch.equal(finite, torch.isfinite(x)), name
        assert torch.equal(x[~finite].nan_to_num(7), y[~finite].float().nan_to_num(7)), name
        close(x[finite], y[finite], (chain + 8 * U) * (1 + scale[finite] + y[finite].abs()))

    big = torch.where(torch.isfinite(want["lse"]), want["lse"].abs(), 0.0) * 1.0
    zero = torch.zeros_like(big)
    check("lse", big)
    check("entropy", zero + 2 * np.log(vocab + 1))  # sum p (log p): magnitudes up to lse - x, weighted by p
    if tokens is not None:
        check("logprob", zero)
    if top:
        assert torch.equal(got.top_index.long(), want["top_index"])
        check("top_logprob", zero[:, None].expand(-1, top))
    assert inv > 0


TOKEN_SHAPES = [  # rows, vocab, top
    (1, 1, 1), (1, 2, 2), (3, 7, 7), (2, 64, 64), (5, 100, 3), (1, 1000, 20), (4, 4099, 64), (300, 513, 5),
    (1, 32003, 20), (3, 65537, 20), (17, 50000, 1), (2, 200001, 40), (160, 8191, 8), (700, 1027, 0), (9, 131072, 8),
    (40, 40000, 64),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab,top", TOKEN_SHAPES)
def test_token_logprobs(rows, vocab, top, dtype):
    seed = rows + vocab
    temperature = (1.0, 0.7, 2.5)[seed % 3]
    logits = rnd(seed, rows, vocab, dtype=dtype, scale=3.0)
    g = torch.Generator("cpu").manual_seed(seed)
    tokens = torch.randint(0, vocab, (rows,), generator=g).cuda() if seed % 4 else None
    if seed % 2 and vocab > 8:  # masked entries
        logits.masked_fill_((torch.rand(rows, vocab, generator=g) < 0.3).cuda(), float("-inf"))
        logits[:, 3] = 1.0
    got = bc.token_logprobs(logits, tokens, top=top, temperature=temperature)
    assert (got.logprob is None) == (tokens is None) and (got.top_index is None) == (top == 0)
    token_check(got, logits, tokens, top, temperature)
    again = bc.token_logprobs(logits, tokens, top=top, temperature=temperature)
    assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [2, 400])
def test_token_logprobs_order_of_hard_rows(rows, dtype):
    """Rows that defeat a bound taken from their first elements, long runs of equal logits, both zeros."""
    vocab = 9000
    ramp = torch.arange(vocab, dtype=torch.float32, device="cuda") / 1000
    kinds = [ramp, ramp.flip(0), torch.zeros(vocab, device="cuda"), torch.full((vocab,), -3.0, device="cuda"),
             torch.where(torch.arange(vocab, device="cuda") % 2 == 0, 0.0, -0.0),
             torch.where(torch.arange(vocab, device="cuda") < 8000, -50.0, 4.0)]
    logits = torch.stack([kinds[i % len(kinds)] for i in range(rows * len(kinds) // 2)]).to(dtype)
    tokens = torch.arange(logits.shape[0], device="cuda") * 13 % vocab
    for top in (1, 20, 64):
        token_check(bc.token_logprobs(logits, tokens, top=top), logits, tokens, top, 1.0)


@pytest.mark.parametrize("dtype", TYPES)
def test_token_logprobs_masks_and_missing_tokens(dtype):
    vocab = 5000
    lowest = torch.finfo(dtype).min
    logits = rnd(1, 8, vocab, dtype=dtype)
    logits[0] = float("-inf")                 # nothing left
    logits[1] = float("-inf")
    logits[1, 4321] = 2.0                     # one entry left
    logits[2] = lowest                        # masked with the lowest value, all of it ...
    logits[3, 10:] = lowest                   # ... and all but ten entries
    logits[4, :4990] = lowest
    tokens = torch.tensor([5, 4321, 7, 3, 4995, -1, vocab, -(1 << 40)], device="cuda")
    logits[5, ::2] = float("-inf")
    tokens[5] = 4                             # a masked token
    for temperature in (1.0, 1.7):
        got = bc.token_logprobs(logits, tokens, top=12, temperature=temperature)
        token_check(got, logits, tokens, 12, temperature)
    assert got.lse[0] == float("-inf") and got.entropy[0] == 0 and got.logprob[0] == float("-inf")
    assert got.top_index[0].tolist() == list(range(12)) and got.logprob[5] == float("-inf")
    assert got.logprob[6].isnan() and got.logprob[7] == 0 and got.logprob[1] == 0 and got.entropy[1] == 0


@pytest.mark.parametrize("vocab", [50, 3000, 40000])
def test_token_logprobs_nan_and_infinity(vocab):
    logits = rnd(2, 4, vocab)
    logits[0, 17] = float("nan")
    logits[1, 18] = float("inf")
    logits[2, [4, 40]] = torch.tensor([float("nan"), float("inf")], device="cuda")
    got = bc.token_logprobs(logits, torch.zeros(4, dtype=torch.int64, device="cuda"), top=3)
    for x in (got.lse, got.entropy, got.logprob):
        assert x[:3].isnan().all() and torch.isfinite(x[3])
    assert got.top_logprob[:3].isnan().all()
    assert got.top_index[0, 0] == 17 and got.top_index[1, 0] == 18 and got.top_index[2, :2].tolist() == [4, 40]
    token_check(bc.token_logprobs(logits[3:], None, top=3), logits[3:], None, 3, 1.0)


@pytest.mark.parametrize("dtype", TYPES)
def test_token_logprobs_strides(dtype):
    base = rnd(3, 6, 5011, dtype=dtype)
    tokens = torch.tensor([0, 1, 2, 3, 4, 4998], device="cuda")
    for x in (base[:, :4999], base[:, 5:5004], base[:, 12:5011], base.t().contiguous().t()[:, :4999]):
        got = bc.token_logprobs(x, tokens, top=9)
        token_check(got, x, tokens, 9, 1.0)
        d = bc.token_logprobs_backward(x, tokens, got.lse, got.entropy, d_logprob=torch.ones(6, device="cuda"))
        assert d.is_contiguous() and d.shape == x.shape
    shaped = bc.token_logprobs(base.reshape(2, 3, -1), tokens.reshape(2, 3), top=2)
    assert shaped.lse.shape == (2, 3) and shaped.top_index.shape == (2, 3, 2)


def token_grad_ref(logits, tokens, g, ge, temperature):
    x = logits.double() / temperature
    logp = x - x.logsumexp(1, keepdim=True)
    p = logp.exp()
    h = -torch.special.xlogy(p, p).sum(1, keepdim=True)
    d, mag = torch.zeros_like(p), torch.zeros_like(p)
    if g is not None:
        has = (tokens >= 0).double()
        d -= p * (g.double() * has)[:, None]
        d.scatter_add_(1, tokens.clamp_min(0)[:, None], (g.double() * has)[:, None])
        mag += p * g.double().abs()[:, None]
        mag.scatter_add_(1, tokens.clamp_min(0)[:, None], (g.double() * has).abs()[:, None])
    if ge is not None:
        lp = torch.where(p > 0, logp, 0.0)
        d -= ge.double()[:, None] * p * (lp + h)
        mag += ge.double().abs()[:, None] * p * (lp.abs() + h)
    return d / temperature, mag / temperature


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab,which", [(1, 1, "both"), (3, 7, "both"), (200, 513, "logprob"), (5, 32003, "both"),
                                              (2, 65536, "entropy"), (33, 8200, "both"), (1, 200001, "both")])
def test_token_logprobs_backward(rows, vocab, which, dtype):
    temperature = (1.0, 0.7, 2.5)[(rows + vocab) % 3]
    logits = rnd(rows, rows, vocab, dtype=dtype, scale=3.0)
    gen = torch.Generator("cpu").manual_seed(rows)
    tokens = torch.randint(0, vocab, (rows,), generator=gen).cuda()
    if vocab > 100:
        keep = logits.gather(1, tokens[:, None])
        logits[:, ::3] = float("-inf")
        logits.scatter_(1, tokens[:, None], keep)
    if rows > 2:
        tokens[1] = -1
    g = rnd(rows + 1, rows) if which != "entropy" else None
    ge = rnd(rows + 2, rows) if which != "logprob" else None
    f = bc.token_logprobs(logits, tokens, temperature=temperature)
    got = bc.token_logprobs_backward(logits, tokens, f.lse, f.entropy, d_logprob=g, d_entropy=ge,
                                     temperature=temperature)
    want, mag = token_grad_ref(logits, tokens, g, ge, temperature)
    # p carries the roundings of lse and of x - lse (magnitudes up to 60 here) and exp2's; the entropy its own
    bound = U * (200 + vocab / 512) * mag + U * (vocab / 512 + 200) * want.abs()
    if ge is not None:
        p = (logits.double() / temperature).log_softmax(1).exp()
        bound = bound + p * ge.double().abs()[:, None] / temperature * U * 200 * 12
    close(got, want, bound)
    assert (got[logits == float("-inf")] == 0).all()


def test_token_logprobs_gradient_against_differences():
    rows, vocab, temperature, h = 4, 33, 0.8, 1e-5
    logits, tokens = rnd(4, rows, vocab, scale=2.0), torch.tensor([3, 0, 32, -1], device="cuda")
    g, ge = rnd(5, rows), rnd(6, rows)
    f = bc.token_logprobs(logits, tokens, temperature=temperature)
    got = bc.token_logprobs_backward(logits, tokens, f.lse, f.entropy, d_logprob=g, d_entropy=ge,
                                     temperature=temperature).double()

    def loss(x):
        r = token_ref(x, tokens, 0, temperature)
        return (r["logprob"] * g.double()).sum() + (r["entropy"] * ge.double()).sum()

    v = rnd(7, rows, vocab).double()
    slope = (loss(logits.double() + h * v) - loss(logits.double() - h * v)) / (2 * h)
    assert abs((got * v).sum() - slope) <= 1e-6 * (got * v).abs().sum() + 1e-6


def test_token_logprobs_backward_edges():
    logits = torch.full((3, 600), float("-inf"), device="cuda")
    logits[1, 5] = 1.0
    logits[2] = 0.0
    tokens = torch.tensor([4, 5, 600], device="cuda")
    f = bc.token_logprobs(logits, tokens)
    one = torch.ones(3, device="cuda")
    d = bc.token_logprobs_backward(logits, tokens, f.lse, f.entropy, d_entropy=one)
    assert (d == 0).all()
    d = bc.token_logprobs_backward(logits, tokens, f.lse, f.entropy, d_logprob=one)
    assert (d[0, :4] == 0).all() and (d[0, 5:] == 0).all() and (d[1] == 0).all() and d[2].isnan().all()
    # in place
    from binarized_convolution_b200 import _native as nat

    x = rnd(8, 40, 1003, dtype=torch.bfloat16)
    t = torch.arange(40, device="cuda")
    f = bc.token_logprobs(x, t)
    one = torch.ones(40, device="cuda")
    want = bc.token_logprobs_backward(x, t, f.lse, f.entropy, d_logprob=one, d_entropy=one)
    desc = nat.bconv_token_desc_t(40, 1003, 1003, nat.DTYPE_BF16, 0, 1.0)
    bc.bconv_token_logprobs_backward(desc, x.data_ptr(), t.data_ptr(), f.lse.data_ptr(), f.entropy.data_ptr(),
                                     one.data_ptr(), one.data_ptr(), x.data_ptr(), 1003,
                                     torch.cuda.current_stream().cuda_stream)
    assert torch.equal(x, want)
    empty = bc.token_logprobs(x[:0], t[:0], top=4)
    assert empty.lse.shape == (0,) and empty.top_index.shape == (0, 4)


def test_token_logprobs_refusals():
    x, t = torch.zeros(2, 50, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        bc.token_logprobs(x, t.int())
    with pytest.raises(TypeError):
        bc.token_logprobs(x, t.cpu())
    with pytest.raises(ValueError):
        bc.token_logprobs(x, t[:1])
    with pytest.raises(TypeError):
        bc.token_logprobs(x.double())
    for kw in (dict(top=51), dict(top=65), dict(top=-1), dict(temperature=0.0)):
        with pytest.raises(bc.BconvError):
            bc.token_logprobs(x, t, **kw)
    one = torch.ones(2, device="cuda")
    for args, kw in (((x, None, one, one), dict(d_logprob=one)), ((x, t, one, None), dict(d_entropy=one)),
                     ((x, t, None, one), dict(d_logprob=one))):
        with pytest.raises(ValueError):
            bc.token_logprobs_backward(*args, **kw)


def test_token_logprobs_graph_and_streams():
    x = rnd(9, 3, 70001, dtype=torch.bfloat16)
    t = torch.tensor([1, 2, 3], device="cuda")
    bc.token_logprobs(x, t, top=10)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = bc.token_logprobs(x, t, top=10)
        grad = bc.token_logprobs_backward(x, t, held.lse, held.entropy, d_logprob=held.lse, d_entropy=held.lse)
    x.copy_(rnd(10, 3, 70001, dtype=torch.bfloat16))
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        now = bc.token_logprobs(x, t, top=10)
        now_grad = bc.token_logprobs_backward(x, t, now.lse, now.entropy, d_logprob=now.lse, d_entropy=now.lse)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, now)) and torch.equal(grad, now_grad)


def test_token_logprobs_past_two_gigabytes_of_offsets():
    stride = (1 << 30) + 7
    base = torch.empty(2 * stride + 900, dtype=torch.bfloat16, device="cuda")
    x = base.as_strided((3, 900), (stride, 1))
    x.copy_(rnd(11, 3, 900, dtype=torch.bfloat16))
    t = torch.tensor([0, 5, 899], device="cuda")
    token_check(bc.token_logprobs(x, t, top=5), x, t, 5, 1.0)


# ---------------------------------------------------------------------------------- together


@pytest.mark.parametrize("tokens", [1, 12, 70])
def test_a_block_and_the_answer(tokens):
    """The operators as they are used: norm, a low-bit layer (binary, then 4-bit), the norm behind it with gate and
    residual, the vocabulary in 4 bits and what its logits say -- each step against its definition on the
    values that the step before really gave."""
    width, hidden, vocab = 256, 384, 1003
    rng = np.random.default_rng(tokens)
    x = rnd(1, tokens, width)
    pre, post, last = (1 + 0.1 * rnd(i, width) for i in (2, 3, 4))
    gate = rnd(5, 1, width)
    wbits = (rng.random((hidden, 1, 1, width)) < 0.5).astype(np.uint8)
    down = quant_case(6, hidden, width, 128, True, False)
    head = quant_case(7, width, vocab, 64, False, True)
    up_layer = bc.BinaryFC(tokens, 1, 1, width, hidden, wbits=wbits, op="xnor", use_beta=True, relu=True,
                           scale=np.full(hidden, 1 / 16, np.float32))
    down_layer = bc.QuantFC(hidden, width, codes=down[0], scale=down[1], zero=down[2], dtype="f32")
    head_layer = bc.QuantFC(width, vocab, codes=head[0], scale=head[1], bias=head[3], group_size=64, dtype="f32")

    _, normed = bc.block_norm(x, pre_weight=pre)
    mid = up_layer(normed.reshape(tokens, 1, 1, width)).reshape(tokens, hidden)
    sign = torch.where(normed < 0, -1.0, 1.0).double()
    s = sign @ (2.0 * torch.from_numpy(wbits.reshape(hidden, width)).double().cuda() - 1).t()
    beta = normed.double().abs().mean(1, keepdim=True)
    want = (s / 16 * beta).clamp_min(0)
    close(mid, want, 300 * U * (s / 16 * beta).abs())
    block = down_layer(mid)
    quant_check(block, mid, down[4], None, 128)
    out, normed2 = bc.block_norm(x, block, pre_weight=last, post_weight=post, gate=gate, rows_per_gate=tokens,
                                 residual_scale=0.5)
    want, want_n = norm_ref(*opt64(x, block, last, post, gate), tokens, 0.5, 1e-6)
    mag = x.double().abs() + (want - x.double()).abs()
    close(out, want, ROW * mag)
    logits = head_layer(normed2)
    quant_check(logits, normed2, head[4], head[3], 64)
    picked = logits.argmax(1)
    answer = bc.token_logprobs(logits, picked, top=8)
    token_check(answer, logits, picked, 8, 1.0)
    assert torch.equal(answer.top_logprob[:, 0], answer.logprob)
    for layer in (up_layer, down_layer, head_layer):
        layer.sync_status()
        layer.close()
