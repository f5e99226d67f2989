"""What is measured of the library's operators around a low-bit layer of a language model.

Three operators, each in the directions it is used in:

``quant_fc``        out = act(x . W^T + bias) with W[c][f] = scale[c][f / g] * (code[c][f] - zero[c][f / g]),
                    4-bit codes, one scale (and one zero code) per group of g input channels: every size of
                    call from one token to a long prompt.
``block_norm``      r' = r + a * gate * rms(b) * post_weight, n = rms(r') * pre_weight: the norm behind a block,
                    its gate and residual scale, the residual sum and the norm before the next block; and the
                    gradient of that.
``token_logprobs``  what a row of logits says: the log probability of a given token, the entropy, the
                    log-sum-exp and the top alternatives; and the gradient of log probability and entropy.

``run`` computes them with elementary torch operations in 32 bits where ``own`` is false and calls this
package where it is true; ``exact`` computes them in 64 bits.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}

# The largest calls: drawn cases stay within them.
_FC_MACS = 2000 * 8192 * 4096
_FC_WEIGHTS = 65537 * 4000
_NORM_ELEMENTS = 8192 * 4096
_LOGITS = 1024 * 131072


def _fc(name, rows, k, n, group, dtype, out, zero, bias, relu):
    return {"name": name, "op": "quant_fc", "rows": rows, "k": k, "n": n, "group": group, "dtype": dtype, "out": out,
            "zero": zero, "bias": bias, "relu": relu}


def _norm(name, backward, rows, width, per_gate, dtype, post):
    return {"name": name, "op": "block_norm", "backward": backward, "rows": rows, "width": width,
            "per_gate": per_gate, "dtype": dtype, "post": post}


def _logp(name, backward, rows, vocab, top, dtype, temperature, masked):
    return {"name": name, "op": "token_logprobs", "backward": backward, "rows": rows, "vocab": vocab, "top": top,
            "dtype": dtype, "temperature": temperature, "masked": masked}


def listed():
    return [
        # one token through a square projection: launch latency and 8 MB of weights
        _fc("fc 1 row 4096-4096 bf16", 1, 4096, 4096, 128, "bf16", "bf16", False, False, False),
        # one token through a vocabulary projection of odd size, its logits in fp32
        _fc("fc 1 row 4000-65537 f16", 1, 4000, 65537, 64, "f16", "f32", True, False, False),
        # a few images through the first fully-connected layer behind a 7 x 7 x 512 image, fp32 like the binary layers
        _fc("fc 9 rows 25088-4096 f32", 9, 25088, 4096, 128, "f32", "f32", False, True, True),
        # decoding a batch of requests
        _fc("fc 160 rows 4096-16384 bf16", 160, 4096, 16384, 128, "bf16", "bf16", True, False, False),
        # a prompt
        _fc("fc 2000 rows 4096-8192 bf16", 2000, 4096, 8192, 128, "bf16", "bf16", False, True, False),
        # between two blocks of one token
        _norm("norm 1 row 4096 bf16", False, 1, 4096, 1, "bf16", True),
        # between two blocks of 8 sequences of 1024 tokens, the gate given per sequence
        _norm("norm 8192 rows 4096 bf16", False, 8192, 4096, 1024, "bf16", True),
        # training, the same in batches of 4 sequences
        _norm("norm back 4096 rows 4096 bf16", True, 4096, 4096, 1024, "bf16", True),
        # training at an odd width in fp32, no norm behind the block
        _norm("norm back 777 rows 1001 f32", True, 777, 1001, 777, "f32", False),
        # sampling three requests: log probabilities with 20 alternatives
        _logp("logprobs 3 rows 65537 f32", False, 3, 65537, 20, "f32", 0.7, True),
        # scoring a prompt
        _logp("logprobs 1024 rows 131072 bf16", False, 1024, 131072, 8, "bf16", 1.0, False),
        # training on log probabilities with an entropy term, rows of odd length
        _logp("logprobs back 1000 rows 32003 bf16", True, 1000, 32003, 0, "bf16", 1.0, True),
    ]


def _log_uniform(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["quant_fc", "block_norm", "token_logprobs"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "quant_fc":
        while True:
            rows, k, n = _log_uniform(rng, 1, 4096), _log_uniform(rng, 33, 25088), _log_uniform(rng, 1, 65537)
            if rng.random() < 0.5:
                k, n = max(32, k // 64 * 64), max(8, n // 8 * 8)
            if rows * n * k <= _FC_MACS and 1 << 16 <= n * k <= _FC_WEIGHTS and rows * (k + n) <= 1 << 26:
                break
        c = _fc("", rows, k, n, rng.choice([32, 64, 128, 128, 256]), dtype, rng.choice([dtype, "f32"]),
                rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.3)
    elif op == "block_norm":
        while True:
            rows, width = _log_uniform(rng, 1, 16384), _log_uniform(rng, 64, 16384)
            if rng.random() < 0.5:
                width = max(64, width // 64 * 64)
            if rows * width <= _NORM_ELEMENTS // (2 if dtype == "f32" else 1):
                break
        backward = rng.random() < 0.5
        c = _norm("", backward, rows, width, rng.choice([0, rows, -(-rows // 3)]), dtype, rng.random() < 0.7)
    else:
        while True:
            rows, vocab = _log_uniform(rng, 1, 8192), _log_uniform(rng, 1000, 200000)
            if rng.random() < 0.5:
                vocab = vocab // 64 * 64 + 64
            if rows * vocab <= _LOGITS // (4 if dtype == "f32" else 2):
                break
        backward = rng.random() < 0.5
        c = _logp("", backward, rows, vocab, 0 if backward else rng.choice([0, 1, 5, 20]), dtype,
                  rng.choice([1.0, 0.7, 1.3]), rng.random() < 0.5)
    del c["name"]
    return c


# ---- inputs ----


def _prepare_fc(c, g):
    rows, k, n = c["rows"], c["k"], c["n"]
    groups = -(-k // c["group"])
    kb = (k + 1) // 2
    code = (torch.randn(n, 2 * kb, generator=g, device="cuda", dtype=torch.float16) * 2.6).round_().clamp_(-8, 7) + 8
    code = code.to(torch.uint8)
    if k % 2:
        code[:, k:] = 0
    s = {"packed": code[:, 0::2] | (code[:, 1::2] << 4)}
    del code
    s["scale"] = 0.02 / 2.6 * (0.5 + torch.rand(n, groups, generator=g, device="cuda"))
    s["zero"] = torch.randint(6, 11, (n, groups), generator=g, device="cuda", dtype=torch.uint8) if c["zero"] else None
    s["bias"] = torch.randn(n, generator=g, device="cuda") if c["bias"] else None
    s["x"] = torch.randn(rows, k, generator=g, device="cuda").to(_TYPES[c["dtype"]])
    if own:
        import binarized_convolution_b200 as bc

        s["layer"] = bc.QuantFC(k, n, packed=s["packed"], scale=s["scale"], zero=s["zero"], bias=s["bias"],
                                group_size=c["group"], relu=c["relu"], dtype=c["dtype"], out_dtype=c["out"])
    return s


def _prepare_norm(c, g):
    rows, width, t = c["rows"], c["width"], _TYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"residual": (2 * normal(rows, width)).to(t), "block": normal(rows, width).to(t),
         "pre_weight": 1 + 0.1 * normal(width), "post_weight": 1 + 0.1 * normal(width) if c["post"] else None,
         "gate": (0.5 + 0.2 * normal(-(-rows // c["per_gate"]), width)).to(t) if c["per_gate"] else None}
    if c["backward"]:
        s["d_residual_out"], s["d_normed"] = normal(rows, width).to(t), normal(rows, width).to(t)
    return s


def _prepare_logp(c, g):
    rows, vocab = c["rows"], c["vocab"]
    x = (3 * torch.randn(rows, vocab, generator=g, device="cuda")).to(_TYPES[c["dtype"]])
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    if c["masked"]:  # a part of the vocabulary is not allowed; the row's own token always is
        banned = torch.rand(vocab, generator=g, device="cuda") < 0.25
        own_logits = x.gather(1, tokens[:, None])
        x.masked_fill_(banned[None, :], float("-inf"))
        x.scatter_(1, tokens[:, None], own_logits)
    s = {"logits": x, "tokens": tokens}
    if c["backward"]:
        s["lse"], s["entropy"] = _lse_entropy(x, c["temperature"])
        s["d_logprob"] = torch.randn(rows, generator=g, device="cuda")
        s["d_entropy"] = 0.1 * torch.randn(rows, generator=g, device="cuda")
    return s


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    make = {"quant_fc": _prepare_fc, "block_norm": _prepare_norm, "token_logprobs": _prepare_logp}[case["op"]]
    return {**make(case, g), "case": case}


# ---- the plain forms ----


def _plain_fc(s, c):
    k = c["k"]
    code = torch.stack((s["packed"] & 15, s["packed"] >> 4), dim=-1).reshape(c["n"], -1)[:, :k].float()
    scale = s["scale"].repeat_interleave(c["group"], dim=1)[:, :k]
    zero = 8.0 if s["zero"] is None else s["zero"].float().repeat_interleave(c["group"], dim=1)[:, :k]
    y = s["x"].float() @ ((code - zero) * scale).t()
    if s["bias"] is not None:
        y = y + s["bias"]
    if c["relu"]:
        y = y.clamp_min(0)
    return y.to(_TYPES[c["out"]])


_EPS, _ALPHA = 1e-6, 0.7


def _gate_rows(s, c):
    if s["gate"] is None:
        return 1.0
    return s["gate"].float().repeat_interleave(c["per_gate"], dim=0)[: c["rows"]]


def _plain_norm(s, c):
    b = s["block"].float()
    if s["post_weight"] is not None:
        b = b * torch.rsqrt((b * b).mean(1, keepdim=True) + _EPS) * s["post_weight"]
    r = s["residual"].float() + _ALPHA * _gate_rows(s, c) * b
    n = r * torch.rsqrt((r * r).mean(1, keepdim=True) + _EPS) * s["pre_weight"]
    return r.to(s["residual"].dtype), n.to(s["residual"].dtype)


def _plain_norm_back(s, c):
    t, r, b = s["residual"].dtype, s["residual"].float(), s["block"].float()
    dn = s["d_normed"].float()
    rstd = torch.rsqrt((r * r).mean(1, keepdim=True) + _EPS)
    dw = dn * s["pre_weight"]
    dr = s["d_residual_out"].float() + rstd * (dw - r * rstd * rstd * (dw * r).mean(1, keepdim=True))
    out = {"d_residual": dr.to(t), "d_pre_weight": (dn * r * rstd).sum(0)}
    gate, p = _gate_rows(s, c), b
    dp = _ALPHA * gate * dr
    if s["post_weight"] is not None:
        bstd = torch.rsqrt((b * b).mean(1, keepdim=True) + _EPS)
        p = b * bstd * s["post_weight"]
        dv = dp * s["post_weight"]
        out["d_post_weight"] = (dp * b * bstd).sum(0)
        out["d_block"] = (bstd * (dv - b * bstd * bstd * (dv * b).mean(1, keepdim=True))).to(t)
    else:
        out["d_block"] = dp.to(t)
    if s["gate"] is not None:
        dg, per, rows = _ALPHA * dr * p, c["per_gate"], c["rows"]
        pad = torch.zeros(-rows % per, c["width"], device=dg.device)
        out["d_gate"] = torch.cat((dg, pad)).reshape(-1, per, c["width"]).sum(1)
    return out


def _lse_entropy(logits, temperature):
    x = logits.float() * (1.0 / temperature)
    top = x.amax(1, keepdim=True)
    e = (x - top).exp()
    total = e.sum(1, keepdim=True)
    shifted = torch.where(e > 0, x - top, 0.0)
    entropy = total.log() - (e * shifted).sum(1, keepdim=True) / total
    return (top + total.log())[:, 0], entropy[:, 0]


def _plain_logp(s, c):
    lse, entropy = _lse_entropy(s["logits"], c["temperature"])
    x = s["logits"].float()
    inv = 1.0 / c["temperature"]
    out = {"logprob": x.gather(1, s["tokens"][:, None])[:, 0] * inv - lse, "entropy": entropy, "lse": lse}
    if c["top"]:
        value, index = x.sort(dim=1, descending=True, stable=True)
        out["top_logprob"] = value[:, : c["top"]] * inv - lse[:, None]
        out["top_index"] = index[:, : c["top"]].int()
    return out


def _plain_logp_back(s, c):
    inv = 1.0 / c["temperature"]
    logp = s["logits"].float() * inv - s["lse"][:, None]
    p = logp.exp()
    d = -p * s["d_logprob"][:, None]
    d = d - s["d_entropy"][:, None] * p * torch.where(p > 0, logp + s["entropy"][:, None], 0.0)
    d.scatter_add_(1, s["tokens"][:, None], s["d_logprob"][:, None])
    return (d * inv).to(s["logits"].dtype)


# ---- the library's calls ----


def _own_norm(s, c):
    import binarized_convolution_b200 as bc

    return bc.block_norm(s["residual"], s["block"], pre_weight=s["pre_weight"], post_weight=s["post_weight"],
                         gate=s["gate"], rows_per_gate=c["per_gate"] or None, residual_scale=_ALPHA, eps=_EPS)


def _own_norm_back(s, c):
    import binarized_convolution_b200 as bc

    g = bc.block_norm_backward(s["residual"], s["block"], pre_weight=s["pre_weight"], post_weight=s["post_weight"],
                               gate=s["gate"], rows_per_gate=c["per_gate"] or None, residual_scale=_ALPHA, eps=_EPS,
                               d_residual_out=s["d_residual_out"], d_normed=s["d_normed"])
    return {name: value for name, value in g._asdict().items() if value is not None}


def _own_logp(s, c):
    import binarized_convolution_b200 as bc

    r = bc.token_logprobs(s["logits"], s["tokens"], top=c["top"], temperature=c["temperature"])
    return {name: value for name, value in r._asdict().items() if value is not None}


def _own_logp_back(s, c):
    import binarized_convolution_b200 as bc

    return bc.token_logprobs_backward(s["logits"], s["tokens"], s["lse"], s["entropy"], d_logprob=s["d_logprob"],
                                      d_entropy=s["d_entropy"], temperature=c["temperature"])


def run(state):
    c = state["case"]
    if c["op"] == "quant_fc":
        return state["layer"](state["x"]) if own else _plain_fc(state, c)
    if c["op"] == "block_norm":
        if c["backward"]:
            return _own_norm_back(state, c) if own else _plain_norm_back(state, c)
        return _own_norm(state, c) if own else _plain_norm(state, c)
    if c["backward"]:
        return _own_logp_back(state, c) if own else _plain_logp_back(state, c)
    return _own_logp(state, c) if own else _plain_logp(state, c)


# ---- work and 64-bit results ----


def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "f16": 2}
    e = size[c["dtype"]]
    if c["op"] == "quant_fc":
        rows, k, n = c["rows"], c["k"], c["n"]
        groups = -(-k // c["group"])
        weights = n * ((k + 1) // 2) + n * groups * (5 if c["zero"] else 4) + (4 * n if c["bias"] else 0)
        return {"bytes": weights + rows * (k * e + n * size[c["out"]]), "flops": 2.0 * rows * k * n}
    rows = c["rows"]
    if c["op"] == "block_norm":
        width = c["width"]
        gates = -(-rows // c["per_gate"]) if c["per_gate"] else 0
        terms = 4 * width * (2 if c["post"] else 1)
        if c["backward"]:
            return {"bytes": rows * width * 6 * e + gates * width * (e + 4) + 2 * terms, "flops": 30.0 * rows * width}
        return {"bytes": rows * width * 4 * e + gates * width * e + terms, "flops": 11.0 * rows * width}
    vocab = c["vocab"]
    if c["backward"]:
        return {"bytes": rows * vocab * 2 * e + rows * 24, "flops": 10.0 * rows * vocab}
    return {"bytes": rows * vocab * e + rows * (8 + 12 + 8 * c["top"]), "flops": 6.0 * rows * vocab}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    rows = c["rows"]
    if c["op"] == "quant_fc":
        k, n = c["k"], c["n"]
        column = torch.arange(k, device="cuda")
        out = torch.empty(rows, n, dtype=torch.float64, device="cuda")
        x = s["x"].double()
        for first in range(0, n, 8192):  # a part of the output channels at a time
            part = slice(first, min(first + 8192, n))
            w = ((s["packed"][part][:, column // 2] >> (4 * (column % 2)).to(torch.uint8)) & 15).double()
            w -= 8 if s["zero"] is None else s["zero"][part].double()[:, column // c["group"]]
            w *= s["scale"][part].double()[:, column // c["group"]]
            out[:, part] = torch.einsum("rk,nk->rn", x, w)
        if s["bias"] is not None:
            out += s["bias"].double()
        return torch.where(out > 0, out, torch.zeros_like(out)) if c["relu"] else out
    if c["op"] == "block_norm":
        gate = None
        if s["gate"] is not None:
            gate = s["gate"].double().detach().requires_grad_()
        pre = s["pre_weight"].double().requires_grad_()
        post = s["post_weight"].double().requires_grad_() if s["post_weight"] is not None else None
        block = s["block"].double().requires_grad_()
        branch = block
        if post is not None:
            branch = branch / ((branch ** 2).sum(1, keepdim=True) / c["width"] + _EPS).sqrt() * post
        if gate is not None:
            branch = branch * gate[torch.arange(rows, device="cuda") // c["per_gate"]]
        if not c["backward"]:
            out = s["residual"].double() + _ALPHA * branch
            norm = (out ** 2).sum(1, keepdim=True) / c["width"] + _EPS
            return out.detach(), (out / norm.sqrt() * pre).detach()
        # the given "residual" is the sum that the forward stored: differentiate there
        start = s["residual"].double() - _ALPHA * branch.detach()
        start.requires_grad_()
        out = start + _ALPHA * branch
        normed = out / ((out ** 2).sum(1, keepdim=True) / c["width"] + _EPS).sqrt() * pre
        leaves = {"d_residual": start, "d_block": block, "d_pre_weight": pre, "d_post_weight": post, "d_gate": gate}
        leaves = {name: v for name, v in leaves.items() if v is not None}
        grads = torch.autograd.grad((out, normed), list(leaves.values()),
                                    (s["d_residual_out"].double(), s["d_normed"].double()))
        return dict(zip(leaves, grads))
    x = s["logits"].double() / c["temperature"]
    lse = x.logsumexp(1)
    token = x.gather(1, s["tokens"][:, None])[:, 0]
    logp = x.sub_(lse[:, None])
    p = logp.exp()
    entropy = -torch.special.xlogy(p, p).sum(1)
    if c["backward"]:
        d = (logp.masked_fill_(p == 0, 0.0) + entropy[:, None]).mul_(s["d_entropy"].double()[:, None])
        d = d.add_(s["d_logprob"].double()[:, None]).mul_(p).neg_()
        at = torch.arange(rows, device="cuda")
        d[at, s["tokens"]] += s["d_logprob"].double()
        return d.div_(c["temperature"])
    out = {"logprob": token - lse, "entropy": entropy, "lse": lse}
    if c["top"]:
        out["top_logprob"] = torch.topk(logp, c["top"], dim=1).values
        out["top_index"] = None
    return out
