"""The cases that the norm operators and the 8-bit product are measured on.

Three operators, all on channels-last rows:

* ``group_norm``: group norm per frame with an optional SiLU, written as bf16 or as e4m3 with one fp32 scale per
  row and block of 128 channels;
* ``rms_norm``: RMS norm over the channels of each position with an optional SiLU, the same two outputs;
* ``gemm``: the product of e4m3 rows and e4m3 weights, one scale per row (activations) or per 128 rows (weights)
  and block of 128 channels, plus bias and residual; ``quantize`` makes its left operand from bf16 rows.

``own`` selects the library's kernels; otherwise the same results come from elementary torch operations in fp32.
"""

import math

import torch

own = False

BLOCK = 128          # channels that share a scale
E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -126
EPS = 1e-6


# ------------------------------------------------------------------------------------------------------- cases --

def listed():
    return [
        # the toy plane, two frames: a few microseconds, what a call costs
        _gn("gn_toy", 2, 96, 64, 32, "silu", "bf16"),
        # the norm in front of the mid block's attention: four latent frames, e4m3 for the projections
        _gn("gn_mid_fp8", 4, 3432, 1024, 32, "none", "fp8"),
        # odd plane, groups of 15 channels: nothing divides evenly
        _gn("gn_odd", 3, 3555, 480, 32, "silu", "bf16"),
        # in front of the output head: sixteen full frames, each larger than half of L2
        _gn("gn_head", 16, 219648, 256, 32, "silu", "bf16"),
        # the residual blocks' norm at the last resampler's output
        _rms("rms_res", 439296, 512, "silu", "bf16"),
        # a few rows: the latency of the fused norm and quantisation
        _rms("rms_few_fp8", 17, 2048, "none", "fp8"),
        # the attention's output on its way into the output projection
        _quant("quant_attn", 13728, 1024),
        # few, short rows that end inside a block
        _quant("quant_few", 5, 1000),
        # a single row through a square projection: the weights' bytes
        _gemm("gemm_one_row", 1, 4096, 4096, True, False),
        # the attention's output projection with the residual, four latent frames
        _gemm("gemm_proj", 13728, 1024, 1024, True, True),
        # a channel-halving 1x1x1 shortcut over eight frames: bound by its rows' bytes
        _gemm("gemm_shortcut", 439296, 256, 512, True, False),
        # a large square product: bound by the tensor cores
        _gemm("gemm_large", 16384, 4096, 4096, False, False),
    ]


def _gn(name, n, p, c, groups, act, out):
    return {"name": name, "op": "group_norm", "n": n, "p": p, "c": c, "groups": groups, "act": act, "out": out}


def _rms(name, rows, c, act, out):
    return {"name": name, "op": "rms_norm", "rows": rows, "c": c, "act": act, "out": out}


def _quant(name, rows, c):
    return {"name": name, "op": "quantize", "rows": rows, "c": c}


def _gemm(name, m, n, k, bias, residual):
    return {"name": name, "op": "gemm", "m": m, "n": n, "k": k, "bias": bias, "residual": residual}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["group_norm", "group_norm", "rms_norm", "quantize", "gemm", "gemm"])
    most = 16 * 219648 * 256
    if op == "group_norm":
        while True:
            groups = rng.choice([1, 2, 4, 8, 16, 32])
            c = 8 * _log(rng, 8, 128)
            if c % groups:
                continue
            n, p = _log(rng, 1, 16), _log(rng, 1, 352) * _log(rng, 1, 624)
            if n * p * c <= most:
                break
        return _unnamed(_gn("", n, p, c, groups, rng.choice(["none", "silu"]), rng.choice(["bf16", "fp8"])))
    if op == "rms_norm":
        rows, c = _log(rng, 1, 439296), 8 * _log(rng, 8, 512)
        rows = max(1, min(rows, most // c))
        return _unnamed(_rms("", rows, c, rng.choice(["none", "silu"]), rng.choice(["bf16", "fp8"])))
    if op == "quantize":
        rows, c = _log(rng, 1, 439296), 8 * _log(rng, 8, 512)
        return _unnamed(_quant("", max(1, min(rows, most // c)), c))
    m, n, k = _log(rng, 1, 439296), 8 * _log(rng, 8, 512), 16 * _log(rng, 4, 256)
    m = max(1, min(m, 16384 * 4096 * 4096 // (n * k), 439296 * 768 // (n + k)))
    return _unnamed(_gemm("", m, n, k, rng.random() < 0.5, rng.random() < 0.5))


def _unnamed(case):
    del case["name"]
    return case


# ------------------------------------------------------------------------------------------------------ inputs --

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    bf16 = torch.bfloat16

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def empty(*shape, dtype=bf16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    state = {"case": dict(case)}
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        rows = normal(m, k)
        state["a"], state["sa"] = _quantize_rows(rows)
        del rows
        state["w"], state["sw"] = _quantize_weights(normal(n, k) / math.sqrt(k))
        state["bias"] = (0.1 * normal(n)).to(bf16) if case["bias"] else None
        state["res"] = normal(m, n).to(bf16) if case["residual"] else None
        state["y"] = empty(m, n)
        return state
    rows = case["n"] * case["p"] if case["op"] == "group_norm" else case["rows"]
    c = case["c"]
    # activations with a scale and an offset of each channel's own
    state["x"] = (normal(rows, c) * (0.5 + normal(c).abs()) + 0.5 * normal(c)).to(bf16)
    if case["op"] != "quantize":
        state["gamma"] = (1 + 0.2 * normal(c)).to(bf16)
    if case["op"] == "group_norm":
        state["x"] = state["x"].view(case["n"], case["p"], c)
        state["beta"] = (0.2 * normal(c)).to(bf16)
    if case.get("out", "fp8") == "fp8":
        state["y"] = empty(*state["x"].shape, dtype=torch.float8_e4m3fn)
        state["sy"] = empty(*state["x"].shape[:-1], -(-c // BLOCK), dtype=torch.float32)
    else:
        state["y"] = empty(*state["x"].shape)
    return state


# -------------------------------------------------------------------------------------------------- plain forms --

def _blocks(v):
    """v [..., C] as [..., ceil(C / 128), 128], the last block filled up with zeros."""
    c = v.shape[-1]
    nb = -(-c // BLOCK)
    if nb * BLOCK != c:
        v = torch.cat([v, v.new_zeros(*v.shape[:-1], nb * BLOCK - c)], -1)
    return v.view(*v.shape[:-1], nb, BLOCK)


def _quantize_rows(v):
    """(e4m3 values, fp32 scales) of fp32 rows: scale = max |v| of the block / 448."""
    blocks = _blocks(v)
    scale = (blocks.abs().amax(-1) / E4M3_MAX).clamp(min=MIN_SCALE)
    q = (blocks / scale[..., None]).flatten(-2)[..., :v.shape[-1]].to(torch.float8_e4m3fn)
    return q.contiguous(), scale


def _quantize_weights(w):
    """The same with one scale for each 128 x 128 block of w [N, K]."""
    n, k = w.shape
    nb = -(-n // BLOCK)
    blocks = _blocks(torch.cat([w, w.new_zeros(nb * BLOCK - n, k)])).view(nb, BLOCK, -1, BLOCK)
    scale = (blocks.abs().amax((1, 3)) / E4M3_MAX).clamp(min=MIN_SCALE)
    q = (blocks / scale[:, None, :, None]).reshape(nb * BLOCK, -1)[:n, :k].to(torch.float8_e4m3fn)
    return q.contiguous(), scale


def _silu(v, act):
    return v / (1 + torch.exp(-v)) if act == "silu" else v


def _plain(s):
    case = s["case"]
    if case["op"] == "gemm":
        k, n = case["k"], case["n"]
        a = s["a"].float() * s["sa"].repeat_interleave(BLOCK, 1)[:, :k]
        w = s["w"].float() * s["sw"].repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
        y = a @ w.T
        if s["bias"] is not None:
            y += s["bias"].float()
        if s["res"] is not None:
            y += s["res"].float()
        return y.to(torch.bfloat16)
    x = s["x"].float()
    if case["op"] == "quantize":
        return _quantize_rows(x)
    gamma = s["gamma"].float()
    if case["op"] == "group_norm":
        n, p, c = x.shape
        g = x.view(n, p, case["groups"], -1)
        mean = g.mean((1, 3), keepdim=True)
        var = (g - mean).square().mean((1, 3), keepdim=True)
        y = ((g - mean) / torch.sqrt(var + EPS)).view(n, p, c) * gamma + s["beta"].float()
    else:
        y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma
    y = _silu(y, case["act"])
    return _quantize_rows(y) if case["out"] == "fp8" else y.to(torch.bfloat16)


def run(state):
    if not own:
        return _plain(state)
    from causal_convolution_gb300 import api
    s, case = state, state["case"]
    if case["op"] == "gemm":
        api.cc_gemm_fp8(s["a"], s["sa"], s["w"], s["sw"], s["bias"], s["res"], s["y"])
        return s["y"]
    if case["op"] == "quantize":
        api.cc_fp8_quantize(s["x"], s["y"], s["sy"])
        return s["y"], s["sy"]
    if case["op"] == "rms_norm":
        if case["out"] == "fp8":
            api.cc_rms_norm_act_fp8(s["x"], s["gamma"], s["y"], s["sy"], eps=EPS, act=case["act"])
            return s["y"], s["sy"]
        api.cc_rms_norm_act(s["x"], s["gamma"], s["y"], eps=EPS, act=case["act"])
        return s["y"]
    if "ws" not in s:  # a caller keeps its workspace, like its outputs
        need = api.cc_group_norm_workspace_bytes(case["n"], case["p"], case["c"], case["groups"])
        s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    if case["out"] == "fp8":
        api.cc_group_norm_act_fp8(s["x"], s["gamma"], s["beta"], s["y"], s["sy"], case["groups"], s["ws"], eps=EPS,
                                  act=case["act"])
        return s["y"], s["sy"]
    api.cc_group_norm_act(s["x"], s["gamma"], s["beta"], s["y"], case["groups"], s["ws"], eps=EPS, act=case["act"])
    return s["y"]


# -------------------------------------------------------------------------------------------------- floors, 64 bits --

def work(case):
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // BLOCK)
        nbytes = m * k + 4 * m * kb + n * k + 4 * -(-n // BLOCK) * kb + 2 * m * n
        return {"bytes": nbytes + 2 * n * case["bias"] + 2 * m * n * case["residual"], "flops": 2 * m * n * k}
    rows = case["n"] * case["p"] if case["op"] == "group_norm" else case["rows"]
    c = case["c"]
    out = rows * (c + 4 * -(-c // BLOCK)) if case.get("out", "fp8") == "fp8" else 2 * rows * c
    params = {"group_norm": 4 * c, "rms_norm": 2 * c, "quantize": 0}[case["op"]]
    flops = {"group_norm": 8, "rms_norm": 6, "quantize": 3}[case["op"]] * rows * c
    return {"bytes": 2 * rows * c + out + params, "flops": flops}


def exact(case, seed):
    """The definitions in 64 bits; where the output is e4m3, the values before they are rounded to it. The large
    group norm goes frame by frame, so that its 64-bit values fit beside the result."""
    s = prepare(case, seed)
    if case["op"] == "gemm":
        out = torch.zeros(case["m"], case["n"], dtype=torch.float64, device="cuda")
        for b in range(s["sa"].shape[1]):
            part = slice(b * 128, min((b + 1) * 128, case["k"]))
            row_scale = s["sa"][:, b, None].double()
            col_scale = torch.stack([s["sw"][j // 128, b] for j in range(0, case["n"], 128)]).double()
            col_scale = col_scale[torch.arange(case["n"], device="cuda") // 128]
            out.addcmul_(s["a"][:, part].double() @ s["w"][:, part].double().t(), row_scale * col_scale)
        for extra in (s["bias"], s["res"]):
            if extra is not None:
                out += extra.double()
        return out
    if case["op"] == "group_norm":
        frames = [_exact_frame(s["x"][i], s, case) for i in range(case["n"])]
        if case["out"] == "fp8":
            return torch.stack([f[0] for f in frames]), torch.stack([f[1] for f in frames])
        return torch.stack(frames)
    x = s["x"].double()
    if case["op"] == "rms_norm":
        norm = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
        x = x * s["gamma"].double() / (norm * norm / case["c"] + EPS).sqrt()
        x = x * torch.special.expit(x) if case["act"] == "silu" else x
    return _exact_blocks(x) if case.get("out", "fp8") == "fp8" else x


def _exact_frame(x, s, case):
    p, c = x.shape
    per = c // case["groups"]
    parts = x.double().reshape(p, case["groups"], per)
    var, mean = torch.var_mean(parts, dim=(0, 2), correction=0)
    y = (parts - mean[:, None]) * (var + EPS).rsqrt()[:, None]
    y = torch.addcmul(s["beta"].double(), y.reshape(p, c), s["gamma"].double())
    y = y * torch.special.expit(y) if case["act"] == "silu" else y
    return _exact_blocks(y) if case["out"] == "fp8" else y


def _exact_blocks(v):
    tops, values = [], []
    for lo in range(0, v.shape[-1], 128):
        part = v[..., lo:lo + 128]
        top = torch.maximum(part.max(-1).values, -part.min(-1).values).div(448).clamp_min(2.0 ** -126)
        tops.append(top)
        values.append(part / top[..., None])
    return torch.cat(values, -1), torch.stack(tops, -1)
