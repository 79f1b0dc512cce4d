"""The cases that the operators around a paged cache of keys and values are measured on.

Four operators, all on rows of heads of channels (bf16):

* ``rope``: RMS norm of every query and key head and the rotation of its channel pairs by its position, in one pass;
* ``append``: the same for the new tokens of several sequences, whose keys and values go into a paged cache;
* ``paged``: attention of the sequences' new tokens over that cache, causal by blocks of tokens (a frame, or one);
* ``cross``: attention to an encoder's states, whose number differs from the queries' and from instance to instance.

``own`` selects the library's kernels; otherwise the same results come from elementary torch operations in fp32.
"""

import math

import torch

own = False

EPS = 1e-6
FRAME = 3432         # positions of a latent frame, 44 x 78
MAX_SCORES = 1 << 28  # scores that the plain form holds at a time


# ------------------------------------------------------------------------------------------------------- cases --

def listed():
    return [
        # one new token of two streams, small heads: what a call costs
        _rope("rope_few", 2, 8, 8, 64, 64, "halves"),
        # four latent frames out of a packed projection
        _rope("rope_chunk", 4 * FRAME, 16, 16, 128, 128, "pairs"),
        # single tokens of 48 streams with shared key heads
        _append("append_step", 48, 1, 1, 20000, 32, 8, 128, 128, 64, "halves"),
        # new chunks of odd lengths, a part of the channels rotated, pages that end anywhere
        _append("append_odd", 3, 77, 4001, 9000, 10, 10, 96, 64, 48, "pairs"),
        # a single token over a short cache: latency
        _paged("paged_one", 1, 1, 1, 2000, 2000, 8, 8, 64, 16, 1),
        # single tokens of 64 streams of very different lengths: the cache's bytes
        _paged("paged_many", 64, 1, 1, 100, 8192, 32, 8, 128, 64, 1),
        # a single token of one long stream with few key heads: the cache split over the SMs
        _paged("paged_long", 1, 1, 1, 131072, 131072, 16, 2, 128, 128, 1),
        # chunks of odd lengths behind caches of odd lengths, seven query heads to a key head, odd head size
        _paged("paged_odd", 5, 1, 700, 1, 5000, 14, 2, 80, 48, 1),
        # four new latent frames that see themselves and the frames before them, four of which are cached
        _paged("paged_chunk", 1, 4 * FRAME, 4 * FRAME, 8 * FRAME, 8 * FRAME, 16, 16, 128, 128, FRAME),
        # four latent frames' positions and a text of full length
        _cross("cross_text", 1, 4 * FRAME, 512, 16, 16, 128, False),
        # texts of different lengths (one may be empty), odd sizes
        _cross("cross_ragged", 5, 1111, 77, 10, 10, 64, True),
        # one new token of 32 streams
        _cross("cross_step", 32, 1, 512, 32, 8, 128, True),
    ]


def _rope(name, rows, heads, kv_heads, d, rd, style):
    return {"name": name, "op": "rope", "rows": rows, "heads": heads, "kv_heads": kv_heads, "d": d, "rd": rd,
            "style": style}


def _append(name, seqs, new_lo, new_hi, kv_hi, heads, kv_heads, d, rd, page, style):
    return {"name": name, "op": "append", "seqs": seqs, "new_lo": new_lo, "new_hi": new_hi, "kv_lo": 1, "kv_hi": kv_hi,
            "heads": heads, "kv_heads": kv_heads, "d": d, "rd": rd, "page": page, "style": style}


def _paged(name, seqs, new_lo, new_hi, kv_lo, kv_hi, heads, kv_heads, d, page, block):
    return {"name": name, "op": "paged", "seqs": seqs, "new_lo": new_lo, "new_hi": new_hi, "kv_lo": kv_lo,
            "kv_hi": kv_hi, "heads": heads, "kv_heads": kv_heads, "d": d, "page": page, "block": block}


def _cross(name, n, lq, lk, heads, kv_heads, d, lens):
    return {"name": name, "op": "cross", "n": n, "lq": lq, "lk": lk, "heads": heads, "kv_heads": kv_heads, "d": d,
            "lens": lens}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    tops = [work(c) for c in listed()]
    top_bytes, top_flops = max(w["bytes"] for w in tops), max(w["flops"] for w in tops)
    while True:
        d = 16 * rng.randint(2, 8)
        kv_heads = _log(rng, 1, 16)
        heads = kv_heads * rng.choice([1, 1, 2, 3, 4, 5, 7, 8])
        style, rd = rng.choice(["pairs", "halves"]), rng.choice([d, d, 16 * rng.randint(1, d // 16)])
        page, seqs = 16 * rng.randint(1, 16), _log(rng, 1, 96)
        op = rng.choice(["rope", "append", "paged", "paged", "cross"])
        if op == "rope":
            case = _rope("", _log(rng, 1, 8 * FRAME), heads, kv_heads, d, rd, style)
        elif op == "append":
            new = 1 if rng.random() < 0.3 else _log(rng, 1, FRAME)
            case = _append("", seqs, max(1, new // 4), new, max(new, _log(rng, 16, 8 * FRAME)), heads, kv_heads, d, rd,
                           page, style)
        elif op == "paged":
            new = 1 if rng.random() < 0.4 else _log(rng, 2, 2 * FRAME)
            hi = max(new, _log(rng, 16, 131072))
            case = _paged("", seqs, max(1, new // 4), new, max(1, hi // 8), hi, heads, kv_heads, d, page,
                          rng.choice([0, 1, 1, max(1, new // 3)]))
        else:
            case = _cross("", seqs, _log(rng, 1, 4 * FRAME), _log(rng, 1, 1024), heads, kv_heads, d,
                          rng.random() < 0.6)
        del case["name"]
        w = work(case)
        # scores that the plain form computes and masks count too
        full = 4 * d * heads * sum(a * b for a, b in _lengths(case)) if op == "paged" else w["flops"]
        if w["bytes"] <= top_bytes and full <= 1.2 * top_flops and _pages(case) * page * kv_heads * d <= 1 << 31:
            return case


# ------------------------------------------------------------------------------------------------------ inputs --

def _lengths(case):
    """(new tokens, tokens in the cache with them) of each sequence: spread evenly over their ranges, in an order that
    mixes long and short ones."""
    out, seqs = [], case["seqs"]
    for b in range(seqs):
        f, g = ((b * 7 + 3) % seqs / (seqs - 1), (b * 5 + 1) % seqs / (seqs - 1)) if seqs > 1 else (1.0, 1.0)
        new = case["new_lo"] + round(f * (case["new_hi"] - case["new_lo"]))
        out.append((new, max(new, case["kv_lo"] + round(g * (case["kv_hi"] - case["kv_lo"])))))
    return out


def _pages(case):
    return sum(-(-kv // case["page"]) for _, kv in _lengths(case)) + 3 if "page" in case else 0


def _cross_lengths(case):
    """Of every five instances one is full, one empty where there are more than two, and the others are in between."""
    if not case["lens"]:
        return [case["lk"]] * case["n"]
    return [case["lk"] * ((3 * b + 4) % 5) // 4 for b in range(case["n"])]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    bf16, op = torch.bfloat16, case["op"]
    heads, kv_heads, d = case["heads"], case["kv_heads"], case["d"]

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda", dtype=bf16).mul_(scale)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    s = {"case": dict(case)}
    if op == "cross":
        n, lq, lk = case["n"], case["lq"], case["lk"]
        s["q"] = normal(n, lq, heads, d, scale=2.0)
        packed = normal(n, lk, 2 * kv_heads, d)  # both projections of the encoder's states side by side
        s["k"], s["v"] = packed[:, :, :kv_heads], packed[:, :, kv_heads:]
        s["lens_host"] = _cross_lengths(case)
        s["lens"] = ints(s["lens_host"]) if case["lens"] else None
        s["o"] = torch.zeros_like(s["q"])
        return s
    if op == "rope":
        rows, positions = case["rows"], case["rows"] + 5
    else:
        lengths = _lengths(case)
        rows, positions = sum(new for new, _ in lengths), max(kv for _, kv in lengths)
        s["lengths"] = lengths
        offsets = [0]
        for new, _ in lengths:
            offsets.append(offsets[-1] + new)
        s["offsets_host"] = offsets
        s["offsets"], s["lens"] = ints(offsets), ints([kv for _, kv in lengths])
        page, pages = case["page"], _pages(case)
        per = max(-(-kv // page) for _, kv in lengths)
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        table = torch.full((len(lengths), per), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, (_, kv) in enumerate(lengths):
            used = -(-kv // page)
            table[b, :used] = order[at:at + used]
            at += used
        s["table"] = table
        cache = normal(pages, 2, page, kv_heads, d)  # a page holds its keys and its values
        s["k_cache"], s["v_cache"] = cache[:, 0], cache[:, 1]
    if op == "paged":
        s["q"] = normal(rows, heads, d, scale=2.0)
        s["o"] = torch.zeros_like(s["q"])
        return s
    packed = normal(rows, heads + 2 * kv_heads, d, scale=1.5)  # the projections of a row side by side
    s["q"], s["k"], s["v"] = packed[:, :heads], packed[:, heads:heads + kv_heads], packed[:, heads + kv_heads:]
    s["gamma_q"], s["gamma_k"] = 1 + normal(d, scale=0.2), 1 + normal(d, scale=0.2)
    # angles in 64 bits: position x 10000^(-pair / pairs)
    pairs = case["rd"] // 2
    angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * torch.exp(
        torch.arange(pairs, dtype=torch.float64, device="cuda") * (-math.log(10000.0) / pairs))
    s["rot"] = torch.stack([angle.cos(), angle.sin()], -1).float()
    s["pos"] = None
    if op == "rope":
        s["pos"] = torch.randint(0, positions, (rows,), generator=gen, device="cuda").to(torch.int32)
        s["k_out"] = torch.zeros(rows, kv_heads, d, dtype=bf16, device="cuda")
    s["q_out"] = torch.zeros(rows, heads, d, dtype=bf16, device="cuda")
    return s


# -------------------------------------------------------------------------------------------------- plain forms --

def _norm_rotate(x, gamma, table, case):
    """x [rows, heads, D], table [rows, rd / 2, 2]."""
    x = x.float()
    x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma.float()
    rd = case["rd"]
    head, rest = x[..., :rd], x[..., rd:]
    c, s = table[:, None, :, 0], table[:, None, :, 1]
    if case["style"] == "pairs":
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    else:
        a, b = head[..., :rd // 2], head[..., rd // 2:]
        head = torch.cat([a * c - b * s, a * s + b * c], -1)
    return torch.cat([head, rest], -1).to(torch.bfloat16)


def _token_places(s):
    """(position in its sequence, slot in the cache) of every row."""
    page, pos, slots = s["case"]["page"], [], []
    for b, (new, kv) in enumerate(s["lengths"]):
        p = torch.arange(kv - new, kv, device="cuda")
        pos.append(p)
        slots.append(s["table"][b].long()[p // page] * page + p % page)
    return torch.cat(pos), torch.cat(slots)


def _attend(q, k, v, limit, out):
    """q [n, H, D], k, v [L, Hk, D] -> out [n, H, D]; query i sees the first limit[i] keys (all of them: None)."""
    n, heads, d = q.shape
    length, kv_heads, _ = k.shape
    if length == 0:
        out.zero_()
        return
    group = heads // kv_heads
    step = max(1, MAX_SCORES // (n * group * length))
    for h in range(0, kv_heads, step):
        e = min(kv_heads, h + step)
        qh = q[:, h * group:e * group].float().view(n, e - h, group, d).permute(1, 2, 0, 3).reshape(e - h, -1, d)
        scores = qh @ k[:, h:e].float().permute(1, 2, 0) * (1 / math.sqrt(d))
        if limit is not None:
            hidden = torch.arange(length, device="cuda") >= limit[:, None]
            scores.view(e - h, group, n, length).masked_fill_(hidden, float("-inf"))
        scores -= scores.amax(-1, keepdim=True)
        scores.exp_()
        total = scores.sum(-1, keepdim=True)
        res = scores @ v[:, h:e].float().permute(1, 0, 2) / total
        out[:, h * group:e * group] = res.view(e - h, group, n, d).permute(2, 0, 1, 3).reshape(n, -1, d)


def _limits(case, new, kv):
    """How many keys each of a sequence's new tokens sees: those up to the end of its own block."""
    block = case["block"] or new
    ends = (torch.arange(new, device="cuda") // block + 1) * block
    return kv - new + ends.clamp(max=new)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "rope":
        table = s["rot"][s["pos"].long()]
        s["q_out"].copy_(_norm_rotate(s["q"], s["gamma_q"], table, case))
        s["k_out"].copy_(_norm_rotate(s["k"], s["gamma_k"], table, case))
        return s["q_out"], s["k_out"]
    if op == "append":
        pos, slots = _token_places(s)
        table, page = s["rot"][pos], case["page"]
        s["q_out"].copy_(_norm_rotate(s["q"], s["gamma_q"], table, case))
        s["k_cache"][slots // page, slots % page] = _norm_rotate(s["k"], s["gamma_k"], table, case)
        s["v_cache"][slots // page, slots % page] = s["v"]
        return s["q_out"], s["k_cache"], s["v_cache"]
    if op == "paged":
        for b, (new, kv) in enumerate(s["lengths"]):
            rows = slice(s["offsets_host"][b], s["offsets_host"][b] + new)
            used = s["table"][b, :-(-kv // case["page"])].long()
            k, v = (s[c][used].flatten(0, 1)[:kv] for c in ("k_cache", "v_cache"))
            limit = None if new == 1 or not case["block"] else _limits(case, new, kv)
            _attend(s["q"][rows], k, v, limit, s["o"][rows])
        return s["o"]
    for b, length in enumerate(s["lens_host"]):
        _attend(s["q"][b], s["k"][b, :length], s["v"][b, :length], None, s["o"][b])
    return s["o"]


def run(state):
    if not own:
        return _plain(state)
    from causal_convolution_gb300 import api
    s, case = state, state["case"]
    op = case["op"]
    if op == "rope":
        api.cc_qk_norm_rope(s["q"], s["k"], s["gamma_q"], s["gamma_k"], s["rot"], s["pos"], s["q_out"], s["k_out"],
                            eps=EPS, style=case["style"])
        return s["q_out"], s["k_out"]
    if op == "append":
        api.cc_qk_norm_rope_append(s["q"], s["k"], s["v"], s["gamma_q"], s["gamma_k"], s["rot"], s["pos"], s["q_out"],
                                   s["k_cache"], s["v_cache"], s["offsets"], s["lens"], s["table"], eps=EPS,
                                   style=case["style"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if op == "paged":
        if "ws" not in s:  # a caller keeps its workspace, like its outputs
            need = api.cc_attn_paged_workspace_bytes(s["q"].shape[0], case["seqs"], case["heads"], case["kv_heads"],
                                                     case["d"])
            s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        api.cc_attn_paged(s["q"], s["k_cache"], s["v_cache"], s["o"], s["offsets"], s["lens"], s["table"], s["ws"],
                          causal_block=case["block"])
        return s["o"]
    if "ws" not in s:
        need = api.cc_attn_cross_workspace_bytes(case["n"], case["lq"], case["lk"], case["heads"], case["kv_heads"],
                                                 case["d"])
        s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    api.cc_attn_cross(s["q"], s["k"], s["v"], s["o"], s["lens"], s["ws"])
    return s["o"]


# ---------------------------------------------------------------------------------------------- floors, 64 bits --

def work(case):
    heads, kv_heads, d = case["heads"], case["kv_heads"], case["d"]
    if case["op"] == "cross":
        lens = _cross_lengths(case)
        rows = case["n"] * case["lq"]
        return {"bytes": 4 * rows * heads * d + 4 * sum(lens) * kv_heads * d + 4 * len(lens) * case["lens"],
                "flops": 4 * heads * d * case["lq"] * sum(lens)}
    if case["op"] == "rope":
        rows = case["rows"]
        return {"bytes": 4 * rows * (heads + kv_heads) * d + 4 * rows * case["rd"] + 4 * rows + 4 * d,
                "flops": 8 * rows * (heads + kv_heads) * d}
    lengths = _lengths(case)
    rows = sum(new for new, _ in lengths)
    plan = 4 * (2 * len(lengths) + 1)
    if case["op"] == "append":
        touched = sum((kv - 1) // case["page"] - (kv - new) // case["page"] + 1 for new, kv in lengths)
        return {"bytes": 4 * rows * (heads + 2 * kv_heads) * d + 4 * rows * case["rd"] + plan + 4 * touched + 4 * d,
                "flops": 8 * rows * (heads + kv_heads) * d}
    table = 4 * sum(-(-kv // case["page"]) for _, kv in lengths)
    seen = 0
    for new, kv in lengths:
        block = case["block"] or new
        whole, rest = divmod(new, block)
        seen += new * (kv - new) + block * block * whole * (whole + 1) // 2 + rest * new
    return {"bytes": 4 * rows * heads * d + 4 * sum(kv for _, kv in lengths) * kv_heads * d + table + plan,
            "flops": 4 * heads * d * seen}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return tuple(_exact_rotated(s[x], s["gamma_" + x], s["rot"], s["pos"].tolist(), case) for x in ("q", "k"))
    if op == "append":
        where = [(b, p) for b, (new, kv) in enumerate(s["lengths"]) for p in range(kv - new, kv)]
        pos = [p for _, p in where]
        keys = _exact_rotated(s["k"], s["gamma_k"], s["rot"], pos, case)
        table = s["table"].tolist()
        page_of = torch.tensor([table[b][p // case["page"]] for b, p in where], device="cuda")
        slot_of = torch.tensor([p % case["page"] for p in pos], device="cuda")
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        k_cache.index_put_((page_of, slot_of), keys)
        v_cache.index_put_((page_of, slot_of), s["v"].double())
        return _exact_rotated(s["q"], s["gamma_q"], s["rot"], pos, case), k_cache, v_cache
    if op == "cross":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b, length in enumerate(s["lens_host"]):
            if length:
                _exact_heads(out[b], s["q"][b], s["k"][b, :length], s["v"][b, :length], None)
        return out
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (new, kv) in enumerate(s["lengths"]):
        first = s["offsets_host"][b]
        at = torch.arange(kv, device="cuda")
        pages, slots = s["table"][b, at // case["page"]].long(), at % case["page"]
        sees = None
        if case["block"]:
            token = torch.arange(new, device="cuda")
            sees = kv - new + torch.minimum((token // case["block"] + 1) * case["block"], torch.tensor(new).cuda())
        _exact_heads(out[first:first + new], s["q"][first:first + new], s["k_cache"][pages, slots],
                     s["v_cache"][pages, slots], sees)
    return out


def _exact_rotated(x, gamma, rot, pos, case):
    x = x.double()
    norm = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
    x = x * gamma.double() / (norm * norm / case["d"] + EPS).sqrt()
    rd = case["rd"]
    # pair j's two channels
    j = torch.arange(rd // 2, device="cuda")
    first, second = (2 * j, 2 * j + 1) if case["style"] == "pairs" else (j, j + rd // 2)
    turn = torch.view_as_complex(rot.double()[torch.tensor(pos, device="cuda")])[:, None]
    z = torch.complex(x[..., first], x[..., second]) * turn
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _exact_heads(out, q, k, v, sees):
    """One query head at a time, a few thousand queries at a time: softmax as exp(score - log of the sum of exps)."""
    heads, group, d = q.shape[1], q.shape[1] // k.shape[1], q.shape[2]
    columns = torch.arange(k.shape[0], device="cuda")
    for h in range(heads):
        kt, vh = k[:, h // group].double().t(), v[:, h // group].double()
        for lo in range(0, q.shape[0], 4096):
            scores = (q[lo:lo + 4096, h].double() @ kt).div_(d ** 0.5)
            if sees is not None:
                scores = torch.where(columns < sees[lo:lo + 4096, None], scores, float("-inf"))
            out[lo:lo + 4096, h] = scores.sub_(scores.logsumexp(-1, keepdim=True)).exp_() @ vh
