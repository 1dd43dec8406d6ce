"""Measured cases of the grouped matrix products (with their gradients), the INT8 products and SwiGLU.

A group is an expert: rows offsets[e] .. offsets[e + 1] - 1 of the activations meet weight matrix e.
`run` computes an operator in plain torch operations, or with the package's kernels where `own` is true.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}

# The layer's sizes: hidden 5120, expert width 2560, 256 experts, 8 per token; dense width 20480.
_MOST_WEIGHTS = 256 * 2560 * 5120
_MOST_FLOPS = 3 * 2 * 65536 * 5120 * 2560


def listed():
    mm, i8 = "mm", "i8_mm"
    return [
        # four tokens of a decode batch: 32 rows over 30 experts, bound by the weights of those experts
        dict(name="decode 4 tokens", op=mm, ways="fwd", experts=256, active=30, rows=32, k=5120, n=2560,
             dtype="bf16", out="bf16"),
        # a decode batch of 256 tokens through the second product: every weight once
        dict(name="decode 256 tokens", op=mm, ways="fwd", experts=256, active=250, rows=2048, k=2560, n=5120,
             dtype="bf16", out="bf16"),
        # a prefill chunk of 4096 tokens
        dict(name="prefill", op=mm, ways="fwd", experts=256, active=256, rows=32768, k=5120, n=2560, dtype="bf16",
             out="bf16"),
        # training on one of four expert-parallel ranks: input gradient of the second product, in fp16
        dict(name="input gradient", op=mm, ways="dgrad", experts=64, active=60, rows=16384, k=2560, n=5120,
             dtype="f16", out="f16"),
        # the same rank's weight gradient of a first product, in fp32 for the optimizer
        dict(name="weight gradient", op=mm, ways="wgrad", experts=64, active=60, rows=16384, k=5120, n=2560,
             dtype="bf16", out="f32"),
        # a long training batch over eight experts, forward and both gradients: bound by the products
        dict(name="training step, long", op=mm, ways="all", experts=8, active=8, rows=65536, k=5120, n=2560,
             dtype="bf16", out="bf16"),
        # a small layer with ragged groups and odd tiles, forward and both gradients: latency counts
        dict(name="training step, small", op=mm, ways="all", experts=16, active=13, rows=1501, k=320, n=192,
             dtype="f16", out="f16"),
        # one token through a dense layer's product with INT8 weights, its quantisation included
        dict(name="int8, one token", op=i8, experts=1, active=1, rows=1, k=5120, n=20480, dtype="bf16", out="bf16"),
        # a prefill chunk through the same product
        dict(name="int8, prefill", op=i8, experts=1, active=1, rows=4096, k=5120, n=20480, dtype="bf16", out="bf16"),
        # INT8 experts on one of four expert-parallel ranks: both first products, SwiGLU, the second product
        dict(name="int8 experts", op="i8_ffn", experts=64, active=64, rows=8192, k=5120, n=2560, dtype="bf16",
             out="bf16"),
        # SwiGLU of a prefill-sized training batch, forward and backward
        dict(name="swiglu, training", op="swiglu", rows=32768, width=2560, dtype="bf16"),
        # the same on a few odd rows in fp32
        dict(name="swiglu, few rows", op="swiglu", rows=77, width=192, dtype="f32"),
    ]


def _spread(rng, low, high, step=1):
    """A multiple of `step` in [low, high], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return min(high, max(low, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["mm"] * 5 + ["i8_mm"] * 2 + ["i8_ffn"] + ["swiglu"] * 2)
    if op == "swiglu":
        return dict(op=op, rows=_spread(rng, 1, 32768), width=_spread(rng, 64, 5120, 8),
                    dtype=rng.choice(["bf16", "f16", "f32"]))
    step = 8 if op == "mm" else 16
    while True:
        ways = rng.choice(["fwd", "fwd", "dgrad", "wgrad", "all"]) if op == "mm" else "fwd"
        k, n = _spread(rng, 64, 5120, step), _spread(rng, 64, 5120, step)
        experts = rng.choice([1, _spread(rng, 2, 256), _spread(rng, 2, 256), _spread(rng, 2, 256)])
        rows = _spread(rng, 1, 65536)
        passes = {"all": 3}.get(ways, 1) * (3 if op == "i8_ffn" else 1)
        weights = experts * k * n * (3 if op == "i8_ffn" else 1)
        if weights <= _MOST_WEIGHTS // 2 and passes * 2 * rows * k * n <= _MOST_FLOPS // 2:
            break
    active = max(1, min(experts, rows, int(experts * rng.uniform(0.5, 1.0) + 0.5)))
    dtype = rng.choice(["bf16", "bf16", "f16"])
    case = dict(op=op, experts=experts, active=active, rows=rows, k=k, n=n, dtype=dtype, out=dtype)
    if op == "mm":
        case["ways"] = ways
        if ways == "wgrad":
            case["out"] = rng.choice([dtype, "f32"])
    return case


def _groups(case, seed):
    """Rows of each group: `active` groups get at least one, the others none, with uneven popularity."""
    r = np.random.RandomState(seed % (1 << 31))
    e, a, rows = case["experts"], case["active"], case["rows"]
    p = np.exp(0.5 * r.standard_normal(a))
    counts = np.zeros(e, dtype=np.int64)
    counts[r.permutation(e)[:a]] = 1 + r.multinomial(rows - a, p / p.sum())
    return counts


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(scale)

    def codes(*shape):
        return normal(*shape, scale=32.0, dtype=torch.float16).round_().clamp_(-127, 127).to(torch.int8)

    def channel_scales(e, n, k):
        s = torch.rand(e, n, generator=g, device="cuda")
        return (s + 0.5) / (32.0 * math.sqrt(k))

    s = dict(case=dict(case))
    if case["op"] == "swiglu":
        r, i = case["rows"], case["width"]
        s.update(g=normal(r, i), u=normal(r, i), dh=normal(r, i))
        return s
    e, r, k, n = case["experts"], case["rows"], case["k"], case["n"]
    counts = _groups(case, seed)
    s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)])).cuda() if e > 1 else None
    # the plain form's plan: the groups that have rows, and the place of each row in a padded batch of them
    filled = np.nonzero(counts)[0]
    starts = np.cumsum(counts) - counts
    slot = np.repeat(np.arange(len(filled)), counts[filled])
    place = np.arange(r) - np.repeat(starts[filled], counts[filled])
    s["filled"] = torch.from_numpy(filled).cuda()
    s["slot"], s["place"] = torch.from_numpy(slot).cuda(), torch.from_numpy(place).cuda()
    s["most"] = int(counts.max())
    if case["op"] == "mm":
        s["x"], s["dy"] = normal(r, k), normal(r, n)
        if case["ways"] != "wgrad":
            s["w"] = normal(e, n, k, scale=1.0 / math.sqrt(k))
    else:
        s["x"] = normal(r, k)
        s["w"], s["ws"] = codes(e, n, k), channel_scales(e, n, k)
        if case["op"] == "i8_ffn":
            s["w_up"], s["ws_up"] = codes(e, n, k), channel_scales(e, n, k)
            s["w_down"], s["ws_down"] = codes(e, k, n), channel_scales(e, k, n)
    return s


def _padded(s, rows):
    """The groups' rows as a batch [groups with rows, most rows of one, width] in fp32, zeros behind each."""
    batch = torch.zeros(len(s["filled"]), s["most"], rows.shape[1], device=rows.device)
    batch[s["slot"], s["place"]] = rows.float()
    return batch


def _rows(s, batch):
    return batch[s["slot"], s["place"]]


def _weights(s, w):
    return (w if len(s["filled"]) == w.shape[0] else w[s["filled"]]).float()


def _plain_mm(s):
    c = s["case"]
    out_dtype, got = _DTYPES[c["out"]], {}
    if c["ways"] in ("fwd", "all"):
        got["out"] = _rows(s, torch.bmm(_padded(s, s["x"]), _weights(s, s["w"]).transpose(1, 2))).to(out_dtype)
    if c["ways"] in ("dgrad", "all"):
        got["dx"] = _rows(s, torch.bmm(_padded(s, s["dy"]), _weights(s, s["w"]))).to(out_dtype)
    if c["ways"] in ("wgrad", "all"):
        dw = torch.zeros(c["experts"], c["n"], c["k"], device=s["x"].device, dtype=out_dtype)
        dw[s["filled"]] = torch.bmm(_padded(s, s["dy"]).transpose(1, 2), _padded(s, s["x"])).to(out_dtype)
        got["dw"] = dw
    return got


def _plain_quant(x):
    x = x.float()
    most = x.abs().amax(dim=1, keepdim=True)
    scale = most / torch.full_like(most, 127.0)  # a quotient: a Python number would be multiplied by its reciprocal
    return torch.where(scale > 0, torch.round(x / scale), torch.zeros_like(x)).clamp(-127, 127), scale


def _plain_i8(s, x, w, ws):
    q, scale = _plain_quant(x)
    batch = torch.bmm(_padded(s, q), _weights(s, w).transpose(1, 2))
    batch = batch * (ws if len(s["filled"]) == ws.shape[0] else ws[s["filled"]]).unsqueeze(1)
    return _rows(s, batch) * scale


def _plain_silu(g):
    return g / (1.0 + torch.exp(-g))


def run(s):
    c = s["case"]
    if own:
        return _own(s)
    if c["op"] == "swiglu":
        g, u, dh = s["g"].float(), s["u"].float(), s["dh"].float()
        sig = 1.0 / (1.0 + torch.exp(-g))
        return {"h": (g * sig * u).to(s["g"].dtype), "dg": (dh * u * sig * (1.0 + g * (1.0 - sig))).to(s["g"].dtype),
                "du": (dh * g * sig).to(s["g"].dtype)}
    if c["op"] == "mm":
        return _plain_mm(s)
    if c["op"] == "i8_mm":
        return _plain_i8(s, s["x"], s["w"], s["ws"]).to(_DTYPES[c["out"]])
    h = _plain_silu(_plain_i8(s, s["x"], s["w"], s["ws"])) * _plain_i8(s, s["x"], s["w_up"], s["ws_up"])
    return _plain_i8(s, h, s["w_down"], s["ws_down"]).to(_DTYPES[c["out"]])


def _own(s):
    import group_limited_routing_router_b200 as bm

    c = s["case"]
    if c["op"] == "swiglu":
        dg, du = bm.swiglu_backward(s["dh"], s["g"], s["u"])
        return {"h": bm.swiglu(s["g"], s["u"]), "dg": dg, "du": du}
    off, out_dtype = s["offsets"], _DTYPES[c["out"]]
    if c["op"] == "mm":
        got = {}
        if c["ways"] in ("fwd", "all"):
            got["out"] = bm.grouped_mm(s["x"], s["w"], off, out_dtype=out_dtype)
        if c["ways"] in ("dgrad", "all"):
            got["dx"] = bm.grouped_mm_dgrad(s["dy"], s["w"], off, out_dtype=out_dtype)
        if c["ways"] in ("wgrad", "all"):
            got["dw"] = bm.grouped_mm_wgrad(s["dy"], s["x"], off, out_dtype=out_dtype)
        return got
    q, scale = bm.quant_i8_rows(s["x"])
    if c["op"] == "i8_mm":
        return bm.grouped_mm_i8(q, scale, s["w"], s["ws"], off, out_dtype=out_dtype)
    # fp32 between the products: what is quantised next is not rounded to 16 bits before
    g = bm.grouped_mm_i8(q, scale, s["w"], s["ws"], off, out_dtype=torch.float32)
    u = bm.grouped_mm_i8(q, scale, s["w_up"], s["ws_up"], off, out_dtype=torch.float32)
    q, scale = bm.swiglu_i8(g, u)
    return bm.grouped_mm_i8(q, scale, s["w_down"], s["ws_down"], off, out_dtype=out_dtype)


def work(case):
    b = _SIZE[case["dtype"]]
    if case["op"] == "swiglu":
        # forward and backward share their reads of g and u: three reads, three writes
        return {"bytes": 6.0 * case["rows"] * case["width"] * b, "flops": 20.0 * case["rows"] * case["width"]}
    r, k, n, a, o = case["rows"], case["k"], case["n"], case["active"], _SIZE[case["out"]]
    one = 2.0 * r * k * n
    if case["op"] == "i8_mm":
        return {"bytes": float(a * n * (k + 4) + r * k * b + r * n * o), "flops": one}
    if case["op"] == "i8_ffn":
        return {"bytes": float(a * (2 * n * (k + 4) + k * (n + 4)) + r * k * (b + o)), "flops": 3 * one}
    ways, total, flops = case["ways"], 0.0, 0.0
    if ways in ("fwd", "dgrad", "all"):
        total += a * n * k * b
    if ways in ("fwd", "wgrad", "all"):
        total += r * k * b
    if ways in ("dgrad", "wgrad", "all"):
        total += r * n * b
    if ways in ("fwd", "all"):
        total, flops = total + r * n * o, flops + one
    if ways in ("dgrad", "all"):
        total, flops = total + r * k * o, flops + one
    if ways in ("wgrad", "all"):
        total, flops = total + case["experts"] * n * k * o, flops + one
    return {"bytes": total, "flops": flops}


def exact(case, seed):
    """The definitions in 64 bits, one group after the other."""
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "swiglu":
        g, u, dh = s["g"].to(d), s["u"].to(d), s["dh"].to(d)
        sig = torch.sigmoid(g)
        silu = g * sig
        return {"h": silu * u, "dg": dh * u * (sig + silu - silu * sig), "du": dh * silu}
    ends = np.cumsum(_groups(case, seed))
    spans = [(e, int(ends[e - 1]) if e else 0, int(ends[e])) for e in range(case["experts"])]
    spans = [t for t in spans if t[1] < t[2]]
    r, k, n = case["rows"], case["k"], case["n"]

    def empty(*shape):
        return torch.zeros(*shape, dtype=d, device="cuda")

    if case["op"] == "mm":
        ways, got = case["ways"], {}
        if ways in ("fwd", "all"):
            got["out"] = empty(r, n)
        if ways in ("dgrad", "all"):
            got["dx"] = empty(r, k)
        if ways in ("wgrad", "all"):
            got["dw"] = empty(case["experts"], n, k)
        for e, a, b in spans:
            x, dy = s["x"][a:b].to(d), s["dy"][a:b].to(d)
            if "out" in got:
                got["out"][a:b] = x @ s["w"][e].to(d).t()
            if "dx" in got:
                got["dx"][a:b] = dy @ s["w"][e].to(d)
            if "dw" in got:
                got["dw"][e] = dy.t() @ x
        return got

    def quantised(x):
        # by definition the scale and the quotient are 32-bit numbers (a bf16 row often holds half its own
        # largest magnitude, whose quotient 63.5 is a tie), and the code is the integer nearest to the latter
        x = x.to(torch.float32)
        most = x.abs().max(dim=1).values[:, None]
        scale = torch.true_divide(most, torch.full_like(most, 127.0))
        return torch.nan_to_num(torch.round(x / scale), nan=0.0).clamp(-127, 127).to(d), scale.to(d)

    def product(x, w, ws):
        q, scale = quantised(x)
        y = empty(r, w.shape[1])
        for e, a, b in spans:
            y[a:b] = (q[a:b] @ w[e].to(d).t()) * ws[e].to(d)
        return y * scale

    y = product(s["x"], s["w"], s["ws"])
    if case["op"] == "i8_mm":
        return y
    h = y * torch.sigmoid(y) * product(s["x"], s["w_up"], s["ws_up"])
    return product(h, s["w_down"], s["ws_down"])
