"""Workloads of the gated recurrence and of the 8-bit projections.

A recurrent block is a gated recurrence (``gated_scan``) behind a short causal
convolution, between projections; served, its projections run in 8-bit
integers (``quantize_tokens``, ``project_int8``).  All activations are
channel-first, [batch, channel, time] with time contiguous (NCHW with H = 1).
Each case names an operator, a direction and its sizes; ``run`` makes one pass
through it, either as elementary torch operations in 32 bits (``own`` false;
64 for the borders between two codes) or through the library's entry points
(``own`` true).  ``exact`` is the definition in 64 bits, its gradients by
differentiation.

Keys of a case: op, dtype, B batch items, D channels (of a projection: of its
input), E channels of a projection's output, L positions, S cache lines
(slots), ragged (a length per sequence, one of them zero).
"""
import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_PAD = 128  # a row of codes is a multiple of this many bytes


def listed():
    return [
        # A generation step of a small batch: a few microseconds of work, so latency is what counts.
        {"name": "gated token", "op": "gated_token", "dtype": "bf16", "B": 8, "D": 2048, "S": 32},
        # A generation step of a large serving batch.
        {"name": "gated tokens", "op": "gated_token", "dtype": "bf16", "B": 256, "D": 4096, "S": 320},
        # Prompts of different lengths continued from cached states, one of them empty; rows of odd length.
        {"name": "gated prompts", "op": "gated_prompt", "dtype": "f16", "B": 5, "D": 1000, "L": 1237, "ragged": True},
        # One long prompt: no batch to spread over the chip.
        {"name": "gated long prompt", "op": "gated_prompt", "dtype": "bf16", "B": 1, "D": 4096, "L": 8192,
         "ragged": False},
        # A training step: forward and backward of a batch of equal sequences.
        {"name": "gated training", "op": "gated_train", "dtype": "bf16", "B": 4, "D": 2048, "L": 2048},
        # A small model trained in full precision, odd sizes.
        {"name": "gated training f32", "op": "gated_train", "dtype": "f32", "B": 2, "D": 602, "L": 777},
        # A projection of a generation step's tokens: the weights' traffic and the launch are all there is.
        {"name": "int8 token", "op": "int8_token", "dtype": "bf16", "B": 8, "D": 2048, "E": 4096},
        # The same of a large serving batch and a wide layer.
        {"name": "int8 tokens", "op": "int8_token", "dtype": "bf16", "B": 64, "D": 4096, "E": 8192},
        # Short prompts of different lengths, one of them empty.
        {"name": "int8 prompts", "op": "int8_prompt", "dtype": "f16", "B": 5, "D": 1000, "E": 2000, "L": 301,
         "ragged": True},
        # Sizes that no tile divides, results in full precision.
        {"name": "int8 prompts f32", "op": "int8_prompt", "dtype": "f32", "B": 2, "D": 2051, "E": 1027, "L": 777,
         "ragged": False},
        # A batch of prompts through a square layer.
        {"name": "int8 batch", "op": "int8_prompt", "dtype": "bf16", "B": 4, "D": 2048, "E": 2048, "L": 2048,
         "ragged": False},
        # One long prompt into a wide layer: the matrix cores' rate is what counts.
        {"name": "int8 long prompt", "op": "int8_prompt", "dtype": "bf16", "B": 1, "D": 4096, "E": 8192, "L": 8192,
         "ragged": False},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    op = rng.choice(("gated_token", "gated_prompt", "gated_prompt", "gated_train", "gated_train", "int8_token",
                     "int8_token", "int8_prompt", "int8_prompt", "int8_prompt"))
    case = {"op": op, "dtype": rng.choice(("f32", "bf16", "f16"))}
    D = _log_int(rng, 64, 4096)
    if op == "gated_token":
        case.update(B=_log_int(rng, 1, 256), D=D)
        case["S"] = case["B"] + _log_int(rng, 1, 64)
    elif op == "int8_token":
        case.update(B=_log_int(rng, 1, 64), D=D, E=_log_int(rng, 64, 8192))
    else:
        # At most what the largest listed cases have.
        case.update(B=_log_int(rng, 1, 8), D=D, L=_log_int(rng, 1, 8192))
        if op == "int8_prompt":
            case["E"] = _log_int(rng, 64, 8192)
        most = {"int8_prompt": 2 ** 38, "gated_prompt": 2 ** 25, "gated_train": 2 ** 24}[op]
        while case["B"] * case["D"] * case["L"] * case.get("E", 1) > most:
            key = max(("B", "D", "L"), key=lambda k: case[k] / {"B": 8, "D": 4096, "L": 8192}[k])
            case[key] = max(1, int(case[key] * 0.71))
        if op != "gated_train":
            case["ragged"] = rng.random() < 0.5
    return case


def _lengths(case, rand):
    """A length per sequence: the first whole, the last empty, the others anything between."""
    if not case.get("ragged") or case["B"] < 2:
        return None
    length = (rand(case["B"], uniform=True) * (case["L"] + 1)).to(torch.int32).clamp_(0, case["L"])
    length[0] = case["L"]
    length[-1] = 0
    return length


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T = _DTYPES[case["dtype"]]

    def rand(*shape, uniform=False):
        f = torch.rand if uniform else torch.randn
        return f(*shape, generator=gen, device="cuda", dtype=torch.float32)

    op, B, D = case["op"], case["B"], case["D"]
    L = case.get("L", 1)
    s = {"case": case, "lengths": _lengths(case, rand) if "L" in case else None}
    if op.startswith("int8"):
        E = case["E"]
        # Channels of different spread, as activations have them.
        spread = torch.exp(0.7 * rand(D))
        x = (rand(B, D, L) * spread[:, None]).to(T)
        s["x"] = x[..., 0] if op == "int8_token" else x
        s["bias"] = 0.1 * rand(E)
        # The weights as a server keeps them: codes in rows of whole 128 bytes, a scale for each channel.
        w = rand(E, D) * D ** -0.5
        most = w.abs().amax(1)
        s["w"] = torch.zeros(E, -(-D // _PAD) * _PAD, dtype=torch.int8, device="cuda")
        s["w"][:, :D] = torch.round(w.double() * 127 / most[:, None]).to(torch.int8)
        s["w_scales"] = most / 127
        return s
    # The first half of a projection's output; the other half is the gate of the result.
    xz = rand(B, 2 * D, L).to(T)
    # Both gates are rows of one projection's output.
    ri = rand(B, 2 * D, L).to(T)
    s.update(x=xz[:, :D], z=xz[:, D:], r=ri[:, :D], i=ri[:, D:])
    # Decays between 0.9 and 0.999 a position where the gate is open.
    s["A"] = torch.log(0.9 + 0.099 * rand(D, uniform=True))
    s["r_bias"], s["i_bias"] = 0.5 * rand(D), 0.5 * rand(D)
    if op == "gated_token":
        s.update({k: s[k][..., 0] for k in "xzri"})
        # Cache lines in no particular order; the last rows of a larger batch are its padding.
        slots = torch.randperm(case["S"], generator=gen, device="cuda")[:B].to(torch.int32)
        if B >= 8:
            slots[-1] = -1
        s["slots"] = slots
        # The cache, and one line behind it that takes what a padding row would write.
        s["lines"] = rand(case["S"] + 1, D)
        s["state"] = s["lines"][:-1]
    elif op == "gated_prompt":
        s["state"] = rand(B, D)
    else:
        s["dy"] = rand(B, D, L).to(T)
    return s


def run(s):
    return (_library if own else _plain)[s["case"]["op"]](s)


# ---- the library's operators --------------------------------------------------------------------


def _gi():
    import conv2d_backward_amd
    return conv2d_backward_amd


def _lib_gated_token(s):
    y = _gi().gated_scan_step(s["x"], s["r"], s["i"], s["A"], s["state"], z=s["z"], r_bias=s["r_bias"],
                              i_bias=s["i_bias"], slots=s["slots"])
    return {"y": y, "state": s["state"]}


def _lib_gated_prompt(s):
    y, state, _ = _gi().gated_scan(s["x"], s["r"], s["i"], s["A"], z=s["z"], r_bias=s["r_bias"], i_bias=s["i_bias"],
                                   state=s["state"], lengths=s["lengths"], want_state=True)
    return {"y": y, "state": state}


def _lib_gated_train(s):
    gi = _gi()
    y, _, checkpoints = gi.gated_scan(s["x"], s["r"], s["i"], s["A"], z=s["z"], r_bias=s["r_bias"],
                                      i_bias=s["i_bias"], want_checkpoints=True)
    g = gi.gated_scan_backward(s["dy"], s["x"], s["r"], s["i"], s["A"], checkpoints, z=s["z"], r_bias=s["r_bias"],
                               i_bias=s["i_bias"])
    return {"y": y, "dx": g.dx, "dr": g.dr, "di": g.di, "dz": g.dz, "dA": g.dA, "dr_bias": g.dr_bias,
            "di_bias": g.di_bias}


def _lib_int8_token(s):
    return {"y": _gi().project_int8_step(s["x"], s["w"], s["w_scales"], s["bias"])}


def _lib_int8_prompt(s):
    gi = _gi()
    codes, scales = gi.quantize_tokens(s["x"], lengths=s["lengths"])
    y = gi.project_int8(codes, scales, s["w"], s["w_scales"], s["bias"], dtype=s["x"].dtype, lengths=s["lengths"])
    return {"y": y, "scales": scales}


_library = {"gated_token": _lib_gated_token, "gated_prompt": _lib_gated_prompt, "gated_train": _lib_gated_train,
            "int8_token": _lib_int8_token, "int8_prompt": _lib_int8_prompt}


# ---- their plain forms --------------------------------------------------------------------------


def _inside(lengths, L):
    """[B, 1, L] truth values: the positions that a sequence has; None where all have all."""
    if lengths is None:
        return None
    return (torch.arange(L, device=lengths.device) < lengths[:, None])[:, None]


def _only(inside, v, other=0.0):
    return v if inside is None else torch.where(inside, v, torch.full((), other, dtype=v.dtype, device=v.device))


def _gates(s, column):
    """log of the decay, the decay, the normaliser and the open part of the input; `column` shapes parameters."""
    x, r, i = s["x"].float(), s["r"].float(), s["i"].float()
    sr = torch.sigmoid(r + s["r_bias"].view(column))
    si = torch.sigmoid(i + s["i_bias"].view(column))
    log_a = s["A"].view(column) * sr
    return x, sr, si, torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a))


def _plain_gated_token(s):
    slots = s["slots"].long()
    live = slots >= 0
    h = s["state"][torch.where(live, slots, torch.zeros_like(slots))]
    x, _, si, a, m = _gates(s, (-1,))
    h = a * h + m * (si * x)
    z = s["z"].float()
    y = torch.where(live[:, None], h * z * torch.sigmoid(z), torch.zeros_like(h)).to(s["x"].dtype)
    s["lines"][torch.where(live, slots, torch.full_like(slots, len(s["state"])))] = h
    return {"y": y, "state": s["state"]}


def _linear_scan(a, b):
    """h_t = a_t h_{t-1} + b_t along the last axis, h before it 0, by doubling the span that each position has summed."""
    span = 1
    while span < a.shape[-1]:
        b = torch.cat([b[..., :span], b[..., span:] + a[..., span:] * b[..., :-span]], -1)
        a = torch.cat([a[..., :span], a[..., span:] * a[..., :-span]], -1)
        span *= 2
    return a, b


def _plain_gated_prompt(s):
    inside = _inside(s["lengths"], s["x"].shape[-1])
    x, _, si, a, m = _gates(s, (-1, 1))
    passed, h = _linear_scan(_only(inside, a, 1.0), _only(inside, m * (si * x)))
    h = h + passed * s["state"][..., None]
    z = s["z"].float()
    return {"y": _only(inside, h * z * torch.sigmoid(z)).to(s["x"].dtype), "state": h[..., -1]}


def _plain_gated_train(s):
    x, sr, si, a, m = _gates(s, (-1, 1))
    T = s["x"].dtype
    _, h = _linear_scan(a, m * (si * x))
    z, dy = s["z"].float(), s["dy"].float()
    sz = torch.sigmoid(z)
    # The gradient of the states runs backwards, with the decay of the next position.
    after = torch.cat([a[..., 1:], torch.zeros_like(a[..., :1])], -1)
    q = _linear_scan(after.flip(-1), (dy * z * sz).flip(-1))[1].flip(-1)
    before = torch.cat([torch.zeros_like(h[..., :1]), h[..., :-1]], -1)
    dlog_a = q * (a * before - a * a / m * (si * x))
    dr = dlog_a * s["A"][:, None] * sr * (1 - sr)
    di = q * m * x * si * (1 - si)
    return {"y": (h * z * sz).to(T), "dx": (q * m * si).to(T), "dr": dr.to(T), "di": di.to(T),
            "dz": (dy * h * sz * (1 + z * (1 - sz))).to(T), "dA": (dlog_a * sr).sum(-1).sum(0),
            "dr_bias": dr.sum(-1).sum(0), "di_bias": di.sum(-1).sum(0)}


def _codes(x):
    """Codes of the rows of x [..., D], as the numbers they are, and a scale for each row.  Which of two codes is
    nearest is decided in 64 bits."""
    most = x.float().abs().amax(-1, keepdim=True)
    codes = torch.round(x.double() * 127 / torch.where(most > 0, most, torch.ones_like(most)))
    return codes.float(), most / 127


def _plain_int8_token(s):
    codes, scales = _codes(s["x"])
    w = s["w"][:, :codes.shape[-1]].float()
    return {"y": (codes @ w.t() * (scales * s["w_scales"]) + s["bias"]).to(s["x"].dtype)}


def _plain_int8_prompt(s):
    B, D, L = s["x"].shape
    inside = _inside(s["lengths"], L)
    codes, scales = _codes(s["x"].transpose(1, 2).contiguous())
    w = s["w"][:, :D].float()
    y = w @ codes.view(B * L, D).t()
    y = y * s["w_scales"][:, None] * scales.view(B * L) + s["bias"][:, None]
    y = y.view(-1, B, L).transpose(0, 1)
    scales = scales.view(B, L)
    return {"y": _only(inside, y).to(s["x"].dtype).contiguous(),
            "scales": scales if inside is None else _only(inside[:, 0], scales)}


_plain = {"gated_token": _plain_gated_token, "gated_prompt": _plain_gated_prompt, "gated_train": _plain_gated_train,
          "int8_token": _plain_int8_token, "int8_prompt": _plain_int8_prompt}


# ---- the definitions in 64 bits -----------------------------------------------------------------


def _exact_gated(s, case):
    """Position by position, the recurrence as it is written; gradients by differentiation."""
    op = case["op"]
    train = op == "gated_train"
    v = {k: s[k].double().detach().requires_grad_(train) for k in ("x", "r", "i", "z", "A", "r_bias", "i_bias")}
    steps = {k: (v[k].unbind(-1) if op != "gated_token" else [v[k]]) for k in "xriz"}
    slots = s["slots"].tolist() if op == "gated_token" else None
    if train:
        h = torch.zeros(case["B"], case["D"], device="cuda", dtype=torch.float64)
    elif slots is None:
        h = s["state"].double()
    else:
        h = s["state"].double()[[max(k, 0) for k in slots]]
    ys = []
    for t in range(len(steps["x"])):
        u = v["A"] / (1 + torch.exp(-(steps["r"][t] + v["r_bias"])))
        enter = steps["x"][t] / (1 + torch.exp(-(steps["i"][t] + v["i_bias"])))
        new = torch.exp(u) * h + (1 - torch.exp(2 * u)).sqrt() * enter
        y = new * steps["z"][t] / (1 + torch.exp(-steps["z"][t]))
        if s["lengths"] is not None:
            here = (s["lengths"] > t)[:, None]
            y, new = torch.where(here, y, torch.zeros_like(y)), torch.where(here, new, h)
        h = new
        ys.append(y)
    if slots is not None:
        state = s["state"].double()
        for b, slot in enumerate(slots):
            if slot < 0:
                ys[0][b] = 0
            else:
                state[slot] = h[b]
        return {"y": ys[0], "state": state}
    y = torch.stack(ys, 2)
    if not train:
        return {"y": y, "state": h}
    names = {"dx": "x", "dr": "r", "di": "i", "dz": "z", "dA": "A", "dr_bias": "r_bias", "di_bias": "i_bias"}
    got = torch.autograd.grad((y * s["dy"].double()).sum(), [v[k] for k in names.values()])
    return {"y": y.detach(), **dict(zip(names, got))}


def _exact_int8(s, case):
    x = s["x"].double()
    if x.dim() == 2:
        x = x[..., None]
    B, D, L = x.shape
    w = s["w"].double()[:, :D] * s["w_scales"].double()[:, None]
    y = torch.empty(B, case["E"], L, device="cuda", dtype=torch.float64)
    scales = torch.zeros(B, L, device="cuda", dtype=torch.float64)
    for b in range(B):
        n = L if s["lengths"] is None else int(s["lengths"][b])
        most = x[b, :, :n].abs().amax(0)
        stands_for = torch.round(127 * x[b, :, :n] / most) * (most / 127)
        y[b, :, :n] = w @ stands_for + s["bias"].double()[:, None]
        y[b, :, n:] = 0
        scales[b, :n] = most / 127
    return {"y": y[..., 0]} if case["op"] == "int8_token" else {"y": y, "scales": scales}


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_int8 if case["op"].startswith("int8") else _exact_gated)(s, case)


# ---- what a pass cannot do without --------------------------------------------------------------


def work(case):
    op, e = case["op"], 4 if case["dtype"] == "f32" else 2
    B, D, L = case["B"], case["D"], case.get("L", 1)
    n = B * D * L
    if op.startswith("int8"):
        # The activations, the weights' codes and the parameters read, the result written.
        E = case["E"]
        return {"bytes": e * n + E * D + 8 * E + e * B * E * L, "flops": 2 * n * E}
    if op == "gated_train":
        # x, r, i, z, dy read; y, dx, dr, di, dz written; the parameters and their gradients
        return {"bytes": 10 * e * n + 24 * D, "flops": 70 * n}
    # x, r, i, z read; y written; the state read and written
    return {"bytes": 5 * e * n + 8 * B * D + 12 * D, "flops": 25 * n}
