"""The operators of a selective state-space block, as cases that can be timed.

``conv1d_causal`` / ``conv1d_causal_step``: the short depthwise causal
convolution over whole prompts, and for one new token of every sequence.
``selective_scan`` / ``selective_scan_step``: the selective state space
recurrence that follows it, over prompts and for one new token.

Per sequence, with x_t the token at position t:

  conv  y_t[c] = act(bias[c] + sum_k w[c,k] * x_{t-(K-1)+k}[c]), the positions
        before the first token taken from the state (carry) or zero; the new
        state is the last K-1 inputs
  scan  delta_t[d] = log(1 + exp(dt_t[d] + dt_bias[d]))
        h_t[d,s] = exp(delta_t[d] * a[d,s]) * h_{t-1}[d,s] + delta_t[d] * b_t[g,s] * x_t[d]
        out_t[d] = (sum_s c_t[g,s] * h_t[d,s] + D[d] * x_t[d]) * silu(z_t[d])
        g = d // (D / groups), h_{-1} the state (carry) or zero; the new state
        is h of the last token

A case of a prompt operator is a dense batch (``n`` sequences of ``l`` tokens)
or packed (``n`` sequences of different lengths one after the other in ``l``
rows, the last ``tail`` of them unused).
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
LARGEST_CONV = 4 * 4096 * 4096          # tokens x channels
LARGEST_SCAN = 8192 * 4096 * 16         # tokens x channels x states
LARGEST_CONV_STEP = 256 * 8192          # sequences x channels
LARGEST_SCAN_STEP = 192 * 4096 * 16     # sequences x channels x states
LARGEST_COST = 268e6                    # bytes, or flops / 50


def listed():
    return [
        # a batch of prompts in one wide layer; x is one half of the projection that made x and z
        {"name": "conv prompts bf16", "op": "conv", "n": 4, "l": 4096, "c": 4096, "k": 4, "type": "bf16",
         "packed": False, "carry": False, "silu": True, "bias": True, "gap": 4096, "tail": 0, "cut": 0},
        # prompts of different lengths packed into one buffer padded to a bucket, each continuing from its cache
        {"name": "conv packed f16", "op": "conv", "n": 13, "l": 5120, "c": 1280, "k": 4, "type": "f16",
         "packed": True, "carry": True, "silu": True, "bias": True, "gap": 1280, "tail": 61, "cut": 3},
        # a short odd-sized layer in fp32, no activation: the launch's own time
        {"name": "conv small f32", "op": "conv", "n": 2, "l": 37, "c": 83, "k": 3, "type": "f32",
         "packed": False, "carry": True, "silu": False, "bias": False, "gap": 0, "tail": 0, "cut": 0},
        # one sequence decoding: the launch's own time
        {"name": "conv step 1 bf16", "op": "conv_step", "n": 1, "c": 2048, "k": 4, "type": "bf16",
         "silu": True, "bias": True, "gap": 2048, "slots": 1},
        # a large decoding batch, its windows scattered over a larger cache
        {"name": "conv step 256 bf16", "op": "conv_step", "n": 256, "c": 8192, "k": 4, "type": "bf16",
         "silu": True, "bias": True, "gap": 8192, "slots": 300},
        # one long prompt in a wide layer: the most work
        {"name": "scan prompt bf16", "op": "scan", "n": 1, "l": 8192, "d": 4096, "s": 16, "groups": 1, "type": "bf16",
         "packed": False, "carry": False, "gate": True, "gap": 4096, "tail": 0, "cut": 0},
        # prompts of different lengths in one padded buffer, continuing from their states
        {"name": "scan packed f16", "op": "scan", "n": 9, "l": 4500, "d": 1280, "s": 16, "groups": 1, "type": "f16",
         "packed": True, "carry": True, "gate": True, "gap": 1280, "tail": 33, "cut": 5},
        # a narrow layer over one long sequence: few channels, parallel over the length or not at all
        {"name": "scan long narrow f32", "op": "scan", "n": 1, "l": 16384, "d": 96, "s": 16, "groups": 1,
         "type": "f32", "packed": False, "carry": True, "gate": False, "gap": 0, "tail": 0, "cut": 0},
        # short sequences, an odd number of states shared by groups of channels: the launch's own time
        {"name": "scan small bf16", "op": "scan", "n": 3, "l": 65, "d": 84, "s": 11, "groups": 2, "type": "bf16",
         "packed": False, "carry": True, "gate": True, "gap": 5, "tail": 0, "cut": 0},
        # one sequence decoding
        {"name": "scan step 1 bf16", "op": "scan_step", "n": 1, "d": 2048, "s": 16, "groups": 1, "type": "bf16",
         "gate": True, "gap": 2048, "slots": 1},
        # a large decoding batch, its states scattered over a larger cache
        {"name": "scan step 192 bf16", "op": "scan_step", "n": 192, "d": 4096, "s": 16, "groups": 1, "type": "bf16",
         "gate": True, "gap": 4096, "slots": 256},
        # wide states shared by groups, fp32
        {"name": "scan step wide state f32", "op": "scan_step", "n": 24, "d": 1024, "s": 128, "groups": 8,
         "type": "f32", "gate": False, "gap": 0, "slots": 24},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "conv_step", "scan", "scan_step"])
    case = {"op": op, "type": rng.choice(["f32", "f16", "bf16"])}
    wide = _log_int(rng, 16, 8192)
    if rng.random() < 0.6:
        wide = max(16, wide // 16 * 16)
    if op == "conv":
        n = _log_int(rng, 1, 16)
        packed = rng.random() < 0.5
        case |= {"n": n, "c": wide, "k": rng.choice([2, 3, 4, 4]), "packed": packed, "carry": rng.random() < 0.5,
                 "silu": rng.random() < 0.7, "bias": rng.random() < 0.7, "gap": rng.choice([0, wide, 8, 3])}
        most = max(2, LARGEST_CONV // (wide if packed else n * wide))
        l = _log_int(rng, 1, min(most, 16384 if packed else 8192))
        case |= {"l": l, "tail": rng.randrange(0, l // 8 + 1) if packed else 0, "cut": rng.randrange(1000)}
    elif op == "conv_step":
        n = _log_int(rng, 1, min(256, max(1, LARGEST_CONV_STEP // wide)))
        case |= {"n": n, "c": wide, "k": rng.choice([2, 3, 4, 4]), "silu": rng.random() < 0.7,
                 "bias": rng.random() < 0.7, "gap": rng.choice([0, wide, 8, 3]), "slots": n + rng.randrange(0, 50)}
    else:
        s = _log_int(rng, 4, 64 if op == "scan" else 128)
        if rng.random() < 0.5:
            s = 16
        groups = rng.choice([1, 1, 2, 4])
        wide = max(groups, wide // groups * groups)
        case |= {"d": wide, "s": s, "groups": groups, "gate": rng.random() < 0.7, "gap": rng.choice([0, wide, 8, 3])}
        if op == "scan":
            n = _log_int(rng, 1, 16)
            packed = rng.random() < 0.5
            most = max(2, LARGEST_SCAN // (wide * s * (1 if packed else n)))
            l = _log_int(rng, 1, min(most, 16384 if packed else 8192))
            case |= {"n": n, "l": l, "packed": packed, "carry": rng.random() < 0.5,
                     "tail": rng.randrange(0, l // 8 + 1) if packed else 0, "cut": rng.randrange(1000)}
        else:
            n = _log_int(rng, 1, min(256, max(1, LARGEST_SCAN_STEP // (wide * s))))
            case |= {"n": n, "slots": n + rng.randrange(0, 50)}
    size = "l" if "l" in case else "n"
    while _cost(case) > LARGEST_COST:
        case[size] //= 2
        if case.get("tail"):
            case["tail"] = min(case["tail"], case["l"] // 8)
    return case


def _cost(case):
    return max(work(case)["bytes"], work(case)["flops"] / 50)


def _lengths(case):
    """Tokens of each sequence.  Packed: random cuts of the used rows, one sequence empty where there are three."""
    n, l = case["n"], case["l"]
    if not case["packed"]:
        return [l] * n
    r = random.Random(case["cut"])
    used = l - case["tail"]
    at = [0] + sorted(r.randrange(0, used + 1) for _ in range(n - 1)) + [used]
    if n >= 3:
        at[n // 2] = at[n // 2 + 1]
    return [b - a for a, b in zip(at, at[1:])]


def prepare(case, seed):
    dev, dt = "cuda", TYPES[case["type"]]
    rng = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, kind=dt):
        return torch.randn(shape, generator=rng, device=dev).to(kind)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=rng, device=dev) * (hi - lo) + lo

    def inner(*shape):
        """A tensor whose rows are slices of wider rows, as one output of a joint projection is."""
        return normal(*shape[:-1], shape[-1] + case["gap"])[..., :shape[-1]]

    op, n = case["op"], case["n"]
    s = {"case": case, "op": op}
    step = op.endswith("step")
    if step:
        lead = (n,)
        s["slots"] = torch.randperm(case["slots"], generator=rng, device=dev)[:n].to(torch.int32)
        slots = case["slots"]
    else:
        lens = _lengths(case)
        starts = [sum(lens[:i]) for i in range(n + 1)]
        lead = (case["l"],) if case["packed"] else (n, case["l"])
        slots = n
        s["carry"] = case["carry"]
        s["slots"] = None
        s["offsets"] = torch.tensor(starts, dtype=torch.int32, device=dev) if case["packed"] else None
        s["longest"] = max(lens)
        # where each row's sequence starts, its number, and the sequences that have rows (known to the program that packed them)
        s["start"] = torch.tensor([starts[i] for i in range(n) for _ in range(lens[i])], dtype=torch.int64, device=dev)
        s["seq"] = torch.tensor([i for i in range(n) for _ in range(lens[i])], dtype=torch.int64, device=dev)
        s["lens"] = torch.tensor(lens, dtype=torch.int64, device=dev)
        s["starts"] = torch.tensor(starts[:n], dtype=torch.int64, device=dev)
        s["full"] = torch.tensor([i for i in range(n) if lens[i]], dtype=torch.int64, device=dev)
    if op in ("conv", "conv_step"):
        c, k = case["c"], case["k"]
        s["x"] = inner(*lead, c)
        s["w"] = uniform(-1, 1, c, k).mul_(k ** -0.5).to(dt)
        s["bias"] = uniform(-1, 1, c).mul_(k ** -0.5).to(dt) if case["bias"] else None
        s["activation"] = "silu" if case["silu"] else None
        s["state"] = normal(slots, k - 1, c)
        s["out"] = torch.zeros(*lead, c, dtype=dt, device=dev) if not step and case["packed"] else None
    else:
        d, st, g = case["d"], case["s"], case["groups"]
        s["x"] = inner(*lead, d)
        s["z"] = inner(*lead, d) if case["gate"] else None
        s["dt"] = normal(*lead, d).mul_(0.5)
        # steps from 1e-3 to 1e-1 after the softplus, decay rates 1..S: what such layers begin with
        first = torch.exp(uniform(math.log(1e-3), math.log(1e-1), d))
        s["dt_bias"] = first + torch.log(-torch.expm1(-first))
        s["a"] = -(torch.arange(1, st + 1, device=dev) * uniform(0.5, 1.5, d, st))
        s["d"] = uniform(0.5, 1.5, d)
        both = normal(*lead, 2 * g * st)                 # b and c are slices of one projection
        s["b"] = both[..., :g * st].unflatten(-1, (g, st))
        s["c"] = both[..., g * st:].unflatten(-1, (g, st))
        s["state"] = normal(slots, d, st, kind=torch.float32)
        s["out"] = torch.zeros(*lead, d, dtype=dt, device=dev) if not step and case["packed"] else None
    return s


def run(s):
    if own:
        import dense_convolution_nhwc_b200 as lib
        if s["op"] == "conv":
            out = lib.conv1d_causal(s["x"], s["w"], s["bias"], s["activation"], offsets=s["offsets"], state=s["state"],
                                    carry=s["carry"], out=s["out"])
        elif s["op"] == "conv_step":
            out = lib.conv1d_causal_step(s["x"], s["w"], s["state"], s["bias"], s["activation"], slots=s["slots"])
        elif s["op"] == "scan":
            out = lib.selective_scan(s["x"], s["dt"], s["a"], s["b"], s["c"], s["d"], s["z"], s["dt_bias"],
                                     softplus=True, offsets=s["offsets"], state=s["state"], carry=s["carry"],
                                     out=s["out"])
        else:
            out = lib.selective_scan_step(s["x"], s["dt"], s["a"], s["b"], s["c"], s["state"], s["d"], s["z"],
                                          s["dt_bias"], softplus=True, slots=s["slots"])
        return {"out": out, "state": s["state"]}
    plain = {"conv": _plain_conv, "conv_step": _plain_conv_step, "scan": _plain_scan, "scan_step": _plain_scan_step}
    return {"out": plain[s["op"]](s), "state": s["state"]}


def _silu(v):
    return v / (1 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _rows(t, inner_dims):
    """The tokens of a dense batch or a packed buffer as rows, in 32 bits."""
    return t.reshape(-1, *t.shape[t.dim() - inner_dims:]).float()


def _put_rows(s, y, like):
    """The rows of the sequences, in the layout and type of the input."""
    if s["out"] is None:
        return y.to(like.dtype).view(like.shape)
    s["out"][:y.shape[0]] = y.to(like.dtype)
    return s["out"]


def _plain_conv(s):
    x, state = _rows(s["x"], 1), s["state"]
    w = s["w"].float()
    k = w.shape[1]
    old = state.float() if s["carry"] else torch.zeros_like(state, dtype=torch.float32)
    rows = s["start"].shape[0]
    # the K rows of each token's window: from its sequence, or from the K-1 rows kept from before it
    at = torch.arange(rows, device=x.device)[:, None] + torch.arange(1 - k, 1, device=x.device)
    past = at - s["start"][:, None]
    window = torch.where((past >= 0)[:, :, None], x[torch.clamp(at, min=0)],
                         old[s["seq"][:, None], torch.clamp(past + k - 1, 0, k - 2)])
    y = (window * w.T).sum(1)
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if s["activation"]:
        y = _silu(y)
    # the last K-1 rows of each sequence, from the kept rows where it is shorter
    left = s["lens"][:, None] + torch.arange(1 - k, 0, device=x.device)
    kept = torch.where((left >= 0)[:, :, None], x[torch.clamp(s["starts"][:, None] + left, 0, x.shape[0] - 1)],
                       old[torch.arange(old.shape[0], device=x.device)[:, None], torch.clamp(left + k - 1, 0, k - 2)])
    state.copy_(kept)
    return _put_rows(s, y, s["x"])


def _plain_conv_step(s):
    x, at = s["x"], s["slots"].long()
    window = torch.cat([s["state"][at], x[:, None]], 1)
    y = (window.float() * s["w"].float().T).sum(1)
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if s["activation"]:
        y = _silu(y)
    s["state"][at] = window[:, 1:]
    return y.to(x.dtype)


def _plain_scan(s):
    rows = s["start"].shape[0]
    x, state = _rows(s["x"], 1)[:rows], s["state"]
    delta = _softplus(_rows(s["dt"], 1)[:rows] + s["dt_bias"])
    b, c = _rows(s["b"], 2)[:rows], _rows(s["c"], 2)[:rows]
    g, st = b.shape[1:]
    d = x.shape[1]
    a = torch.exp(delta[:, :, None] * s["a"])
    # h as the sum that each token adds, over all pairs of neighbours, then of fours, eights, ...
    h = ((delta * x).view(rows, g, d // g, 1) * b[:, :, None, :]).view(rows, d, st)
    first = s["starts"][s["full"]]
    if s["carry"]:
        h[first] += a[first] * state[s["full"]]
    a[first] = 0
    reach = 1
    while reach < s["longest"]:
        h[reach:] = h[reach:] + a[reach:] * h[:-reach]
        a[reach:] = a[reach:] * a[:-reach]
        reach *= 2
    del a
    y = (h.view(rows, g, d // g, st) * c[:, :, None, :]).sum(-1).view(rows, d) + s["d"] * x
    if s["z"] is not None:
        y = y * _silu(_rows(s["z"], 1)[:rows])
    if not s["carry"]:
        state.zero_()
    state[s["full"]] = h[first + s["lens"][s["full"]] - 1]
    return _put_rows(s, y, s["x"])


def _plain_scan_step(s):
    at = s["slots"].long()
    x, b, c = s["x"].float(), s["b"].float(), s["c"].float()
    n, d = x.shape
    g, st = b.shape[1:]
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    add = (delta * x).view(n, g, d // g, 1) * b[:, :, None, :]
    h = torch.exp(delta[:, :, None] * s["a"]) * s["state"][at] + add.view(n, d, st)
    y = (h.view(n, g, d // g, st) * c[:, :, None, :]).sum(-1).view(n, d) + s["d"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["state"][at] = h
    return y.to(s["x"].dtype)


def work(case):
    e, n = BYTES[case["type"]], case["n"]
    if case["op"] in ("conv", "conv_step"):
        c, k = case["c"], case["k"]
        tokens = n if case["op"] == "conv_step" else sum(_lengths(case))
        reads = 1 if case.get("carry", True) else 0
        size = e * (2 * tokens * c + c * k + (c if case["bias"] else 0) + (1 + reads) * n * (k - 1) * c)
        return {"bytes": size, "flops": tokens * c * (2 * k + (4 if case["silu"] else 0))}
    d, s, g = case["d"], case["s"], case["groups"]
    tokens = n if case["op"] == "scan_step" else sum(_lengths(case))
    reads = 1 if case.get("carry", True) else 0
    size = e * tokens * ((4 if case["gate"] else 3) * d + 2 * g * s) + 4 * (d * s + 2 * d + (1 + reads) * n * d * s)
    return {"bytes": size, "flops": tokens * d * (7 * s + 8 + (5 if case["gate"] else 0))}


def exact(case, seed):
    """The definitions, token by token in 64 bits."""
    s = prepare(case, seed)
    n, dev, f = case["n"], s["x"].device, torch.float64
    conv = case["op"] in ("conv", "conv_step")
    step = case["op"].endswith("step")
    keep = s["state"].to(f)
    slot = s["slots"].long() if step else torch.arange(n, device=dev)
    if step:
        lens, starts = [1] * n, list(range(n))
    else:
        lens = _lengths(case)
        starts = [sum(lens[:i]) for i in range(n)]
    flat = lambda t, dims: t.reshape(-1, *t.shape[t.dim() - dims:])  # noqa: E731
    x = flat(s["x"], 1)
    out = torch.zeros(x.shape, dtype=f, device=dev)
    now = keep[slot] if step or s["carry"] else torch.zeros_like(keep[slot])
    if not step and case["op"] == "scan" and not s["carry"]:
        keep = torch.zeros_like(keep)
    order = sorted(range(n), key=lambda i: -lens[i])        # the sequences still running are the first ones
    now = now[order]
    begin = torch.tensor([starts[i] for i in order], device=dev)
    for t in range(max(lens)):
        live = sum(1 for i in order if lens[i] > t)
        at = begin[:live] + t
        xt = x[at].to(f)
        if conv:
            seen = torch.cat([now[:live], xt[:, None]], 1)
            y = torch.einsum("nkc,ck->nc", seen, s["w"].to(f))
            y = y if s["bias"] is None else y + s["bias"].to(f)
            y = y * torch.sigmoid(y) if s["activation"] else y
            now[:live] = seen[:, 1:]
        else:
            delta = torch.nn.functional.softplus(flat(s["dt"], 1)[at].to(f) + s["dt_bias"].to(f), threshold=100)
            repeat = case["d"] // case["groups"]
            b = flat(s["b"], 2)[at].to(f).repeat_interleave(repeat, 1)
            c = flat(s["c"], 2)[at].to(f).repeat_interleave(repeat, 1)
            now[:live] = now[:live] * torch.exp(delta[:, :, None] * s["a"].to(f)) + (delta * xt)[:, :, None] * b
            y = torch.einsum("nds,nds->nd", now[:live], c) + s["d"].to(f) * xt
            if s["z"] is not None:
                zt = flat(s["z"], 1)[at].to(f)
                y = y * zt * torch.sigmoid(zt)
        out[at] = y
    keep[slot[torch.tensor(order, device=dev)]] = now
    return {"out": out.view(s["x"].shape), "state": keep}
