"""The sequence operators: the short causal conv1d and the selective scan, over
prompts and for single tokens, against their definitions in 64 bits
(tests/sequence_ref.py, where the tolerances come from)."""
import ctypes

import pytest
import torch

import dense_convolution_nhwc_b200 as dc
from dense_convolution_nhwc_b200 import binding as B
from tests import sequence_ref as ref
from tests.gpu_util import Guarded, guarded_input

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
B200 = B.DeviceProps(148, 10, 0, 183359 * 2 ** 20)


# ------------------------------ no GPU needed ----------------------------------

def flat(fields):
    """Field values, a stride array's elements as values of their own."""
    return [v for f in fields.values() for v in (f if isinstance(f, tuple) else (f,))]


def conv_desc(**over):
    d = dict(n=2, l=5, c=8, k=4, activation=0, carry=1, state_slots=2, x_stride=(40, 8), out_stride=(40, 8))
    d.update(over)
    return B.CausalConvDesc(*flat(d))


# distinct, aligned addresses that no refused call may touch
X, W, BIAS, STATE, OUT, SLOTS, OFFSETS = (0x100000 * i for i in range(1, 8))


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), 1), (dict(l=-1), 1), (dict(l=2 ** 30 + 1), 1), (dict(c=0), 1), (dict(c=2 ** 22 + 1), 1), (dict(k=1), 1), (dict(k=9), 1),
    (dict(activation=2), 1), (dict(state_slots=1), 1), (dict(x_stride=(-1, 8)), 1), (dict(out_stride=(40, 7)), 1),
    (dict(out_stride=(39, 8)), 1), (dict(n=0), 0),
])
def test_conv_descriptor_refusals(over, status):
    assert B.conv1d_causal_forward(X, W, BIAS, 0, STATE, 0, OUT, conv_desc(**over), 0, 0) == status


def test_conv_pointer_refusals():
    call = B.conv1d_causal_forward
    d = conv_desc()
    assert call(0, W, 0, 0, STATE, 0, OUT, d, 0, 0) == 1
    assert call(X, 0, 0, 0, STATE, 0, OUT, d, 0, 0) == 1
    assert call(X, W, 0, 0, STATE, 0, 0, d, 0, 0) == 1
    assert call(X, W, 0, 0, 0, 0, OUT, d, 0, 0) == 1                      # carry without a state
    assert call(X, W, 0, 0, 0, SLOTS, OUT, conv_desc(carry=0), 0, 0) == 1  # slots without a state
    assert call(X, W, 0, 0, STATE, 0, OUT, d, 3, 0) == 1                  # no such type
    assert call(X + 2, W, 0, 0, STATE, 0, OUT, d, 0, 0) == 3
    assert call(X + 1, W, 0, 0, STATE, 0, OUT, d, 2, 0) == 3
    assert call(X, W, 0, OFFSETS + 2, STATE, 0, OUT, d, 0, 0) == 3
    for overlap in (X, X + 300, W, STATE):
        assert call(X, W, 0, 0, STATE, 0, overlap, d, 0, 0) == 1
    assert call(X, W, 0, 0, X + 64, 0, OUT, d, 0, 0) == 1                 # state over x
    assert B.conv1d_causal_step_forward(X, W, 0, 0, 0, OUT, d, 0, 0) == 1
    assert B.conv1d_causal_step_forward(X, W, 0, STATE, 0, X, d, 0, 0) == 1
    assert B._conv1d_causal_forward(X, W, 0, 0, STATE, 0, OUT, None, 0, None) == 1


def scan_desc(**over):
    d = dict(n=2, l=5, d=8, s=16, groups=2, softplus=1, carry=1, state_slots=2, packed=0, x_stride=(40, 8), dt_stride=(40, 8),
             z_stride=(40, 8), b_stride=(160, 32), c_stride=(160, 32), out_stride=(40, 8))
    d.update(over)
    return B.ScanDesc(*flat(d))


def scan_tensors(**over):
    names = [n for n, _ in B.ScanTensors._fields_]
    at = {n: 0x100000 * (i + 1) for i, n in enumerate(names)}
    at.update(offsets=0, slots=0)
    at.update(over)
    return B.ScanTensors(*(at[n] for n in names))


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), 1), (dict(l=-1), 1), (dict(l=2 ** 30 + 1), 1), (dict(d=0), 1), (dict(d=2 ** 22 + 2), 1), (dict(s=0), 1), (dict(s=257), 1),
    (dict(groups=0), 1), (dict(groups=3), 1), (dict(state_slots=1), 1), (dict(b_stride=(160, -1)), 1),
    (dict(out_stride=(40, 7)), 1), (dict(n=0), 0),
])
def test_scan_descriptor_refusals(over, status):
    assert B.selective_scan_forward(scan_tensors(), scan_desc(**over), 0, 0, 0, 0) == status
    if "l" not in over and "out_stride" not in over:
        assert B.selective_scan_step_forward(scan_tensors(), scan_desc(**over), 0, 0) == status


@pytest.mark.parametrize("over,status", [
    (dict(x=0), 1), (dict(dt=0), 1), (dict(a=0), 1), (dict(b=0), 1), (dict(c=0), 1), (dict(out=0), 1), (dict(state=0), 1),
    (dict(x=0x100002), 3), (dict(a=0x600002), 3), (dict(state=0xb00002), 3),
    (dict(offsets=0xd00000), 1), (dict(out=0x100000), 1), (dict(out=0x100040), 1), (dict(out=0xb00000), 1), (dict(state=0x600000), 1),
])
def test_scan_pointer_refusals(over, status):
    assert B.selective_scan_forward(scan_tensors(**over), scan_desc(), 0, 0, 0, 0) == status
    assert B.selective_scan_step_forward(scan_tensors(**over), scan_desc(), 0, 0) == status
    assert B._selective_scan_forward(None, scan_desc(), 0, None, 0, None) == 1


def test_scan_workspace_may_not_overlap():
    assert B.selective_scan_forward(scan_tensors(), scan_desc(), 0, 0x100000, 1024, 0) == 1
    assert B.selective_scan_forward(scan_tensors(), scan_desc(), 0, 0xb00000, 1024, 0) == 1


def scan_plan(**over):
    p = B.ScanPlan()
    assert B.selective_scan_plan_for_props(scan_desc(**over), 0, B200, p) == 0
    return p.as_dict()


def test_scan_plan_is_a_rule_on_sizes():
    """Every state has a lane; sequences are cut only where the channels leave the
    device idle, into chunks that cover them, with a workspace for each chunk's
    state and sum."""
    for s in range(1, 257):
        p = scan_plan(s=s, d=64, groups=1, l=100)
        assert p["lanes"] * p["states_per_lane"] >= s and p["lanes"] in (1, 2, 4, 8, 16, 32)
    wide = scan_plan(n=1, d=8192, groups=1, l=16384)
    assert wide["chunks"] == 1 and wide["workspace_bytes"] == 0
    for n, d, l in [(1, 96, 16384), (2, 64, 5000), (1, 8, 1000)]:
        p = scan_plan(n=n, d=d, groups=1, l=l)
        assert p["chunks"] > 2 and (p["chunks"] - 1) * p["chunk_tokens"] < l <= p["chunks"] * p["chunk_tokens"]
        assert p["workspace_bytes"] >= n * p["chunks"] * d * 17 * 4
    # packed sequences share the rows: shorter chunks, more of them a sequence at most
    dense, packed = scan_plan(n=11, d=48, groups=1, l=10813), scan_plan(n=11, d=48, groups=1, l=10813, packed=1)
    assert 2 < dense["chunks"] < packed["chunks"] <= 128 and packed["chunk_tokens"] >= 64
    assert scan_plan(n=200, d=4096, groups=1, l=10000, packed=1)["chunks"] == 1
    assert scan_plan(n=11, d=300, groups=1, l=10813, packed=1)["chunks"] > 4
    assert scan_plan(n=1, d=8, groups=1, l=1)["chunks"] == 1
    assert scan_plan(n=1, d=8, groups=1, l=0)["chunks"] == 1
    assert scan_plan(n=1, d=8, groups=1, l=2 ** 30)["chunk_tokens"] > 0
    assert B.selective_scan_plan_for_props(scan_desc(), 0, B.DeviceProps(), B.ScanPlan()) == 1


def test_torch_conveniences_refuse_host_tensors():
    x, w, state = torch.zeros(2, 5, 8), torch.zeros(8, 4), torch.zeros(2, 3, 8)
    for call in (lambda: dc.conv1d_causal(x, w), lambda: dc.conv1d_causal_step(x[:, 0], w, state),
                 lambda: dc.selective_scan(x, x, w, x[..., None], x[..., None]),
                 lambda: dc.selective_scan_step(x[:, 0], x[:, 0], w, x[:, 0, None], x[:, 0, None], state)):
        with pytest.raises(TypeError):
            call()


def test_names_are_exported():
    lib = ctypes.CDLL(B.library_path)
    for name in ("conv1d_causal_forward", "conv1d_causal_step_forward", "selective_scan_plan", "selective_scan_plan_for_props",
                 "selective_scan_workspace_size", "selective_scan_forward", "selective_scan_step_forward"):
        assert hasattr(lib, name) and callable(getattr(dc, name))


# ----------------------------------- GPU ---------------------------------------

gpu = pytest.mark.gpu


def draws(seed):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0, gap=0, at=0):
        """Values whose rows are `gap` elements apart, `at` elements into their buffer."""
        wide = torch.randn(*shape[:-1], shape[-1] + gap, generator=g) * scale
        flat = torch.cat([torch.full((at,), float("nan")), wide.flatten()]).to(dtype).cuda()
        return flat[at:].view(wide.shape)[..., :shape[-1]]
    return normal


def split(lens):
    at = [0]
    for v in lens:
        at.append(at[-1] + v)
    return torch.tensor(at, dtype=torch.int32).cuda(), at


def cpu(t):
    return None if t is None else t.detach().cpu()


def check_conv(dtype, k, c, lens, packed, carry, silu, bias, gap=0, at=0, tail=0, slots=None, seed=0):
    """One prompt call against the definition, its buffers between canaries."""
    normal, n = draws(seed), len(lens)
    rows = sum(lens) + tail
    x = normal(rows, c, dtype=dtype, gap=gap, at=at) if packed else normal(n, lens[0], c, dtype=dtype, gap=gap, at=at)
    if tail:
        x[sum(lens):] = float("nan")                       # never read
    w, b = normal(c, k, dtype=dtype), normal(c, dtype=dtype) if bias else None
    cache = n + 2 if slots is not None else n
    g_state = Guarded(cache * (k - 1) * c * x.element_size(), "cuda")
    state = g_state.tensor((cache, k - 1, c), dtype)
    state.copy_(normal(cache, k - 1, c, dtype=dtype))
    if not carry:
        state[:] = float("nan")                            # not read either
    before = state.clone()
    offsets, starts = split(lens)
    g_out = Guarded(x.numel() * x.element_size(), "cuda")
    out = g_out.tensor(tuple(x.shape), dtype)
    out.fill_(7.0)
    at_slots = None if slots is None else torch.tensor(slots, dtype=torch.int32).cuda()
    got = dc.conv1d_causal(x, w, b, "silu" if silu else None, offsets=offsets if packed else None, state=state,
                           slots=at_slots, carry=carry, out=out)
    torch.cuda.synchronize()
    assert got is out
    g_out.assert_intact("out")
    g_state.assert_intact("state")
    out, state, x = out.cpu(), state.cpu(), x.cpu()
    for i, length in enumerate(lens):
        lo = starts[i]
        xi, oi = (x[lo:lo + length], out[lo:lo + length]) if packed else (x[i], out[i])
        slot = i if slots is None else slots[i]
        if not 0 <= slot < cache:
            assert (oi == 7).all()
            continue
        window = before[slot].cpu() if carry else torch.zeros(k - 1, c, dtype=dtype)
        y, bound, kept = ref.causal_conv(xi, w.cpu(), cpu(b), silu, window)
        ref.assert_within(oi, y, bound, f"sequence {i}")
        assert torch.equal(state[slot], kept), f"window {i}"
    if packed and tail:
        assert (out[starts[-1]:] == 7).all()
    untouched = set(range(cache)) - {i if slots is None else slots[i] for i in range(n)}
    for slot in untouched:
        assert torch.equal(state[slot].isnan(), before[slot].cpu().isnan())


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("k", range(2, 9))
@pytest.mark.parametrize("carry", [False, True])
def test_conv_taps(dtype, k, carry):
    for length in (1, k - 1, k, 31, 33, 75):
        check_conv(TYPES[dtype], k, 24, [length] * 2, False, carry, True, True, seed=length)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("c,gap,at", [(1, 0, 0), (7, 0, 0), (8, 3, 0), (40, 8, 1), (83, 0, 0), (264, 264, 0), (520, 4, 8)])
def test_conv_widths_strides_and_alignment(dtype, c, gap, at):
    check_conv(TYPES[dtype], 4, c, [37, 37, 37], False, True, True, True, gap=gap, at=at)
    check_conv(TYPES[dtype], 4, c, [37, 3, 70], True, True, False, False, gap=gap, at=at, tail=2)


@gpu
@pytest.mark.parametrize("carry", [False, True])
@pytest.mark.parametrize("lens,tail", [
    ([0], 0), ([0, 0, 0], 5), ([1], 0), ([1, 1, 1, 1], 0), ([31, 1, 32, 0, 33], 7), ([32, 32, 0, 64, 2], 0),
    ([30, 3, 2, 1, 0, 1, 5, 90], 31), ([200], 1), ([1] * 70, 3), ([0, 63, 0, 0, 1, 0], 0),
])
def test_conv_packed(lens, tail, carry):
    """Sequences that end anywhere in a walk, empty ones, one-token ones, rows behind the last."""
    for k in (2, 4, 8):
        check_conv(torch.bfloat16, k, 16, lens, True, carry, True, True, tail=tail, seed=k)


@gpu
def test_conv_slots():
    check_conv(torch.float16, 4, 32, [5, 40, 3, 7], True, True, True, False, slots=[3, 0, -1, 5], tail=3)
    check_conv(torch.float32, 3, 10, [9, 9, 9], False, False, False, True, slots=[4, 99, 1])


@gpu
def test_conv_without_a_state():
    normal = draws(1)
    x, w = normal(2, 40, 24, dtype=torch.bfloat16), normal(24, 4, dtype=torch.bfloat16)
    got = dc.conv1d_causal(x, w, activation="silu")
    for i in range(2):
        y, bound, _ = ref.causal_conv(x[i].cpu(), w.cpu(), None, True, torch.zeros(3, 24, dtype=x.dtype))
        ref.assert_within(got[i], y, bound)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,c,k,gap", [(1, 1, 2, 0), (1, 2048, 4, 2048), (3, 83, 3, 0), (5, 40, 8, 8), (70, 24, 4, 3)])
def test_conv_step(dtype, n, c, k, gap):
    normal, dt = draws(n + c), TYPES[dtype]
    x, w, b = normal(n, c, dtype=dt, gap=gap), normal(c, k, dtype=dt), normal(c, dtype=dt)
    state = normal(n + 3, k - 1, c, dtype=dt)
    slots = torch.randperm(n + 3)[:n].to(torch.int32)
    if n > 2:
        slots[1] = -1
    before, out = state.cpu(), torch.full((n, c), 7.0, dtype=dt, device="cuda")
    dc.conv1d_causal_step(x, w, state, b, "silu", slots=slots.cuda(), out=out)
    want = before.clone()
    for i, slot in enumerate(slots.tolist()):
        if slot < 0:
            assert (out[i] == 7).all()
            continue
        y, bound, want[slot] = ref.causal_conv(x[i:i + 1].cpu(), w.cpu(), b.cpu(), True, before[slot])
        ref.assert_within(out[i:i + 1], y, bound, f"sequence {i}")
    assert torch.equal(state.cpu(), want)


def scan_inputs(normal, lead, d, s, g, dtype, gate=True, gap=0, at=0, bc_gap=0):
    first = torch.rand(d) * 0.1 + 1e-3
    t = dict(x=normal(*lead, d, dtype=dtype, gap=gap, at=at), dt=normal(*lead, d, dtype=dtype, scale=0.5, gap=gap),
             z=normal(*lead, d, dtype=dtype, gap=gap, at=at) if gate else None,
             a=-(torch.rand(d, s) + 0.5).cuda() * (torch.arange(s, device="cuda") + 1),
             d=normal(d) if gate else None, dt_bias=torch.log(torch.expm1(first)).cuda())
    both = normal(*lead, 2 * g * s, dtype=dtype, gap=bc_gap)
    t["b"], t["c"] = both[..., :g * s].unflatten(-1, (g, s)), both[..., g * s:].unflatten(-1, (g, s))
    return t


def check_scan(dtype, d, s, g, lens, packed, carry, gate=True, gap=0, at=0, bc_gap=0, tail=0, slots=None, softplus=True,
               seed=0):
    normal, n = draws(seed), len(lens)
    torch.manual_seed(seed)
    rows = sum(lens) + tail
    t = scan_inputs(normal, (rows,) if packed else (n, lens[0]), d, s, g, dtype, gate, gap, at, bc_gap)
    if not softplus:
        t["dt"] = (t["dt"].float().abs() * 0.1).to(dtype)
        t["dt_bias"] = None
    if tail:
        for name in ("x", "dt", "z", "b", "c"):
            if t[name] is not None:
                t[name][sum(lens):] = float("nan")         # never read
    cache = n + 2 if slots is not None else n
    g_state = Guarded(cache * d * s * 4, "cuda")
    state = g_state.tensor((cache, d, s), torch.float32)
    state.copy_(normal(cache, d, s))
    if not carry:
        state[:] = float("nan")
    before = state.cpu()
    offsets, starts = split(lens)
    g_out = Guarded(t["x"].numel() * t["x"].element_size(), "cuda")
    out = g_out.tensor(tuple(t["x"].shape), dtype)
    out.fill_(7.0)
    dc.selective_scan(**t, softplus=softplus, offsets=offsets if packed else None, state=state,
                      slots=None if slots is None else torch.tensor(slots, dtype=torch.int32).cuda(), carry=carry, out=out)
    torch.cuda.synchronize()
    g_out.assert_intact("out")
    g_state.assert_intact("state")
    out, state = out.cpu(), state.cpu()
    h = {name: cpu(v) for name, v in t.items()}
    seen = set()
    for i, length in enumerate(lens):
        rows_i = slice(starts[i], starts[i] + length) if packed else i
        slot = i if slots is None else slots[i]
        if not 0 <= slot < cache:
            assert (out[rows_i] == 7).all()
            continue
        seen.add(slot)
        part = {name: h[name] if name in ("a", "d", "dt_bias") or h[name] is None else h[name][rows_i] for name in h}
        y, bound, last, last_bound = ref.scan(**part, softplus=softplus, h=before[slot] if carry else torch.zeros(d, s))
        ref.assert_within(out[rows_i], y, bound, f"sequence {i}")
        ref.assert_within(state[slot], last, last_bound + 1e-30, f"state {i}")
    if packed and tail:
        assert (out[starts[-1]:] == 7).all()
    for slot in set(range(cache)) - seen:
        assert torch.equal(state[slot].nan_to_num(9), before[slot].nan_to_num(9))


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("s", [1, 3, 4, 8, 11, 16, 17, 32, 64, 130, 256])
def test_scan_states(dtype, s):
    check_scan(TYPES[dtype], 24, s, 2, [45, 45], False, True, seed=s)
    check_scan(TYPES[dtype], 5, s, 1, [37, 3], True, False, tail=4, seed=s)


@gpu
@pytest.mark.parametrize("length", [0, 1, 2, 7, 8, 9, 31, 32, 33, 64, 65, 140])
def test_scan_lengths(length):
    for carry in (False, True):
        check_scan(torch.bfloat16, 40, 16, 1, [length] * 2, False, carry, seed=length)
        check_scan(torch.float32, 9, 5, 3, [length] * 2, False, carry, gate=False, seed=length)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,g,gap,at,bc_gap", [(1, 1, 0, 0, 0), (6, 3, 0, 0, 1), (16, 1, 3, 1, 0), (84, 2, 8, 0, 5),
                                               (130, 1, 130, 0, 0), (256, 4, 8, 8, 8), (272, 1, 0, 0, 48)])
def test_scan_widths_strides_and_alignment(dtype, d, g, gap, at, bc_gap):
    for s in (16, 12):
        check_scan(TYPES[dtype], d, s, g, [41, 41], False, True, gap=gap, at=at, bc_gap=bc_gap, seed=d)


@gpu
@pytest.mark.parametrize("carry", [False, True])
@pytest.mark.parametrize("lens,tail", [([0], 0), ([0, 0, 5], 3), ([1, 1, 40], 0), ([33, 0, 64, 7], 9), ([1] * 20, 1)])
def test_scan_packed(lens, tail, carry):
    check_scan(torch.float16, 24, 16, 1, lens, True, carry, tail=tail)
    check_scan(torch.float32, 20, 10, 2, lens, True, carry, tail=tail, softplus=False)


@gpu
def test_scan_slots():
    check_scan(torch.bfloat16, 16, 16, 1, [5, 40, 3, 7], True, True, slots=[3, 0, -1, 5], tail=2)
    check_scan(torch.float32, 10, 6, 1, [9, 9, 9], False, False, slots=[4, 99, 1])


@gpu
@pytest.mark.parametrize("lens,packed", [([700], False), ([530, 530], False), ([400, 0, 3, 333, 64, 65], True)])
@pytest.mark.parametrize("s,d", [(16, 24), (7, 10), (64, 6)])
def test_scan_cut_into_chunks(lens, packed, s, d):
    desc = B.ScanDesc(len(lens), sum(lens) + 3 if packed else lens[0], d, s, 1, packed=int(packed))
    assert B.selective_scan_workspace_size(desc, 0, 0) > 0
    for carry in (False, True):
        check_scan(torch.float32, d, s, 1, lens, packed, carry, tail=3 if packed else 0)
        check_scan(torch.bfloat16, d, s, 1, lens, packed, carry, tail=3 if packed else 0)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d,s,g", [(1, 1, 1, 1), (1, 2048, 16, 1), (3, 20, 11, 2), (5, 64, 128, 4), (9, 33, 200, 1),
                                     (70, 24, 16, 1), (2, 7, 4, 1), (4, 12, 256, 3)])
def test_scan_step(dtype, n, d, s, g):
    check_scan_step(dtype, n, d, s, g)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d,s,g", [
    (30, 2048, 16, 1), (50, 1000, 20, 1), (20, 500, 200, 1), (60, 1000, 10, 1),      # four channels a turn
    (100, 2048, 16, 1), (200, 1000, 12, 1), (64, 1024, 128, 8), (400, 512, 8, 2),    # blocks that walk over sequences
    (120, 1020, 16, 3),                                                              # groups that a warp's channels straddle
])
def test_large_scan_steps(dtype, n, d, s, g):
    check_scan_step(dtype, n, d, s, g)


def check_scan_step(dtype, n, d, s, g):
    normal, dt = draws(n + d + s), TYPES[dtype]
    torch.manual_seed(s)
    t = scan_inputs(normal, (n,), d, s, g, dt, gap=3 if n == 3 else 0)
    state = normal(n + 3, d, s)
    slots = torch.randperm(n + 3)[:n].to(torch.int32)
    if n > 2:
        slots[1] = -1
    before, out = state.cpu(), torch.full((n, d), 7.0, dtype=dt, device="cuda")
    dc.selective_scan_step(**t, state=state, softplus=True, slots=slots.cuda(), out=out)
    h, kept = {name: cpu(v) for name, v in t.items()}, set(range(n + 3))
    for i, slot in enumerate(slots.tolist()):
        if slot < 0:
            assert (out[i] == 7).all()
            continue
        kept.discard(slot)
        part = {name: h[name] if name in ("a", "d", "dt_bias") else h[name][i:i + 1] for name in h}
        y, bound, last, last_bound = ref.scan(**part, softplus=True, h=before[slot])
        ref.assert_within(out[i:i + 1], y, bound, f"sequence {i}")
        ref.assert_within(state[slot], last, last_bound, f"state {i}")
    for slot in kept:
        assert torch.equal(state[slot].cpu(), before[slot])


class Block:
    """A state-space block as a model has it, over the library's operators."""

    def __init__(self, dim, inner, s, rank, dtype):
        normal = draws(11)
        torch.manual_seed(11)
        self.inner, self.s, self.rank = inner, s, rank
        self.w_in = normal(2 * inner, dim, dtype=dtype, scale=dim ** -0.5)
        self.w_conv, self.b_conv = normal(inner, 4, dtype=dtype, scale=0.5), normal(inner, dtype=dtype, scale=0.1)
        self.w_x = normal(rank + 2 * s, inner, dtype=dtype, scale=inner ** -0.5)
        self.w_dt = normal(inner, rank, dtype=dtype, scale=rank ** -0.5)
        self.dt_bias = torch.log(torch.expm1(torch.rand(inner) * 0.1 + 1e-3)).cuda()
        self.a = -(torch.arange(1, s + 1).float().repeat(inner, 1)).cuda()
        self.d = torch.ones(inner, device="cuda")
        self.w_out = normal(dim, inner, dtype=dtype, scale=inner ** -0.5)

    def caches(self, slots, dtype):
        return torch.zeros(slots, 3, self.inner, dtype=dtype, device="cuda"), torch.zeros(slots, self.inner, self.s, device="cuda")

    def scan_inputs(self, u):
        p = u @ self.w_x.T
        dt = p[..., :self.rank] @ self.w_dt.T
        b, c = (p[..., self.rank + i * self.s:self.rank + (i + 1) * self.s].unsqueeze(-2) for i in (0, 1))
        return dt, b, c

    def prompt(self, x, caches, carry, **where):
        xz = x @ self.w_in.T
        u, z = xz[..., :self.inner], xz[..., self.inner:]
        u = dc.conv1d_causal(u, self.w_conv, self.b_conv, "silu", state=caches[0], carry=carry, **where)
        dt, b, c = self.scan_inputs(u)
        y = dc.selective_scan(u, dt, self.a, b, c, self.d, z, self.dt_bias, softplus=True, state=caches[1], carry=carry, **where)
        return y @ self.w_out.T

    def token(self, x, caches, slots=None):
        xz = x @ self.w_in.T
        u, z = xz[..., :self.inner], xz[..., self.inner:]
        u = dc.conv1d_causal_step(u, self.w_conv, caches[0], self.b_conv, "silu", slots=slots)
        dt, b, c = self.scan_inputs(u)
        y = dc.selective_scan_step(u, dt, self.a, b, c, caches[1], self.d, z, self.dt_bias, softplus=True, slots=slots)
        return y @ self.w_out.T


@gpu
def test_block_prompt_then_tokens():
    """The operators together: a prompt, a second part continuing it, packed with
    another sequence, then single tokens, against the whole sequence at once.  In
    fp32 the parts differ by fp32 rounding alone, and by the matrix products' order."""
    torch.backends.cuda.matmul.allow_tf32 = False
    block = Block(32, 48, 16, 4, torch.float32)
    x = draws(3)(2, 90, 32)
    want = block.prompt(x, block.caches(2, torch.float32), False)
    caches = block.caches(5, torch.float32)
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    got = [block.prompt(x[:, :41].contiguous(), caches, False, slots=slots)]
    # 30 tokens of the first, 20 of the second, in one packed call
    packed = torch.cat([x[0, 41:71], x[1, 41:61]])
    part = block.prompt(packed, caches, True, slots=slots, offsets=torch.tensor([0, 30, 50], dtype=torch.int32, device="cuda"))
    tol = 2 ** -24 * 2000 * want.abs().max().item()      # about 100 tokens of memory, some 20 roundings each
    assert (got[0] - want[:, :41]).abs().max() <= tol
    assert (part[:30] - want[0, 41:71]).abs().max() <= tol and (part[30:] - want[1, 41:61]).abs().max() <= tol
    for t in range(19):
        rows = torch.stack([x[0, 71 + t], x[1, 61 + t]])
        y = block.token(rows, caches, slots)
        assert (y - torch.stack([want[0, 71 + t], want[1, 61 + t]])).abs().max() <= tol, t


@gpu
def test_prompt_call_of_one_token_is_the_step():
    """A prompt of one token and a step compute the same."""
    normal = draws(5)
    torch.manual_seed(5)
    t = scan_inputs(normal, (6, 1), 40, 16, 1, torch.bfloat16)
    first = normal(6, 40, 16)
    s1, s2 = first.clone(), first.clone()
    whole = dc.selective_scan(**t, softplus=True, state=s1, carry=True)
    one = {k: v if k in ("a", "d", "dt_bias") else v[:, 0] for k, v in t.items()}
    step = dc.selective_scan_step(**one, softplus=True, state=s2)
    assert (whole[:, 0].float() - step.float()).abs().max() <= 2 ** -8 * whole.float().abs().max()
    assert (s1 - s2).abs().max() <= 2 ** -20 * s1.abs().max()


@gpu
def test_capture_streams_and_replay():
    """On a side stream, captured, and replayed on new inputs: the results of eager calls."""
    block = Block(32, 48, 16, 4, torch.bfloat16)
    slots = torch.tensor([2, 0, -1], dtype=torch.int32, device="cuda")
    x = draws(7)(3, 32, dtype=torch.bfloat16)
    caches, again = block.caches(4, torch.bfloat16), block.caches(4, torch.bfloat16)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.token(x, again, slots)
        for t in again:
            t.zero_()
        with torch.cuda.graph(graph, stream=side):
            y = block.token(x, again, slots)
    torch.cuda.current_stream().wait_stream(side)
    for t in again:
        t.zero_()
    for i in range(5):
        x.copy_(draws(20 + i)(3, 32, dtype=torch.bfloat16))
        want = block.token(x, caches, slots)
        graph.replay()
        assert torch.equal(y[:2], want[:2])
    assert all(torch.equal(p, q) for p, q in zip(caches, again))


@gpu
def test_chunked_prompt_captured():
    """A cut scan, with its workspace, captured and replayed."""
    normal = draws(9)
    torch.manual_seed(9)
    t = scan_inputs(normal, (1, 600), 24, 16, 1, torch.float32)
    want = dc.selective_scan(**t, softplus=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = dc.selective_scan(**t, softplus=True)
    got.fill_(float("nan"))
    graph.replay()
    assert torch.equal(got, want)
    t["x"].copy_(normal(1, 600, 24))
    graph.replay()
    assert torch.equal(got, dc.selective_scan(**t, softplus=True))


@gpu
def test_infinities_and_nans_stay_in_their_sequence():
    normal = draws(13)
    torch.manual_seed(13)
    t = scan_inputs(normal, (3, 40), 16, 11, 1, torch.float32)
    clean = dc.selective_scan(**t, softplus=True)
    bad = {k: v if v is None else v.clone() for k, v in t.items()}
    bad["x"][1, 5, 3] = float("inf")
    bad["x"][1, 20, 4] = float("nan")
    got = dc.selective_scan(**bad, softplus=True)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])
    others = [i for i in range(16) if i not in (3, 4)]
    assert torch.equal(got[1][:, others], clean[1][:, others])
    assert torch.equal(got[1, :5], clean[1, :5]) and got[1, 20:, 4].isnan().all()
    w = normal(16, 4)
    y, good = dc.conv1d_causal(bad["x"], w), dc.conv1d_causal(t["x"], w)
    assert torch.equal(y[0], good[0]) and torch.equal(y[1, 9:20, 3], good[1, 9:20, 3]) and not y[1, 5:9, 3].isfinite().any()


@gpu
def test_a_decay_of_minus_infinity_forgets():
    """a = -inf: each token's state is what it adds, ragged tiles included."""
    normal = draws(15)
    torch.manual_seed(15)
    t = scan_inputs(normal, (1, 45), 10, 6, 1, torch.float32, gate=False)
    t["a"] = torch.full_like(t["a"], -float("inf"))
    state = normal(1, 10, 6)
    got = dc.selective_scan(**t, softplus=True, state=state, carry=True)
    delta = torch.nn.functional.softplus(t["dt"] + t["dt_bias"]).double()
    h = (delta * t["x"])[..., None] * t["b"].double()
    want = (h * t["c"].double()).sum(-1)
    assert (got - want).abs().max() <= 2 ** -24 * 64 * (h * t["c"]).abs().sum(-1).max()
    assert (state - h[:, -1]).abs().max() <= 2 ** -24 * 64 * h.abs().max()


@gpu
def test_far_slots_and_far_rows():
    """A cache of more than 2^31 values and rows more than 2^31 values apart."""
    d, s = 2048, 128
    slots = 2 ** 31 // (d * s) + 2
    state = torch.empty(slots, d, s, device="cuda")
    normal = draws(17)
    torch.manual_seed(17)
    t = scan_inputs(normal, (1,), d, s, 1, torch.bfloat16)
    start = normal(1, d, s)
    state[-1:] = start
    near = start.clone()
    want = dc.selective_scan_step(**t, state=near, softplus=True)
    got = dc.selective_scan_step(**t, state=state, softplus=True, slots=torch.tensor([slots - 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(got, want) and torch.equal(state[-1:], near)
    del state
    wide = 2 ** 30 + 64
    buffer = torch.empty(2 * wide + 64, dtype=torch.bfloat16, device="cuda")
    x = buffer.as_strided((3, 64), (wide, 1))
    x.copy_(normal(3, 64, dtype=torch.bfloat16))
    w = normal(64, 4, dtype=torch.bfloat16)
    assert torch.equal(dc.conv1d_causal(x[None], w), dc.conv1d_causal(x.contiguous()[None], w))
    near = scan_inputs(normal, (1, 3), 64, 16, 1, torch.bfloat16)
    near["x"] = x.contiguous()[None]
    far = dict(near, x=x[None])
    assert torch.equal(dc.selective_scan(**far, softplus=True), dc.selective_scan(**near, softplus=True))


@gpu
def test_bad_offsets_stay_inside():
    """Offsets that descend or leave the buffer: unspecified rows, no access outside (canaries and NaN bands)."""
    normal = draws(19)
    torch.manual_seed(19)
    rows, d, s = 50, 16, 16
    t = scan_inputs(normal, (rows,), d, s, 1, torch.float32, gate=False)
    x_guard, x = guarded_input(t["x"].contiguous())
    w = normal(d, 4)
    for offsets in ([0, 40, 20, 50], [-5, 10, 900, 50], [60, 70, 80, 90], [50, 30, 10, 0], [-9, -8, -7, -6]):
        off = torch.tensor(offsets, dtype=torch.int32).cuda()
        g_out, g_state = Guarded(rows * d * 4, "cuda"), Guarded(3 * d * s * 4, "cuda")
        out, state = g_out.tensor((rows, d), torch.float32), g_state.tensor((3, d, s), torch.float32)
        state.zero_()
        dc.selective_scan(**dict(t, x=x), softplus=True, offsets=off, state=state, carry=True, out=out)
        window = torch.zeros(3, 3, d, device="cuda")
        dc.conv1d_causal(x, w, offsets=off, state=window, carry=True, out=out)
        torch.cuda.synchronize()
        g_out.assert_intact("out")
        g_state.assert_intact("state")
        x_guard.assert_intact("x")


@gpu
def test_gpu_refusals():
    normal = draws(21)
    x, w = normal(2, 8, 16), normal(16, 4)
    with pytest.raises(ValueError):
        dc.conv1d_causal(x, w, offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))    # dense x
    with pytest.raises(TypeError):
        dc.conv1d_causal(x[0], w, offsets=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        dc.conv1d_causal(x, w, carry=True)
    with pytest.raises(ValueError):
        dc.conv1d_causal(x, w[:8])
    with pytest.raises(TypeError):
        dc.conv1d_causal(x, w.half())
    with pytest.raises(TypeError):
        dc.conv1d_causal(x.double(), w.double())
    with pytest.raises(ValueError):
        dc.conv1d_causal(x.transpose(1, 2), normal(8, 4))
    with pytest.raises(ValueError):
        dc.conv1d_causal(x, w, activation="gelu")
    with pytest.raises(ValueError):
        dc.conv1d_causal(x, w, state=torch.zeros(1, 3, 16, device="cuda"))                  # fewer slots than sequences
    with pytest.raises(B.ConvError):
        dc.conv1d_causal(x, normal(16, 1))
    with pytest.raises(B.ConvError):
        dc.conv1d_causal(x, w, out=x)
    torch.manual_seed(0)
    t = scan_inputs(normal, (2, 8), 16, 4, 1, torch.float32)
    for name, value in [("a", t["a"].half()), ("b", t["b"][:, :4]), ("c", t["c"].half()), ("d", t["d"][:8]),
                        ("dt", t["dt"][:1]), ("z", t["z"].cpu()), ("dt_bias", t["dt_bias"].double())]:
        with pytest.raises((TypeError, ValueError)):
            dc.selective_scan(**dict(t, **{name: value}))
    with pytest.raises(ValueError):
        dc.selective_scan(**t, state=torch.zeros(2, 16, 5, device="cuda"))
    with pytest.raises(B.ConvError):
        dc.selective_scan(**t, out=t["z"])
    long = scan_inputs(normal, (1, 600), 16, 4, 1, torch.float32)
    with pytest.raises(ValueError):
        dc.selective_scan(**long, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


@gpu
def test_empty_calls():
    x = torch.empty(0, 5, 8, device="cuda")
    w = torch.zeros(8, 4, device="cuda")
    assert dc.conv1d_causal(x, w).shape == (0, 5, 8)
    assert dc.conv1d_causal_step(x[:, 0], w, torch.zeros(1, 3, 8, device="cuda")).shape == (0, 8)
    b = torch.empty(0, 5, 1, 4, device="cuda")
    assert dc.selective_scan(x, x, w, b, b).shape == (0, 5, 8)
    empty = torch.empty(0, 8, device="cuda")
    off = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert dc.conv1d_causal(empty, w, offsets=off).shape == (0, 8)


@gpu
def test_many_short_sequences():
    """Thousands of packed sequences of none to three tokens, and slots in any order."""
    torch.manual_seed(23)
    lens = torch.randint(0, 4, (2500,)).tolist()
    order = torch.randperm(2502)[:2500].tolist()
    check_conv(torch.float16, 4, 16, lens, True, True, True, True, tail=5, slots=order)
    check_scan(torch.bfloat16, 9, 6, 1, lens, True, True, tail=5, slots=order)


@gpu
@pytest.mark.parametrize("lens,slots", [([300, 0, 5, 270], [5, -1, 0, 2]), ([500, 40], [7, 1])])
def test_cut_scan_with_slots(lens, slots):
    assert B.selective_scan_workspace_size(B.ScanDesc(len(lens), sum(lens) + 2, 12, 16, 2, packed=1), 0, 0) > 0
    for carry in (False, True):
        check_scan(torch.float16, 12, 16, 2, lens, True, carry, tail=2, slots=slots, gap=3)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_scan_wide_states_over_many_tiles(dtype):
    """More tiles than the rings of b and c hold, at the widest states."""
    for s in (100, 200, 256):
        check_scan(TYPES[dtype], 70, s, 1, [200, 131], True, True, seed=s)


@gpu
def test_broadcast_inputs_and_strided_outputs():
    """One x for every sequence (batch stride 0), outputs into a slice of wider rows."""
    normal = draws(25)
    torch.manual_seed(25)
    x = normal(1, 50, 24, dtype=torch.bfloat16).expand(3, 50, 24)
    w = normal(24, 4, dtype=torch.bfloat16)
    wide = torch.full((3, 50, 40), 7.0, dtype=torch.bfloat16, device="cuda")
    got = dc.conv1d_causal(x, w, out=wide[..., 8:32])
    assert torch.equal(got, dc.conv1d_causal(x.contiguous(), w))
    assert (wide[..., :8] == 7).all() and (wide[..., 32:] == 7).all()
    t = scan_inputs(normal, (3, 50), 24, 16, 1, torch.bfloat16)
    want = dc.selective_scan(**dict(t, x=x.contiguous()), softplus=True)
    wide.fill_(7.0)
    got = dc.selective_scan(**dict(t, x=x), softplus=True, out=wide[..., 3:27])
    assert torch.equal(got, want) and (wide[..., :3] == 7).all() and (wide[..., 27:] == 7).all()


@gpu
def test_two_calls_at_once():
    """Cut scans, each with a workspace of its own, side by side on two streams."""
    normal = draws(27)
    torch.manual_seed(27)
    inputs = [scan_inputs(normal, (1, 4000), 32, 16, 1, torch.float32) for _ in range(2)]
    want = [dc.selective_scan(**t, softplus=True) for t in inputs]
    streams = [torch.cuda.Stream() for _ in inputs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for t, s in zip(inputs, streams):
            with torch.cuda.stream(s):
                got.append(dc.selective_scan(**t, softplus=True))
        torch.cuda.synchronize()
        assert all(torch.equal(g, v) for g, v in zip(got, want))


@gpu
def test_infinite_input_with_states_that_do_not_fill_the_lanes():
    """An infinite x gives the states that exist infinities and the others nothing: the
    outputs are infinite, not NaN, where b and c agree in sign; prompt and step alike."""
    normal = draws(29)
    torch.manual_seed(29)
    for s in (3, 5, 11, 20, 70):
        t = scan_inputs(normal, (2, 20), 8, s, 1, torch.float32, gate=False)
        t["b"], t["c"] = t["b"].abs() + 0.1, t["c"].abs() + 0.1
        t["x"] = t["x"].abs()
        t["x"][0, 7, 2] = float("inf")
        got = dc.selective_scan(**t, softplus=True)
        assert (got[0, 7:, 2] == float("inf")).all() and got[0, :7].isfinite().all() and got[1].isfinite().all()
        state = torch.zeros(2, 8, s, device="cuda")
        one = {k: v if k in ("a", "d", "dt_bias") or v is None else v[:, 7] for k, v in t.items()}
        step = dc.selective_scan_step(**one, state=state, softplus=True)
        assert step[0, 2] == float("inf") and state[0, 2].eq(float("inf")).all() and step[1].isfinite().all()


@gpu
def test_the_same_slot_twice_stays_inside():
    """What such a slot holds is unspecified; nothing else changes."""
    normal = draws(31)
    torch.manual_seed(31)
    t = scan_inputs(normal, (3,), 16, 16, 1, torch.float32)
    guard = Guarded(5 * 16 * 16 * 4, "cuda")
    state = guard.tensor((5, 16, 16), torch.float32)
    state.copy_(normal(5, 16, 16))
    before = state.clone()
    dc.selective_scan_step(**t, state=state, softplus=True, slots=torch.tensor([1, 1, 4], dtype=torch.int32, device="cuda"))
    window = normal(5, 3, 16)
    kept = window.clone()
    dc.conv1d_causal_step(t["x"], normal(16, 4), window, slots=torch.tensor([2, 2, 0], dtype=torch.int32, device="cuda"))
    guard.assert_intact("state")
    assert torch.equal(state[[0, 2, 3]], before[[0, 2, 3]]) and torch.equal(window[[1, 3, 4]], kept[[1, 3, 4]])


@gpu
def test_log_line(capfd, monkeypatch):
    """B200CONV_LOG=1 prints one line a call, like the convolutions."""
    monkeypatch.setenv("B200CONV_LOG", "1")
    normal = draws(33)
    torch.manual_seed(33)
    t = scan_inputs(normal, (1, 700), 16, 16, 1, torch.bfloat16)
    dc.selective_scan(**t, softplus=True)
    dc.conv1d_causal(t["x"], normal(16, 4, dtype=torch.bfloat16), activation="silu")
    lines = [line for line in capfd.readouterr().err.splitlines() if line.startswith("b200conv:")]
    assert len(lines) == 2 and "selective_scan n1 l700 d16 s16 g1 bf16" in lines[0] and "chunks=" in lines[0]
    assert "conv1d_causal n1 l700 c16 k4 bf16" in lines[1]


@gpu
def test_kernels_are_timed_by_name():
    normal = draws(35)
    torch.manual_seed(35)
    t = scan_inputs(normal, (1, 30), 16, 16, 1, torch.bfloat16)
    assert B.conv_profile_begin() == 0
    dc.selective_scan(**t, softplus=True)
    dc.conv1d_causal(t["x"], normal(16, 4, dtype=torch.bfloat16))
    times = B.profile_end()
    assert times["selective_scan"][0] == 1 and times["causal_conv"][0] == 1


@gpu
def test_conv_long_walks():
    """Calls large enough for walks of 64, 32 and 16 rows."""
    check_conv(torch.bfloat16, 4, 4096, [3001, 3001], False, True, True, True, gap=64)
    check_conv(torch.float16, 3, 4096, [700, 0, 1, 1500, 897], True, True, False, True, tail=2)
    check_conv(torch.float32, 4, 512, [3000, 31, 33, 2, 3134], True, False, True, False, tail=1)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_scan_more_blocks_than_sms(dtype):
    check_scan(TYPES[dtype], 40, 16, 1, [70] * 90, False, True)
    check_scan(TYPES[dtype], 2400, 16, 1, [33, 100, 0, 64], True, False, tail=1)
