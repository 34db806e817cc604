"""The sequence operators at the edges of fp32's range, against their definitions
in 64 bits (tests/sequence_ref.py, where the tolerances come from)."""
import pytest
import torch

import dense_convolution_nhwc_b200 as dc
from dense_convolution_nhwc_b200 import binding as B
from tests import sequence_ref as ref
from tests.gpu_util import Guarded, guarded_input
from tests.test_sequence import (BIAS, OUT, STATE, TYPES, W, X, check_scan, conv_desc, cpu, draws, scan_desc, scan_inputs,
                                 scan_tensors)

B200 = B.DeviceProps(148, 10, 0, 183359 * 2 ** 20)
gpu = pytest.mark.gpu


def chunk_tokens(n, l, d, s, packed=False):
    """Tokens of a chunk, or None for a call that is not cut."""
    plan = B.ScanPlan()
    assert B.selective_scan_plan_for_props(B.ScanDesc(n, l, d, s, 1, packed=int(packed)), 0, B200, plan) == 0
    return plan.chunk_tokens if plan.chunks > 1 else None


# ------------------------- cut scans: a chunk's decay ---------------------------
#
# A cut scan carries a state over a chunk of 64 tokens with exp(a times the sum of
# delta).  That leaves fp32's range where no token's own decay does, and the result
# has to be the definition's all the same.  Bounds: the reference's, token by token.  The three
# factors of a third of the exponent are off by 3 * 4 u and, through their arguments,
# by 3 |arg| u and the sum's own rounding; with their 3 u, that is below what the reference
# counts for 64 tokens one after the other, 64 (4 + 2) u + 3 |arg| u.

def exponents(dtype, length, per_token, seed):
    """Inputs without a gate whose token t multiplies state s by exp(per_token[t] (s + 1) / 16)."""
    normal = draws(seed)
    t = dict(x=normal(1, length, 24, dtype=dtype), b=normal(1, length, 1, 16, dtype=dtype),
             c=normal(1, length, 1, 16, dtype=dtype))
    t["dt"] = -per_token.to(dtype).cuda()[None, :, None].expand(1, length, 24).contiguous()
    t["a"] = -(torch.arange(1, 17) / 16.0).repeat(24, 1).cuda()
    assert chunk_tokens(1, length, 24, 16) == 64
    return t


def check(t, state=None):
    carry = state is not None
    start = state.cpu() if carry else torch.zeros(1, 24, 16)
    state = state.clone() if carry else torch.full((1, 24, 16), float("nan"), device="cuda")
    got = dc.selective_scan(**t, state=state, carry=carry)
    part = {name: cpu(v) if name == "a" else cpu(v)[0] for name, v in t.items()}
    y, bound, last, last_bound = ref.scan(**part, d=None, z=None, dt_bias=None, softplus=False, h=start[0])
    ref.assert_within(got[0], y, bound, "out")
    ref.assert_within(state[0], last, last_bound + 2.0 ** -149, "state")


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_zero_states_through_growing_chunks(dtype):
    """exp(96) over a chunk, and nothing to multiply by it until the last 40 tokens."""
    t = exponents(TYPES[dtype], 700, torch.full((700,), 1.5), 1)
    t["x"][:, :660] = 0
    check(t)


@gpu
@pytest.mark.parametrize("size,rate", [(1e-30, 1.5), (1e-40, 2.375), (0.0, 6.0)])
def test_small_states_through_a_growing_chunk(size, rate):
    """States, a subnormal one too, that a growth past fp32's range brings back into it; later tokens leave them be."""
    per_token = torch.zeros(200)
    per_token[:64] = rate
    t = exponents(torch.float32, 200, per_token, 3)
    t["x"].zero_()
    check(t, (torch.randn(1, 24, 16, generator=torch.Generator().manual_seed(3)) * size).cuda())


@gpu
def test_large_states_through_a_decaying_chunk():
    """A decay of exp(-102), below fp32's range, of states of 1e30 is not nothing."""
    per_token = torch.zeros(200)
    per_token[:64] = -1.59375
    t = exponents(torch.float32, 200, per_token, 5)
    t["x"].zero_()
    check(t, (torch.randn(1, 24, 16, generator=torch.Generator().manual_seed(5)) * 1e30).cuda())


@gpu
def test_exponents_of_both_signs():
    """Chunks that grow by exp(48) and shrink again."""
    per_token = torch.tensor([1.5] * 32 + [-1.5] * 32).repeat(5)
    check(exponents(torch.float32, 320, per_token, 7), draws(7)(1, 24, 16))


@gpu
@pytest.mark.parametrize("carried", [False, True])
def test_infinite_states_through_decaying_chunks(carried):
    """An infinite input, or a carried infinity, stays one to the sequence's end although
    a chunk decays by exp(-150): cut and uncut calls give the same outputs."""
    torch.manual_seed(9)
    t = scan_inputs(draws(9), (1, 700), 24, 16, 1, torch.float32, gate=False)
    t["b"], t["c"], t["x"] = t["b"].abs() + 0.1, t["c"].abs() + 0.1, t["x"].abs()
    t["dt"], t["dt_bias"] = torch.full_like(t["dt"], 0.125), None
    state = torch.zeros(1, 24, 16, device="cuda")
    if carried:
        state[0, 2] = float("inf")
    else:
        t["x"][0, 7, 2] = float("inf")
    assert chunk_tokens(1, 700, 24, 16) == 64 and chunk_tokens(90, 700, 24, 16) is None
    many = {name: v if name == "a" or v is None else v.expand(90, *v.shape[1:]) for name, v in t.items()}
    states = state.repeat(90, 1, 1)
    got, want = dc.selective_scan(**t, state=state, carry=True), dc.selective_scan(**many, state=states, carry=True)
    first = 0 if carried else 7
    for y, h in ((got[0], state[0]), (want[89], states[89])):
        assert (y[first:, 2] == float("inf")).all() and (h[2] == float("inf")).all()
        others = [i for i in range(24) if i != 2]
        assert y[:, others].isfinite().all() and h[others].isfinite().all() and y[:first].isfinite().all()


# -------------------------------- silu, far out ---------------------------------
#
# exp(-v) leaves fp32's range from v = -88.7 on, and the reciprocal of 1 + exp(-v) from
# -87.3, where silu(v) is still a normal number (down to -91.9; above 2^-149 to -108).
# The reference's bound is relative, with the type's smallest step at the final
# rounding (2^-149 of fp32).  A gate's sigmoid, and for steps the gate, is held in fp32
# before it is multiplied on.  Below 2^-126, for z < -87.3, that is a multiple of 2^-149
# and off by up to 2^-150, which the z and the 0.75 that it meets here multiply.

FAR = [-80.0, -84.0, -87.0, -87.5, -88.0, -88.75, -89.0, -90.0, -91.5, -92.0, -95.0, -100.0, -103.0, -104.0, -106.0, -112.0,
       -130.0, -1e4, -1e30, 80.0, 88.0, 100.0, 1e4, 1e30, 0.0, -0.0, 2.0 ** -120, -2.0 ** -120, -1.0, 1.0, -20.0, 20.0]


def far_values(dtype):
    """Each of FAR beside ordinary values, and in the place of both neighbours of a pair."""
    v = torch.tensor(FAR)
    v = v[v.abs() <= torch.finfo(dtype).max]
    return torch.cat([v, v.repeat_interleave(2), torch.stack([v, torch.full_like(v, 0.5)]).T.flatten()]).to(dtype)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [0, 3])
def test_activation_far_out(dtype, width):
    """silu of a conv that passes its input on, over prompts and steps, 16-byte accesses and single elements."""
    v = far_values(TYPES[dtype])
    v = v[:v.numel() // 8 * 8 - width]
    w = torch.tensor([0.0, 1.0]).repeat(v.numel(), 1).to(v.dtype)
    y, bound = ref._silu(v.double()[None], torch.zeros(1, v.numel(), dtype=torch.float64))      # 0 x' + 1 x is exact
    bound = ref._cast(y, bound, v.dtype)
    got = dc.conv1d_causal(v.cuda()[None, None], w.cuda(), activation="silu")
    ref.assert_within(got[0], y, bound, "prompt")
    got = dc.conv1d_causal_step(v.cuda()[None], w.cuda(), torch.zeros(1, 1, v.numel(), dtype=v.dtype, device="cuda"),
                                activation="silu")
    ref.assert_within(got, y, bound, "step")


def held(z):
    return torch.where(z < -87.3, 0.75 * z.double().abs() * 2.0 ** -150, 0.0)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 64])
def test_gate_far_out(dtype, n):
    """silu(z) 0.75: b is zero and d x is 0.75, over prompts and steps (64: blocks that walk over sequences)."""
    z = far_values(TYPES[dtype])
    dim, s = z.numel(), 16
    one = dict(x=torch.ones(1, dim), dt=torch.zeros(1, dim), b=torch.zeros(1, 1, s), c=torch.ones(1, 1, s), z=z[None])
    one = {name: v.to(z.dtype) for name, v in one.items()}
    fixed = dict(a=-torch.ones(dim, s), d=torch.full((dim,), 0.75))
    y, bound, _, _ = ref.scan(**one, **fixed, dt_bias=None, softplus=True, h=torch.zeros(dim, s))
    bound = bound + held(one["z"])
    fixed = {name: v.cuda() for name, v in fixed.items()}
    many = {name: v.cuda().expand(n, *v.shape[1:]).contiguous() for name, v in one.items()}
    got = dc.selective_scan(**{name: v[:, None] for name, v in many.items()}, **fixed, softplus=True)
    ref.assert_within(got[:, 0], y.expand(n, dim), bound.expand(n, dim), "prompt")
    got = dc.selective_scan_step(**many, **fixed, state=torch.zeros(n, dim, s, device="cuda"), softplus=True)
    ref.assert_within(got, y.expand(n, dim), bound.expand(n, dim), "step")


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("c", [24, 21])
@pytest.mark.parametrize("carry", [False, True])
def test_activations_far_out_anywhere_in_a_prompt(dtype, c, carry):
    """Whole and half numbers, whose sums are exact: some 15 % of them lie below -80, in
    the first rows that read the old window, at a sequence's end, between two walks."""
    g = torch.Generator().manual_seed(11)
    lens = [37, 3, 0, 1, 150]
    x = torch.randint(-90, 91, (sum(lens) + 2, c), generator=g).to(TYPES[dtype])
    w = (torch.randint(0, 2, (c, 4), generator=g) - 0.5).to(x.dtype)
    w[:, 3] = 1
    bias = torch.randint(-4, 5, (c,), generator=g).to(x.dtype)
    window = torch.randint(-90, 91, (len(lens), 3, c), generator=g).to(x.dtype)
    offsets = [sum(lens[:i]) for i in range(len(lens) + 1)]
    state, out = window.cuda(), torch.full_like(x, 7.0, device="cuda")
    dc.conv1d_causal(x.cuda(), w.cuda(), bias.cuda(), "silu", offsets=torch.tensor(offsets, dtype=torch.int32).cuda(),
                     state=state, carry=carry, out=out)
    far = 0
    for i, lo in enumerate(offsets[:-1]):
        old = window[i] if carry else torch.zeros_like(window[i])
        rows = x[lo:lo + lens[i]]
        v, _, kept = ref.causal_conv(rows, w, bias, False, old)
        y, bound = ref._silu(v, torch.zeros_like(v))
        far += int((v < -87.4).sum())
        ref.assert_within(out[lo:lo + lens[i]], y, ref._cast(y, bound, x.dtype), f"sequence {i}")
        assert torch.equal(state[i].cpu(), kept)
    assert far > 200 and (out[offsets[-1]:] == 7).all()


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [40, 37])
def test_gates_far_out_anywhere_in_a_prompt(dtype, dim):
    """Several tiles of tokens, whole vectors of channels and the ends of them."""
    far, g = far_values(TYPES[dtype]), torch.Generator().manual_seed(13)
    z = far[torch.randint(0, far.numel(), (2, 75, dim), generator=g)]
    t = dict(x=torch.ones(2, 75, dim), dt=torch.zeros(2, 75, dim), b=torch.zeros(2, 75, 1, 16), c=torch.ones(2, 75, 1, 16), z=z)
    t = {name: v.to(z.dtype) for name, v in t.items()}
    fixed = dict(a=-torch.ones(dim, 16), d=torch.full((dim,), 0.75))
    got = dc.selective_scan(**{name: v.cuda() for name, v in (t | fixed).items()}, softplus=True)
    for i in range(2):
        part = {name: v[i] for name, v in t.items()}
        y, bound, _, _ = ref.scan(**part, **fixed, dt_bias=None, softplus=True, h=torch.zeros(dim, 16))
        ref.assert_within(got[i], y, bound + held(z[i]), f"sequence {i}")


# ------------------------------- layouts of out ---------------------------------

@pytest.mark.parametrize("stride", [(8, 15), (15, 8), (7, 40), (40, 7), (0, 8), (8, 8), (39, 8), (8, 0)])
def test_rows_of_out_may_not_overlap(stride):
    """Two sequences of five rows of eight: neither within its own span."""
    assert B.conv1d_causal_forward(X, W, BIAS, 0, STATE, 0, OUT, conv_desc(out_stride=stride), 0, 0) == 1
    assert B.selective_scan_forward(scan_tensors(), scan_desc(out_stride=stride), 0, 0, 0, 0) == 1


@pytest.mark.parametrize("stride", [(2 ** 62, 8), (40, 2 ** 61), (2 ** 60, 8), (40, 2 ** 58)])
def test_strides_past_any_memory(stride):
    """Spans that 64 bits do not hold, or no memory has, are refused, not wrapped around."""
    for name in ("x_stride", "out_stride"):
        assert B.conv1d_causal_forward(X, W, BIAS, 0, STATE, 0, OUT, conv_desc(n=3, state_slots=3, **{name: stride}), 0, 0) == 1
    for name in ("x_stride", "dt_stride", "z_stride", "b_stride", "c_stride", "out_stride"):
        desc = scan_desc(n=3, state_slots=3, **{name: stride})
        assert B.selective_scan_forward(scan_tensors(), desc, 0, 0, 0, 0) == 1
    step = conv_desc(n=3, state_slots=3, x_stride=(2 ** 62, 0))
    assert B.conv1d_causal_step_forward(X, W, 0, STATE, 0, OUT, step, 0, 0) == 1


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim,gap", [(24, 0), (24, 8), (21, 3)])
def test_out_token_by_token(dtype, dim, gap):
    """Outputs, and inputs, that are transposed [L, N, C] buffers."""
    normal, n, l = draws(15), 3, 70
    torch.manual_seed(15)
    buffer = torch.full((l, n, dim + gap), 7.0, dtype=TYPES[dtype], device="cuda")
    out = buffer[..., :dim].transpose(0, 1)
    x, w = normal(n, l, dim, dtype=buffer.dtype), normal(dim, 4, dtype=buffer.dtype)
    want = dc.conv1d_causal(x, w, activation="silu")
    across = x.transpose(0, 1).contiguous().transpose(0, 1)
    assert dc.conv1d_causal(across, w, activation="silu", out=out) is out
    assert torch.equal(out, want) and (buffer[..., dim:] == 7).all()
    t = scan_inputs(normal, (n, l), dim, 16, 1, buffer.dtype)
    want = dc.selective_scan(**t, softplus=True)
    buffer.fill_(7.0)
    dc.selective_scan(**dict(t, x=t["x"].transpose(0, 1).contiguous().transpose(0, 1)), softplus=True, out=out)
    assert torch.equal(out, want) and (buffer[..., dim:] == 7).all()


# ----------------------- chunks that are no multiple of 64 ----------------------

def test_chunks_are_whole_tiles_of_32():
    assert chunk_tokens(1, 380, 1900, 16) == 96 and chunk_tokens(11, 10813, 48, 16, packed=True) == 96


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("carry", [False, True])
def test_chunks_of_an_odd_number_of_tiles(dtype, carry):
    """Four chunks of 96 tokens, the last one of 92; and packed, 97 tokens and one chunk exactly."""
    check_scan(TYPES[dtype], 1900, 16, 1, [380], False, carry)
    lens = [97, 0, 96, 350]
    assert chunk_tokens(4, sum(lens) + 2, 1000, 16, packed=True) == 96
    check_scan(TYPES[dtype], 1000, 16, 1, lens, True, carry, tail=2)


# ------------------- what a call has no business to read or write ----------------

@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [50, 700])
def test_bad_offsets_read_and_write_nothing_outside(dtype, rows):
    """Every input between NaN bands and every output between canaries, offsets that
    descend, are negative or point behind the rows: all that is there stays finite.
    700 rows: scans that are cut."""
    dtype, d, s = TYPES[dtype], 16, 16
    assert (chunk_tokens(3, rows, d, s, packed=True) is not None) == (rows == 700)
    normal = draws(41)
    torch.manual_seed(41)
    t = scan_inputs(normal, (rows,), d, s, 1, dtype)
    w, bias = normal(d, 4, dtype=dtype), normal(d, dtype=dtype)
    first = [normal(3, 3, d, dtype=dtype), normal(3, d, s)]
    guards = {}
    for name, v in t.items():
        guards[name], t[name] = guarded_input(v.contiguous())
    guards["w"], w = guarded_input(w)
    guards["bias"], bias = guarded_input(bias)
    for offsets in ([0, 40, 20, 50], [-5, 10, 900, 50], [60, 70, 80, 90], [50, 30, 10, 0], [-9, -8, -7, -6],
                    [0, rows, rows // 3, rows], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, -2 ** 31], [-2 ** 31, 2 ** 31 - 1, 0, 5]):
        guards["offsets"], off = guarded_input(torch.tensor(offsets, dtype=torch.int32).cuda())
        for carry in (False, True):
            def buffers(like):
                g_out, g_state = Guarded(rows * d * t["x"].element_size(), "cuda"), Guarded(like.numel() * like.element_size(), "cuda")
                out, state = g_out.tensor((rows, d), dtype), g_state.tensor(tuple(like.shape), like.dtype)
                out.fill_(7.0)
                state.copy_(like)
                return g_out, g_state, out, state
            made = [buffers(like) for like in first]
            dc.conv1d_causal(t["x"], w, bias, "silu", offsets=off, state=made[0][3], carry=carry, out=made[0][2])
            dc.selective_scan(**t, softplus=True, offsets=off, state=made[1][3], carry=carry, out=made[1][2])
            torch.cuda.synchronize()
            for what, (g_out, g_state, out, state) in zip(("conv", "scan"), made):
                g_out.assert_intact(f"{what} out {offsets}")
                g_state.assert_intact(f"{what} state {offsets}")
                assert out.isfinite().all() and state.isfinite().all(), (what, offsets)
            for name, guard in guards.items():
                guard.assert_intact(name)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("carry", [False, True])
def test_windows_of_other_slots_keep_their_values(dtype, carry):
    """Prompts and steps into scattered slots, one left out: every other window is the same to the bit."""
    normal, dtype = draws(43), TYPES[dtype]
    lens, slots = [5, 40, 3, 0, 7, 33], [8, 0, -1, 3, 99, 5]
    x, w = normal(sum(lens), 32, dtype=dtype), normal(32, 4, dtype=dtype)
    offsets = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32).cuda()
    where = torch.tensor(slots, dtype=torch.int32).cuda()
    before = normal(10, 3, 32, dtype=dtype)
    others = [i for i in range(10) if i not in slots]
    state = before.clone()
    dc.conv1d_causal(x, w, offsets=offsets, state=state, slots=where, carry=carry)
    assert torch.equal(state[others], before[others]) and not torch.equal(state[[8, 0, 5]], before[[8, 0, 5]])
    assert torch.equal(state[3], before[3] if carry else torch.zeros_like(before[3]))
    state = before.clone()
    dc.conv1d_causal_step(x[:6], w, state, slots=where)
    assert torch.equal(state[others], before[others]) and torch.equal(state[[8, 0, 3, 5], 2], x[[0, 1, 3, 5]])
