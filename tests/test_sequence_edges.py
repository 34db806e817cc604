"""The sequence operators at the edges of fp32's range, against their definitions
in 64 bits (tests/sequence_ref.py, where the tolerances come from)."""
import pytest
import torch

import dense_convolution_nhwc_b200 as dc
from dense_convolution_nhwc_b200 import binding as B
from tests import sequence_ref as ref
from tests.test_sequence import TYPES, cpu, draws, scan_inputs

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
