"""Gated delta rule on the GPU against the fp64 token recurrence.

Tolerances (2-norm of the error over that of the result), from the roundings
the kernels make:

- fp32 results of bf16 inputs (states): every fp32 operand enters a product as
  two bf16 terms, off by at most 2^-18 of its value, and a product of two such
  operands drops lo * lo, another 2^-18.  A state passes three products a chunk
  (K S, T' X, K^T U) with two, three and two such errors: 8 * 2^-18 = 2^-15.
- bf16 outputs: the result and three operands are rounded to bf16, each by at
  most 2^-8; independent errors of that size, uniform within a step, add up to
  sqrt(4) * 2^-8 / sqrt(3) < 1.2 * 2^-8: 2^-7 holds them.
- fp32 inputs: sums of up to 128 products a token in fp32, 2^-24 each and
  random: sqrt(128) * 2^-24 per token and up to 16 tokens' worth of memory:
  2^-18."""
import pytest
import torch

import gated_delta_rule_22_amd as ck
from _gdr_ref import gdr, inputs, rel

pytestmark = pytest.mark.gpu

TOL = {torch.bfloat16: (2.0 ** -7, 2.0 ** -15), torch.float32: (2.0 ** -18, 2.0 ** -18)}
BF, F32 = torch.bfloat16, torch.float32


def dev(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def run(x, lens, **kw):
    d = dev(x)
    lead = {n: d[n][None] for n in ("q", "k", "v", "g", "beta")}
    o, S = ck.gdr_forward(**lead, S0=d["S0"], cu_seqlens=offsets(lens), **kw)
    torch.cuda.synchronize()
    return o[0], S


def check(x, lens, dtype):
    print("gdr_forward", lens, dtype, flush=True)
    o, S = run(x, lens)
    ro, rS = gdr(x["q"], x["k"], x["v"], x["g"], x["beta"], x["S0"], lens)
    to, ts = TOL[dtype]
    assert rel(o, ro) < to and rel(S, rS) < ts, (rel(o, ro), rel(S, rS))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens", [[1], [2], [17], [63], [64], [65], [128], [200], [0, 5, 0, 64, 1, 130, 0]])
def test_lengths(lens, dtype):
    check(inputs(len(lens) + lens[-1], lens, 1, 2, 128, 128, dtype), lens, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("hk,hv", [(1, 1), (2, 6), (3, 3)])
def test_heads_and_dims(hk, hv, dk, dv, dtype):
    check(inputs(3, [97, 33], hk, hv, dk, dv, dtype), [97, 33], dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("gate", ["one", "fast", "resets"])
@pytest.mark.parametrize("beta", [1.0, 2.0])
def test_gates(gate, beta, dtype):
    check(inputs(5, [150], 2, 4, 128, 64, dtype, gate, beta), [150], dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_rows_and_no_states(dtype):
    """Equal rows without cu_seqlens or S0, and without a final state."""
    B, T = 3, 70
    x = inputs(7, [T] * B, 2, 4, 64, 128, dtype, s0=False)
    d = dev(x)
    lead = {n: d[n].reshape(B, T, *d[n].shape[1:]) for n in ("q", "k", "v", "g", "beta")}
    o, S = ck.gdr_forward(**lead)
    o2, none = ck.gdr_forward(**lead, output_final_state=False)
    ro, rS = gdr(x["q"], x["k"], x["v"], x["g"], x["beta"], None, [T] * B)
    assert none is None and torch.equal(o, o2)
    assert rel(o.reshape(B * T, 4, 128), ro) < TOL[dtype][0]
    assert rel(S, rS) < TOL[dtype][1]


def test_many_sequences_and_heads():
    """More (sequence, head) pairs than a multiple of 8, longest first."""
    lens = [3, 0, 70, 1, 128, 9, 64, 65, 2, 31, 5]
    check(inputs(9, lens, 1, 3, 64, 64, BF), lens, BF)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_rows_behind_the_last_sequence_stay(dtype):
    x = inputs(11, [100], 1, 2, 64, 64, dtype, s0=False)
    d = dev(x)
    lead = {n: d[n][None] for n in ("q", "k", "v", "g", "beta")}
    out = torch.full((1, 100, 2, 64), 7.0, dtype=dtype, device="cuda")
    cu = torch.tensor([10, 40, 30, 80], dtype=torch.int32, device="cuda")   # decreases once
    o, S = ck.gdr_forward(**lead, cu_seqlens=cu, out=out)
    assert bool((o[0, :10] == 7).all()) and bool((o[0, 80:] == 7).all())
    part = {n: t[10:40] for n, t in x.items() if t is not None}
    ro, rS = gdr(**part, S0=None, lens=[30])
    assert rel(o[0, 10:40], ro) < TOL[dtype][0] and rel(S[0], rS[0]) < TOL[dtype][1]
    assert not S[1].any()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_nan_stays_in_its_head(dtype):
    x = inputs(13, [80, 80], 1, 2, 64, 64, dtype)
    clean, _ = run(x, [80, 80])
    for name in ("v", "g", "beta"):
        y = {n: None if t is None else t.clone() for n, t in x.items()}
        y[name][20, 1] = float("nan")
        o, S = run(y, [80, 80])
        assert torch.equal(o[:, 0], clean[:, 0]) and torch.equal(o[80:], clean[80:]), name
        assert bool(torch.isnan(o[20:80, 1].float()).any()), name
        assert not torch.isnan(S[:, 0]).any() and not torch.isnan(S[1]).any(), name


@pytest.mark.parametrize("dtype", [F32, BF])
def test_split_and_in_place_state(dtype):
    """Two calls with the state handed on, in place, against one call."""
    x = inputs(15, [192], 1, 2, 128, 128, dtype)
    o, S = run(x, [192])
    first = {n: (t if n == "S0" else t[:128]) for n, t in x.items()}
    d = dev(first)
    lead = {n: d[n][None] for n in ("q", "k", "v", "g", "beta")}
    state = d["S0"]
    a, _ = ck.gdr_forward(**lead, S0=state, final_state=state)
    d = dev({n: t[128:] for n, t in x.items() if n != "S0"})
    lead = {n: d[n][None] for n in ("q", "k", "v", "g", "beta")}
    b, _ = ck.gdr_forward(**lead, S0=state, final_state=state)
    assert torch.equal(torch.cat([a[0], b[0]]), o) and torch.equal(state, S)


def test_other_stream_and_repeat():
    x = inputs(17, [300, 20], 2, 4, 128, 128, BF)
    o, S = run(x, [300, 20])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o2, S2 = run(x, [300, 20])
    s.synchronize()
    assert torch.equal(o, o2) and torch.equal(S, S2)


# ------------------------------------------------------------------ single tokens
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("n,hk,hv", [(1, 1, 1), (3, 2, 6), (9, 1, 4)])
def test_step(n, hk, hv, dk, dv, dtype):
    x = inputs(19 + n, [1] * n, hk, hv, dk, dv, dtype)
    pool = n + 3
    S = 0.3 * torch.randn(pool, hv, dk, dv, generator=torch.Generator().manual_seed(1))
    slots = torch.randperm(pool, generator=torch.Generator().manual_seed(2))[:n].to(torch.int32)
    ro, rS = gdr(x["q"], x["k"], x["v"], x["g"], x["beta"], S[slots.long()], [1] * n)
    d = dev(x)
    Sd = S.cuda()
    print("gdr_decode_step", n, hk, hv, dk, dv, dtype, flush=True)
    o = ck.gdr_decode_step(d["q"], d["k"], d["v"], d["g"], d["beta"], Sd, slots=slots.cuda())
    assert rel(o, ro) < (2.0 ** -8 if dtype == BF else 2.0 ** -20)
    assert rel(Sd[slots.long().cuda()], rS) < 2.0 ** -20
    rest = [i for i in range(pool) if i not in slots.tolist()]
    assert torch.equal(Sd[rest].cpu(), S[rest])
    # without slots: row n has state n
    Sn = S[slots.long()].contiguous().cuda()
    o2 = ck.gdr_decode_step(d["q"], d["k"], d["v"], d["g"], d["beta"], Sn)
    assert torch.equal(o, o2) and torch.equal(Sn, Sd[slots.long().cuda()])


def test_step_padded_and_repeated_slots():
    """Slots outside the pool, and a slot named twice: padding, in order."""
    n, pool = 6, 4
    x = inputs(23, [1] * n, 1, 2, 64, 64, BF)
    S = 0.3 * torch.randn(pool, 2, 64, 64, generator=torch.Generator().manual_seed(3))
    slots = [2, -1, 0, 2, 4, 2 ** 31 - 1]
    d = dev(x)
    Sd = S.cuda()
    o = ck.gdr_decode_step(d["q"], d["k"], d["v"], d["g"], d["beta"], Sd,
                           slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    live = [0, 2]
    ro, rS = gdr(*(x[m][live] for m in ("q", "k", "v", "g", "beta")), S[[2, 0]], [1, 1])
    assert rel(o[live], ro) < 2.0 ** -8 and rel(Sd[[2, 0]], rS) < 2.0 ** -20
    assert not o[[1, 3, 4, 5]].any() and torch.equal(Sd[[1, 3]].cpu(), S[[1, 3]])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_prefill_then_steps(dtype):
    """A prompt, then tokens one by one, against one forward over all of them."""
    x = inputs(29, [90], 2, 4, 128, 64, dtype)
    ro, rS = gdr(x["q"], x["k"], x["v"], x["g"], x["beta"], x["S0"], [90])
    d = dev(x)
    lead = {n: d[n][None, :80] for n in ("q", "k", "v", "g", "beta")}
    o, S = ck.gdr_forward(**{n: t.contiguous() for n, t in lead.items()}, S0=d["S0"])
    out = [o[0]]
    for t in range(80, 90):
        out.append(ck.gdr_decode_step(*(d[n][t:t + 1] for n in ("q", "k", "v", "g", "beta")), S))
    assert rel(torch.cat(out), ro) < TOL[dtype][0] and rel(S, rS) < TOL[dtype][1]


@pytest.mark.parametrize("lens", [[900, 3, 0, 70, 64, 1, 33, 200, 65], [130] * 9, [2000] + [1] * 8,
                                  [3900, 3, 0, 170, 64, 1, 33, 200, 65], [470] * 9])
def test_packed_batches_long_and_even(lens):
    """More than 128 blocks of 64 columns: from 64 chunks on, how even the lengths are decides
    how a head's columns are cut, and results are the sequences' own either way."""
    hk, hv = 4, 16
    x = inputs(41, lens, hk, hv, 64, 64, BF)
    check(x, lens, BF)
    o, S = run(x, lens)
    at, n = sum(lens[:3]), lens[3]
    one = {m: x[m][at:at + n] for m in ("q", "k", "v", "g", "beta")}
    one["S0"] = x["S0"][3:4]
    oo, SS = run(one, [n])
    assert torch.equal(o[at:at + n], oo) and torch.equal(S[3:4], SS)
