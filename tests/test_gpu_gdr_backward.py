"""Backward of the gated delta rule on the GPU against fp64 autograd of the
token recurrence, and against differences of its forward.

Tolerances (2-norm, relative), as for the forward: an fp32 gradient of bf16
inputs passes the forward's chain, the reverse chain and the gradient's own
products, three times the roundings of a state, rounded up to a power of two:
2^-13; bf16 gradients add one rounding of 2^-8.  fp32 inputs (and bf16 calls of
at most 128 token-head pairs, held to the same bounds as longer ones) run in
fp64 and round their gates (2^-24, over up to 2^8 tokens), intermediates to fp32 and the
result once: 2^-18."""
import pytest
import torch

import gated_delta_rule_22_amd as ck
from _gdr_ref import gdr, inputs, rel

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dS0")


def tol(name, dtype):
    if dtype == F32:
        return 2.0 ** -18
    return 2.0 ** -8 + 2.0 ** -13 if name in ("dq", "dk", "dv") else 2.0 ** -13


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def upstream(seed, x, lens, dtype, with_state=True):
    r = torch.Generator().manual_seed(seed)
    do = torch.randn(x["v"].shape, generator=r).to(dtype)
    n, (hv, dv), dk = len(lens), x["v"].shape[1:], x["q"].shape[2]
    return do, 0.3 * torch.randn(n, hv, dk, dv, generator=r) if with_state else None


def wanted(x, do, dS, lens):
    leaves = [x[n].double().requires_grad_() for n in ("q", "k", "v", "g", "beta")]
    S0 = x["S0"]
    if S0 is None:
        S0 = torch.zeros(len(lens), x["v"].shape[1], x["q"].shape[2], x["v"].shape[2])
    S0 = S0.double().requires_grad_()
    o, S = gdr(*leaves, S0, lens)
    loss = (o * do.double()).sum()
    if dS is not None:
        loss = loss + (S * dS.double()).sum()
    got = torch.autograd.grad(loss, leaves + [S0], allow_unused=True)
    return [torch.zeros_like(y) if z is None else z for y, z in zip(leaves + [S0], got)]


def run(x, do, dS, lens, cu=None, **kw):
    d = {n: None if t is None else t.cuda() for n, t in x.items()}
    lead = [d[n][None] for n in ("q", "k", "v", "g", "beta")]
    print("gdr_backward", lens, x["q"].dtype, tuple(x["q"].shape), tuple(x["v"].shape), flush=True)
    got = ck.gdr_backward(*lead, do.cuda()[None], S0=d["S0"], dS_T=None if dS is None else dS.cuda(),
                          cu_seqlens=offsets(lens) if cu is None else cu, **kw)
    torch.cuda.synchronize()
    return [t[0] for t in got[:5]] + [got[5]]


def check(x, lens, dtype, seed=0, with_state=True):
    do, dS = upstream(seed, x, lens, dtype, with_state)
    got, want = run(x, do, dS, lens), wanted(x, do, dS, lens)
    for n, a, b in zip(NAMES, got, want):
        assert rel(a, b) < tol(n, dtype), (n, rel(a, b))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens", [[1], [2], [16], [63], [64], [65], [128], [150], [0, 5, 0, 64, 1, 130, 0]])
def test_lengths(lens, dtype):
    check(inputs(len(lens) + lens[-1], lens, 1, 2, 128, 128, dtype), lens, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("hk,hv", [(1, 1), (2, 6), (3, 3)])
def test_heads_and_dims(hk, hv, dk, dv, dtype):
    """Gradients of shared query/key heads are sums over their value heads."""
    check(inputs(3, [97, 33], hk, hv, dk, dv, dtype), [97, 33], dtype, 1)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("beta", [1.0, 2.0])
@pytest.mark.parametrize("gate", ["one", "fast"])
def test_gates(gate, beta, dtype):
    """Includes a token with beta = 0 (inputs() puts one in the middle)."""
    check(inputs(5, [150], 2, 4, 128, 64, dtype, gate, beta), [150], dtype, 2)


# Calls of more than 1024 tokens times value heads: bf16 takes the chunkwise path.
@pytest.mark.parametrize("lens", [[1025], [64] * 17, [63, 0, 65, 1, 700, 2, 200], [1] * 1030])
def test_lengths_in_chunks(lens):
    check(inputs(23 + len(lens), lens, 1, 1, 128, 128, BF), lens, BF)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("hk,hv", [(1, 4), (3, 9), (5, 5)])
def test_heads_and_dims_in_chunks(hk, hv, dk, dv):
    check(inputs(25, [197, 133], hk, hv, dk, dv, BF), [197, 133], BF)


@pytest.mark.parametrize("gate", ["one", "fast", "resets"])
@pytest.mark.parametrize("beta", [1.0, 2.0])
def test_gates_in_chunks(gate, beta):
    lens = [350]
    x = inputs(27, lens, 2, 4, 128, 64, BF, gate, beta)
    x["g"] = x["g"].clamp(min=-1e4)      # the reference has no derivative at -infinity
    check(x, lens, BF)


def test_chunks_repeat_and_keep_to_their_rows():
    """Rows outside the sequences stay, a head's NaN stays in it, reruns give the same bits."""
    lens = [300, 170]
    x = inputs(29, [600], 2, 4, 64, 128, BF)
    x["S0"] = x["S0"].repeat(2, 1, 1, 1)
    do, dS = upstream(11, x, lens, BF)
    cu = torch.tensor([0, 300, 470], dtype=torch.int32, device="cuda")
    one = run(x, do, dS, lens, cu=cu)
    two = run(x, do, dS, lens, cu=cu)
    for a, b in zip(one[:5], two[:5]):
        assert torch.equal(a[:470], b[:470])
    assert torch.equal(one[5], two[5])
    x["v"][20, 1] = float("nan")
    got = run(x, do, dS, lens, cu=cu)
    for a, b, n in zip(got[:5], one[:5], NAMES):
        assert torch.equal(a[300:470], b[300:470]), n
    for i in (2, 3, 4):                  # dv, dg, dbeta of the other heads
        assert torch.equal(got[i][:300, [0, 2, 3]], one[i][:300, [0, 2, 3]])
    assert torch.isnan(got[3][:300, 1]).any()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_no_states(dtype):
    check(inputs(7, [70, 129], 2, 2, 64, 128, dtype, s0=False), [70, 129], dtype, 3, False)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens", [[1, 0, 1], [1] * 70, [70, 0, 129]])
def test_first_gate_of_a_zero_state(lens, dtype):
    """It scales nothing: its gradient is zero itself, not a rounding off."""
    x = inputs(11, lens, 1, 2, 64, 64, dtype, s0=False)
    do, dS = upstream(5, x, lens, dtype)
    dg = run(x, do, dS, lens)[3]
    first = [sum(lens[:i]) for i, n in enumerate(lens) if n]
    assert not dg[first].any()
    want = wanted(x, do, dS, lens)[3]
    assert rel(dg, want) < tol("dg", dtype)


@pytest.mark.parametrize("lens", [[140], [20]])
def test_resets(lens):
    """Log-gates of -infinity forget everything and have no gradient (the
    chunkwise path, and the fp64 one that short calls take)."""
    x = inputs(9, lens, 1, 2, 128, 128, BF, "resets")
    do, dS = upstream(4, x, lens, BF)
    got = run(x, do, dS, lens)
    y = dict(x, g=torch.where(torch.isinf(x["g"]), torch.full_like(x["g"], -1e4), x["g"]))
    want = wanted(y, do, dS, lens)
    assert not got[3][torch.isinf(x["g"]).cuda()].any()
    for n, a, b in zip(NAMES, got, want):
        assert rel(a, b) < tol(n, BF), (n, rel(a, b))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_against_differences(dtype):
    """The gradient along a random direction against a central difference of
    the fp64 forward: step 1e-5, error of order 1e-10 relative to the third
    derivative, far below the gradient's own tolerance (which is taken on the
    whole: the direction mixes all inputs, sizes within a factor of 2^4)."""
    lens = [75]
    x = inputs(11, lens, 1, 2, 64, 64, dtype)
    do, dS = upstream(5, x, lens, dtype)
    got = run(x, do, dS, lens)
    r = torch.Generator().manual_seed(6)
    names = ("q", "k", "v", "g", "beta", "S0")
    for name, grad in zip(names, got):
        step = torch.randn(x[name].shape, generator=r, dtype=torch.float64)
        # along the gradient itself, so that the sum is no small difference
        step = step * 0.1 + grad.double().cpu() / grad.double().cpu().norm() * step.norm() * 0.9

        def loss(sign):
            y = {n: t.double() for n, t in x.items()}
            y[name] = y[name] + sign * 1e-5 * step
            o, S = gdr(y["q"], y["k"], y["v"], y["g"], y["beta"], y["S0"], lens)
            return ((o * do.double()).sum() + (S * dS.double()).sum()).item()

        diff = (loss(1) - loss(-1)) / 2e-5
        mine = (grad.double().cpu() * step).sum().item()
        assert abs(diff - mine) <= 4 * tol("d" + name, dtype) * abs(diff), (name, diff, mine)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_rows_outside_sequences_and_skipped_state(dtype):
    x = inputs(13, [100], 1, 2, 64, 64, dtype, s0=False)
    do, _ = upstream(7, x, [100], dtype, False)
    cu = torch.tensor([10, 40, 30, 80], dtype=torch.int32, device="cuda")
    got = run(x, do, None, [100], cu=cu, need_dS0=False)
    part = {n: None if t is None else t[10:40] for n, t in x.items()}
    want = wanted(part, do[10:40], None, [30])
    assert got[5] is None
    for n, a, b in zip(NAMES[:5], got, want):
        assert rel(a[10:40], b) < tol(n, dtype), n


def test_repeat_and_other_stream():
    """The same bits again, and on another stream."""
    lens = [200, 64, 3]
    x = inputs(15, lens, 2, 4, 128, 128, BF)
    do, dS = upstream(8, x, lens, BF)
    a = run(x, do, dS, lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = run(x, do, dS, lens)
    s.synchronize()
    for y, z in zip(a, b):
        assert torch.equal(y, z)


def test_nan_stays_in_its_head():
    lens = [80, 80]
    x = inputs(17, lens, 2, 2, 64, 64, BF)
    do, dS = upstream(9, x, lens, BF)
    clean = run(x, do, dS, lens)
    x["v"][20, 1] = float("nan")
    got = run(x, do, dS, lens)
    for a, b in zip(got[:5], clean[:5]):
        assert torch.equal(a[:, 0], b[:, 0]) and torch.equal(a[80:], b[80:])
    assert torch.isnan(got[0][20:80, 1].float()).any()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_layer_run_through(dtype):
    """As a layer uses them: norm and rotation of a projection's q and k, the
    recurrence, and the gradients back to the projection and the weights."""
    from _gdr_ref import norm, rotate
    T, hk, hv, d = 100, 2, 4, 64
    r = torch.Generator().manual_seed(21)
    proj = torch.randn(1, T, 2 * hk, d, generator=r).to(dtype)
    x = inputs(22, [T], hk, hv, d, d, dtype)
    wq, wk = (1 + 0.1 * torch.randn(d, generator=r) for _ in range(2))
    pos = torch.arange(T, dtype=torch.int32)[None]
    f, _ = ck.rotary_frequencies(32)
    do = torch.randn(1, T, hv, d, generator=r).to(dtype)
    P, W, pd, fd = proj.cuda(), [wq.cuda(), wk.cuda()], pos.cuda(), f.cuda()
    opts = dict(norm="l2", q_weight=W[0], k_weight=W[1], q_scale=d ** -0.5)
    q, k = ck.qk_norm_rotary(P[:, :, :hk], P[:, :, hk:], pd, fd, **opts)
    rest = [x[n].cuda()[None] for n in ("v", "g", "beta")]
    o, S = ck.gdr_forward(q, k, *rest, S0=x["S0"].cuda())
    gq, gk, gv, gg, gb, gS = ck.gdr_backward(q, k, *rest, do.cuda(), S0=x["S0"].cuda())
    grad = torch.zeros_like(P)
    out = ck.qk_norm_rotary_backward(gq, gk, P[:, :, :hk], P[:, :, hk:], pd, fd, dq=grad[:, :, :hk],
                                     dk=grad[:, :, hk:], **opts)
    # In fp64 from the operands as the kernels hand them on (q and k rounded).
    p = proj.double().requires_grad_()
    w = [wq.double().requires_grad_(), wk.double().requires_grad_()]
    rq = rotate(norm(p[:, :, :hk], "l2", w[0]), pos, f, "half") * d ** -0.5
    rk = rotate(norm(p[:, :, hk:], "l2", w[1]), pos, f, "half")
    ro, _ = gdr(rq[0], rk[0], x["v"], x["g"], x["beta"], x["S0"], [T])
    want = torch.autograd.grad((ro * do[0].double()).sum(), [p, *w])
    # bf16: q and k are rounded on their way (2^-8 each, through keys twice),
    # their gradients on the way back, results once: 6 * 2^-8 at most
    t = 6 * 2.0 ** -8 if dtype == BF else 2.0 ** -17
    assert rel(o[0], ro) < t
    for a, b in zip((grad, out[2], out[3]), want):
        assert rel(a, b) < t, rel(a, b)
