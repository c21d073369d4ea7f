"""Norm of queries and keys with the rotation, its backward, and the rotation
alone, against fp64.

Tolerances: results are computed in fp32 and rounded once, so a bf16 result is
within half a step, 2^-8 of its size, and its fp32 part adds 2^-20 at most (a
sum of 256 squares, a root, cos and sin to 2^-22, four products); the same
2^-20 holds fp32 results and the weights' gradients (sums of up to 2^12 rows,
random errors)."""
import math

import pytest
import torch

import gated_delta_rule_22_amd as ck
from _gdr_ref import norm, rel, rotate

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL = {BF: 2.0 ** -8 + 2.0 ** -20, F32: 2.0 ** -20}
NO = torch.Generator


def data(seed, tokens, hq, hk, d, rd, dtype, packed=True, far=5000, weight=True):
    r = NO().manual_seed(seed)
    both = torch.randn(tokens, hq + 2 * hk, d, generator=r).to(dtype)
    q, k = both[:, :hq], both[:, hq:hq + hk]
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    pos = torch.randint(0, far, (tokens,), generator=r).to(torch.int32)
    freqs = 10000.0 ** (-torch.arange(0, rd, 2, dtype=torch.float64) / rd) if rd else None
    w = [1 + 0.2 * torch.randn(d, generator=r) for _ in range(2)] if weight else [None, None]
    return q, k, pos, freqs, *w


def cu(x, base=None):
    if x is None:
        return None
    if x.is_contiguous():
        return x.cuda()
    y = torch.empty(x.shape[0], x.stride(0), dtype=x.dtype, device="cuda")
    v = y[:, :x.shape[1] * x.shape[2]].unflatten(1, x.shape[1:])
    v.copy_(x)
    return v


SHAPES = [(1, 1, 1, 128, 128), (5, 4, 2, 64, 64), (37, 3, 1, 128, 64), (9, 2, 2, 96, 96),
          (9, 2, 2, 96, 24), (7, 2, 1, 256, 256), (7, 2, 1, 256, 34), (6, 1, 3, 80, 6),
          (11, 2, 2, 10, 4), (3, 2, 1, 2, 2), (4100, 2, 1, 128, 128), (33, 5, 0, 64, 32),
          (8, 0, 2, 128, 0)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,hq,hk,d,rd", SHAPES)
def test_norm_rotary_both_ways(tokens, hq, hk, d, rd, layout, dtype):
    kind = ["rms", "l2", "none"][(tokens + d) % 3]
    packed, weight = tokens % 2 == 1, d % 3 != 2
    q, k, pos, freqs, wq, wk = data(tokens + d, tokens, hq, hk, d, rd, dtype, packed, weight=weight)
    qs, rs = 0.37, 1.25
    opts = dict(norm=kind, layout=layout, q_scale=qs, rotary_scale=rs)
    print("qk_norm_rotary", tokens, hq, hk, d, rd, layout, kind, dtype, flush=True)
    dq, dk, dp, df = cu(q), cu(k), pos.cuda(), cu(freqs)
    dw = [cu(wq), cu(wk)]
    a, b = ck.qk_norm_rotary(dq, dk, dp, df, q_weight=dw[0], k_weight=dw[1], **opts)

    leaves = [q.double().requires_grad_(), k.double().requires_grad_()]
    ws = [None if w is None else w.double().requires_grad_() for w in (wq, wk)]
    ra = rotate(norm(leaves[0], kind, ws[0]), pos, freqs, layout, rs) * qs
    rb = rotate(norm(leaves[1], kind, ws[1]), pos, freqs, layout, rs)
    assert rel(a, ra) < TOL[dtype] and rel(b, rb) < TOL[dtype], (rel(a, ra), rel(b, rb))

    r = NO().manual_seed(1)
    ga, gb = torch.randn(ra.shape, generator=r).to(dtype), torch.randn(rb.shape, generator=r).to(dtype)
    got = ck.qk_norm_rotary_backward(ga.cuda(), gb.cuda(), dq, dk, dp, df, q_weight=dw[0],
                                     k_weight=dw[1], **opts)
    want = torch.autograd.grad((ra * ga.double()).sum() + (rb * gb.double()).sum(),
                               leaves + [w for w in ws if w is not None], allow_unused=True)
    assert rel(got[0], want[0]) < TOL[dtype] and rel(got[1], want[1]) < TOL[dtype]
    if weight:
        for x, y in zip(got[2:], want[2:]):
            y = torch.zeros_like(x.cpu()) if y is None else y
            assert rel(x, y) < 2.0 ** -20, rel(x, y)
    else:
        assert got[2] is None and got[3] is None


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rd", [(128, 64), (64, 64), (96, 48), (40, 18)])
def test_rotary(d, rd, layout, dtype):
    q, _, pos, freqs, _, _ = data(d, 51, 3, 1, d, rd, dtype, far=2 ** 31 - 1)
    x = cu(q)
    y = ck.rotary(x, pos.cuda(), freqs.cuda(), layout=layout, rotary_scale=1.1)
    # freqs * pos of positions near 2^31 is off by 2^-53 of 3e8 turns in either
    # form: 4e-8 turns, 2^-22 of a unit vector
    assert rel(y, rotate(q.double(), pos, freqs, layout, 1.1)) < TOL[dtype]
    back = ck.rotary(x, pos.cuda(), freqs.cuda(), layout=layout, inverse=True)
    assert rel(back, rotate(q.double(), pos, freqs, layout, inverse=True)) < TOL[dtype]
    ck.rotary(x, pos.cuda(), freqs.cuda(), layout=layout, rotary_scale=1.1, out=x)
    assert torch.equal(x, y)
    assert torch.equal(y[..., rd:].cpu(), q[..., rd:])


def test_in_place_in_a_projection():
    """q and k rotated where they lie; the values behind them are untouched."""
    q, k, pos, freqs, wq, wk = data(3, 20, 4, 2, 128, 128, BF)
    p = torch.randn(20, 8, 128, generator=NO().manual_seed(4)).to(BF)
    want = ck.qk_norm_rotary(p[:, :4].cuda(), p[:, 4:6].cuda(), pos.cuda(), freqs.cuda(),
                             q_weight=wq.cuda(), k_weight=wk.cuda())
    d = p.cuda()
    ck.qk_norm_rotary(d[:, :4], d[:, 4:6], pos.cuda(), freqs.cuda(), q_weight=wq.cuda(),
                      k_weight=wk.cuda(), q_out=d[:, :4], k_out=d[:, 4:6])
    assert torch.equal(d[:, :4], want[0]) and torch.equal(d[:, 4:6], want[1])
    assert torch.equal(d[:, 6:].cpu(), p[:, 6:])


def test_unaligned_rows():
    """Rows that start at an odd element."""
    q, k, pos, freqs, wq, wk = data(5, 12, 2, 2, 64, 32, BF)
    flat = torch.zeros(12, 2 * 64 + 5, dtype=BF, device="cuda")
    odd = flat[:, 3:131].unflatten(1, (2, 64))
    odd.copy_(q)
    a, b = ck.qk_norm_rotary(odd, cu(k), pos.cuda(), freqs.cuda(), norm="l2")
    c, e = ck.qk_norm_rotary(cu(q), cu(k), pos.cuda(), freqs.cuda(), norm="l2")
    assert rel(a, rotate(norm(q, "l2"), pos, freqs, "half")) < TOL[BF]
    assert torch.equal(b, e) and rel(a, c.double()) < 2.0 ** -8


def test_no_tokens():
    q, k, pos, freqs, wq, wk = (x.cuda() for x in data(6, 0, 2, 1, 64, 64, BF, packed=False))
    a, b = ck.qk_norm_rotary(q, k, pos, freqs, q_weight=wq, k_weight=wk)
    got = ck.qk_norm_rotary_backward(a, b, q, k, pos, freqs, q_weight=wq, k_weight=wk)
    assert a.shape == (0, 2, 64) and b.shape == (0, 1, 64)
    assert not got[2].any() and not got[3].any()


def test_batched_leading_dimensions_and_zero_rows():
    r = NO().manual_seed(8)
    x = torch.randn(2, 3, 4, 64, generator=r)
    x[1, 2, 3] = 0.0                      # a row of zeros has norm sqrt(eps)
    pos = torch.arange(6, dtype=torch.int32).reshape(2, 3)
    f = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    a, b = ck.qk_norm_rotary(x.cuda(), x[:, :, :1].contiguous().cuda(), pos.cuda(), f.cuda(), norm="l2")
    assert rel(a, rotate(norm(x, "l2"), pos, f, "half")) < TOL[F32]
    g = torch.ones_like(x).cuda()
    back = ck.qk_norm_rotary_backward(g, g[:, :, :1].contiguous(), x.cuda(),
                                      x[:, :, :1].contiguous().cuda(), pos.cuda(), f.cuda(), norm="l2")
    assert bool(torch.isfinite(back[0]).all())


def test_frequencies_give_the_plain_rotation():
    f, scale = ck.rotary_frequencies(64, device="cuda")
    x = torch.randn(4, 2, 64, generator=NO().manual_seed(9))
    pos = torch.tensor([0, 1, 1000, 10 ** 6], dtype=torch.int32)
    y = ck.rotary(x.cuda(), pos.cuda(), f, rotary_scale=scale)
    a = pos.double()[:, None] * 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
    u, w = x.double()[..., :32], x.double()[..., 32:]
    assert rel(y, torch.cat([u * c - w * s, w * c + u * s], -1)) < TOL[F32]
    assert math.isclose(scale, 1.0)


@pytest.mark.parametrize("tokens", [1023, 1024, 1025, 1031])
def test_where_tiles_of_tokens_begin(tokens):
    """One token a workgroup below 1024 tokens, tiles of eight from there on, the last one partial."""
    q, k, pos, freqs, wq, wk = data(tokens, tokens, 3, 1, 64, 48, BF, packed=False)
    a, b = ck.qk_norm_rotary(q.cuda(), k.cuda(), pos.cuda(), freqs.cuda(), q_weight=wq.cuda(),
                             k_weight=wk.cuda())
    assert rel(a, rotate(norm(q, "rms", wq), pos, freqs, "half")) < TOL[BF]
    assert rel(b, rotate(norm(k, "rms", wk), pos, freqs, "half")) < TOL[BF]
    x = ck.rotary(q.cuda(), pos.cuda(), freqs.cuda())
    assert rel(x, rotate(q.double(), pos, freqs, "half")) < TOL[BF]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("kind", ["rms", "l2"])
def test_gradients_against_differences(kind, layout):
    """Along a random direction u of all inputs, central differences of the fp32
    operator.  With steps h u of 2^-7 of a row's length the third-order term is
    within 2^-14 of the scale |g| |u| and the rounding of outputs (2^-23, over
    2 h) within 2^-16; the bound is 2^-11 of that scale, where the derivative
    itself is about 2^-3 of it."""
    tokens, d, rd = 2, 16, 12
    q, k, pos, freqs, wq, wk = data(31, tokens, 2, 1, d, rd, F32, packed=False)
    r = NO().manual_seed(32)
    leaves = [q, k, wq, wk]
    step = [torch.randn(t.shape, generator=r) for t in leaves]
    out = [torch.randn(q.shape, generator=r), torch.randn(k.shape, generator=r)]
    opts = dict(norm=kind, layout=layout, q_scale=0.5, rotary_scale=1.5)
    h = 2.0 ** -7

    def loss(s):
        q, k, wq, wk = (t.double().add(u.double(), alpha=s).float().cuda() for t, u in zip(leaves, step))
        a, b = ck.qk_norm_rotary(q, k, pos.cuda(), freqs.cuda(), q_weight=wq, k_weight=wk, **opts)
        return float((a.cpu().double() * out[0].double()).sum() + (b.cpu().double() * out[1].double()).sum())

    got = ck.qk_norm_rotary_backward(out[0].cuda(), out[1].cuda(), q.cuda(), k.cuda(), pos.cuda(),
                                     freqs.cuda(), q_weight=wq.cuda(), k_weight=wk.cuda(), **opts)
    dot = sum(float((g.cpu().double() * u.double()).sum()) for g, u in zip(got, step))
    scale = math.sqrt(sum(float(g.double().square().sum()) for g in got)
                      * sum(float(u.double().square().sum()) for u in step))
    assert abs((loss(h) - loss(-h)) / (2 * h) - dot) < 2.0 ** -11 * scale
