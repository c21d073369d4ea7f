"""The gated delta rule and the norm with rotation as programs use them: in
captured graphs, on two streams at once, beyond 32-bit offsets, and in debug
mode.  The kernels have a fixed order of operations, so every comparison with
another run of the same call is bit for bit."""
import os

import pytest
import torch

import gated_delta_rule_22_amd as ck
from _gdr_ref import gdr, inputs, rel

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
LENS = [70, 1, 193, 0, 64]
CU = [0, 70, 71, 264, 264, 328]


def seq(seed, dtype, lens=LENS, hk=2, hv=4, dk=128, dv=64):
    """Device inputs of one packed batch, and upstream gradients."""
    x = {n: t.cuda() for n, t in inputs(seed, lens, hk, hv, dk, dv, dtype).items()}
    r = torch.Generator().manual_seed(seed + 1)
    x["do"] = torch.randn(x["v"].shape, generator=r).to(dtype).cuda()
    x["dS"] = 0.3 * torch.randn(x["S0"].shape, generator=r).cuda()
    for n in ("q", "k", "v", "g", "beta", "do"):
        x[n] = x[n][None]
    return x


def rows(seed, dtype, tokens=45, hq=4, hk=2, d=128, rd=64):
    r = torch.Generator().manual_seed(seed)
    p = torch.randn(tokens, hq + 2 * hk, d, generator=r).to(dtype).cuda()
    return dict(p=p, pos=torch.randint(0, 9000, (tokens,), generator=r).to(torch.int32).cuda(),
                wq=1 + 0.2 * torch.randn(d, generator=r).cuda(),
                wk=1 + 0.2 * torch.randn(d, generator=r).cuda(),
                dq=torch.randn(tokens, hq, d, generator=r).to(dtype).cuda(),
                dk=torch.randn(tokens, hk, d, generator=r).to(dtype).cuda())


def calls(dtype):
    """name -> (inputs of a seed, call on them)."""
    cu = torch.tensor(CU, dtype=torch.int32, device="cuda")
    freqs = ck.rotary_frequencies(64, device="cuda")[0]
    five = ("q", "k", "v", "g", "beta")

    def forward(x):
        return ck.gdr_forward(*(x[n] for n in five), S0=x["S0"], cu_seqlens=cu)

    def forward_rows(x):
        return ck.gdr_forward(*(x[n].unflatten(1, (2, 164))[0] for n in five))

    def backward(x):
        return ck.gdr_backward(*(x[n] for n in five), x["do"], S0=x["S0"], dS_T=x["dS"],
                               cu_seqlens=cu)

    def backward_few(x):
        return ck.gdr_backward(*(x[n][:, :20].contiguous() for n in five),
                               x["do"][:, :20].contiguous())

    def step(x):
        S = x["S0"].clone()
        slots = torch.arange(4, -1, -1, dtype=torch.int32, device="cuda")
        o = ck.gdr_decode_step(*(x[n][0, :5].contiguous() for n in five), S, slots=slots)
        return o, S

    def prepare(x):
        return ck.qk_norm_rotary(x["p"][:, :4], x["p"][:, 4:6], x["pos"], freqs,
                                 q_weight=x["wq"], k_weight=x["wk"])

    def prepare_back(x):
        return ck.qk_norm_rotary_backward(x["dq"], x["dk"], x["p"][:, :4], x["p"][:, 4:6],
                                          x["pos"], freqs, q_weight=x["wq"], k_weight=x["wk"])

    def turn(x):
        return ck.rotary(x["dq"], x["pos"], freqs)

    return {f.__name__: (seq if f in (forward, forward_rows, backward, backward_few, step) else rows, f)
            for f in (forward, forward_rows, backward, backward_few, step, prepare, prepare_back, turn)}


NAMES = ("forward", "forward_rows", "backward", "backward_few", "step", "prepare", "prepare_back", "turn")


def outputs(got):
    return [t.clone() for t in (got if isinstance(got, tuple) else (got,)) if t is not None]


def same(a, b, what):
    for i, (x, y) in enumerate(zip(outputs(a), outputs(b))):
        assert torch.equal(x, y), (what, i)


def capture(fn, x):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn(x)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fn(x)
    torch.cuda.synchronize()
    return graph, got


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("name", NAMES)
def test_replays_are_the_eager_call(name, dtype):
    make, fn = calls(dtype)[name]
    x = make(1, dtype)
    print("graph of", name, dtype, flush=True)
    graph, got = capture(fn, x)
    for r in range(4):
        for n, t in make(10 + r, dtype).items():
            x[n].copy_(t)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = outputs(got)
        same(tuple(kept), fn(x), (name, r))
        torch.cuda.synchronize()


def test_replays_with_other_lengths():
    """The offsets are read on the device: a captured call serves even and uneven batches, which
    take their columns differently, and empty ones."""
    n, T = 9, 4608
    x = seq(21, BF, lens=[512] * n, hk=4, hv=16, dk=64)
    five = [x[m] for m in ("q", "k", "v", "g", "beta")]
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    batches = [[512] * n, [4500] + [1] * 8, [0] * 8 + [T], [0] * n, [700, 3, 0, 64, 1000, 1, 900, 65, 1875]]

    def fill(lens):
        cu.copy_(torch.tensor([0] + lens).cumsum(0).to(torch.int32))

    def call(_):
        o = torch.zeros_like(x["v"])     # rows outside every sequence stay as they are
        return ck.gdr_forward(*five, S0=x["S0"], cu_seqlens=cu, out=o)

    fill(batches[0])
    graph, got = capture(call, None)
    for lens in batches + batches[:1]:
        fill(lens)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same(tuple(outputs(got)), call(None), lens)
        torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["forward", "backward", "prepare_back"])
def test_two_graphs_at_once(name):
    """Two captured graphs of one call, each with its own workspace, replayed on two streams."""
    make, fn = calls(BF)[name]
    xs = [make(3, BF), make(4, BF)]
    print("two graphs of", name, flush=True)
    graphs = [capture(fn, x) for x in xs]
    want = [outputs(fn(x)) for x in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        torch.cuda.synchronize()
        for s, (g, _got) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for w, (_g, got) in zip(want, graphs):
            same(tuple(w), got, name)


@pytest.mark.parametrize("name", NAMES)
def test_two_streams_at_once(name):
    make, fn = calls(BF)[name]
    xs = [make(5, BF), make(6, BF)]
    want = [outputs(fn(x)) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(outputs(fn(xs[i])))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for r in runs:
            same(tuple(w), tuple(r), name)


def test_caller_workspace_and_outputs():
    """One workspace for a forward and its backward after each other, outputs in given tensors."""
    x = seq(7, BF)
    cu = torch.tensor(CU, dtype=torch.int32, device="cuda")
    five = [x[n] for n in ("q", "k", "v", "g", "beta")]
    want, wantb = ck.gdr_forward(*five, S0=x["S0"], cu_seqlens=cu), ck.gdr_backward(
        *five, x["do"], S0=x["S0"], cu_seqlens=cu)
    sizes = (1, 328, 2, 4, 128, 64, 5, BF)
    ws = torch.full((max(ck.gdr_forward_workspace_bytes(*sizes),
                         ck.gdr_backward_workspace_bytes(*sizes)),), 255, dtype=torch.uint8, device="cuda")
    out, S = torch.empty_like(x["v"]), x["S0"].clone()
    for _ in range(2):
        S.copy_(x["S0"])
        a = ck.gdr_forward(*five, S0=S, cu_seqlens=cu, out=out, final_state=S, workspace=ws)
        assert a[0] is out and a[1] is S
        b = ck.gdr_backward(*five, x["do"], S0=x["S0"], cu_seqlens=cu, workspace=ws)
        same(a, want, "forward")
        same(b, wantb, "backward")


@pytest.mark.parametrize("dtype", [F32, BF])
def test_no_tokens(dtype):
    x = seq(8, dtype, lens=[0, 0])
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    five = [x[n] for n in ("q", "k", "v", "g", "beta")]
    o, S = ck.gdr_forward(*five, S0=x["S0"], cu_seqlens=cu)
    assert o.numel() == 0 and torch.equal(S, x["S0"])
    got = ck.gdr_backward(*five, x["do"], S0=x["S0"], dS_T=x["dS"], cu_seqlens=cu)
    assert torch.equal(got[5], x["dS"])


def test_tensors_elsewhere_are_refused():
    x = seq(15, BF)
    five = [x[n] for n in ("q", "k", "v", "g", "beta")]
    for i in range(5):
        bad = list(five)
        bad[i] = bad[i].cpu()
        with pytest.raises((TypeError, ValueError)):
            ck.gdr_forward(*bad)
        bad[i] = five[i].transpose(0, 1)
        with pytest.raises((TypeError, ValueError)):
            ck.gdr_forward(*bad)
    with pytest.raises((TypeError, ValueError)):
        ck.gdr_backward(*five, x["do"].float())
    with pytest.raises((TypeError, ValueError)):
        ck.gdr_decode_step(*(t[0].contiguous() for t in five), x["S0"].cpu())
    p = rows(16, BF)
    f = ck.rotary_frequencies(64, device="cuda")[0]
    with pytest.raises((TypeError, ValueError)):
        ck.qk_norm_rotary(p["dq"], p["dk"], p["pos"].cpu(), f)
    with pytest.raises((TypeError, ValueError)):
        ck.rotary(p["dq"], p["pos"], f.float())


def test_debug_mode_changes_nothing():
    """CKDA_DEBUG fills the workspace with NaN patterns first."""
    todo = calls(BF)
    want = {n: outputs(fn(make(9, BF))) for n, (make, fn) in todo.items()}
    torch.cuda.synchronize()
    os.environ["CKDA_DEBUG"] = "1"
    try:
        for n, (make, fn) in todo.items():
            same(tuple(want[n]), fn(make(9, BF)), n)
        torch.cuda.synchronize()
        x = seq(9, BF)
        bad = torch.tensor([0, 70, 60, 264, 264, 328], dtype=torch.int32, device="cuda")
        with pytest.raises(RuntimeError):
            ck.gdr_forward(*(x[n] for n in ("q", "k", "v", "g", "beta")), cu_seqlens=bad)
    finally:
        os.environ.pop("CKDA_DEBUG")


def test_offsets_that_go_backwards_stay_inside():
    """Without debug mode the device makes them monotone: 60 behind 70 counts as 70, 999 as T."""
    x = seq(10, BF)
    five = [x[n] for n in ("q", "k", "v", "g", "beta")]
    bad = torch.tensor([-5, 70, 60, 264, 264, 999], dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 70, 70, 264, 264, 328], dtype=torch.int32, device="cuda")
    same(ck.gdr_forward(*five, cu_seqlens=bad), ck.gdr_forward(*five, cu_seqlens=good), "offsets")
    same(ck.gdr_backward(*five, x["do"], cu_seqlens=bad),
         ck.gdr_backward(*five, x["do"], cu_seqlens=good), "offsets")


# ------------------------------------------------------ offsets past 32 bits
def far(B, T, hk, hv, d, seed):
    r = torch.Generator("cuda").manual_seed(seed)
    kw = dict(generator=r, device="cuda")
    q = (0.1 * torch.randn(B, T, hk, d, **kw)).to(BF)
    k = (d ** -0.5 * torch.randn(B, T, hk, d, **kw)).to(BF)
    v = torch.randn(B, T, hv, d, **kw).to(BF)
    return q, k, v, -0.05 * torch.rand(B, T, hv, **kw), torch.rand(B, T, hv, **kw)


def test_sequences_past_32_bits():
    """2^31 elements of v and 2^33 bytes of kept states: the last row is the row alone."""
    B, T, H, d = 17, 16384, 64, 128
    x = far(B, T, 16, H, d, 11)
    assert x[2].numel() > 2 ** 31
    do = torch.randn_like(x[2])
    one = [t[-1:].clone() for t in x]
    print("gdr_forward", tuple(x[2].shape), flush=True)
    o, S = ck.gdr_forward(*x)
    oo, SS = ck.gdr_forward(*one)
    assert torch.equal(o[-1], oo[0]) and torch.equal(S[-1], SS[0])
    print("gdr_backward", tuple(x[2].shape), flush=True)
    need = ck.gdr_backward_workspace_bytes(B, T, 16, H, d, d, B, BF)
    assert need < torch.cuda.mem_get_info()[0]
    got = ck.gdr_backward(*x, do)
    alone = ck.gdr_backward(*one, do[-1:].clone())
    for a, b in zip(got[:5], alone):
        assert torch.equal(a[-1], b[0])


def test_pool_past_32_bits():
    """A slot behind 2^31 elements of the pool."""
    pool, H, d = 4100, 32, 128
    S = torch.zeros(pool, H, d, d, device="cuda")
    assert S.numel() > 2 ** 31
    x = inputs(13, [1, 1], 8, H, d, d, BF)
    S[4099], S[1] = x["S0"][0].cuda(), x["S0"][1].cuda()
    want = gdr(x["q"], x["k"], x["v"], x["g"], x["beta"], x["S0"], [1, 1])
    o = ck.gdr_decode_step(*(x[n].cuda() for n in ("q", "k", "v", "g", "beta")), S,
                           slots=torch.tensor([4099, 1], dtype=torch.int32, device="cuda"))
    assert rel(o, want[0]) < 2.0 ** -8 and rel(S[[4099, 1]], want[1]) < 2.0 ** -20
    assert not S[2:4099].any()


def test_rows_past_32_bits():
    """q and k in a projection of more than 2^31 elements; the last tokens are the tokens alone."""
    tokens, heads, d = 1 << 19, 36, 128
    p = torch.randn(tokens, heads, d, generator=torch.Generator("cuda").manual_seed(14),
                    device="cuda", dtype=BF)
    assert p.numel() > 2 ** 31
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    f = ck.rotary_frequencies(d, device="cuda")[0]
    w = torch.ones(d, device="cuda")
    q, k = p[:, :20], p[:, 32:]
    a, b = ck.qk_norm_rotary(q, k, pos, f, q_weight=w)
    last = slice(tokens - 9, tokens)
    c, e = ck.qk_norm_rotary(q[last], k[last], pos[last], f, q_weight=w)
    assert torch.equal(a[last], c) and torch.equal(b[last], e)
    ga = ck.qk_norm_rotary_backward(a, b, q, k, pos, f, q_weight=w)
    gb = ck.qk_norm_rotary_backward(c, e, q[last], k[last], pos[last], f, q_weight=w)
    assert torch.equal(ga[0][last], gb[0]) and torch.equal(ga[1][last], gb[1])
