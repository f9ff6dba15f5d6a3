"""hq_rope against the float64 oracle.

Tolerance per element of a pair (u, v), output y in type t: half a step of the
output, eps(t)/2 |y| (and half the smallest subnormal of fp16, 2^-25), plus the
float32 arithmetic: the angle is off by at most pi 2^-25 (24 bits of half-turns)
and sincospif by 2 ulp (2^-23), so cos and sin are off by less than 2^-22; two
products and a sum add 3 roundings of 2^-24, the factor one to each: below
2^-21 amp (|u| + |v|) together.
"""
import numpy as np
import pytest
import torch

from oracle import rope as orope

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -149}


def _hq():
    from hybrid_precision_attention_b200 import hq
    return hq


def _table(rot, kind="plain", base=10000.0, factor=8.0, orig_len=2048):
    hq = _hq()
    t = hq.RopeTable(rot, base, kind=orope.KINDS.index(kind), factor=factor, orig_len=orig_len)
    return t, orope.frequencies(rot, base, kind, factor, orig_len)


def _check(x, y, pos, wa, layout, dtype, grad=False):
    w, amp = wa
    xd = x.double().cpu().numpy()
    want = orope.rotate(xd, pos.cpu().numpy(), w, amp, layout, grad)
    n = len(w)
    size = np.zeros_like(xd)
    if layout == "half":
        size[..., :n] = size[..., n:2 * n] = np.abs(xd[..., :n]) + np.abs(xd[..., n:2 * n])
    else:
        size[..., 0:2 * n:2] = size[..., 1:2 * n:2] = np.abs(xd[..., 0:2 * n:2]) + np.abs(xd[..., 1:2 * n:2])
    tol = torch.finfo(TYPES[dtype]).eps / 2 * np.abs(want) * (1 + 2.0 ** -20) + 2.0 ** -21 * amp * size + TINY[dtype]
    got = y.double().cpu().numpy()
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()
    assert np.array_equal(got[..., 2 * n:], xd[..., 2 * n:])


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot,kind", [(128, 128, "plain"), (128, 64, "yarn"), (80, 80, "bands"), (64, 18, "ntk"), (96, 26, "linear"),
                                        (256, 256, "yarn"), (6, 4, "plain"), (7, 2, "plain"), (512, 512, "linear"), (511, 34, "plain")])
def test_rope(dtype, layout, D, rot, kind):
    hq = _hq()
    torch.manual_seed(D + rot)
    B, T, Hq, Hkv = 2, 37, 6, 3
    q = torch.randn(B, T, Hq, D, device="cuda").to(TYPES[dtype])
    k = torch.randn(B, T, Hkv, D, device="cuda").to(TYPES[dtype])
    pos = torch.randint(0, 200000, (B, T), dtype=torch.int32, device="cuda")
    t, wa = _table(rot, kind)
    for grad in (False, True):
        yq, yk = hq.hq_rope(q, k, pos, t, layout=("half", "interleaved").index(layout), grad=grad)
        _check(q, yq, pos, wa, layout, dtype, grad)
        _check(k, yk, pos, wa, layout, dtype, grad)


@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 1, 1, 0), (1, 1, 32, 8), (16, 1, 32, 8), (1, 3000, 5, 1), (7, 61, 4, 4), (1, 700, 64, 8)])
def test_sizes_from_one_token_to_many(B, T, Hq, Hkv):
    hq = _hq()
    q = torch.randn(B, T, Hq, 128, device="cuda").half()
    k = torch.randn(B, T, Hkv, 128, device="cuda").half() if Hkv else None
    pos = torch.arange(B * T, dtype=torch.int32, device="cuda").reshape(B, T) * 31
    t, wa = _table(128)
    yq, yk = hq.hq_rope(q, k, pos, t)
    _check(q, yq, pos, wa, "half", "f16")
    if Hkv:
        _check(k, yk, pos, wa, "half", "f16")
    else:
        assert yk is None


def test_far_positions():
    hq = _hq()
    pos = torch.tensor([0, 1, -1, 131071, 1000003, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    x = torch.randn(7, 2, 128, device="cuda")
    for kind in orope.KINDS:
        t, wa = _table(128, kind, base=500000.0)
        y, _ = hq.hq_rope(x, None, pos, t)
        _check(x, y, pos, wa, "half", "f32")


def test_strides_in_place_and_transposed_output():
    """Views into the fused projection's rows, in place; and written as [B, H, T, D], the layout of the prefill call."""
    hq = _hq()
    B, T, Hq, Hkv, D = 2, 50, 8, 2, 128
    row = torch.randn(B, T, Hq + 2 * Hkv, D, device="cuda").half()
    q, k, v = row[:, :, :Hq], row[:, :, Hq:Hq + Hkv], row[:, :, Hq + Hkv:]
    pos = torch.arange(T, dtype=torch.int32, device="cuda").repeat(B, 1)
    t, wa = _table(64, "bands")
    out = torch.full((B, Hq, T, D), 7.0, device="cuda", dtype=torch.float16)
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    yq, _ = hq.hq_rope(q, k, pos, t, q_out=out.transpose(1, 2), k_out=k)
    _check(q0, yq, pos, wa, "half", "f16")
    _check(k0, k, pos, wa, "half", "f16")
    assert torch.equal(q, q0) and torch.equal(v, v0) and yq.data_ptr() == out.data_ptr()
    # rows that no 16-byte access fits: an odd offset and odd strides
    wide = torch.randn(T * 3 * 131 + 5, device="cuda").half()
    x = wide[5:5 + T * 3 * 131].reshape(T, 3, 131)[..., 1:129]
    y, _ = hq.hq_rope(x, None, pos[0], t, layout=hq.ROPE_INTERLEAVED)
    _check(x, y, pos[0], wa, "interleaved", "f16")
    keep = wide.clone()
    y, _ = hq.hq_rope(x, None, pos[0], t, layout=hq.ROPE_INTERLEAVED, q_out=x)
    rest = torch.ones_like(wide, dtype=torch.bool)
    rest[5:5 + T * 3 * 131].reshape(T, 3, 131)[..., 1:65] = False
    assert torch.equal(wide[rest], keep[rest])


def test_in_place_leaves_the_rest_of_one_tensor_and_copies_the_other():
    hq = _hq()
    x, z = torch.randn(9, 2, 128, device="cuda").half(), torch.randn(9, 3, 128, device="cuda").half()
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    t, wa = _table(32)
    x0 = x.clone()
    _, yz = hq.hq_rope(x, z, pos, t, q_out=x)
    _check(x0, x, pos, wa, "half", "f16")
    _check(z, yz, pos, wa, "half", "f16")


def test_not_finite_values_stay_in_their_pair():
    hq = _hq()
    x = torch.randn(4, 2, 128, device="cuda").half()
    x[1, 0, 3], x[2, 1, 70] = float("inf"), float("nan")
    pos = torch.arange(4, dtype=torch.int32, device="cuda") + 5
    t, _ = _table(128)
    y, _ = hq.hq_rope(x, None, pos, t)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[1, 0, 3] = want[1, 0, 67] = want[2, 1, 6] = want[2, 1, 70] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("layout", [0, 1])
def test_gradient_against_differences(layout):
    """The rotation is linear: (f(x + e) - f(x - e)) / 2 contracted with g equals e contracted with the gradient,
    up to float32 roundings: each of the n = 2 x 768 products' factors is off by less than 2^-21 of its pair."""
    hq = _hq()
    torch.manual_seed(3)
    x, e, g = (torch.randn(3, 2, 128, device="cuda") for _ in range(3))
    pos = torch.tensor([3, 999, 70001], dtype=torch.int32, device="cuda")
    t, (w, amp) = _table(64, "yarn")
    f = lambda z: hq.hq_rope(z, None, pos, t, layout=layout)[0].double()
    d = ((f(x + e) - f(x - e)) / 2 * g.double()).sum()
    grad, _ = hq.hq_rope(g, None, pos, t, layout=layout, grad=True)
    size = (x.abs() + e.abs()).max().double() * g.abs().double().sum()
    assert abs(d - (grad.double() * e.double()).sum()) <= 2.0 ** -19 * amp * size


def test_autograd_function_of_a_user():
    """A training program's rotary step: forward and backward through the two calls, against torch's own gradient."""
    hq = _hq()
    t, (w, amp) = _table(128, "linear")
    pos = torch.arange(40, dtype=torch.int32, device="cuda").reshape(2, 20)

    class Rope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k):
            return hq.hq_rope(q, k, pos, t)

        @staticmethod
        def backward(ctx, gq, gk):
            return hq.hq_rope(gq, gk, pos, t, grad=True)

    q = torch.randn(2, 20, 4, 128, device="cuda", requires_grad=True)
    k = torch.randn(2, 20, 1, 128, device="cuda", requires_grad=True)
    yq, yk = Rope.apply(q, k)
    s = (yq.reshape(2, 20, 4, 128) * yk).square().sum()
    s.backward()
    ang = pos.double().cpu().numpy()[..., None] * w.astype(np.float64)
    c, n = (torch.from_numpy(z).cuda()[:, :, None] for z in (np.cos(ang), np.sin(ang)))
    q2, k2 = q.detach().double().requires_grad_(), k.detach().double().requires_grad_()
    turn = lambda x: torch.cat((x[..., :64] * c - x[..., 64:] * n, x[..., 64:] * c + x[..., :64] * n), -1)
    (turn(q2) * turn(k2)).square().sum().backward()
    for a, b in ((q, q2), (k, k2)):
        # a product of four float32 factors, each within 2^-20 of its size, summed over at most 4 heads
        assert torch.linalg.norm(a.grad.double() - b.grad) <= 2.0 ** -17 * torch.linalg.norm(b.grad)


def test_streams_and_graph():
    hq = _hq()
    t, wa = _table(128)
    x = torch.randn(16, 32, 128, device="cuda").half()
    pos = torch.arange(16, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, _ = hq.hq_rope(x, None, pos, t, stream=s)
    s.synchronize()
    _check(x, y, pos, wa, "half", "f16")
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hq.hq_rope(x, None, pos, t, q_out=out)
    x.copy_(torch.randn_like(x))
    pos += 1000
    graph.replay()
    torch.cuda.synchronize()
    _check(x, out, pos, wa, "half", "f16")


def test_refusals_of_the_binding():
    hq = _hq()
    t, _ = _table(64)
    x = torch.randn(4, 2, 64, device="cuda").half()
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    for a in ((x.int(), None, pos), (x, x.float(), pos), (x[0], None, pos), (x, None, pos.long()), (x, None, pos[:3]), (x, None, pos.cpu()),
              (x.cpu(), None, pos), (x.transpose(1, 2), None, pos), (x[..., :32], None, pos)):
        with pytest.raises(hq.HqError):
            hq.hq_rope(*a, t)
    with pytest.raises(hq.HqError):
        hq.hq_rope(x, None, pos, t, q_out=x[:3])
    empty, _ = hq.hq_rope(x[:0], None, pos[:0], t)
    assert empty.shape == (0, 2, 64)


# ----------------------------------------------------------------------------- in a graph

@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_gradients_flow(layout, dtype):
    """The gradient is the transposed call's, to the bit, whichever of q and k ask and however the gradients come."""
    hq = _hq()
    torch.manual_seed(11)
    t, wa = _table(64, "yarn")
    q, k = torch.randn(2, 9, 4, 96, device="cuda").to(TYPES[dtype]), torch.randn(2, 9, 2, 96, device="cuda").to(TYPES[dtype])
    pos = torch.randint(0, 5000, (2, 9), dtype=torch.int32, device="cuda")
    gq, gk = torch.randn_like(q), torch.randn_like(k)
    plain = hq.hq_rope(q, k, pos, t, layout=layout)
    want = hq.hq_rope(gq, gk, pos, t, layout=layout, grad=True)
    _check(gq, want[0], pos, wa, ("half", "interleaved")[layout], dtype, grad=True)
    for asks in ((True, True), (True, False), (False, True)):
        a, b = q.clone().requires_grad_(asks[0]), k.clone().requires_grad_(asks[1])
        yq, yk = hq.hq_rope(a, b, pos, t, layout=layout)
        assert torch.equal(yq, plain[0]) and torch.equal(yk, plain[1]) and yq.requires_grad
        torch.autograd.backward((yq, yk), (gq, gk))
        for x, w, ask in ((a, want[0], asks[0]), (b, want[1], asks[1])):
            assert torch.equal(x.grad, w) if ask else x.grad is None
    for use in (0, 1):                     # one output unused; a sum's gradient, expanded
        a, b = q.clone().requires_grad_(), k.clone().requires_grad_()
        hq.hq_rope(a, b, pos, t, layout=layout)[use].sum().backward()
        ones = hq.hq_rope(torch.ones_like(q), torch.ones_like(k), pos, t, layout=layout, grad=True)
        assert torch.equal((a, b)[use].grad, ones[use]) and ((a, b)[1 - use].grad is None or not (a, b)[1 - use].grad.any())
    a = q.clone().requires_grad_()         # without k, without a batch, and grad=True of it
    y, none = hq.hq_rope(a[0], None, pos[0], t, layout=layout, grad=True)
    assert none is None
    y.backward(gq[0])
    assert torch.equal(a.grad[0], hq.hq_rope(gq[0], None, pos[0], t, layout=layout)[0]) and not a.grad[1].any()


def test_gradients_of_gradients_shared_heads_and_changed_positions():
    hq = _hq()
    t, _ = _table(64)
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    one = torch.randn(5, 1, 64, device="cuda", requires_grad=True)
    y, _ = hq.hq_rope(one.expand(5, 3, 64), None, pos, t)      # a head shared by three: its gradient is their sum
    g = torch.randn(5, 3, 64, device="cuda", requires_grad=True)
    d, = torch.autograd.grad(y, one, g, create_graph=True)
    assert torch.equal(d, hq.hq_rope(g.detach(), None, pos, t, grad=True)[0].sum(1, keepdim=True))
    z = torch.randn_like(d)
    back, = torch.autograd.grad(d, g, z)                         # linear in g: the rotation of z
    assert torch.equal(back, hq.hq_rope(z.expand(5, 3, 64), None, pos, t)[0])
    y, _ = hq.hq_rope(one, None, pos, t)
    pos += 1
    with pytest.raises(RuntimeError):                            # the positions of the forward call are gone
        y.sum().backward()


def test_outputs_of_the_caller_have_no_gradient():
    hq = _hq()
    t, _ = _table(64)
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    x = torch.randn(5, 2, 64, device="cuda", requires_grad=True)
    for kw in (dict(q_out=torch.empty_like(x)), dict(q_out=x)):
        with pytest.raises(hq.HqError):
            hq.hq_rope(x, None, pos, t, **kw)
    with torch.no_grad():
        y, _ = hq.hq_rope(x, None, pos, t, q_out=torch.empty(5, 2, 64, device="cuda"))
        assert not y.requires_grad and torch.equal(y, hq.hq_rope(x, None, pos, t)[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, _ = hq.hq_rope(x, None, pos, t, stream=s)
    with torch.cuda.stream(s):
        y.sum().backward()
    torch.cuda.synchronize()
    assert torch.equal(x.grad, hq.hq_rope(torch.ones(5, 2, 64, device="cuda"), None, pos, t, grad=True)[0])


def test_windows_over_one_another():
    """Heads and tokens one element apart in memory: read as they are, the outputs rows of their own."""
    hq = _hq()
    t, wa = _table(8)
    pos = torch.arange(5, dtype=torch.int32, device="cuda") * 100
    x = torch.randn(200, device="cuda")
    for strides in ((1, 1, 1), (1, 7, 1), (9, 1, 1), (0, 1, 1), (1, 0, 1), (0, 0, 1)):
        q = x.as_strided((5, 3, 8), strides)
        y, z = hq.hq_rope(q, q[:, :2], pos, t)
        assert y.stride(-1) == 1 and z.stride(-1) == 1
        _check(q, y, pos, wa, "half", "f32")
        _check(q[:, :2], z, pos, wa, "half", "f32")


@pytest.mark.parametrize("T", [50, 20000])
@pytest.mark.parametrize("layout", [0, 1])
def test_sines_to_their_last_bits(T, layout):
    """Pairs (1, 0) become (cos a, sin a) in float32: sincospif is good to 2 ulp (2^-22 of the value), the factor's and the
    sum's roundings add 2^-23 of it, and the angle is cut off at 2^-31 half-turns (pi 2^-31 < 2^-29, twice that for the
    first-order step): also where the value is near 0 nothing else is lost."""
    hq = _hq()
    g = torch.Generator(device="cuda").manual_seed(5)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (T,), dtype=torch.int64, device="cuda", generator=g)
    pos[::3] = torch.arange(pos[::3].numel(), device="cuda")
    pos[:8] = torch.tensor([0, 1, -1, 355, 710, 103993, 2 ** 31 - 1, -2 ** 31])  # numerators of pi's convergents among them
    pos = pos.int()
    t, (w, amp) = _table(16, "plain", base=10000.0)
    x = torch.zeros(T, 1, 16, device="cuda")
    first = torch.arange(8) if layout == 0 else torch.arange(8) * 2
    x[..., first] = 1
    y, _ = hq.hq_rope(x, None, pos, t, layout=layout)
    want = orope.rotate(x.double().cpu().numpy(), pos.cpu().numpy(), w, amp, ("half", "interleaved")[layout])
    err = np.abs(y.double().cpu().numpy() - want)
    tol = (2.0 ** -22 + 2.0 ** -23) * np.abs(want) + 2.0 ** -28
    assert (err <= tol).all(), (err / tol).max()


# ----------------------------------------------------------------------------- many tokens: heads that share their sines

@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (256, 32), (80, 20), (80, 40), (96, 24), (64, 18), (34, 34), (66, 2), (7, 6), (512, 256)])
def test_many_tokens(dtype, layout, D, rot):
    """The block's tokens and heads in every access width: out of views into fused rows with a copied rest, into a
    transposed output, in place, and one tensor in place beside one that is copied."""
    hq = _hq()
    B, T, Hq, Hkv = 2, 2503, 5, 2
    torch.manual_seed(D * rot)
    row = torch.randn(B, T, Hq + 2 * Hkv, D, device="cuda").to(TYPES[dtype])
    q, k, v = row[:, :, :Hq], row[:, :, Hq:Hq + Hkv], row[:, :, Hq + Hkv:]
    pos = torch.randint(0, 100000, (B, T), dtype=torch.int32, device="cuda")
    t, wa = _table(rot, "bands" if rot > 2 else "plain")
    lay = ("half", "interleaved").index(layout)
    yq, yk = hq.hq_rope(q, k, pos, t, layout=lay)
    _check(q, yq, pos, wa, layout, dtype)
    _check(k, yk, pos, wa, layout, dtype)
    out = torch.full((B, Hq + 1, T, D), 7.0, device="cuda", dtype=TYPES[dtype])
    hq.hq_rope(q, None, pos, t, layout=lay, q_out=out[:, :Hq].transpose(1, 2))
    # (not the same to the bit: the kernels for few and for many tokens fuse a product each with their sum)
    _check(q, out[:, :Hq].transpose(1, 2), pos, wa, layout, dtype)
    assert (out[:, Hq] == 7).all()
    v0, q0, k0 = v.clone(), q.clone(), k.clone()
    z, _ = hq.hq_rope(q, k, pos, t, layout=lay, k_out=k)            # k in place, q copied
    _check(q, z, pos, wa, layout, dtype)
    _check(k0, k, pos, wa, layout, dtype)
    assert torch.equal(q, q0) and torch.equal(v, v0)
    hq.hq_rope(q, None, pos, t, layout=lay, q_out=q)                  # in place
    _check(q0, q, pos, wa, layout, dtype)
    _check(k0, k, pos, wa, layout, dtype)
    assert torch.equal(v, v0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 0), (8, 1), (9, 8), (33, 8), (70, 10)])
def test_many_tokens_of_many_heads(dtype, Hq, Hkv):
    """Heads that the block's threads share out unevenly, rows at an odd offset (single elements), the gradient."""
    hq = _hq()
    T = 1501
    torch.manual_seed(Hq)
    wide = torch.randn(T, Hq + Hkv, 131, device="cuda").to(TYPES[dtype])
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 37
    t, wa = _table(96)
    for x in (wide[..., :128], wide[..., 1:129], wide[..., :128].contiguous()):
        for grad in (False, True):
            yq, yk = hq.hq_rope(x[:, :Hq], x[:, Hq:] if Hkv else None, pos, t, grad=grad)
            _check(x[:, :Hq], yq, pos, wa, "half", dtype, grad)
            if Hkv:
                _check(x[:, Hq:], yk, pos, wa, "half", dtype, grad)


def test_a_captured_step_with_its_gradient():
    """Forward and gradient captured into a graph, and replayed on other inputs.  (While an eager graph of the same leaf
    lives, torch itself ends such a capture, whatever the operators: it synchronises with the leaf's stream.)"""
    hq = _hq()
    t, wa = _table(64)
    pos = torch.arange(7, dtype=torch.int32, device="cuda")
    x = torch.randn(7, 2, 64, device="cuda", requires_grad=True)
    g = torch.randn(7, 2, 64, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.autograd.grad(hq.hq_rope(x, None, pos, t)[0], x, g)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = hq.hq_rope(x, None, pos, t)
        d, = torch.autograd.grad(y, x, g)
    for i in range(3):
        with torch.no_grad():
            x.copy_(torch.randn_like(x))
        g.copy_(torch.randn_like(g))
        pos += 1000
        graph.replay()
        torch.cuda.synchronize()
        _check(x.detach(), y.detach(), pos, wa, "half", "f32")
        _check(g, d, pos, wa, "half", "f32", grad=True)
