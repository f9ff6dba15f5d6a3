"""The 8-bit block cache on the GPU against the float64 oracle.

Codes, scales and the 16-bit tail are exact.  Read back: code * scale is one
float32 product (2^-24), then half a step of the output type.

Attention, for row r with weights p and values v:
    |out - want| <= eps(t)/2 |want| + (2^-11 + 2^-15 + 3 dS) sum_j p_j |v_j|
  eps(t)/2   the output's rounding
  2^-11      the weights' rounding to fp16
  2^-15      float32 sums of the weights and products, the exponentials' 2^-22
             and the running references' rescalings, a few per block
  dS         a score's error in nats: 128 float32 products and sums of size at
             most S = sum_d |q_d k_d| sm_scale, 2^-18 S with the scales' and the
             base-2 factor's roundings; a weight's relative error is twice that
             (its own and the denominator's), and half as much again for the bound's
             own slack
The denominator's log: (dS + 2^-15) / ln 2 and its own rounding.
"""
import numpy as np
import pytest
import torch

from oracle import kv8 as okv

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _hq():
    from hybrid_precision_attention_b200 import hq
    return hq


def _fmt(fmt):
    return {"e4m3": _hq().KV8_E4M3, "int8": _hq().KV8_INT8}[fmt]


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Pair:
    """A cache on the GPU and its sequences' oracles, fed the same rows."""

    def __init__(self, B, Hkv, cap, fmt="e4m3", dtype="f16", paged=True, seed=0, spread=1.0):
        hq = _hq()
        self.rng = np.random.default_rng(seed)
        self.B, self.Hkv, self.fmt, self.dtype, self.spread = B, Hkv, fmt, dtype, spread
        order = self.rng.permutation(B * Hkv * ((cap + 127) // 128 * 2)) if paged else None
        self.c = hq.Kv8Cache(B, Hkv, cap, fmt=_fmt(fmt), paged=paged, page_order=order)
        self.ref = [okv.Kv8Ref(Hkv, fmt) for _ in range(B)]

    def rows(self, n):
        x = self.rng.standard_normal((n, self.Hkv, 128)) * self.spread
        return torch.from_numpy(x).to(TYPES[self.dtype])

    def append(self, news, at=None, k=None, v=None, stream=None):
        """news[b] rows to each sequence; at[b]: position of the first (default: the end)."""
        hq = _hq()
        N = sum(news)
        k = self.rows(N) if k is None else k
        v = self.rows(N) if v is None else v
        cu = np.concatenate(([0], np.cumsum(news)))
        for b, n in enumerate(news):
            self.ref[b].append(k[cu[b]:cu[b + 1]].double().numpy(), v[cu[b]:cu[b + 1]].double().numpy(), None if at is None else at[b])
        self.cu, self.len = _ints(cu.tolist()), _ints([r.len for r in self.ref])
        hq.hq_kv8_append(self.c, k.cuda(), v.cuda(), self.cu, self.len, stream=stream)

    def check_stored(self):
        """Codes, scales and tail of every position, exactly."""
        hq = _hq()
        pages = self.c.pages.reshape(-1, hq.KV8_PAGE_BYTES).cpu().numpy()
        table = self.c.page_table.cpu().numpy() if self.c.page_table is not None else \
            np.arange(self.B * self.Hkv * self.c.npg).reshape(self.B, self.Hkv, -1)
        tails = [self.c.tail_k.cpu().numpy(), self.c.tail_v.cpu().numpy()]
        unit = self.c.tail_scale.cpu().numpy()
        r, d = np.arange(64)[:, None], np.arange(128)[None]
        for b, ref in enumerate(self.ref):
            for which in range(2):
                codes, scales = ref.blocks(which)
                full = codes.shape[1]
                p = pages[table[b, :, :full]]
                got = okv.code_values(okv.page_rows(p[..., 8192 * which:8192 * which + 8192], which), self.fmt)
                s = np.ascontiguousarray(p[..., 16384 + 4 * which:16388 + 4 * which]).view(np.float32)[..., 0]
                assert np.array_equal(s, scales, equal_nan=True) and np.array_equal(got, codes)
                x = ref.x[which][:, full * 64:]
                n = x.shape[1]
                if n:
                    t = tails[which][b, :, full % 2][:, (okv.k_index, okv.v_index)[which](r, d)][:, :n].astype(np.float64)
                    u = unit[b, :, which, full % 2 * 64:full % 2 * 64 + n].astype(np.float64)
                    fine = np.isfinite(x).all(-1)
                    assert np.array_equal(np.isfinite(u), fine) and np.isfinite(t).all() and not t[~fine].any()
                    assert np.array_equal((t * np.where(fine, u, 0)[..., None])[fine], x[fine])
                    if self.dtype == "f16":
                        assert (u[fine] == 1).all()

    def attend(self, G, n, window=0, q=None, check=True, sm=None, **kw):
        """The newest n[b] positions of each sequence attend; compared with the oracle."""
        hq = _hq()
        N, Hq = sum(n), G * self.Hkv
        cu = np.concatenate(([0], np.cumsum(n)))
        if q is None:
            q = torch.from_numpy(self.rng.standard_normal((N, Hq, 128))).to(TYPES[self.dtype])
        sm = 128 ** -0.5 if sm is None else sm
        out, lse = hq.hq_kv8_attn(self.c, q.cuda(), _ints(cu.tolist()), _ints([r.len for r in self.ref]), max(n), sm_scale=sm,
                                  window=window, return_lse=True, **kw)
        torch.cuda.synchronize()
        assert not any(self.c.errors())
        if check:
            for b, ref in enumerate(self.ref):
                if n[b]:
                    check_rows(out[cu[b]:cu[b + 1]], lse[cu[b]:cu[b + 1]], ref, q[cu[b]:cu[b + 1]].double().numpy(), sm, window,
                               self.dtype)
        return q, out, lse


def check_rows(out, lse, ref, q, sm, window, dtype):
    want, wlse, mass, size = ref.attend(q, sm, window)
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    dS = 2.0 ** -18 * size
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    tol = torch.finfo(TYPES[dtype]).eps / 2 * np.abs(want) + (2.0 ** -11 + 2.0 ** -15 + 3 * dS[..., None]) * mass + 2.0 ** -25
    err = np.abs(got - want)
    assert (err[~nan] <= tol[~nan]).all(), (err / tol)[~nan].max()
    fine = ~np.isnan(wlse)
    assert np.array_equal(~np.isnan(glse), fine)
    ltol = (dS + 2.0 ** -15) * 1.4427 + 2.0 ** -22 * np.abs(wlse)
    assert (np.abs(glse - wlse)[fine] <= ltol[fine]).all()


FORMS = [("e4m3", "f16"), ("int8", "f16"), ("e4m3", "bf16"), ("int8", "bf16")]


# ----------------------------------------------------------------------------- write and read back

@pytest.mark.parametrize("fmt,dtype", FORMS)
@pytest.mark.parametrize("paged", [True, False])
def test_append_in_any_split(fmt, dtype, paged):
    """The same store whatever the calls: single tokens, odd runs, runs over several blocks from mid-block, none."""
    p = Pair(5, 3, 700, fmt, dtype, paged, seed=1, spread=3.0)
    p.append([64, 1, 0, 200, 130])
    p.check_stored()
    p.append([1, 62, 3, 0, 129])
    p.check_stored()
    p.append([63, 1, 250, 327, 5])
    p.check_stored()
    for n in ([1, 1, 1, 1, 1], [1, 0, 1, 0, 0], [5, 2, 8, 61, 127], [60, 100, 300, 5, 64]):
        p.append(n)
        p.check_stored()
    assert not any(p.c.errors())


@pytest.mark.parametrize("fmt,dtype", FORMS)
def test_token_by_token(fmt, dtype):
    p = Pair(2, 2, 256, fmt, dtype, seed=2, spread=0.01)
    for i in range(200):
        p.append([1, i % 2])
        if i % 21 == 0 or i in (62, 63, 64, 127, 128, 199):
            p.check_stored()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_take_back_drafted_tokens(dtype):
    """An append that starts up to 64 positions before the end replaces what followed, over block borders too."""
    p = Pair(4, 2, 512, "e4m3", dtype, seed=3)
    p.append([100, 130, 64, 191])
    p.append([8, 8, 8, 64])
    p.append([5, 61, 3, 3], at=[103, 131, 64, 192])
    p.check_stored()
    p.append([64, 1, 64, 1], at=[104, 128, 3, 192])
    p.check_stored()
    p.append([30, 70, 1, 130])
    p.check_stored()
    assert not any(p.c.errors())


def test_values_at_the_edges_of_the_types():
    """Zero blocks, subnormals, the largest values, one outlier a block; scales from 2^-30 to 2^7."""
    for dtype in ("f16", "bf16"):
        for fmt in ("e4m3", "int8"):
            p = Pair(1, 1, 640, fmt, dtype, seed=4)
            big = torch.finfo(TYPES[dtype]).max
            x = torch.zeros(640, 1, 128, dtype=torch.float64)
            g = torch.Generator().manual_seed(5)
            r = torch.randn(640, 1, 128, generator=g, dtype=torch.float64)
            x[64:128] = r[64:128] * 2.0 ** -24
            x[128:192] = r[128:192].clamp(-1, 1) * (60000.0 if dtype == "f16" else 1e30)
            x[192:256] = r[192:256]
            x[200, 0, 5] = big if dtype == "f16" else 3e38
            x[256:320] = torch.sign(r[256:320]) * 2.0 ** -14
            x[320:384] = r[320:384] * 2.0 ** torch.randint(-12, 8, (64, 1, 1), generator=g)
            x[384:448, 0, 0] = 448.0
            x[384:448, 0, 1:100] = torch.arange(99) * 0.5 + 0.25          # ties of both formats' codes
            x[448:600] = r[448:600] * 1e-3
            x = x.to(TYPES[dtype])
            p.append([600], k=x[:600], v=-x[:600])
            p.check_stored()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_scales_at_the_ends_of_float32(fmt):
    """bf16 blocks whose scale is subnormal (the quotients pass the format's largest value and are clipped), tiny, and
    as large as the type allows: codes by the division of the definition."""
    p = Pair(1, 1, 512, fmt, "bf16", seed=30)
    g = torch.Generator().manual_seed(31)
    x = torch.randn(384, 1, 128, generator=g, dtype=torch.float64)
    for i, s in enumerate((1e-39, 3e-38, 2.0 ** -100, 2.0 ** 90, 1e37, 1.0)):
        x[64 * i:64 * i + 64] *= s
    x = x.to(torch.bfloat16)
    p.append([384], k=x, v=-x)
    p.check_stored()


def test_not_finite_rows_mark_their_block():
    p = Pair(2, 2, 256, "e4m3", "f16", seed=6)
    k, v = p.rows(200 + 70), p.rows(200 + 70)
    k[3, 1, 7], v[130, 0, 100] = float("inf"), float("nan")
    v[200 + 66, 1, 0] = float("-inf")                                    # in the second sequence's tail
    p.append([200, 70], k=k, v=v)
    p.check_stored()
    hq = _hq()
    K, V = hq.hq_kv8_read(p.c, p.len, n=200)
    bad = torch.isnan(K[0]).any(-1).nonzero().tolist()
    assert bad == [[1, i] for i in range(64)]
    assert torch.isnan(V[0]).any(-1).nonzero().tolist() == [[0, i] for i in range(128, 192)]
    assert torch.isnan(V[1]).any(-1).nonzero().tolist() == [[1, 66]]
    p.append([0, 58])                                                     # the tail's row makes its block NaN
    p.check_stored()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("start,n", [(0, 300), (0, 1), (37, 200), (64, 64), (250, 6), (299, 1), (0, 0), (383, 1)])
def test_read_back(fmt, out, start, n):
    hq = _hq()
    p = Pair(4, 2, 384, fmt, "f16", seed=7)
    p.append([300, 0, 64, 129])
    want = [[r.cached(i) for i in range(2)] for r in p.ref]
    K, V = hq.hq_kv8_read(p.c, p.len, start=start, n=n, dtype=TYPES[out])
    # into the caller's own padded buffers, the rest left as it is
    buf = torch.full((2, 4, n, 3, 136), 9.0, dtype=TYPES[out], device="cuda")
    k2, v2 = buf[0, :, :, :2, :128].transpose(1, 2), buf[1, :, :, :2, :128].transpose(1, 2)
    hq.hq_kv8_read(p.c, p.len, start=start, n=n, k_out=k2, v_out=v2, zero_rest=False)
    for which, (x, y) in enumerate(((K, k2), (V, v2))):
        for b in range(4):
            w = want[b][which][:, start:start + n]
            m = w.shape[1]
            got = x[b].double().cpu().numpy()
            tol = (torch.finfo(TYPES[out]).eps / 2 + 2.0 ** -24) * np.abs(w) * (1 + 2.0 ** -9) + 2.0 ** -25
            assert (np.abs(got[:, :m] - w) <= tol).all() and not got[:, m:].any()
            assert torch.equal(y[b, :, :m], x[b, :, :m]) and (y[b, :, m:] == 9).all()
    assert (buf[..., 2, :] == 9).all() and (buf[..., 128:] == 9).all()
    assert not any(p.c.errors())


def test_strided_rows_of_the_fused_projection():
    hq = _hq()
    row = torch.randn(75, 8 + 2 * 2, 128, device="cuda").half()
    c = hq.Kv8Cache(2, 2, 128)
    cu, n = _ints([0, 70, 75]), _ints([70, 5])
    hq.hq_kv8_append(c, row[:, 8:10], row[:, 10:], cu, n)
    d = hq.Kv8Cache(2, 2, 128)
    hq.hq_kv8_append(d, row[:, 8:10].contiguous(), row[:, 10:].contiguous(), cu, n)
    assert torch.equal(c.pages, d.pages) and torch.equal(c.tail_k, d.tail_k) and torch.equal(c.tail_v, d.tail_v)
    q = row[:, :8]
    buf = torch.full((75, 10, 128), 3.0, device="cuda").half()
    o = hq.hq_kv8_attn(c, q, cu, n, 70, out=buf[:, 1:9])
    assert torch.equal(o, hq.hq_kv8_attn(d, q.contiguous(), cu, n, 70)) and (buf[:, [0, 9]] == 3).all()


# ----------------------------------------------------------------------------- attention

@pytest.mark.parametrize("fmt,dtype", FORMS)
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 2), (3, 4), (1, 5), (2, 8), (1, 16)])
def test_single_tokens(fmt, dtype, Hkv, G):
    """One token of each sequence, at lengths around the block borders."""
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 100, 127, 128, 129, 192, 333, 0, 640]
    p = Pair(len(lens), Hkv, 640, fmt, dtype, seed=8)
    p.append(lens)
    p.attend(G, [min(n, 1) for n in lens])


@pytest.mark.parametrize("fmt,dtype", FORMS)
@pytest.mark.parametrize("G,n", [(1, 2), (4, 2), (8, 1), (4, 5), (8, 8), (3, 7), (1, 17), (2, 40)])
def test_drafted_tokens(fmt, dtype, G, n):
    lens = [n, n + 1, 63, 64, 65, 70, 128, 131, 200, 0]
    lens = [0 if m == 0 else max(m, n) for m in lens]
    p = Pair(len(lens), 2, 256, fmt, dtype, seed=9)
    p.append(lens)
    p.attend(G, [min(m, max(1, n - b)) for b, m in enumerate(lens)])


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 100, 1000])
@pytest.mark.parametrize("n", [1, 6, 70])
def test_window(window, n):
    lens = [n, 64 + n, 128, 300, 257]
    lens = [max(m, n) for m in lens]
    p = Pair(len(lens), 2, 384, "e4m3", "f16", seed=10)
    p.append(lens)
    p.attend(4, [n] * len(lens), window=window)


@pytest.mark.parametrize("fmt,dtype", FORMS)
@pytest.mark.parametrize("L,n,G", [(128, 128, 4), (200, 200, 2), (333, 150, 8), (700, 300, 1), (1111, 129, 4)])
def test_chunks(fmt, dtype, L, n, G):
    """Chunks of a prompt: from the first position, from inside a block, alone and beside a shorter one."""
    p = Pair(2, 1, 1152, fmt, dtype, seed=11)
    p.append([L, L // 2])
    p.attend(G, [n, min(n, L // 2) // 3 + 1])


@pytest.mark.parametrize("fmt,dtype", [("e4m3", "f16"), ("int8", "bf16")])
def test_long_contexts_split_over_the_grid(fmt, dtype):
    p = Pair(2, 2, 9000, fmt, dtype, seed=12)
    p.append([8999, 4100])
    p.attend(4, [1, 1])
    p.attend(4, [3, 1])
    p.attend(8, [2, 16], window=5000)


def test_sharp_and_flat_softmax():
    """Scores far apart (one key takes all the weight) and all alike, at several scales."""
    for sm in (1e-6, 0.05, 2.0):
        p = Pair(2, 1, 512, "e4m3", "f16", seed=13, spread=2.0)
        p.append([500, 321])
        p.attend(4, [2, 2], sm=sm)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_blocks_whose_scales_lie_far_apart(dtype):
    """Values of 2^-20 in some blocks and 2^12 in others, the weight on either: the accumulators keep both."""
    p = Pair(1, 1, 512, "e4m3", dtype, seed=14)
    k, v = p.rows(400).double(), p.rows(400).double()
    q = torch.zeros(1, 4, 128, dtype=torch.float64)
    q[0, :, 0] = torch.tensor([6.0, -6.0, 3.0, 0.0])
    k[:, 0, 0] = torch.where(torch.arange(400) // 64 % 2 == 0, 30.0, -30.0)
    v = v * torch.where(torch.arange(400) // 64 % 2 == 0, 2.0 ** -13, 2.0 ** 12)[:, None, None]
    p.append([400], k=k.to(TYPES[dtype]), v=v.to(TYPES[dtype]))
    p.attend(4, [1], q=q.to(TYPES[dtype]))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_large_and_small_queries(dtype):
    p = Pair(1, 1, 256, "int8", dtype, seed=15)
    p.append([200])
    q = torch.from_numpy(p.rng.standard_normal((3, 4, 128)))
    q[:, 1] *= 2.0 ** -14
    q[:, 2] *= 1000.0 if dtype == "f16" else 1e6
    q[:, 3] = 0
    p.attend(4, [3], q=q.to(TYPES[dtype]))
    if dtype == "bf16":
        q = torch.from_numpy(p.rng.standard_normal((1, 4, 128)))
        q[0, 0] *= 1e30
        q[0, 1] *= 1e-38
        p.attend(4, [1], q=q.to(torch.bfloat16), sm=1e-30)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_not_finite_values_behind_the_mask(fmt):
    """Rows that a query must not see (later drafted tokens, positions before its window) do not reach it; rows that
    it sees do."""
    p = Pair(1, 1, 512, fmt, "f16", seed=16)
    k, v = p.rows(330), p.rows(330)
    k[10, 0, 3], v[20, 0, 5] = float("nan"), float("inf")                # block 0
    k[328, 0, 1], v[329, 0, 2] = float("inf"), float("nan")              # the last two of four new tokens
    p.append([330], k=k, v=v)
    _, out, lse = p.attend(4, [4], window=100)
    assert torch.isfinite(out[:2]).all() and torch.isnan(out[2:]).all()
    _, out, _ = p.attend(4, [4])
    assert torch.isnan(out).all()
    # a window that starts inside the marked block: the block's scale marks all its rows
    p2 = Pair(1, 1, 512, fmt, "f16", seed=17)
    k, v = p2.rows(130), p2.rows(130)
    v[0, 0, 0] = float("inf")
    p2.append([130], k=k, v=v)
    _, out, _ = p2.attend(2, [1], window=66)
    assert torch.isfinite(out).all()
    _, out, _ = p2.attend(2, [1], window=67)
    assert torch.isnan(out).all()


def test_a_query_that_is_not_finite_stays_alone():
    p = Pair(1, 1, 256, "e4m3", "bf16", seed=18)
    p.append([150])
    q = torch.from_numpy(p.rng.standard_normal((2, 4, 128))).bfloat16()
    q[0, 1, 5], q[1, 2, 0] = float("nan"), float("nan")
    _, out, lse = p.attend(4, [2], q=q, check=False)
    bad = torch.isnan(out).all(-1)
    assert bad.nonzero().tolist() == [[0, 1], [1, 2]] and torch.equal(torch.isnan(lse), bad)
    assert torch.equal(torch.isnan(out).any(-1), bad)


def test_rows_that_no_sequence_has_are_left():
    """Rows before cu[0], behind cu[B], and of sequences that are refused keep what they held."""
    hq = _hq()
    p = Pair(4, 2, 256, "e4m3", "f16", seed=19)
    p.append([100, 60, 30, 200])
    q = torch.randn(20, 8, 128, device="cuda").half()
    out, lse = torch.full_like(q, 5.0), torch.full((20, 8), 5.0, device="cuda")
    cu = _ints([2, 4, 4, 10, 13])
    hq.hq_kv8_attn(p.c, q, cu, _ints([100, 60, 5, 257]), 6, out=out, lse=lse)
    assert p.c.errors() == [0, 0, hq.DEVERR_ROWS, hq.DEVERR_CAPACITY]
    keep = [0, 1] + list(range(4, 20))
    assert (out[keep] == 5).all() and (lse[keep] == 5).all() and (out[2:4] != 5).any()
    check_rows(out[2:4], lse[2:4], p.ref[0], q[2:4].double().cpu().numpy(), 128 ** -0.5, 0, "f16")


def test_inconsistent_rows_are_refused_on_the_device():
    hq = _hq()
    p = Pair(3, 1, 256, "e4m3", "f16", seed=20)
    p.append([64, 64, 64])
    before = [t.clone() for t in (p.c.pages, p.c.tail_k, p.c.tail_v, p.c.tail_scale)]
    k = torch.randn(6, 1, 128, device="cuda").half()
    q = torch.randn(6, 2, 128, device="cuda").half()
    for cu, lens, want in (([0, 7, 7, 7], [70, 64, 64], [32, 32, 32]), ([0, 3, 1, 6], [67, 64, 69], [0, 32, 0]),
                           ([-4, 2, 2, 2], [70, 64, 64], [32, 0, 0]), ([0, 2, 4, 6], [1, -5, 300], [32, 32, 2])):
        p.c.err.zero_()
        out = torch.full_like(q, 5.0)
        hq.hq_kv8_attn(p.c, q, _ints(cu), _ints(lens), 6, out=out)
        assert p.c.errors() == want
        if 0 not in want:
            assert (out == 5).all()
        p.c.err.zero_()
        if 0 in want:                      # the sequences that fit are written: only the flags are compared
            d = hq.Kv8Cache(3, 1, 256)
            hq.hq_kv8_append(d, k, k, _ints(cu), _ints(lens))
            assert d.errors() == want
        else:
            hq.hq_kv8_append(p.c, k, k, _ints(cu), _ints(lens))
            assert p.c.errors() == want
            assert all(torch.equal(a, b) for a, b in zip(before, (p.c.pages, p.c.tail_k, p.c.tail_v, p.c.tail_scale)))
    p.c.err.zero_()                        # more new tokens than the call allows
    out = torch.full_like(q, 5.0)
    hq.hq_kv8_attn(p.c, q, _ints([0, 2, 4, 6]), _ints([64, 64, 64]), 1, out=out)
    assert p.c.errors() == [32, 32, 32] and (out == 5).all()


def test_bad_page_entries():
    hq = _hq()
    c = hq.Kv8Cache(2, 1, 256, paged=True, n_pages=8)
    c.page_table[0, 0, 1], c.page_table[1, 0, 0] = 8, -1
    k = torch.randn(260, 1, 128, device="cuda").half()
    pages = c.pages.clone()
    hq.hq_kv8_append(c, k, k, _ints([0, 130, 260]), _ints([130, 130]))
    assert c.errors() == [hq.DEVERR_PAGE] * 2
    changed = (c.pages != pages).any(-1).nonzero().flatten().tolist()
    assert changed == [0, 5]               # the good entries' pages alone
    c.err.zero_()
    hq.hq_kv8_read(c, _ints([130, 130]), n=130)
    assert c.errors() == [hq.DEVERR_PAGE] * 2
    c.err.zero_()
    hq.hq_kv8_attn(c, torch.randn(2, 2, 128, device="cuda").half(), _ints([0, 1, 2]), _ints([130, 130]), 1)
    assert c.errors() == [hq.DEVERR_PAGE] * 2


def test_pages_beyond_two_gigabytes():
    """A pool whose last pages start past 2^31 bytes."""
    hq = _hq()
    n = (1 << 31) // hq.KV8_PAGE_BYTES + 40
    p = Pair(1, 2, 512, "e4m3", "f16", paged=False, seed=21)
    p.c = hq.Kv8Cache(1, 2, 512, paged=True, n_pages=n, page_order=list(range(n - 16, n)))
    p.append([450])
    p.check_stored()
    p.attend(4, [1])
    p.attend(4, [30])
    K, _ = hq.hq_kv8_read(p.c, p.len, n=450, dtype=torch.float32)
    assert np.abs(K[0].double().cpu().numpy() - p.ref[0].cached(0)).max() <= 2.0 ** -20


def test_many_sequences():
    lens = [(37 * i) % 150 for i in range(600)]
    p = Pair(600, 1, 256, "int8", "f16", seed=22)
    p.append(lens)
    p.check_stored()
    _, out, _ = p.attend(2, [min(1, n) for n in lens])
    p.append([1] * 600)
    p.attend(2, [1] * 600)


def test_shared_full_pages():
    """Two sequences over the same prefix pages, each with its own continuation."""
    hq = _hq()
    p = Pair(2, 1, 256, "e4m3", "f16", seed=23)
    k, v = p.rows(128), p.rows(128)
    p.c.page_table[0, 0] = _ints([0, 1, 2, 3])
    p.c.page_table[1, 0] = _ints([0, 1, 4, 5])
    p.append([128, 0], k=k, v=v)
    p.ref[1].append(k.double().numpy(), v.double().numpy())
    p.append([70, 5])
    p.check_stored()
    p.attend(4, [2, 1])


# ----------------------------------------------------------------------------- streams, graphs, repeated calls

def test_repeated_calls_give_the_same_bits():
    p = Pair(3, 2, 4096, "e4m3", "f16", seed=24)
    p.append([4000, 1500, 70])
    for n in ([1, 1, 1], [5, 3, 1], [200, 64, 70]):
        q, out, lse = p.attend(4, n, check=False)
        for _ in range(5):
            _, o, z = p.attend(4, n, q=q, check=False)
            assert torch.equal(o, out) and torch.equal(z, lse)


def test_two_streams_at_once():
    p = Pair(2, 4, 8192, "e4m3", "f16", seed=25)
    p.append([8000, 5001])
    q, out, _ = p.attend(4, [1, 1], check=False)
    q2, out2, _ = p.attend(4, [4, 4], check=False)
    hq = _hq()
    cu, cu2, n = _ints([0, 1, 2]), _ints([0, 4, 8]), _ints([8000, 5001])
    qd, qd2 = q.cuda(), q2.cuda()
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        got[0].append(hq.hq_kv8_attn(p.c, qd, cu, n, 1, stream=s[0]))
        got[1].append(hq.hq_kv8_attn(p.c, qd2, cu2, n, 4, stream=s[1]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, out) for x in got[0]) and all(torch.equal(x, out2) for x in got[1])


def test_captured_steps():
    """A decode step (append and attend) captured once and replayed as the lengths advance; two graphs replayed at the
    same time share no scratch."""
    hq = _hq()
    p = Pair(3, 2, 512, "e4m3", "f16", seed=26)
    p.append([62, 130, 1])
    k, v = torch.empty(3, 2, 128, device="cuda").half(), torch.empty(3, 2, 128, device="cuda").half()
    q = torch.randn(3, 8, 128, device="cuda").half()
    cu, n = _ints([0, 1, 2, 3]), p.len.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n += 1
        hq.hq_kv8_append(p.c, k, v, cu, n)
        out, lse = hq.hq_kv8_attn(p.c, q, cu, n, 1, return_lse=True)
    for _ in range(5):
        x, y = p.rows(3), p.rows(3)
        k.copy_(x)
        v.copy_(y)
        for b in range(3):
            p.ref[b].append(x[b:b + 1].double().numpy(), y[b:b + 1].double().numpy())
        graph.replay()
        torch.cuda.synchronize()
        for b in range(3):
            check_rows(out[b:b + 1], lse[b:b + 1], p.ref[b], q[b:b + 1].double().cpu().numpy(), 128 ** -0.5, 0, "f16")
    p.check_stored()
    both, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in both:
        with torch.cuda.graph(g):
            outs.append(hq.hq_kv8_attn(p.c, q, cu, n, 1))
    want = hq.hq_kv8_attn(p.c, q, cu, n, 1)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for g, st in zip(both, s):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_workspace_of_the_caller():
    hq = _hq()
    p = Pair(1, 2, 4096, "e4m3", "f16", seed=27)
    p.append([4000])
    q, out, _ = p.attend(4, [1], check=False)
    need = hq._lib.hq_kv8_attn_workspace_bytes(p.c.ref, 8, 1)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(hq.hq_kv8_attn(p.c, q.cuda(), _ints([0, 1]), p.len, 1, ws=ws), out)
    with pytest.raises(hq.HqError, match="workspace"):
        hq.hq_kv8_attn(p.c, q.cuda(), _ints([0, 1]), p.len, 1, ws=ws[:-16])


def test_refusals_of_the_binding():
    hq = _hq()
    c = hq.Kv8Cache(2, 2, 128)
    k = torch.randn(4, 2, 128, device="cuda").half()
    q = torch.randn(4, 4, 128, device="cuda").half()
    cu, n = _ints([0, 2, 4]), _ints([2, 2])
    for a in ((k.float(), k.float(), cu, n), (k, k.bfloat16(), cu, n), (k[:, :1], k[:, :1], cu, n), (k, k[:3], cu, n),
              (k, k, cu.long(), n), (k, k, cu[:2], n), (k, k, cu, n.cpu()), (k.transpose(1, 2), k, cu, n), (k.cpu(), k.cpu(), cu, n)):
        with pytest.raises(hq.HqError):
            hq.hq_kv8_append(c, *a)
    for a, kw in (((q.float(), cu, n, 2), {}), ((q[:, :3], cu, n, 2), {}), ((q, cu, n, -1), {}), ((q, cu, n, 2), dict(window=-1)),
                  ((q, cu, n, 2), dict(out=q[:3])), ((q, cu, n, 2), dict(out=q.bfloat16())), ((q, cu, n, 2), dict(sm_scale=0.0)),
                  ((q, cu, n, 2), dict(lse=torch.empty(4, 3, device="cuda"))), ((q[..., :64], cu, n, 2), {})):
        with pytest.raises(hq.HqError):
            hq.hq_kv8_attn(c, *a, **kw)
    for kw in (dict(n=129), dict(start=-1), dict(n=-2), dict(zero_rest=False), dict(k_out=k), dict(start=128, n=1)):
        with pytest.raises(hq.HqError):
            hq.hq_kv8_read(c, n, **kw)
    with pytest.raises(hq.HqError):
        hq.Kv8Cache(2, 2, 128, D=64)
    with pytest.raises(hq.HqError):
        hq.Kv8Cache(2, 2, 128, page_table=_ints([0]))
    hq.hq_kv8_append(c, k[:0], k[:0], _ints([0, 0, 0]), _ints([0, 0]))
    assert hq.hq_kv8_attn(c, q[:0], _ints([0, 0, 0]), _ints([0, 0]), 1).shape == (0, 4, 128)
    assert not any(c.errors())


# ----------------------------------------------------------------------------- where the kernels change

@pytest.mark.parametrize("fmt,dtype", FORMS)
@pytest.mark.parametrize("G,n", [(8, 3), (5, 5), (2, 13), (8, 16), (1, 129), (3, 43), (2, 128), (1, 257), (16, 17), (7, 40)])
def test_row_counts_around_the_kernels_borders(fmt, dtype, G, n):
    """24 and 25 rows of a kv head (a second task), 128 and 129 (the tcgen05 kernel's second row tile), 256 and more
    (further tasks), with sequences of fewer rows beside."""
    p = Pair(3, 2, 640, fmt, dtype, seed=32)
    p.append([600, max(n, 129), 300])
    p.attend(G, [n, n, max(1, n // 3)])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("G,n", [(8, 4), (3, 11), (1, 47), (16, 3), (4, 12), (7, 7), (8, 8)])
def test_row_counts_of_two_tasks(dtype, G, n):
    """25 to 48 rows are two tasks of a kv head, 49 go to the tcgen05 kernel; sequences of one task, of none and of
    cut tasks beside, with windows."""
    p = Pair(5, 2, 4096, "e4m3", dtype, seed=42)
    p.append([4000, 100, 77, 1, 2000])
    p.attend(G, [n, max(1, 24 // G), 0, 1, n])
    p.attend(G, [n, n, 1, 0, min(n, 3)], window=65)
    p.append([1, 28, 0, 0, 48])
    p.attend(G, [n, n, n, 1, 1], window=1500)


@pytest.mark.parametrize("window", [1, 30, 64, 129, 500])
def test_window_of_many_rows(window):
    p = Pair(2, 1, 1024, "int8", "f16", seed=33)
    p.append([1000, 333])
    p.attend(8, [100, 30], window=window)
    p.attend(2, [50, 17], window=window)


def test_many_rows_over_a_long_context():
    """Pieces of one task on many CTAs, one and two row tiles."""
    p = Pair(1, 1, 20096, "e4m3", "bf16", seed=34)
    p.append([20001])
    p.attend(4, [10])
    p.attend(4, [40], window=15000)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_many_rows_and_blocks_whose_scales_lie_far_apart(dtype):
    p = Pair(1, 1, 512, "e4m3", dtype, seed=35)
    k, v = p.rows(400).double(), p.rows(400).double()
    q = torch.zeros(8, 8, 128, dtype=torch.float64)
    q[:, :, 0] = torch.tensor([6.0, -6.0, 3.0, 0.0, 1.0, -1.0, 0.1, -3.0])
    k[:, 0, 0] = torch.where(torch.arange(400) // 64 % 2 == 0, 30.0, -30.0)
    v = v * torch.where(torch.arange(400) // 64 % 2 == 0, 2.0 ** -13, 2.0 ** 12)[:, None, None]
    p.append([400], k=k.to(TYPES[dtype]), v=v.to(TYPES[dtype]))
    p.attend(8, [8], q=q.to(TYPES[dtype]))
    p.attend(8, [8], q=(-q).to(TYPES[dtype]), window=100)


def test_scores_that_rise_block_by_block():
    """Each block's scores pass the last one's by far more than the references allow: they are set anew every time."""
    for n in (1, 4, 40):
        p = Pair(1, 1, 1024, "e4m3", "f16", seed=36)
        k, v = p.rows(900), p.rows(900)
        k[:, 0, 0] = torch.arange(900) // 64 * 4.0
        q = torch.from_numpy(p.rng.standard_normal((n, 8, 128))).half()
        q[:, :4, 0], q[:, 4:, 0] = 60.0, -60.0
        p.append([900], k=k, v=v)
        p.attend(8, [n], q=q)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_many_rows_and_not_finite_values_behind_the_mask(fmt):
    p = Pair(1, 1, 512, fmt, "f16", seed=37)
    k, v = p.rows(330), p.rows(330)
    k[10, 0, 3], v[20, 0, 5] = float("nan"), float("inf")                # block 0
    k[325, 0, 1], v[328, 0, 2] = float("inf"), float("nan")              # among 20 new tokens, in the tail
    p.append([330], k=k, v=v)
    _, out, _ = p.attend(8, [20], window=200)
    assert torch.isfinite(out[:15]).all() and torch.isnan(out[15:]).all()
    _, out, _ = p.attend(8, [20])
    assert torch.isnan(out).all()
    q = torch.from_numpy(p.rng.standard_normal((20, 8, 128))).half()     # a query that is not finite stays alone
    q[3, 2, 9] = float("nan")
    _, out, _ = p.attend(8, [20], window=200, q=q, check=False)
    assert torch.isnan(out[3, 2]).all() and torch.isfinite(out[3, :2]).all() and torch.isfinite(out[:3]).all()


def test_many_rows_to_strided_outputs_and_untouched_ones():
    hq = _hq()
    p = Pair(3, 2, 512, "e4m3", "bf16", seed=38)
    p.append([300, 90, 500])
    q = torch.randn(140, 12, 128, device="cuda").bfloat16()[:, 2:10]
    buf, lse = torch.full((140, 9, 136), 5.0, device="cuda", dtype=torch.bfloat16), torch.full((140, 8), 5.0, device="cuda")
    cu = _ints([3, 60, 60, 130])
    hq.hq_kv8_attn(p.c, q, cu, p.len, 70, out=buf[:, :8, :128], lse=lse)
    assert p.c.errors() == [0, 0, 0]
    keep = [0, 1, 2] + list(range(130, 140))
    assert (buf[keep] == 5).all() and (lse[keep] == 5).all() and (buf[:, 8] == 5).all() and (buf[:, :, 128:] == 5).all()
    for b, (lo, hi) in ((0, (3, 60)), (2, (60, 130))):
        check_rows(buf[lo:hi, :8, :128], lse[lo:hi], p.ref[b], q[lo:hi].double().cpu().numpy(), 128 ** -0.5, 0, "bf16")


def test_calls_of_every_kernel_share_a_stream_and_its_scratch():
    """One token, drafts and chunks in turn on one stream and on two at once, and captured: the same bits as alone."""
    hq = _hq()
    p = Pair(2, 2, 4096, "e4m3", "f16", seed=39)
    p.append([4000, 2500])
    cases = []
    for G, n in ((4, [1, 1]), (8, [2, 1]), (4, [5, 6]), (4, [9, 20]), (4, [100, 300])):
        q, out, _ = p.attend(G, n, check=False)
        cases.append((q.cuda(), _ints([0, n[0], n[0] + n[1]]), max(n), out.clone()))
    call = lambda x, **kw: hq.hq_kv8_attn(p.c, x[0], x[1], p.len, x[2], **kw)
    for _ in range(3):
        for x in cases + cases[::-1]:
            assert torch.equal(call(x), x[3])
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    got = [(call(x, stream=s[i % 2]), x[3]) for i, x in enumerate(cases * 4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in got)
    graphs = []
    for x in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call(x)
        graphs.append((g, out, x[3]))
    for _ in range(3):
        for i, (g, _, _) in enumerate(graphs):
            with torch.cuda.stream(s[i % 2]):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for _, a, b in graphs)


def test_scratch_after_a_wait_that_gave_up():
    """errors() that tells of a timeout lets go of scratch whose counters may not be zero."""
    hq = _hq()
    p = Pair(1, 1, 4096, "e4m3", "f16", seed=40)
    p.append([4000])
    q, out, _ = p.attend(4, [1])
    assert len(p.c._ws) == 1
    for w in p.c._ws.values():
        w[:hq.KV8_WS_ZERO] = 1
    p.c.err[0] = hq.DEVERR_TIMEOUT
    assert p.c.errors() == [hq.DEVERR_TIMEOUT]
    p.c.err.zero_()
    assert torch.equal(hq.hq_kv8_attn(p.c, q.cuda(), _ints([0, 1]), p.len, 1), out)


def test_output_in_the_queries_place_is_refused():
    hq = _hq()
    p = Pair(1, 1, 128, "e4m3", "f16", seed=41)
    p.append([5])
    q = torch.randn(1, 4, 128, device="cuda").half()
    with pytest.raises(hq.HqError, match="hq_kv8_attn"):
        hq.hq_kv8_attn(p.c, q, _ints([0, 1]), p.len, 1, out=q)


# ----------------------------------------------------------------------------- together

@pytest.mark.parametrize("fmt,dtype", [("e4m3", "f16"), ("int8", "bf16")])
def test_a_layer_generates(fmt, dtype):
    """Rotary positions, append and attention as a serving loop calls them: two ragged prompts in chunks, then decode
    steps with drafted tokens, some of them taken back; each output against the oracle fed the rotated rows."""
    hq = _hq()
    Hq, Hkv, t = 8, 2, TYPES[dtype]
    p = Pair(2, Hkv, 512, fmt, dtype, seed=28)
    table = hq.RopeTable(64, 10000.0, kind=hq.ROPE_YARN, factor=4.0, orig_len=256)
    at = [0, 0]
    for news, kept in (([100, 37], [100, 37]), ([130, 0], [130, 0]), ([1, 1], [1, 1]), ([4, 4], [2, 4]), ([4, 4], [1, 1]), ([1, 64], [1, 64])):
        N = sum(news)
        row = torch.from_numpy(p.rng.standard_normal((N, Hq + 2 * Hkv, 128))).to(t).cuda()
        pos = _ints([at[b] + i for b in range(2) for i in range(news[b])])
        q, k = hq.hq_rope(row[:, :Hq], row[:, Hq:Hq + Hkv], pos, table)
        p.append(news, at=at, k=k.cpu(), v=row[:, Hq + Hkv:].cpu())
        p.attend(Hq // Hkv, news, q=q.cpu())
        at = [a + n for a, n in zip(at, kept)]
        for b in range(2):
            for i in range(2):
                p.ref[b].x[i] = p.ref[b].x[i][:, :at[b]]
    assert not any(p.c.errors())


def test_read_back_installs_a_hybrid_cache():
    """The read-back rows are the dense prefix that the hybrid cache's selection and install take."""
    hq = _hq()
    p = Pair(1, 2, 512, "e4m3", "f16", seed=29)
    p.append([400])
    K, V = hq.hq_kv8_read(p.c, p.len, n=400)
    h = hq.HybridCache(1, 8, 2, 512, W=64)
    q_tail = torch.randn(1, 8, 64, 128, device="cuda").half()
    hq.hq_select_vlines(h, K, q_tail)
    hq.hq_pack_merge(h, K, V)
    st = h.state()
    assert st["T"] == 400 and st["err"] == 0
    assert torch.equal(h.kr[0, :, 399 % h.R], K[0, :, 399]) and torch.equal(h.vr[0, :, 399 % h.R], V[0, :, 399])


# ----------------------------------------------------------------------------- values of any magnitude

# half the smallest number of the output's type: where the outputs themselves are small, check_rows' 2^-25 would pass anything
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def check_relative(p, b, q, out, sm=128 ** -0.5, window=0):
    """check_rows' bound on the output, relative to sum p |v| alone, with the weights' smallest step.

    A weight w_j = p_j s_j (s_j the scale of key j's value, c_j = v_j / s_j what the product takes) is rounded to fp16 at
    2^6 / E, E the reference of such weights, at most their largest (it is set to the largest met so far, and otherwise
    stays).  Below 2^-14 the step of fp16 is 2^-24 whatever the weight, its half 2^-25 = 2^-31 E: the sum over j of that
    times |c_j|, 2^-31 max_j w_j sum_j |c_j|, is beyond what 2^-11 of each weight counts.  It tells only where values of
    one channel lie below the others' by more than the weights' 2^20.  s_j is the block's scale, and for 16-bit rows
    between 2^-15 and 2^-14 of the row's largest value: the larger counts in w_j, the smaller in c_j."""
    ref, q = p.ref[b], q.double().cpu().numpy()
    want, _, mass, size = ref.attend(q, sm, window)
    got = out.double().cpu().numpy()
    K, V = ref.cached(0), ref.cached(1)
    codes, scale = ref.blocks(1)
    scale = np.where(codes.any(axis=(-1, -2)), scale.astype(np.float64), 0).repeat(64, axis=-1)  # zeros have no magnitude
    top = np.abs(V[:, scale.shape[1]:]).max(-1)
    large, small = np.concatenate((scale, top * 2.0 ** -14), 1), np.concatenate((scale, top * 2.0 ** -15), 1)
    code = np.abs(V) / np.where(small == 0, 1, small)[..., None]
    n, Hq, _ = q.shape
    G, step = Hq // K.shape[0], np.zeros_like(want)
    for i in range(n):
        t = ref.len - n + i
        lo = max(0, t - window + 1) if window > 0 else 0
        for h in range(Hq):
            s = K[h // G, lo:t + 1] @ q[i, h] * sm
            w = np.exp(s - s.max())
            step[i, h] = 2.0 ** -31 * (w * large[h // G, lo:t + 1]).max() / w.sum() * code[h // G, lo:t + 1].sum(0)
    tol = torch.finfo(TYPES[p.dtype]).eps / 2 * np.abs(want) + (2.0 ** -11 + 2.0 ** -15 + 3 * 2.0 ** -18 * size[..., None]) * mass + step + TINY[p.dtype]
    err = np.abs(got - want)
    assert (err <= tol).all(), (err / tol).max()


# rows of a kv head: one task of the first kernel, two of them, one row tile of the second, two tiles
ROWS = [(4, 1), (4, 5), (8, 5), (8, 8), (8, 32)]


@pytest.mark.parametrize("G,n", ROWS)
@pytest.mark.parametrize("L", [40, 63, 65, 100])
def test_an_incomplete_block_of_small_values(G, n, L):
    """bf16 rows of the 16-bit tail stand at a scale of their own, far below 1: positions past the length, and those that
    a query does not see yet, leave no trace in the weights' reference."""
    for window in (0, 20):
        for size in (1e-2, 1e-3, 1e-4, 1e-6, 1e-20):
            p = Pair(1, 1, 256, "e4m3", "bf16", seed=43)
            k, v = p.rows(L), p.rows(L).double() * size
            p.append([L], k=k, v=v.bfloat16())
            q, out, _ = p.attend(G, [n], window=window, check=False)
            check_relative(p, 0, q, out, window=window)


@pytest.mark.parametrize("G,n", [(8, 8), (8, 32)])
def test_new_tokens_of_unlike_size(G, n):
    """Each token's values are 4 times the one's before: what a query does not see yet is far above what it sees."""
    p = Pair(1, 1, 256, "e4m3", "bf16", seed=44)
    v = p.rows(40).double() * 2.0 ** (2.0 * (torch.arange(40) - 29))[:, None, None]
    p.append([40], k=p.rows(40), v=v.bfloat16())
    q, out, _ = p.attend(G, [n], check=False)
    check_relative(p, 0, q, out)


@pytest.mark.parametrize("G,n", ROWS)
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_values_at_the_ends_of_float32(G, n, fmt):
    """Values whose scales lie at 2^-117 and above (bf16): the factor that the weights take and what undoes it agree."""
    for L in (320, 350):
        for e in (60, -80, -95, -104):
            p = Pair(1, 1, 384, fmt, "bf16", seed=45)
            k, v = p.rows(L), p.rows(L).double() * 2.0 ** e
            p.append([L], k=k, v=v.bfloat16())
            q, out, _ = p.attend(G, [n], check=False)
            check_relative(p, 0, q, out)
    # blocks and rows from one end to the other, the newest the smallest
    p = Pair(1, 1, 384, fmt, "bf16", seed=46)
    v = p.rows(350).double() * 2.0 ** (-20.0 * (torch.arange(350) // 64))[:, None, None]
    p.append([350], k=p.rows(350), v=v.bfloat16())
    for window in (0, 20):
        q, out, _ = p.attend(G, [n], window=window, check=False)
        check_relative(p, 0, q, out, window=window)


@pytest.mark.parametrize("G,n", ROWS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_zero_rows_beside_small_values(G, n, dtype):
    """Rows of the 16-bit tail whose values are all zero (a padding token's) have no magnitude; fp16 rows, stored as they
    are, have their own: neither sets the reference of the others' weights."""
    for L, zero in ((40, [3, 39]), (100, [70]), (100, list(range(64, 99))), (65, [64]), (300, [256, 270]), (47, list(range(47)))):
        for size in (1e-1, 1e-2, 1e-4, 1e-6) if dtype == "bf16" else (1.0, 1e-2, 1e-3):
            p = Pair(1, 1, 384, "e4m3", dtype, seed=47)
            k, v = p.rows(L), p.rows(L).double() * size
            v[zero] = 0
            p.append([L], k=k, v=v.to(TYPES[dtype]))
            q, out, _ = p.attend(G, [n], check=False)
            check_relative(p, 0, q, out)


@pytest.mark.parametrize("G,n", ROWS)
def test_not_finite_and_zero_rows_of_the_tail(G, n):
    """A row that is not finite still marks what sees it where the others are zero or tiny."""
    p = Pair(1, 1, 256, "e4m3", "bf16", seed=48)
    k, v = p.rows(100), p.rows(100).double() * 1e-4
    v[64:99] = 0
    v[99, 0, 3] = float("nan")
    p.append([100], k=k, v=v.bfloat16())
    _, out, _ = p.attend(G, [n], check=False)
    assert torch.isnan(out[-1]).all() and torch.isfinite(out[:-1]).all()


@pytest.mark.parametrize("G,n", ROWS)
@pytest.mark.parametrize("fmt,dtype", FORMS)
def test_zero_blocks_beside_small_values(G, n, fmt, dtype):
    """A block whose values are all zero (of either sign) has scale 1 and no magnitude, wherever it stands; a block whose
    scale is 1 with some rows of zeros has that of the others."""
    for zero in ([0], [2], [4], [0, 1, 2, 3], [0, 3, 4]):
        for size in (1e-2, 1e-4, 1e-6) if dtype == "bf16" else (1.0, 1e-3):
            p = Pair(1, 1, 384, fmt, dtype, seed=49)
            k, v = p.rows(340), p.rows(340).double() * size
            for z in zero:
                v[64 * z:64 * z + 64] *= 0  # 0 and -0
            p.append([340], k=k, v=v.to(TYPES[dtype]))
            q, out, _ = p.attend(G, [n], check=False)
            check_relative(p, 0, q, out)
    for place in (0, 40, 63):  # the block's scale is 1 by one row
        p = Pair(1, 1, 384, fmt, dtype, seed=50)
        k, v = p.rows(340), p.rows(340).double() * 1e-2
        v[64:128] *= 0
        v[64 + place] = {"e4m3": 448.0, "int8": 127.0}[fmt]
        p.append([340], k=k, v=v.to(TYPES[dtype]))
        for window in (0, 250):
            q, out, _ = p.attend(G, [n], window=window, check=False)
            check_relative(p, 0, q, out, window=window)


@pytest.mark.parametrize("G,n", ROWS)
@pytest.mark.parametrize("where", [0, 64, 339])
def test_a_key_without_values_takes_the_weight(G, n, where):
    """One key takes nearly all of the weight, by 2^40 to 2^105, and its values are zero: what the others, of values up to
    2^40, add up to is the output."""
    for far in (40.0, 80.0, 105.0):
        for size in (2.0 ** -20, 1.0, 2.0 ** 40):
            p = Pair(1, 1, 384, "e4m3", "bf16", seed=51)
            k, v = p.rows(340).double(), p.rows(340).double() * size
            k[:, 0, 0] = 0
            k[where, 0], v[where] = 0, 0
            k[where, 0, 0] = 16.0
            q = torch.from_numpy(p.rng.standard_normal((n, 8 if G == 8 else 4, 128)))
            q[..., 0] = far * np.log(2) / 16 * 128 ** 0.5
            p.append([340], k=k.bfloat16(), v=v.bfloat16())
            q = q.bfloat16()
            _, out, _ = p.attend(G, [n], q=q, check=False)
            check_relative(p, 0, q, out)


# ----------------------------------------------------------------------------- element types in turn

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("first,then", [("f16", "bf16"), ("bf16", "f16")])
@pytest.mark.parametrize("size", [1.0, 1e6, 1e-7])
def test_element_types_in_turn(fmt, first, then, size):
    """Rows of one element type completed by rows of the other: the codes come from the values as they were appended,
    whether the later type holds them (bf16 rows of 1e6 are no fp16 numbers, fp16 rows have three bits more than bf16)."""
    if first == "f16" and size != 1:
        size = 1e4 if size > 1 else 1e-4
    p = Pair(3, 2, 512, fmt, first, seed=52)

    def append(n, dtype, scale):
        p.dtype = dtype
        p.append(n, k=(p.rows(sum(n)).double() * scale).to(TYPES[dtype]), v=(p.rows(sum(n)).double() * scale).to(TYPES[dtype]))
        p.dtype = "both"
        p.check_stored()

    append([40, 100, 1], first, size)
    append([24, 28, 200], then, 1.0)
    append([10, 63, 1], first, size)
    append([1, 1, 1], then, 1.0)
    append([60, 64, 53], then, 1.0)
    append([70, 1, 2], first, size)
    append([1, 127, 64], then, 1.0)
    assert not any(p.c.errors())


def test_element_types_in_turn_and_a_row_that_is_not_finite():
    p = Pair(1, 1, 256, "e4m3", "bf16", seed=53)
    k, v = (p.rows(40).double() * 1e6).bfloat16(), p.rows(40)
    k[7, 0, 3], v[9, 0, 1] = float("inf"), float("nan")
    p.append([40], k=k, v=v)
    p.dtype = "f16"
    p.append([30])
    p.dtype = "both"
    p.check_stored()


def test_attention_over_element_types_in_turn():
    """Queries of either type over a cache whose tail holds rows of both."""
    p = Pair(2, 1, 256, "int8", "f16", seed=54)
    p.append([90, 70])
    p.dtype = "bf16"
    p.append([20, 25], k=(p.rows(45).double() * 4).bfloat16())
    for dtype in ("bf16", "f16"):
        p.dtype = dtype
        p.attend(4, [1, 1])
        p.attend(8, [20, 9])


# ----------------------------------------------------------------------------- queries that are not finite

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("L,n,G", [(40, 1, 4), (200, 1, 4), (200, 5, 8), (40, 8, 8), (300, 8, 8), (300, 40, 8)])
def test_an_infinite_query_whose_scores_are_all_minus_infinity(dtype, L, n, G):
    """Its softmax is 0 / 0, whichever pages it sees.  The other rows stay within their bound (not the same to the bit: the
    rows of a warp have their references set anew together)."""
    p = Pair(1, 1, 512, "e4m3", dtype, seed=55)
    k = p.rows(L)
    k[:, 0, 3] = -1.0
    p.append([L], k=k)
    q = torch.from_numpy(p.rng.standard_normal((n, G, 128))).to(TYPES[dtype])
    fine = q.clone()
    q[n // 2, 1, 3] = float("inf")
    for window in (0, 30):
        _, out, lse = p.attend(G, [n], q=q, window=window, check=False)
        bad = torch.isnan(out).all(-1)
        assert bad.nonzero().tolist() == [[n // 2, 1]] and torch.equal(torch.isnan(out).any(-1), bad)
        assert torch.equal(torch.isnan(lse), bad)
        _, want, wlse = p.attend(G, [n], q=fine, window=window)
        out[bad], lse[bad] = want[bad], wlse[bad]
        check_rows(out, lse, p.ref[0], fine.double().numpy(), 128 ** -0.5, window, dtype)


# ----------------------------------------------------------------------------- outputs in places of their own

def test_outputs_that_share_places_are_refused():
    """An output that overlaps the queries, the other output or itself; neighbours and interleaved views are taken."""
    hq = _hq()
    p = Pair(2, 2, 256, "e4m3", "f16", seed=56)
    p.append([200, 100])
    cu = _ints([0, 1, 2])
    row = torch.randn(2, 26, 128, device="cuda").half()
    want = hq.hq_kv8_attn(p.c, row[:, :8].clone(), cu, p.len, 1)
    for out in (row[:, 4:12], row[:, :8], row.as_strided((2, 8, 128), row.stride(), 8), row.as_strided((2, 8, 128), (128, 256, 1), 512),
                torch.empty(1, 8, 128, device="cuda").half().expand(2, 8, 128)):
        with pytest.raises(hq.HqError):
            hq.hq_kv8_attn(p.c, row[:, :8], cu, p.len, 1, out=out)
    assert torch.equal(hq.hq_kv8_attn(p.c, row[:, :8], cu, p.len, 1, out=row[:, 8:16]), want)
    kv = torch.zeros(2, 2, 2, 200, 128, device="cuda", dtype=torch.float16)
    K, V = hq.hq_kv8_read(p.c, p.len, n=200)
    whole = (2, 2, 200, 128)
    for a, b in ((kv[:, 0], kv[:, 0]), (kv[:, :, 0], kv.as_strided(whole, kv[:, :, 0].stride(), 128 * 199)),
                 (kv.view(-1)[:128].expand(whole), kv.view(-1)[128:256].expand(whole))):
        with pytest.raises(hq.HqError):
            hq.hq_kv8_read(p.c, p.len, n=200, k_out=a, v_out=b)
    for a, b in ((kv[:, 0], kv[:, 1]), (kv[:, :, 0], kv[:, :, 1]), (kv.view(2, 200, 2, 2, 128)[:, :, 0].transpose(1, 2),
                                                                  kv.view(2, 200, 2, 2, 128)[:, :, 1].transpose(1, 2))):
        hq.hq_kv8_read(p.c, p.len, n=200, k_out=a, v_out=b)
        assert torch.equal(a, K) and torch.equal(b, V)
    x = torch.randn(4, 12, 128, device="cuda").half()
    t, pos = hq.RopeTable(128), _ints([0, 1, 2, 3])
    q, k = hq.hq_rope(x[:, :4].clone(), x[:, 4:6].clone(), pos, t)
    for kw in (dict(q_out=x[:, 2:6]), dict(q_out=x[:, 6:10], k_out=x[:, 5:7]), dict(q_out=x[:1, 6:10].expand(4, 4, 128))):
        with pytest.raises(hq.HqError):
            hq.hq_rope(x[:, :4], x[:, 4:6], pos, t, **kw)
    a, b = hq.hq_rope(x[:, :4], x[:, 4:6], pos, t, q_out=x[:, 6:10], k_out=x[:, 4:6])
    assert torch.equal(a, q) and torch.equal(b, k)


def test_strides_of_dimensions_of_one():
    """A single token, kv head or query head may have any stride there (torch gives such tensors odd ones)."""
    hq = _hq()
    odd = lambda x, dim: x.as_strided(x.shape, [s if i != dim else 3 for i, s in enumerate(x.stride())])
    for H, N in ((1, 5), (2, 1), (1, 1)):
        k, v = torch.randn(N, H, 128, device="cuda").half(), torch.randn(N, H, 128, device="cuda").half()
        q = torch.randn(N, H, 128, device="cuda").half()
        cu, n = _ints([0, N]), _ints([N])
        c, d = hq.Kv8Cache(1, H, 128), hq.Kv8Cache(1, H, 128)
        hq.hq_kv8_append(c, k, v, cu, n)
        K, V = hq.hq_kv8_read(c, n, n=N)
        want = hq.hq_kv8_attn(c, q, cu, n, N)
        dims = [i for i, m in enumerate((N, H)) if m == 1]
        for i in dims:
            k, v, q = odd(k, i), odd(v, i), odd(q, i)
        out, K2, V2 = torch.empty(N, H, 128, device="cuda").half(), odd(torch.empty_like(K), 0), odd(torch.empty_like(V), 0)
        for i in dims:
            out = odd(out, i)
            K2, V2 = odd(K2, 2 - i), odd(V2, 2 - i)
        hq.hq_kv8_append(d, k, v, cu, n)
        assert torch.equal(hq.hq_kv8_attn(d, q, cu, n, N, out=out), want)
        hq.hq_kv8_read(d, n, n=N, k_out=K2, v_out=V2)
        assert torch.equal(K, K2) and torch.equal(V, V2)


def test_layers_share_one_scratch_of_a_stream():
    """The scratch of a prompt chunk is kept once for the stream, not once for each layer's cache; calls of the layers in
    turn, and on another stream, give what they give alone."""
    hq = _hq()
    layers = [Pair(1, 2, 2048, "e4m3", "f16", seed=60 + i) for i in range(4)]
    q = torch.randn(300, 8, 128, device="cuda").half()
    calls, want = [], []
    for p in layers:
        p.append([2000])
        for n in (1, 20, 300):
            calls.append((p.c, q[:n].contiguous(), _ints([0, n]), p.len, n))
            need = hq._lib.hq_kv8_attn_workspace_bytes(p.c.ref, 8, n)
            want.append(hq.hq_kv8_attn(*calls[-1], ws=torch.zeros(need, dtype=torch.uint8, device="cuda")))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for stream in (None, s):
        for _ in range(3):
            for a, w in zip(calls, want):
                out = hq.hq_kv8_attn(*a, stream=stream)
                torch.cuda.synchronize()
                assert torch.equal(out, w)
    del out
    most = hq._lib.hq_kv8_attn_workspace_bytes(layers[0].c.ref, 8, 300)
    assert torch.cuda.memory_allocated() - before <= 2 * most + (1 << 20)
    layers[0].c.err[0] = hq.DEVERR_TIMEOUT   # scratch of a call that gave up goes, the other layers' calls get new
    assert layers[0].c.errors() == [hq.DEVERR_TIMEOUT]
    layers[0].c.err.zero_()
    for a, w in zip(calls, want):
        assert torch.equal(hq.hq_kv8_attn(*a), w)


@pytest.mark.parametrize("G,n", [(8, 8), (8, 17)])
def test_many_sequences_of_many_rows(G, n):
    """More sequences than threads that plan the work, one and two row tiles; every ninth against the oracle."""
    lens = [(37 * i) % 150 for i in range(700)]
    p = Pair(700, 1, 256, "e4m3", "bf16", seed=61)
    p.append(lens)
    news = [min(m, 1 + (n + i) % n) if i % 3 else min(m, n) for i, m in enumerate(lens)]
    q, out, lse = p.attend(G, news, check=False)
    cu = np.concatenate(([0], np.cumsum(news)))
    for b in range(0, 700, 9):
        if news[b]:
            check_rows(out[cu[b]:cu[b + 1]], lse[cu[b]:cu[b + 1]], p.ref[b], q[cu[b]:cu[b + 1]].double().numpy(), 128 ** -0.5, 0, "bf16")
    again = hq_again(p, q, news, n)
    assert torch.equal(out, again)


def hq_again(p, q, news, n):
    cu = np.concatenate(([0], np.cumsum(news)))
    return _hq().hq_kv8_attn(p.c, q.cuda(), _ints(cu.tolist()), p.len, n)


@pytest.mark.parametrize("G,n", ROWS)
@pytest.mark.parametrize("fmt,dtype", [("e4m3", "bf16"), ("int8", "f16")])
def test_pieces_of_unlike_magnitude(G, n, fmt, dtype):
    """A long context cut over the grid whose pieces lie far apart: values of 2^-60 to 1 (2^-8 to 1) by turns of 11 blocks,
    zero blocks among them, a tail of small values with a zero row; the weight on the small ones too."""
    p = Pair(1, 1, 9088, fmt, dtype, seed=62)
    L, far = 9011, 60.0 if dtype == "bf16" else 8.0
    at = torch.arange(L) // 64
    k, v = p.rows(L).double(), p.rows(L).double() * 2.0 ** (-far * (at // 11 % 5) / 4)[:, None, None]
    v[at % 17 == 3] = 0
    v[-19:] *= 2.0 ** -10
    v[-4] = 0
    k[:, 0, 0] = torch.where(at // 11 % 5 == 4, 12.0, -12.0)
    p.append([L], k=k.to(TYPES[dtype]), v=v.to(TYPES[dtype]))
    q = torch.from_numpy(p.rng.standard_normal((n, G, 128)))
    q[:, ::2, 0] = 6.0
    q = q.to(TYPES[dtype])
    for window in (0, 5000):
        _, out, _ = p.attend(G, [n], q=q, window=window, check=False)
        check_relative(p, 0, q, out, window=window)
        _, again, _ = p.attend(G, [n], q=q, window=window, check=False)
        assert torch.equal(out, again)


def test_taken_back_again_and_started_again():
    """Drafted tokens taken back several times, up to 64 positions before the furthest one; a slot started again at a
    multiple of 64 far before its end, and taken back from there."""
    for dtype in ("f16", "bf16"):
        p = Pair(3, 2, 512, "e4m3", dtype, seed=63)
        p.append([130, 300, 191])
        p.append([30, 40, 10])                                   # 160, 340, 201 the furthest
        for at, n in (([140, 300, 190], [3, 1, 2]), ([100, 277, 137], [1, 5, 1]), ([96, 276, 138], [64, 64, 64]), ([128, 280, 201], [2, 1, 7])):
            p.append(n, at=at)
            p.check_stored()
        p.append([70, 10, 65], at=[0, 64, 128])
        p.check_stored()
        p.append([9, 30, 1], at=[61, 70, 192])
        p.check_stored()
        p.append([100, 1, 64])
        p.check_stored()
        p.attend(4, [1, 1, 1])
        assert not any(p.c.errors())


def test_empty_rows_of_any_stride():
    """No new rows, as torch makes them out of an empty array (strides of 0)."""
    hq = _hq()
    c = hq.Kv8Cache(2, 3, 128)
    none = torch.empty(0, 3, 128, device="cuda").half().as_strided((0, 3, 128), (0, 0, 0))
    cu, n = _ints([0, 0, 0]), _ints([0, 0])
    hq.hq_kv8_append(c, none, none, cu, n)
    assert hq.hq_kv8_attn(c, none, cu, n, 1).shape == (0, 3, 128) and not any(c.errors())
    y, _ = hq.hq_rope(none, none, _ints([]), hq.RopeTable(64))
    assert y.shape == (0, 3, 128)


def test_strides_beyond_32_bits():
    """Tokens 2^30 elements apart: rows of every call (rotary positions, append, read back, queries and outputs of both
    kernels) at offsets past 2^31 elements."""
    hq = _hq()
    far, n, G = 1 << 30, 3, 17
    buf = torch.empty((n - 1) * far + 6 * (G + 2) * 128, dtype=torch.bfloat16, device="cuda")
    at = lambda i, h: buf.as_strided((n, h, 128), (far, 128, 1), i * (G + 2) * 128)
    small = lambda h: torch.randn(n, h, 128, device="cuda").bfloat16()
    q, k, v = small(G), small(1), small(1)
    qf, kf, vf = at(0, G), at(1, 1), at(2, 1)
    t, pos = hq.RopeTable(128), _ints([5, 6, 7])
    cu, L = _ints([0, n]), _ints([n])
    for x, y in ((qf, q), (kf, k), (vf, v)):
        x.copy_(y)
    q2, k2 = hq.hq_rope(q, k, pos, t)
    hq.hq_rope(qf, kf, pos, t, q_out=at(3, G), k_out=kf)
    assert torch.equal(at(3, G), q2) and torch.equal(kf, k2) and torch.equal(qf, q)
    a, b = hq.Kv8Cache(1, 1, 128), hq.Kv8Cache(1, 1, 128)
    hq.hq_kv8_append(a, k2, v, cu, L)
    hq.hq_kv8_append(b, kf, vf, cu, L)
    assert torch.equal(a.tail_k, b.tail_k) and torch.equal(a.tail_v, b.tail_v) and torch.equal(a.tail_scale, b.tail_scale)
    for h in (G, 5, 1):                                       # 51 rows, 15, 3
        want = hq.hq_kv8_attn(a, q2[:, :h].contiguous(), cu, L, n)
        out = hq.hq_kv8_attn(b, at(3, h), cu, L, n, out=at(4, h))
        assert torch.equal(out, want)
    K, V = hq.hq_kv8_read(a, L, n=n, dtype=torch.bfloat16)
    shape, strides = (1, 1, n, 128), (128, 128, far, 1)
    K2, V2 = (buf.as_strided(shape, strides, i * (G + 2) * 128) for i in (4, 5))
    hq.hq_kv8_read(b, L, n=n, k_out=K2, v_out=V2)
    assert torch.equal(K, K2) and torch.equal(V, V2)


def test_the_largest_batch():
    """1024 sequences, one to three tokens each, and 20 of some: every plan's last entries."""
    lens = [1 + (53 * i) % 90 for i in range(1024)]
    p = Pair(1024, 1, 128, "int8", "f16", seed=64)
    p.append(lens)
    for G, news in ((3, [1 + i % min(3, m) for i, m in enumerate(lens)]), (8, [min(m, 20 if i % 7 == 0 else 1) for i, m in enumerate(lens)])):
        q, out, lse = p.attend(G, news, check=False)
        cu = np.concatenate(([0], np.cumsum(news)))
        for b in list(range(0, 1024, 23)) + [1022, 1023]:
            check_rows(out[cu[b]:cu[b + 1]], lse[cu[b]:cu[b + 1]], p.ref[b], q[cu[b]:cu[b + 1]].double().numpy(), 128 ** -0.5, 0, "f16")
