"""Pins of the oracle's rotary positions and 8-bit block cache, and of the
library's host-side frequency table.  CPU only."""
import ctypes
import math

import numpy as np
import pytest

from oracle import kv8, rope


def test_page_orders_are_permutations():
    r, d = np.arange(64)[:, None], np.arange(128)[None]
    for f in (kv8.k_index, kv8.v_index):
        assert np.array_equal(np.sort(f(r, d).ravel()), np.arange(8192))
    # hand-worked: token 9, element 70 of K: row group 1, second half, row 1
    assert kv8.k_index(9, 70) == (1 * 2 + 1) * 512 + 64 + 6
    # token 27 = 16 + 8 + 2 + 1, element 45 = 32 + 8 + 5 of V
    assert kv8.v_index(27, 45) == 2048 + 512 + (5 * 4 + 1) * 16 + 0 + 4 + 2 + 1


def test_quantise_by_hand():
    x = np.zeros((64, 128))
    x[0, 0], x[1, 1], x[2, 2] = 127.0, -63.5, 0.4
    c, s = kv8.quantise(x, "int8")
    assert s == 1.0 and c[0, 0] == 127 and c[1, 1] == -64 and c[2, 2] == 0      # -63.5 ties to even
    x[0, 0] = 448.0
    c, s = kv8.quantise(x, "e4m3")
    assert s == 1.0 and c[0, 0] == 448 and c[1, 1] == -64 and c[2, 2] == 0.40625
    c, s = kv8.quantise(np.zeros((64, 128)), "e4m3")
    assert s == 1.0 and not c.any()
    x[5, 5] = np.inf
    c, s = kv8.quantise(x, "int8")
    assert np.isnan(s) and not c.any()


def test_codes_values_round_trip():
    for fmt in ("e4m3", "int8"):
        v = kv8.code_values(np.arange(256), fmt)
        if fmt == "int8":
            assert np.array_equal(v, np.arange(256).astype(np.int8))
        else:
            ok = np.arange(256) % 128 != 127                                    # not the NaN codes
            assert np.array_equal(kv8.e4m3_round(v[ok]), v[ok]) and v[ok].max() == 448


def test_attend_is_a_softmax_over_the_window():
    rng = np.random.default_rng(0)
    ref = kv8.Kv8Ref(2, "e4m3")
    ref.append(rng.standard_normal((70, 2, 128)), rng.standard_normal((70, 2, 128)))
    q = rng.standard_normal((3, 4, 128))
    out, lse, mass, _ = ref.attend(q, 0.1, window=5)
    k, v = ref.cached(0), ref.cached(1)
    for i in range(3):
        t = 67 + i
        w = np.exp(0.1 * k[1, t - 4:t + 1] @ q[i, 3])
        assert np.allclose(out[i, 3], w @ v[1, t - 4:t + 1] / w.sum())
        assert np.isclose(2 ** lse[i, 3], w.sum())
    assert (mass >= np.abs(out) - 1e-12).all()


def test_rotation_by_hand_and_its_transpose():
    w, amp = rope.frequencies(4, 100.0)
    assert np.allclose(w.astype(float), [1.0, 0.1]) and amp == 1.0
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    y = rope.rotate(x, np.array([2]), w, 1.0, "half")
    c, s = math.cos(2), math.sin(2)
    assert np.allclose(y[0, 0], [c - 3 * s, 2 * math.cos(.2) - 4 * math.sin(.2), 3 * c + s, 4 * math.cos(.2) + 2 * math.sin(.2), 5])
    y = rope.rotate(x, np.array([2]), w, 1.0, "interleaved")
    assert np.allclose(y[0, 0], [c - 2 * s, 2 * c + s, 3 * math.cos(.2) - 4 * math.sin(.2), 4 * math.cos(.2) + 3 * math.sin(.2), 5])
    rng = np.random.default_rng(1)
    for layout in ("half", "interleaved"):
        x, z, pos = rng.standard_normal((3, 2, 12)), rng.standard_normal((3, 2, 12)), np.array([0, 7, 100000])
        w, amp = rope.frequencies(8, 1e4, "yarn", 4.0, 2048)
        a = (rope.rotate(x, pos, w, amp, layout) * z).sum()
        b = (x * rope.rotate(z, pos, w, amp, layout, grad=True)).sum()
        assert np.isclose(a, b)


def test_scaled_frequencies():
    plain, _ = rope.frequencies(64, 1e4)
    lin, _ = rope.frequencies(64, 1e4, "linear", 4.0)
    assert np.allclose((plain / lin).astype(float), 4)
    ntk, _ = rope.frequencies(64, 1e4, "ntk", 4.0)
    assert np.isclose(float(plain[0] / ntk[0]), 1) and np.isclose(float(plain[-1] / ntk[-1]), 4)
    for kind, high in (("yarn", 32), ("bands", 4)):
        w, amp = rope.frequencies(64, 1e4, kind, 8.0, 4096)
        turns = (4096 * plain / (2 * math.pi)).astype(float)
        ratio = (plain / w).astype(float)
        assert np.allclose(ratio[turns > high * 2], 1) and np.allclose(ratio[turns < 0.5], 8)
        assert (np.diff(ratio) >= -1e-12).all()
        assert np.isclose(amp, 1 + 0.1 * math.log(8) if kind == "yarn" else 1)


@pytest.mark.parametrize("kind", range(5))
@pytest.mark.parametrize("rot", [4, 34, 128])
def test_library_table_holds_the_frequencies(kind, rot):
    from hybrid_precision_attention_b200 import hq
    t = hq.RopeTable(rot, 500000.0, kind=kind, factor=8.0, orig_len=8192, device="cpu")
    w, amp = rope.frequencies(rot, 500000.0, rope.KINDS[kind], 8.0, 8192.0)
    turns = w / (8 * np.arctan(np.longdouble(1)))
    got = t.freqs.numpy().view(np.uint64).astype(np.longdouble) / np.longdouble(2) ** 64
    # a fraction of a turn per position: half a unit of 2^-64, and long double powers good to a few units of 2^-63 relative
    assert np.abs((got - turns).astype(float)).max() <= 2.0 ** -64 + 2.0 ** -60 * float(turns.max())
    assert abs(t.amp - amp) <= 2.0 ** -23


def test_table_refusals():
    from hybrid_precision_attention_b200 import hq
    for kw in (dict(rot=0), dict(rot=3), dict(rot=-2), dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")),
               dict(kind=5), dict(kind=-1), dict(kind=1, factor=0.5), dict(kind=1, factor=float("inf")),
               dict(kind=2, factor=2.0, rot=2), dict(kind=3, factor=2.0), dict(kind=4, factor=2.0, orig_len=100, low=4.0, high=2.0),
               dict(kind=3, factor=2.0, orig_len=100, low=-1.0)):
        a = dict(rot=64, base=1e4, device="cpu")
        a.update(kw)
        with pytest.raises(hq.HqError):
            hq.RopeTable(**a)


# ----------------------------------------------------------------------------- refusals before any launch

OK, INVALID, UNSUPPORTED, WORKSPACE, CAPACITY, CUDA = range(6)


@pytest.fixture(scope="module")
def mem():
    buf = ctypes.create_string_buffer(1 << 16)
    return buf, (ctypes.addressof(buf) + 255) & ~255


def _cache(base, **kw):
    from hybrid_precision_attention_b200 import hq
    f = dict(B=2, Hkv=4, D=128, cap=1024, fmt=0, n_pages=0, pages=base, page_table=None, tail_k=base, tail_v=base,
             tail_scale=base, err=base)
    f.update(kw)
    return hq.HqKv8CacheStruct(*[f[n] for n, _ in hq.HqKv8CacheStruct._fields_])


def test_kv8_descriptor(mem):
    from hybrid_precision_attention_b200 import hq
    base = mem[1]
    check = lambda **kw: hq._lib.hq_kv8_validate(ctypes.byref(_cache(base, **kw)))
    assert check() == OK and check(fmt=1) == OK and check(page_table=base + 4, n_pages=3, err=base + 4) == OK
    assert hq._lib.hq_kv8_validate(None) == INVALID
    for kw, want in ((dict(D=64), UNSUPPORTED), (dict(B=0), INVALID), (dict(B=4097), UNSUPPORTED), (dict(Hkv=0), INVALID),
                     (dict(Hkv=1025), UNSUPPORTED), (dict(cap=64), INVALID), (dict(cap=0), INVALID), (dict(fmt=2), INVALID),
                     (dict(fmt=-1), INVALID), (dict(pages=None), INVALID), (dict(pages=base + 8), INVALID),
                     (dict(tail_k=None), INVALID), (dict(tail_v=base + 2), INVALID), (dict(tail_scale=base + 4), INVALID),
                     (dict(err=None), INVALID), (dict(err=base + 2), INVALID), (dict(page_table=base, n_pages=0), INVALID),
                     (dict(page_table=base + 2, n_pages=3), INVALID)):
        assert check(**kw) == want, kw


def test_kv8_call_refusals(mem):
    from hybrid_precision_attention_b200 import hq
    L, base = hq._lib, mem[1]
    c = ctypes.byref(_cache(base))

    def append(**kw):
        a = dict(dtype=0, k=base, kt=512, kh=128, v=base, vt=512, vh=128, N=0, cu=base, kv=base)
        a.update(kw)
        return L.hq_kv8_append(c, *a.values(), None)

    assert append() == OK                                              # no new rows: nothing is launched
    for kw in (dict(dtype=2), dict(dtype=-1), dict(N=-1), dict(cu=None), dict(kv=base + 2), dict(N=3, k=None),
               dict(N=3, v=base + 8), dict(N=3, kt=100), dict(N=3, vh=4)):
        assert append(**kw) == INVALID, kw
    assert L.hq_kv8_append(ctypes.byref(_cache(base, D=64)), 0, base, 512, 128, base, 512, 128, 0, base, base, None) == UNSUPPORTED

    def read(**kw):
        a = dict(dtype=0, kv=base, start=0, n=0, k=base, v=base, ob=4096, oh=1024, ot=128, z=1)
        a.update(kw)
        return L.hq_kv8_read(c, *a.values(), None)

    assert read() == OK
    for kw, want in ((dict(dtype=3), INVALID), (dict(start=-1), INVALID), (dict(n=-1), INVALID), (dict(kv=None), INVALID),
                     (dict(n=1025), CAPACITY), (dict(start=1000, n=25), CAPACITY), (dict(start=2 ** 31 - 1, n=2 ** 31 - 1), CAPACITY),
                     (dict(n=5, k=None), INVALID), (dict(n=5, v=base + 4), INVALID), (dict(n=5, ot=130), INVALID)):
        assert read(**kw) == want, kw

    need = L.hq_kv8_attn_workspace_bytes(c, 8, 4)
    assert need > 0 and L.hq_kv8_attn_workspace_bytes(c, 6, 1) == 0 and L.hq_kv8_attn_workspace_bytes(c, 0, 1) == 0
    assert L.hq_kv8_attn_workspace_bytes(c, 8, -1) == 0

    def attn(**kw):
        a = dict(dtype=0, q=base, qt=1024, qh=128, Hq=8, N=0, cu=base, kv=base, new=4, window=0, scale=0.1, out=base, ot=1024,
                 oh=128, lse=None, ws=base, wsb=need)
        a.update(kw)
        return L.hq_kv8_attn(c, *a.values(), None)

    assert attn() == OK and attn(N=3, new=0) == OK
    for kw, want in ((dict(dtype=2), INVALID), (dict(N=-1), INVALID), (dict(window=-1), INVALID), (dict(scale=0.0), INVALID),
                     (dict(scale=float("nan")), INVALID), (dict(Hq=6), INVALID), (dict(Hq=0), INVALID), (dict(new=-1), INVALID),
                     (dict(new=2 ** 30), INVALID), (dict(cu=None), INVALID), (dict(kv=base + 1), INVALID), (dict(lse=base + 2), INVALID),
                     (dict(N=3, q=None), INVALID), (dict(N=3, q=base + 8), INVALID), (dict(N=3, out=base + 2), INVALID),
                     (dict(N=3, qt=1020), INVALID), (dict(N=3, oh=12), INVALID)):
        assert attn(**kw) == want, kw


def test_rope_call_refusals(mem):
    from hybrid_precision_attention_b200 import hq
    base = mem[1]

    def t(**kw):
        a = dict(x=base, y=base + 4096, xb=512, xt=128, xh=64, yb=512, yt=128, yh=64, H=2, r=0)
        a.update(kw)
        return hq.HqRopeTensor(*a.values())

    def call(q=None, k=None, **kw):
        a = dict(dtype=0, B=1, T=2, D=64, rot=64, layout=0, grad=0)
        a.update({n: v for n, v in kw.items() if n in a})
        return hq._lib.hq_rope(*a.values(), q, k, kw.get("pos", base), kw.get("freqs", base), 1.0, None)

    assert call(t(), B=0) == OK and call(t(), T=0) == OK and call(t(H=0)) == OK and call(t(x=None, H=0), t(H=0)) == OK
    for q, k, kw, want in ((None, None, {}, INVALID), (t(), None, dict(dtype=3), INVALID), (t(), None, dict(layout=2), INVALID),
                           (t(), None, dict(rot=0), INVALID), (t(), None, dict(rot=7), INVALID), (t(), None, dict(rot=66), INVALID),
                           (t(), None, dict(D=514, rot=64), UNSUPPORTED), (t(), None, dict(D=0, rot=2), INVALID),
                           (t(), None, dict(B=-1), INVALID), (t(), None, dict(T=-1), INVALID), (t(H=-1), None, {}, INVALID),
                           (t(x=None), None, {}, INVALID), (t(y=base + 1), None, {}, INVALID), (t(), t(x=None), {}, INVALID),
                           (t(y=base, yh=72), None, {}, INVALID), (t(), None, dict(pos=None), INVALID),
                           (t(), None, dict(pos=base + 2), INVALID), (t(), None, dict(freqs=base + 4), INVALID)):
        assert call(q, k, **kw) == want, kw


def test_kv8_workspace_for_more_tokens_serves_fewer(mem):
    """A caller that sizes scratch for its largest max_new may call with any smaller one."""
    from hybrid_precision_attention_b200 import hq
    c = ctypes.byref(_cache(mem[1]))
    for Hq in (4, 12, 20, 32, 64):
        need = [hq._lib.hq_kv8_attn_workspace_bytes(c, Hq, n) for n in range(0, 300)]
        assert all(a <= b for a, b in zip(need, need[1:])) and need[0] > 0


class _Elsewhere:
    """A tensor of another device."""
    is_cuda, device = True, "cuda:1"

    def __init__(self, t):
        self.dtype, self.shape, self.nbytes = t.dtype, t.shape, t.nbytes

    def is_contiguous(self):
        return True

    def get_device(self):
        return 1

    def data_ptr(self):
        return 0


def test_attention_takes_scratch_and_lse_on_its_device_alone(monkeypatch):
    """Checked before the library is called, which takes their addresses as they are."""
    from types import SimpleNamespace

    from hybrid_precision_attention_b200 import hq
    import torch
    called = []
    for name, f in (("_rows", lambda *a, **k: None), ("_ints", lambda *a: None), ("_device", lambda: 0), ("_raw_stream", lambda d: 0)):
        monkeypatch.setattr(hq, name, f)
    monkeypatch.setattr(hq._lib, "hq_kv8_attn", lambda *a: called.append(a) or 0)
    cache = SimpleNamespace(index=0, B=1, D=128, ref=None, workspace=lambda *a: torch.zeros(64, dtype=torch.uint8))
    q, cu, n = torch.zeros(2, 4, 128).half(), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    ws, lse = torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(2, 4)
    hq.hq_kv8_attn(cache, q, cu, n, 1)
    assert len(called) == 1
    for kw in (dict(ws=ws), dict(ws=_Elsewhere(ws)), dict(lse=_Elsewhere(lse)), dict(lse=lse)):
        with pytest.raises(hq.HqError):
            hq.hq_kv8_attn(cache, q, cu, n, 1, **kw)
    assert len(called) == 1
