"""Cases of the 8-bit block cache and of rotary positions, with each operator's plain form.

Four operators that a serving loop calls around the attention of one layer:

  rope    rotary positions of q and k in one call
  write   new keys and values appended to the 8-bit cache (quantised a block of
          64 positions at a time, the incomplete last block kept in 16 bits)
  read    keys and values read back, dequantised, as [B, Hkv, n, D]
  attend  attention of each sequence's newest tokens over its cache

``own`` selects the library's calls; otherwise ``run`` computes the same in
elementary float32 torch operations.

The cache, as both forms see it (D = 128):
  pages  uint8 [n_pages, 16448], one page per 64 positions of one (sequence, kv
         head): 8192 K codes, 8192 V codes, the K scale and the V scale
         (float32).  K codes stand as [token / 8][d / 64][token % 8][d % 64],
         V codes as [token / 16][d / 32][d % 8][token % 8 / 2][d / 16 % 2]
         [d / 8 % 2][token / 8 % 2][token % 2].
  scale  amax / 448 (e4m3) or amax / 127 (int8) over the page's 64 x 128 values
         in float32, 1 where amax is 0; code = round(x / scale) in that type
  tail   fp16 [B, Hkv, 2, 8192] for K and for V: positions of the two newest
         blocks (block % 2) in the page's element order, with a float32 scale
         per position; a block of which all 64 positions are cached is read
         from its page, the incomplete last one from the tail
"""
import math
import random

import torch

own = False

D, BLOCK, PAGE = 128, 64, 16448
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
TOP = {"e4m3": 448.0, "int8": 127.0}


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a small batch: 16 tokens, heads of an 8B-class layer (32 query, 8 kv heads of 128)
        dict(name="rope decode", op="rope", B=16, T=1, Hq=32, Hkv=8, D=128, rot=128, layout="half", scaling="bands",
             dtype="f16", far=32768, grad=False),
        # a long prompt read from the fused projection's rows, half of each head rotated, stretched context
        dict(name="rope prompt", op="rope", B=1, T=8192, Hq=32, Hkv=8, D=128, rot=64, layout="interleaved",
             scaling="yarn", dtype="bf16", far=131072, grad=False),
        # the gradient of rotated queries and keys of a ragged-length training batch
        dict(name="rope gradient", op="rope", B=3, T=1777, Hq=16, Hkv=8, D=128, rot=128, layout="half",
             scaling="linear", dtype="f32", far=16384, grad=True),
        # each of 64 running sequences appends its new token
        dict(name="write token", op="write", B=64, n=1, lo=100, hi=16000, Hkv=8, fmt="e4m3", dtype="f16"),
        # prompts of different lengths installed in one call
        dict(name="write prompts", op="write", B=5, n=8191, lo=0, hi=0, Hkv=8, fmt="int8", dtype="bf16"),
        # a short conversation's cache read back
        dict(name="read short", op="read", B=3, lo=150, hi=700, Hkv=8, fmt="int8", dtype="f16"),
        # a 32K prompt's cache read back, as the input of another cache's install
        dict(name="read 32K", op="read", B=2, lo=32768, hi=32801, Hkv=8, fmt="e4m3", dtype="f16"),
        # decode of short conversations: launch and latency
        dict(name="attend short", op="attend", B=4, n=1, lo=33, hi=700, Hq=32, Hkv=8, fmt="e4m3", dtype="f16", window=0),
        # decode of one 32K context
        dict(name="attend 32K", op="attend", B=1, n=1, lo=32768, hi=32768, Hq=32, Hkv=8, fmt="e4m3", dtype="f16", window=0),
        # decode of a large ragged batch
        dict(name="attend batch", op="attend", B=64, n=1, lo=1000, hi=16001, Hq=64, Hkv=8, fmt="int8", dtype="bf16", window=0),
        # drafted tokens of a batch checked in one pass, sliding window
        dict(name="attend drafts", op="attend", B=16, n=5, lo=3000, hi=16384, Hq=32, Hkv=8, fmt="e4m3", dtype="f16", window=4096),
        # the last chunk of a long prompt over what is cached of it
        dict(name="attend chunk", op="attend", B=1, n=2048, lo=16384, hi=16384, Hq=32, Hkv=8, fmt="e4m3", dtype="bf16", window=0),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attend", "attend"])
    fmt, dtype = rng.choice(["e4m3", "int8"]), rng.choice(["f16", "bf16"])
    if op == "rope":
        head = rng.choice([64, 80, 96, 128, 256])
        hq = rng.choice([1, 2, 4]) * (hkv := rng.choice([1, 3, 8]))
        most = max(1, 8192 * 40 * 128 // (head * (hq + hkv)))
        b = _log(rng, 1, min(64, most))
        return dict(op="rope", B=b, T=_log(rng, 1, min(8192, most // b)), Hq=hq, Hkv=hkv, D=head,
                    rot=rng.choice([head, head // 2, head // 4 // 2 * 2 + 2]), layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["plain", "linear", "ntk", "yarn", "bands"]), dtype=rng.choice(["f16", "bf16", "f32"]),
                    far=_log(rng, 10000, 1000000), grad=rng.random() < 0.3)
    hkv = rng.choice([1, 2, 5, 8])
    if op == "write":
        if rng.random() < 0.5:  # a few new tokens of running sequences
            return dict(op="write", B=_log(rng, 1, 128), n=rng.choice([1, 1, 2, 5, 8, 61]), lo=_log(rng, 1, 500),
                        hi=_log(rng, 500, 16000), Hkv=hkv, fmt=fmt, dtype=dtype)
        b = _log(rng, 1, 16)  # prompts, or their next chunks
        at = 64 * rng.choice([0, 0, 1, 7, 40])
        return dict(op="write", B=b, n=_log(rng, 64, min(8192, 40000 // b)), lo=at, hi=at, Hkv=hkv, fmt=fmt, dtype=dtype)
    if op == "read":
        b = _log(rng, 1, 16)
        hi = _log(rng, 64, 64000 // b)
        return dict(op="read", B=b, lo=rng.randint(0, hi), hi=hi, Hkv=hkv, fmt=fmt, dtype=rng.choice(["f16", "bf16", "f32"]))
    hq = hkv * rng.choice([1, 2, 4, 8])
    n = rng.choice([1, 1, 1, 2, 4, 8, _log(rng, 9, 64), _log(rng, 64, 1500)])
    b = _log(rng, 1, max(1, min(64, 64 // n + 1)))
    hi = max(n, _log(rng, 64, max(64, min(32768, 500000 // b // max(1, n // 40)))))
    return dict(op="attend", B=b, n=n, lo=rng.randint(n, hi), hi=hi, Hq=hq, Hkv=hkv, fmt=fmt, dtype=dtype,
                window=rng.choice([0, 0, 0, 100, 4096]))


def _lengths(case):
    """Lengths of the sequences (new tokens included) and how many tokens each has new: by the case alone."""
    rng = random.Random(97 * case["B"] + 31 * case["lo"] + case["hi"])
    lens = [rng.randint(case["lo"], max(case["lo"], case["hi"])) for _ in range(case["B"])]
    lens[0] = max(case["lo"], case["hi"])
    if case["op"] == "read":
        return lens, [0] * case["B"]
    n = case["n"]
    news = [n if n <= 8 or i == 0 else rng.randint(max(1, n // 2), n) for i in range(case["B"])]
    if case["op"] == "write":
        return [x + y for x, y in zip(lens, news)], news
    return [max(x, y) for x, y in zip(lens, news)], news


# ----------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "rope":
        return _prepare_rope(case, g)
    lens, news = _lengths(case)
    B, H, dtype = case["B"], case["Hkv"], DTYPES[case["dtype"]]
    npg = max(1, -(-max(lens) // 128) * 2)  # capacity: a multiple of 128 positions
    total = B * H * npg
    s = dict(case=case, npg=npg, longest=max(lens), most=max(news),
             kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             cu=torch.tensor([sum(news[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda"))
    # the pool has a page more than the cache is told of: where the plain form writes what is not to be kept
    s["pages"] = torch.zeros(total + 1, PAGE, dtype=torch.uint8, device="cuda")
    s["table"] = torch.randperm(total, device="cuda", generator=g).int().reshape(B, H, npg)
    for t in ("tail_k", "tail_v"):
        s[t] = torch.zeros(B, H, 2, BLOCK * D, dtype=torch.float16, device="cuda")
    s["tail_scale"] = torch.ones(B, H, 2, 2 * BLOCK, device="cuda")
    channel = torch.exp(0.5 * torch.randn(H, 1, D, device="cuda", generator=g))  # keys: some channels are larger
    if case["op"] != "write" or case["lo"] > 0:
        _fill(s, case, g, channel, [x - y if case["op"] == "write" else x for x, y in zip(lens, news)])
    N = sum(news)
    if case["op"] == "write":
        s["k"] = (torch.randn(N, H, D, device="cuda", generator=g) * channel.reshape(1, H, D)).to(dtype)
        s["v"] = torch.randn(N, H, D, device="cuda", generator=g).to(dtype)
    elif case["op"] == "attend":
        s["q"] = torch.randn(N, case["Hq"], D, device="cuda", generator=g).to(dtype)
    if own:
        from hybrid_precision_attention_b200 import hq
        s["cache"] = hq.Kv8Cache(B, H, npg * BLOCK, fmt={"e4m3": hq.KV8_E4M3, "int8": hq.KV8_INT8}[case["fmt"]],
                                 pages=s["pages"][:total], page_table=s["table"], tail_k=s["tail_k"], tail_v=s["tail_v"],
                                 tail_scale=s["tail_scale"])
    return s


def _fill(s, case, g, channel, lens):
    """Caches that hold lens[b] positions: every block of every sequence, a few blocks of all at a time."""
    B, H, top = case["B"], case["Hkv"], TOP[case["fmt"]]
    n = torch.tensor(lens, device="cuda")
    step = max(1, 200_000_000 // (B * H * BLOCK * D))
    for j in range(0, s["npg"], step):
        m = min(step, s["npg"] - j)
        k = torch.randn(B, H, m * BLOCK, D, device="cuda", generator=g).mul_(channel).to(DTYPES[case["dtype"]])
        v = torch.randn(B, H, m * BLOCK, D, device="cuda", generator=g).to(DTYPES[case["dtype"]])
        for at, x, order, word in ((0, k, _order_k, 16384), (8192, v, _order_v, 16388)):
            x = x.float().reshape(B, H, m, BLOCK, D)
            amax = x.abs().amax((-1, -2))
            scale = torch.where(amax == 0, 1.0, amax / torch.full_like(amax, top))
            idx = s["table"][:, :, j:j + m].reshape(-1).long()
            s["pages"][idx, at:at + 8192] = order(_code(x / scale[..., None, None], case["fmt"])).reshape(-1, BLOCK * D)
            s["pages"][idx, word:word + 4] = scale.reshape(-1, 1).view(torch.uint8)
            for b in range(B):  # the two newest blocks in 16 bits
                for blk in range(max(0, (lens[b] - 1) // BLOCK - 1), -(-lens[b] // BLOCK)):
                    if j <= blk < j + m:
                        rows = torch.where((blk * BLOCK + torch.arange(BLOCK, device="cuda") < n[b])[:, None], x[b, :, blk - j], 0.0)
                        s["tail_v" if at else "tail_k"][b, :, blk % 2] = order(rows.half()).reshape(H, -1)


def _prepare_rope(case, g):
    B, T, Hq, Hkv, head = case["B"], case["T"], case["Hq"], case["Hkv"], case["D"]
    dtype = DTYPES[case["dtype"]]
    # the fused projection's rows: q, k and v of a token side by side
    row = torch.randn(B, T, Hq + 2 * Hkv, head, device="cuda", generator=g).to(dtype)
    start = torch.randint(0, case["far"], (B, 1), device="cuda", generator=g)
    s = dict(case=case, q=row[:, :, :Hq], k=row[:, :, Hq:Hq + Hkv],
             pos=(start + torch.arange(T, device="cuda")).clamp(max=case["far"]).int())
    inv, amp = _frequencies(case)
    s["inv"], s["amp"] = inv.cuda(), amp
    if own:
        from hybrid_precision_attention_b200 import hq
        kind = dict(plain=hq.ROPE_PLAIN, linear=hq.ROPE_LINEAR, ntk=hq.ROPE_NTK, yarn=hq.ROPE_YARN, bands=hq.ROPE_BANDS)
        s["rope"] = hq.RopeTable(case["rot"], 500000.0, kind=kind[case["scaling"]], factor=8.0, orig_len=8192)
    return s


def _frequencies(case):
    """Radians per position of each pair, float64, and the factor of the rotated values; base 500000, contexts
    stretched 8 times from 8192.  `yarn` (Peng et al. 2023) blends over the pairs that turn 1 to 32 times in the
    original context, linearly in the pair's index; `bands` over those that turn 1 to 4 times, linearly in the turns."""
    rot, base, factor, orig = case["rot"], 500000.0, 8.0, 8192.0
    i = torch.arange(rot // 2, dtype=torch.float64)
    if case["scaling"] == "ntk":
        base = base * factor ** (rot / (rot - 2))
    inv = base ** (-2 * i / rot)
    amp = 1.0
    if case["scaling"] == "linear":
        inv = inv / factor
    elif case["scaling"] == "yarn":
        place = [rot * math.log(orig / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32, 1)]
        low, high = max(math.floor(place[0]), 0), min(math.ceil(place[1]), rot - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        inv = inv / factor * ramp + inv * (1 - ramp)
        amp = 0.1 * math.log(factor) + 1
    elif case["scaling"] == "bands":
        keep = ((orig * inv / (2 * math.pi) - 1) / (4 - 1)).clamp(0, 1)
        inv = (1 - keep) * inv / factor + keep * inv
    return inv, amp


# ----------------------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if own:
        from hybrid_precision_attention_b200 import hq
        if case["op"] == "rope":
            return hq.hq_rope(s["q"], s["k"], s["pos"], s["rope"], grad=case["grad"],
                              layout=hq.ROPE_HALF if case["layout"] == "half" else hq.ROPE_INTERLEAVED)
        if case["op"] == "write":
            hq.hq_kv8_append(s["cache"], s["k"], s["v"], s["cu"], s["kv_len"])
            return _cached(s)
        if case["op"] == "read":
            return hq.hq_kv8_read(s["cache"], s["kv_len"], n=s["longest"], dtype=DTYPES[case["dtype"]], zero_rest=True)
        return hq.hq_kv8_attn(s["cache"], s["q"], s["cu"], s["kv_len"], s["most"], window=case["window"], return_lse=True)
    return {"rope": _rope, "write": _write, "read": _read, "attend": _attend}[case["op"]](s)


def _rope(s):
    case = s["case"]
    angle = s["pos"].double()[..., None, None] * s["inv"]
    cos, sin = (angle.cos() * s["amp"]).float(), (angle.sin() * s["amp"]).float()
    if case["grad"]:  # the transposed rotation
        sin = -sin

    def turn(x):
        rot, out = case["rot"], x.clone(memory_format=torch.contiguous_format)
        y = x[..., :rot].float()
        if case["layout"] == "half":
            a, b = y[..., :rot // 2], y[..., rot // 2:]
            out[..., :rot] = torch.cat((a * cos - b * sin, b * cos + a * sin), -1).to(x.dtype)
        else:
            a, b = y[..., 0::2], y[..., 1::2]
            out[..., :rot] = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2).to(x.dtype)
        return out

    return turn(s["q"]), turn(s["k"])


def _order_k(x):
    """[..., 64, 128] in the page's order of keys."""
    return x.reshape(*x.shape[:-2], 8, 8, 2, 64).transpose(-3, -2).flatten(-4)


def _order_v(x):
    """[..., 64, 128] in the page's order of values."""
    x = x.reshape(*x.shape[:-2], 4, 2, 4, 2, 4, 2, 2, 8)  # token: /16, /8, /2, %2; d: /32, /16, /8, %8
    n = x.dim() - 8
    return x.permute(*range(n), n, n + 4, n + 7, n + 2, n + 5, n + 6, n + 1, n + 3).flatten(-8)


def _rows_k(x):
    """Keys of a page, [..., 8192], as [..., 64, 128]."""
    return x.reshape(*x.shape[:-1], 8, 2, 8, 64).transpose(-3, -2).reshape(*x.shape[:-1], 64, 128)


def _rows_v(x):
    y = x.reshape(*x.shape[:-1], 4, 4, 8, 4, 2, 2, 2, 2)
    n = y.dim() - 8
    return y.permute(*range(n), n, n + 6, n + 3, n + 7, n + 1, n + 4, n + 5, n + 2).reshape(*x.shape[:-1], 64, 128)


def _code(x, fmt):
    if fmt == "e4m3":
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)


def _value(codes, fmt):
    return codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).float()


def _cached(s):
    """What the cache holds: the codes' values, the blocks' scales and the newest blocks in 16 bits."""
    t = torch.float8_e4m3fn if s["case"]["fmt"] == "e4m3" else torch.int8
    p = s["pages"][:-1]
    return dict(codes=p[:, :16384].view(t), scales=p[:, 16384:16392].view(torch.float32), tail_k=s["tail_k"],
                tail_v=s["tail_v"], tail_scale=s["tail_scale"])


def _write(s):
    case, H, dev = s["case"], s["case"]["Hkv"], s["k"].device
    B, n = s["kv_len"].numel(), s["kv_len"].long()
    cu = s["cu"].long()
    first = n - (cu[1:] - cu[:-1])  # position of the first new token
    M = (s["most"] + 62) // BLOCK + 1
    blk = (first // BLOCK)[:, None] + torch.arange(M, device=dev)  # [B, M] blocks that the new tokens touch
    pos = blk[..., None] * BLOCK + torch.arange(BLOCK, device=dev)  # [B, M, 64]
    new = (pos >= first[:, None, None]) & (pos < n[:, None, None])
    rows = (cu[:-1, None, None] + pos - first[:, None, None]).clamp(0, s["k"].shape[0] - 1)
    full = (blk + 1) * BLOCK <= n[:, None]
    page = s["table"].long().gather(2, blk.clamp(max=s["npg"] - 1)[:, None].expand(B, H, M))
    page = torch.where(full[:, None], page, s["pages"].shape[0] - 1).reshape(-1)
    b, h = torch.arange(B, device=dev)[:, None, None], torch.arange(H, device=dev)[None, :, None]
    halves = []
    for x, t, order, back, at, word, which in ((s["k"], "tail_k", _order_k, _rows_k, 0, 16384, 0),
                                               (s["v"], "tail_v", _order_v, _rows_v, 8192, 16388, 1)):
        x = x.float()
        # the block's positions: the new ones, and the earlier ones from the tail
        old = back(s[t])[b, h, (blk % 2)[:, None]].float()  # [B, H, M, 64, 128]
        old = old * s["tail_scale"][:, :, which].reshape(B, H, 2, BLOCK)[b, h, (blk % 2)[:, None]][..., None]
        block = torch.where(new[:, None, ..., None], x[rows].permute(0, 3, 1, 2, 4), old)
        amax = block.abs().amax((-1, -2))
        scale = torch.where(amax == 0, 1.0, amax / torch.full_like(amax, TOP[case["fmt"]]))
        s["pages"][page, at:at + 8192] = order(_code(block / scale[..., None, None], case["fmt"])).reshape(-1, BLOCK * D)
        s["pages"][page, word:word + 4] = scale.reshape(-1, 1).view(torch.uint8)
        halves.append((x, t, order, back, which))
    # the newest two blocks of each sequence in 16 bits
    last = (n - 1) // BLOCK
    both = last[:, None] - (last[:, None] - torch.arange(2, device=dev)) % 2  # [B, 2]: the block of each half
    pos = both[..., None] * BLOCK + torch.arange(BLOCK, device=dev)
    new = ((pos >= first[:, None, None]) & (pos < n[:, None, None]))[:, None]
    rows = (cu[:-1, None, None] + pos - first[:, None, None]).clamp(0, s["k"].shape[0] - 1)
    for x, t, order, back, which in halves:
        y = x[rows].permute(0, 3, 1, 2, 4)
        unit = torch.ones_like(y[..., 0])
        if case["dtype"] == "bf16":  # the row's largest value comes to 2^14 .. 2^15
            top = y.abs().amax(-1)
            unit = torch.where(top == 0, unit, torch.ldexp(unit, (torch.frexp(top)[1] - 15).clamp(min=-126)))
        s[t].copy_(order(torch.where(new[..., None], (y / unit[..., None]).half(), back(s[t]))))
        ts = s["tail_scale"][:, :, which].reshape(B, H, 2, BLOCK)
        s["tail_scale"][:, :, which] = torch.where(new, unit, ts).reshape(B, H, 2 * BLOCK)
    return _cached(s)


def _dense(s, longest):
    """Keys and values as cached, float32 [B, H, blocks * 64, 128]."""
    case, out = s["case"], []
    m = -(-longest // BLOCK)
    B, H = s["kv_len"].numel(), case["Hkv"]
    n, idx = s["kv_len"].long(), s["table"][:, :, :m].long()
    blk = torch.arange(m, device=idx.device)
    tail = (blk[None] == n[:, None] // BLOCK)[:, None, :, None, None]  # the incomplete last block
    p = s["pages"][idx]
    for t, back, at, word, which in (("tail_k", _rows_k, 0, 16384, 0), ("tail_v", _rows_v, 8192, 16388, 1)):
        x = back(_value(p[..., at:at + 8192], case["fmt"])) * p[..., word:word + 4].contiguous().view(torch.float32)[..., None]
        y = back(s[t]).float() * s["tail_scale"][:, :, which].reshape(B, H, 2, BLOCK, 1)
        x = torch.where(tail, y[:, :, blk % 2], x)
        out.append(x.reshape(B, H, m * BLOCK, D))
    return out


def _read(s):
    longest = s["longest"]
    held = (torch.arange(longest, device="cuda") < s["kv_len"][:, None])[:, None, :, None]
    return tuple(torch.where(held, x[:, :, :longest], 0.0).to(DTYPES[s["case"]["dtype"]]) for x in _dense(s, longest))


def _attend(s):
    case, q = s["case"], s["q"]
    B, H, n = s["kv_len"].numel(), case["Hkv"], s["most"]
    G = case["Hq"] // H
    k, v = _dense(s, s["longest"])
    cu = s["cu"].long()
    i = torch.arange(n, device=q.device)
    row = cu[:-1, None] + i  # [B, n] rows of q, those of shorter sequences clamped
    real = row < cu[1:, None]
    at = s["kv_len"].long()[:, None] - (cu[1:] - cu[:-1])[:, None] + i  # position of each query
    x = q[row.clamp(max=q.shape[0] - 1)].float().reshape(B, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, D)
    w = torch.matmul(x, k.transpose(-1, -2)).reshape(B, H, G, n, -1).mul_(D ** -0.5)
    j = torch.arange(k.shape[2], device=q.device)
    seen = (j <= at[..., None]) & real[..., None]
    if case["window"]:
        seen &= j > at[..., None] - case["window"]
    w.masked_fill_(~seen[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True).clamp(min=-3e38)
    w = w.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.reshape(B, H, G * n, -1), v).reshape(B, H, G, n, D) / total
    lse = (top + total.log())[..., 0] / math.log(2)
    o, lse = o.permute(0, 3, 1, 2, 4).reshape(B, n, -1, D), lse.permute(0, 3, 1, 2).reshape(B, n, -1)
    # the sequences' rows one behind another, as q has them
    where = torch.arange(q.shape[0], device=q.device)
    b = torch.searchsorted(cu[1:], where, right=True)
    return o[b, where - cu[b]].to(q.dtype), lse[b, where - cu[b]]


# ----------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "rope":
        n = case["B"] * case["T"] * (case["Hq"] + case["Hkv"])
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * n * case["D"] * size + 4 * case["B"] * case["T"] + 8 * case["rot"] // 2, "flops": 3 * n * case["rot"]}
    lens, news = _lengths(case)
    H, size = case["Hkv"], 4 if case["dtype"] == "f32" else 2
    if case["op"] == "write":
        read = sum(news) * 2 * size * D * H
        wrote = 0
        for L, n in zip(lens, news):
            first = L - n
            blocks = L // BLOCK - first // BLOCK  # blocks that become complete
            wrote += H * blocks * 16392
            if blocks:
                read += H * (first % BLOCK) * 2 * (2 * D + 4)  # their earlier positions
            wrote += H * min(n, (L - 1) % BLOCK + 1 + BLOCK) * 2 * (2 * D + 4)  # the newest two blocks in 16 bits
        return {"bytes": read + wrote, "flops": 0}
    if case["op"] == "read":
        cached = sum(L // BLOCK * 16392 + L % BLOCK * 2 * (2 * D + 4) for L in lens) * H
        return {"bytes": cached + case["B"] * H * max(lens) * 2 * D * size, "flops": sum(lens) * H * 2 * D}
    total, pairs = 0, 0
    for L, n in zip(lens, news):
        w = case["window"] or L
        begin = max(0, L - n + 1 - w) // BLOCK * BLOCK  # the first block that a query sees
        total += H * ((L // BLOCK * BLOCK - begin) // BLOCK * 16392 + L % BLOCK * 2 * (2 * D + 4))
        pairs += sum(min(L - n + i + 1, w) for i in range(n))
    rows = sum(news) * case["Hq"]
    return {"bytes": total + rows * (4 * D + 4), "flops": 4 * D * case["Hq"] * pairs}


# ----------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "write": _exact_write, "read": _exact_read, "attend": _exact_attend}[case["op"]](case, s)


def _exact_rope(case, s):
    rot, z = case["rot"], s["pos"].double()[..., None] * s["inv"]
    turn = torch.polar(torch.full_like(z, s["amp"]), -z if case["grad"] else z)[:, :, None]
    out = []
    for x in (s["q"], s["k"]):
        y = x.double()
        a, b = (y[..., :rot // 2], y[..., rot // 2:rot]) if case["layout"] == "half" else (y[..., 0:rot:2], y[..., 1:rot:2])
        c = torch.complex(a.contiguous(), b.contiguous()) * turn
        first = torch.cat((c.real, c.imag), -1) if case["layout"] == "half" else torch.view_as_real(c).flatten(-2)
        out.append(torch.cat((first, y[..., rot:]), -1))
    return tuple(out)


def _places():
    """Where (token, d) stands in a page's keys and in its values, each [64, 128]."""
    t, d = torch.arange(64, device="cuda")[:, None], torch.arange(128, device="cuda")[None]
    k = ((t // 8 * 2 + d // 64) * 8 + t % 8) * 64 + d % 64
    v = t // 16 * 2048 + d // 32 * 512 + (d % 8 * 4 + t % 8 // 2) * 16 + d // 16 % 2 * 8 + d // 8 % 2 * 4 + t // 8 % 2 * 2 + t % 2
    return k, v


def _e4m3_table():
    c = torch.arange(256, dtype=torch.float64, device="cuda")
    e, m = c % 128 // 8, c % 8
    x = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10))
    return torch.where(c >= 128, -x, x)


def _exact_kv(case, s, b):
    """Keys and values of sequence b as cached: float64 [H, len, 128] each."""
    L, both = int(s["kv_len"][b]), []
    m = -(-L // BLOCK)
    p = s["pages"][s["table"][b, :, :m].long()]
    for place, at, t, which in zip(_places(), (0, 8192), ("tail_k", "tail_v"), (0, 1)):
        c = p[..., place + at].long()
        x = _e4m3_table()[c] if case["fmt"] == "e4m3" else torch.where(c > 127, c - 256, c).double()
        x = x * p[..., 16384 + 4 * which:16388 + 4 * which].contiguous().view(torch.float32).double()[..., None]
        if L % BLOCK:
            half = L // BLOCK % 2
            x[:, -1] = s[t][b, :, half][:, place].double() * s["tail_scale"][b, :, which, half * 64:half * 64 + 64, None].double()
        both.append(x.reshape(x.shape[0], m * BLOCK, D)[:, :L])
    return both


def _exact_read(case, s):
    k = torch.zeros(case["B"], case["Hkv"], s["longest"], D, dtype=torch.float64, device="cuda")
    v = torch.zeros_like(k)
    for b in range(case["B"]):
        x, y = _exact_kv(case, s, b)
        k[b, :, :x.shape[1]], v[b, :, :x.shape[1]] = x, y
    return k, v


def _exact_attend(case, s):
    G, out, lse = case["Hq"] // case["Hkv"], [], []
    cu = s["cu"].tolist()
    for b in range(case["B"]):
        k, v = _exact_kv(case, s, b)
        n, L = cu[b + 1] - cu[b], k.shape[1]
        at = torch.arange(L - n, L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")
        hide = (j > at) | (j <= at - case["window"]) if case["window"] else j > at
        o = torch.empty(n, case["Hq"], D, dtype=torch.float64, device="cuda")
        z = torch.empty(n, case["Hq"], dtype=torch.float64, device="cuda")
        for h in range(case["Hq"]):
            w = (s["q"][cu[b]:cu[b + 1], h].double() @ k[h // G].T / math.sqrt(D)).masked_fill_(hide, -math.inf)
            z[:, h] = torch.logsumexp(w, -1)
            o[:, h] = (w - z[:, h, None]).exp_() @ v[h // G]
        out.append(o)
        lse.append(z / math.log(2))
    return torch.cat(out), torch.cat(lse)


def _exact_write(case, s):
    """Codes by rounding the quotient by the stored (float32) scale in 64 bits; int8 codes are whole numbers and have
    no place here."""
    place = _places()
    codes, scales = torch.zeros(s["pages"].shape[0] - 1, 16384, dtype=torch.float64, device="cuda"), None
    codes[:] = _e4m3_table()[s["pages"][:-1, :16384].long()]
    scales = s["pages"][:-1, 16384:16392].contiguous().view(torch.float32).double()
    tails, unit = [s["tail_k"].double(), s["tail_v"].double()], s["tail_scale"].double()
    cu, lens = s["cu"].tolist(), s["kv_len"].tolist()
    for b in range(case["B"]):
        n, L = cu[b + 1] - cu[b], lens[b]
        begin = (L - n) // BLOCK * BLOCK  # from the first block that changes
        for which, x in enumerate((s["k"], s["v"])):
            new = x[cu[b]:cu[b + 1]].double().transpose(0, 1)  # [H, n, 128]
            half, keep = begin // BLOCK % 2, (L - n) - begin
            old = (s["tail_v" if which else "tail_k"][b, :, half][:, place[which]].double()
                   * s["tail_scale"][b, :, which, half * 64:half * 64 + 64, None].double())[:, :keep]
            rows = torch.cat((old, new), 1)
            full = rows.shape[1] // BLOCK
            if full:
                block = rows[:, :full * BLOCK].reshape(-1, full, BLOCK, D)
                amax = block.abs().amax((-1, -2))
                scale = torch.where(amax == 0, 1.0, amax / TOP[case["fmt"]]).float().double()
                idx = s["table"][b, :, begin // BLOCK:begin // BLOCK + full].long()
                scales[idx, which] = scale
                y = block / scale[..., None, None]
                step = 2.0 ** (torch.frexp(y)[1] - 4).clamp(min=-9).double()  # the distance of e4m3's values near y
                y = (torch.round(y / step) * step).clamp(-448, 448)
                flat = torch.empty(*idx.shape, BLOCK * D, dtype=torch.float64, device="cuda")
                flat[..., place[which]] = y
                codes[idx, 8192 * which:8192 * which + 8192] = flat
            for p in range(max(L - n, (L - 1) // BLOCK * BLOCK - BLOCK), L):
                y = new[:, p - (L - n)]
                u = torch.ones_like(y[:, 0])
                if case["dtype"] == "bf16":
                    top = y.abs().amax(-1)
                    u = torch.where(top == 0, u, 2.0 ** (torch.frexp(top)[1] - 15).clamp(min=-126).double())
                tails[which][b, :, p // BLOCK % 2, place[which][p % BLOCK]] = y / u[:, None]
                unit[b, :, which, p % (2 * BLOCK)] = u
    return dict(codes=codes if case["fmt"] == "e4m3" else None, scales=scales, tail_k=tails[0], tail_v=tails[1], tail_scale=unit)
