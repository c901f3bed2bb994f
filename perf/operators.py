"""The paged K/V cache operators as cases to measure: writing a cache (bf16 or
e4m3 with a scale per token and head), reading it back, and attention of new
tokens over it (causal, bidirectional, sliding window with sinks).

With ``own`` false, ``run`` computes them from elementary torch operations in
32 bits; with ``own`` true it calls ``block_decoding_gb300``.
"""

import math
import random

import torch

own = False

E_MIN, E_MAX = -117, 120      # exponents a scale can have
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _case(op, **kw):
    c = dict(op=op, B=1, heads=8, group=1, dh=128, page=64, fp8=False, lo=1, hi=1, w_lo=1, w_hi=1, left=-1, right=-1,
             sinks=0, ragged=1)
    c.update(kw)
    return c


def listed():
    return [
        # one decode step's new tokens of 64 requests enter an 8-bit cache: latency
        _case("write", name="write_token_e4m3", B=64, heads=8, dh=128, page=16, fp8=True, lo=1, hi=8192, w_lo=1, w_hi=1,
              ragged=11),
        # the refresh of 16 requests (prompt, block and vicinity rows of the 32 x 128 heads) into an 8-bit cache
        _case("write", name="write_refresh_e4m3", B=16, heads=32, dh=128, page=32, fp8=True, lo=320, hi=1120, w_lo=320,
              w_hi=1120, ragged=12),
        # one request of the 16 x 64 heads leaves a bf16 cache, an odd number of rows: latency
        _case("read", name="read_small_bf16", B=1, heads=16, dh=64, page=16, fp8=False, lo=257, hi=257, w_lo=257, w_hi=257,
              ragged=13),
        # 16 requests handed from an 8-bit cache to contiguous bf16 K/V
        _case("read", name="read_requests_e4m3", B=16, heads=32, dh=128, page=64, fp8=True, lo=257, hi=1984, w_lo=257,
              w_hi=1984, ragged=14),
        # the smallest call: one new token of one request of the 16 x 64 heads
        _case("attn", name="attn_token_one", B=1, heads=16, group=1, dh=64, page=16, lo=257, hi=257, right=0, ragged=15),
        # a decode step of 64 ragged requests, grouped heads, 8-bit cache
        _case("attn", name="attn_token_b64_e4m3", B=64, heads=8, group=4, dh=128, page=64, fp8=True, lo=1, hi=8192, right=0,
              ragged=16),
        # a decode step of a few long requests, bf16 cache in small pages
        _case("attn", name="attn_token_long", B=4, heads=8, group=4, dh=128, page=16, lo=20000, hi=40000, right=0, ragged=17),
        # a denoising step of 16 requests: block and vicinity rows of the 32 x 128 heads, every key visible
        _case("attn", name="attn_block_b16", B=16, heads=32, group=1, dh=128, page=32, lo=352, hi=1120, w_lo=64, w_hi=96,
              ragged=18),
        # a piece of two long prompts, causal, grouped heads
        _case("attn", name="attn_chunk", B=2, heads=8, group=4, dh=128, page=64, lo=9001, hi=12001, w_lo=1200, w_hi=1537,
              right=0, ragged=19),
        # pieces of four prompts over an 8-bit cache
        _case("attn", name="attn_chunk_e4m3", B=4, heads=8, group=4, dh=128, page=128, fp8=True, lo=1500, hi=8000, w_lo=300,
              w_hi=512, right=0, ragged=20),
        # a decode step of long requests that see a window and the first tokens
        _case("attn", name="attn_window_token_e4m3", B=32, heads=4, group=8, dh=128, page=64, fp8=True, lo=3000, hi=50000,
              left=4095, right=0, sinks=4, ragged=21),
        # a piece of a long prompt under a window, 64-wide heads
        _case("attn", name="attn_window_chunk", B=1, heads=16, group=1, dh=64, page=32, lo=16001, hi=16001, w_lo=2000,
              w_hi=2000, left=1023, right=0, sinks=4, ragged=22),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "window"])
    c = _case("attn" if op == "window" else op, dh=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
              fp8=rng.random() < 0.5, ragged=rng.randrange(1000, 1 << 20))
    if op in ("write", "read"):
        c["heads"] = rng.choice([1, 2, 4, 5, 8, 16, 32])
        rows = _log_int(rng, 1, 20000)
        c["B"] = min(rows, _log_int(rng, 1, 64))
        w = max(1, min(rows // c["B"], 11000 * 16 // (c["B"] * c["heads"])))
        c["w_lo"], c["w_hi"] = max(1, w // 3), w
        c["lo"], c["hi"] = w, max(w, _log_int(rng, 1, 8192))
        return c
    c["heads"] = rng.choice([1, 2, 4, 8, 16, 32])
    c["group"] = rng.choice([1, 1, 2, 3, 4, 7, 8])
    while c["heads"] * c["group"] > 64:
        c["group"] = (c["group"] + 1) // 2
    form = rng.choice(["token", "block", "chunk"])
    w = {"token": 1, "block": _log_int(rng, 2, 128), "chunk": _log_int(rng, 129, 2048)}[form]
    c["B"] = _log_int(rng, 1, {"token": 64, "block": 16, "chunk": 4}[form])
    c["w_lo"], c["w_hi"] = max(1, w // 2), w
    hi = _log_int(rng, max(1, w // 2), 50000)
    # no dearer than the largest listed cases: score values, and K/V values that the plain form gathers
    hi = min(hi, 1_000_000_000 // (c["B"] * c["heads"] * c["group"] * w), 800_000_000 // (c["B"] * c["heads"] * c["dh"]))
    c["hi"] = max(1, hi)
    c["lo"] = rng.choice([max(1, c["hi"] // 8), c["hi"]])
    c["right"] = rng.choice([0, 0, -1]) if op == "attn" else rng.choice([0, 0, 0, 64])
    if op == "window":
        c["left"] = _log_int(rng, 1, 4096)
        c["sinks"] = rng.choice([0, 1, 4, 64, 200])
    return c


def _lengths(case):
    """(kv_len, new rows) of every request."""
    r = random.Random(case["ragged"])
    kv = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    w = [r.randint(case["w_lo"], case["w_hi"]) for _ in range(case["B"])]
    if case["op"] != "attn":
        kv = [max(a, b) for a, b in zip(kv, w)]
    return kv, w


def work(case):
    kv, w = _lengths(case)
    per = 1 if case["fp8"] else 2
    row = case["heads"] * (case["dh"] * per + (1 if case["fp8"] else 0))       # one cached row of K or of V
    if case["op"] != "attn":
        return {"bytes": sum(w) * 2 * (case["heads"] * case["dh"] * 2 + row), "flops": 0}
    hq = case["heads"] * case["group"]
    pairs = rows = 0
    for n, m in zip(kv, w):
        first, last = n, -1
        for p in range(n - m, n):
            a, b = _span(case, p, n)
            s = min(case["sinks"], a, b) if case["left"] >= 0 else 0
            pairs += max(0, b - a) + max(0, s)
            first, last = min(first, a), max(last, b)
        seen = max(0, last - first)
        rows += seen + (max(0, min(case["sinks"], first, last)) if case["left"] >= 0 else 0)
    total = sum(w)
    return {"bytes": rows * 2 * row + total * hq * (case["dh"] * 4 + 4), "flops": 4 * case["dh"] * hq * pairs}


def _span(case, p, n):
    """The keys [a, b) that a row at position p sees apart from the sinks."""
    b = n if case["right"] < 0 else min(n, p + case["right"] + 1)
    a = 0 if case["left"] < 0 else max(0, p - case["left"])
    return a, max(b, 0)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _pow2(e):
    """2^e in float32, exactly, for whole e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """(codes, biased exponents) of float32 x [..., dh]."""
    a = x.abs().amax(-1)
    m, e = torch.frexp(a)                           # a = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(a > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)
    return (x * _pow2(-e)[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _pool(gen, pages, case, scale):
    """One page pool [pages][heads][page][dh] and its scales: normal rows, channels of several sizes."""
    h, ps, dh = case["heads"], case["page"], case["dh"]
    out = torch.empty((pages, h, ps, dh), dtype=torch.float8_e4m3fn if case["fp8"] else torch.bfloat16, device=DEV)
    sc = torch.empty((pages, h, ps), dtype=torch.uint8, device=DEV) if case["fp8"] else None
    size = scale * torch.exp(0.5 * torch.randn((h, 1, dh), generator=gen, device=DEV))
    step = max(1, (1 << 27) // (h * ps * dh))
    for a in range(0, pages, step):
        b = min(pages, a + step)
        x = torch.randn((b - a, h, ps, dh), generator=gen, device=DEV) * size
        if case["fp8"]:
            out[a:b], sc[a:b] = _quantise(x)
        else:
            out[a:b] = x
    return out, sc


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    kv, w = _lengths(case)
    ps, B, h, dh = case["page"], case["B"], case["heads"], case["dh"]
    need = [-(-n // ps) for n in kv]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=DEV)[:sum(need)].to(torch.int32).cpu()
    table = torch.zeros((B, max(need)), dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    off = [0]
    for n in w:
        off.append(off[-1] + n)
    s = dict(case=dict(case), table=table.to(DEV), off=torch.tensor(off, dtype=torch.int32, device=DEV), rows=off[-1],
             kv_len=torch.tensor(kv, dtype=torch.int32, device=DEV),
             pos0=torch.tensor([a - b for a, b in zip(kv, w)], dtype=torch.int32, device=DEV),
             max_q=max(w), max_kv=max(kv))
    s["k_pages"], s["k_scale"] = _pool(gen, pages, case, 1.0)
    s["v_pages"], s["v_scale"] = _pool(gen, pages, case, 1.0)
    if case["op"] == "write":
        # K and V lie side by side in one projection's output
        both = torch.randn((s["rows"], 2, h, dh), generator=gen, device=DEV)
        both *= torch.exp(0.7 * torch.randn((1, 2, h, dh), generator=gen, device=DEV))
        both = both.to(torch.bfloat16)
        s["k"], s["v"] = both[:, 0], both[:, 1]
    elif case["op"] == "attn":
        s["q"] = (1.5 * torch.randn((s["rows"], h * case["group"], dh), generator=gen, device=DEV)).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return _write(s) if op == "write" else _read(s) if op == "read" else _attn(s)


def _own(s, op):
    import block_decoding_gb300 as bd
    c = s["case"]
    cache = bd.KVPages(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
    if op == "write":
        bd.kv_write(cache, s["k"], s["v"], s["off"], s["pos0"], s["table"])
        return [t for t in (s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]) if t is not None]
    if op == "read":
        return list(bd.kv_read(cache, s["off"], s["pos0"], s["table"], s["rows"]))
    return list(bd.paged_attn(s["q"], cache, s["off"], s["kv_len"], s["table"], s["max_q"], s["max_kv"], left=c["left"],
                              right=c["right"], sinks=c["sinks"], return_lse=True))


def _places(s):
    """Page and slot of every row of the ragged batch."""
    r = torch.arange(s["rows"], device=DEV)
    i = torch.searchsorted(s["off"][1:], r.to(torch.int32), right=True)
    pos = s["pos0"][i] + r - s["off"][i]
    ps = s["case"]["page"]
    return s["table"][i, pos // ps].long(), pos % ps


def _write(s):
    page, slot = _places(s)
    outs = []
    for name in ("k", "v"):
        if s["case"]["fp8"]:
            codes, e = _quantise(s[name].float())
            s[name + "_pages"].view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
            s[name + "_scale"][page, :, slot] = e
        else:
            s[name + "_pages"][page, :, slot] = s[name]
        outs.append(s[name + "_pages"])
    return outs + [t for t in (s["k_scale"], s["v_scale"]) if t is not None]


def _gather(s, name, page, slot):
    """Cached rows as float32 [..., heads, dh]."""
    if not s["case"]["fp8"]:
        return s[name + "_pages"][page, :, slot].float()
    codes = s[name + "_pages"].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn)
    return codes.float() * _pow2(s[name + "_scale"][page, :, slot].to(torch.int32) - 127)[..., None]


def _read(s):
    page, slot = _places(s)
    return [_gather(s, "k", page, slot).to(torch.bfloat16), _gather(s, "v", page, slot).to(torch.bfloat16)]


def _attn(s):
    c = s["case"]
    B, h, g, dh, ps, W, L = c["B"], c["heads"], c["group"], c["dh"], c["page"], s["max_q"], s["max_kv"]
    u = torch.arange(L, device=DEV)
    page = s["table"][:, u // ps].long()                                   # [B][L]
    slot = (u % ps).expand(B, L)
    k = _gather(s, "k", page, slot).permute(0, 2, 3, 1)                    # [B][h][dh][L]
    v = _gather(s, "v", page, slot).permute(0, 2, 1, 3)                    # [B][h][L][dh]
    t = torch.arange(W, device=DEV)
    n = s["off"][1:] - s["off"][:-1]
    live = t < n[:, None]                                                  # [B][W]
    row = torch.where(live, s["off"][:-1, None] + t, 0).long()
    q = s["q"][row].float().view(B, W, h, g, dh).permute(0, 2, 3, 1, 4)    # [B][h][g][W][dh]
    p = s["kv_len"][:, None] - n[:, None] + t                              # [B][W]
    see = (u < s["kv_len"][:, None])[:, None, :] & live[:, :, None]
    if c["right"] >= 0:
        see = see & (u <= p[:, :, None] + c["right"])
    if c["left"] >= 0:
        see = see & ((u >= p[:, :, None] - c["left"]) | (u < c["sinks"]))
    x = torch.matmul(q.reshape(B, h, g * W, dh), k).view(B, h, g, W, L)
    x = (x * (1.0 / math.sqrt(dh))).masked_fill_(~see[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    none = m == float("-inf")
    x = x.sub_(torch.where(none, 0.0, m)).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, h, g * W, L), v).view(B, h, g, W, dh) / torch.where(none, 1.0, l)
    lse = (m + l.log()).squeeze(-1)                                        # an empty row: -inf
    i = torch.searchsorted(s["off"][1:], torch.arange(s["rows"], device=DEV, dtype=torch.int32), right=True)
    at = torch.arange(s["rows"], device=DEV) - s["off"][i]
    out = o.permute(0, 3, 1, 2, 4).reshape(B, W, h * g, dh)[i, at].to(torch.bfloat16)
    return [out, lse.permute(0, 3, 1, 2).reshape(B, W, h * g)[i, at]]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _two(e):
    """2^e in float64, exactly, for whole e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _e4m3(x):
    """float64 x, |x| <= 448, rounded to the nearest e4m3 value (ties to even)."""
    step = _two((torch.frexp(x)[1] - 1).clamp(min=-6) - 3)               # |x| in [2^e, 2^(e+1)): 2^(e-3)
    return torch.round(x / step) * step


def _cached(s, name, i, n):
    """The first n cached rows of request i in float64 [n][heads][dh]."""
    c = s["case"]
    pages = s["table"][i, :-(-n // c["page"])].long()
    x = s[name + "_pages"][pages].to(torch.float64)
    if c["fp8"]:
        x = x * _two(s[name + "_scale"][pages].to(torch.int64) - 127)[..., None]
    return x.transpose(1, 2).reshape(-1, c["heads"], c["dh"])[:n]


def exact(case, seed):
    s = prepare(case, seed)
    kv, w = _lengths(case)
    off = s["off"].tolist()
    if case["op"] == "write":
        outs, scales = [], []
        for name in ("k", "v"):
            pool = s[name + "_pages"].to(torch.float64)
            for i in range(case["B"]):
                x = s[name][off[i]:off[i + 1]].to(torch.float64)
                pos = torch.arange(kv[i] - w[i], kv[i], device=DEV)
                page, slot = s["table"][i, pos // case["page"]].long(), pos % case["page"]
                if case["fp8"]:
                    top = x.abs().amax(-1)
                    e = torch.round(torch.log2(torch.where(top > 0, top / 448, 2.0 ** E_MIN)))
                    e = e + (top > 448 * _two(e)).double()          # the least e with top <= 448 * 2^e
                    e = e - (top <= 448 * _two(e - 1)).double()
                    e = e.clamp(E_MIN, E_MAX)
                    x = _e4m3(x / _two(e)[..., None])
                    s[name + "_scale"][page, :, slot] = (e + 127).to(torch.uint8)
                pool[page, :, slot] = x
            outs.append(pool)
            if case["fp8"]:
                scales.append(s[name + "_scale"])
        return outs + scales
    if case["op"] == "read":
        return [torch.cat([_cached(s, name, i, kv[i])[kv[i] - w[i]:] for i in range(case["B"])]) for name in ("k", "v")]
    h, g, dh = case["heads"], case["group"], case["dh"]
    out = torch.zeros((s["rows"], h * g, dh), dtype=torch.float64, device=DEV)
    lse = torch.full((s["rows"], h * g), float("-inf"), dtype=torch.float64, device=DEV)
    for i in range(case["B"]):
        k, v = _cached(s, "k", i, kv[i]), _cached(s, "v", i, kv[i])
        u = torch.arange(kv[i], device=DEV)
        for a in range(off[i], off[i + 1], 512):
            b = min(off[i + 1], a + 512)
            p = (torch.arange(a, b, device=DEV) - off[i] + kv[i] - w[i])[:, None]
            hidden = torch.zeros((b - a, kv[i]), dtype=torch.bool, device=DEV)
            if case["right"] >= 0:
                hidden |= u > p + case["right"]
            if case["left"] >= 0:
                hidden |= (u < p - case["left"]) & (u >= case["sinks"])
            for j in range(h):
                x = s["q"][a:b, j * g:(j + 1) * g].to(torch.float64) @ k[:, j].T / math.sqrt(dh)
                x = x.masked_fill(hidden[:, None], float("-inf"))
                z = torch.logsumexp(x, -1)
                y = torch.exp(x - z[..., None]).nan_to_num(0.0) @ v[:, j]
                out[a:b, j * g:(j + 1) * g], lse[a:b, j * g:(j + 1) * g] = y, z
    return [out, lse]
