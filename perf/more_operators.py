"""What a server does around the attention of a paged K/V cache, as cases to
measure: rotary positions with several axes on the way into the cache,
attention for a tree of drafted tokens, the weight that attention gave to every
cached row, eviction by that weight, and moving rows within the cache.

With ``own`` false, ``run`` computes them from elementary torch operations;
with ``own`` true it calls ``block_decoding_gb300``.
"""

import math
import random

import numpy as np
import torch

own = False

E_MIN, E_MAX = -117, 120      # exponents a scale of the 8-bit rows can have
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _case(op, **kw):
    c = dict(op=op, B=1, heads=8, group=1, dh=128, page=64, fp8=False, lo=1, hi=1, w_lo=1, w_hi=1, ragged=1)
    if op == "rope":
        c.update(rot=c["dh"], axes=3, interleaved=False, base=10000.0, far=0)
    if op == "mass":
        c.update(right=-1, decay=1.0)
    if op == "evict":
        c.update(budget=1, sinks=0, recent=0, in_place=True, move_mass=False)
    if op == "move":
        c.update(per_head=False, with_mass=False)
    c.update(kw)
    return c


def listed():
    return [
        # the new tokens of 64 requests of a model for text and images, one denoising or decode step: latency
        _case("rope", name="rope_token", B=64, heads=8, group=4, rot=128, lo=1, hi=8192, page=16, ragged=11),
        # the patches of images (an odd number of them) and the text around them enter a bf16 cache
        _case("rope", name="rope_image", B=4, heads=8, group=4, rot=128, lo=1300, hi=2600, w_lo=1300, w_hi=2600, page=64,
              ragged=12),
        # frames of long videos, far positions, half of each head rotated, into an 8-bit cache and from there to the
        # contiguous rows that a block's attention reads
        _case("rope", name="rope_video_e4m3", B=8, heads=32, group=1, rot=64, interleaved=True, base=1000000.0, far=1000000,
              fp8=True, lo=900, hi=1800, w_lo=900, w_hi=1800, page=32, ragged=13),
        # one request's short draft, 16 x 64 heads: latency
        _case("tree", name="tree_one", B=1, heads=16, dh=64, page=16, lo=300, hi=300, w_lo=13, w_hi=13, ragged=14),
        # the drafts of 32 ragged requests, grouped heads, 8-bit cache
        _case("tree", name="tree_batch_e4m3", B=32, heads=8, group=4, page=64, fp8=True, lo=70, hi=8192, w_lo=20, w_hi=64,
              ragged=15),
        # a few long requests whose drafts are small
        _case("tree", name="tree_long", B=4, heads=8, group=4, page=16, lo=20000, hi=40000, w_lo=5, w_hi=8, ragged=16),
        # a decode step of 64 ragged requests adds its weights to an 8-bit cache's rows
        _case("mass", name="mass_token_e4m3", B=64, heads=8, group=4, page=64, fp8=True, lo=1, hi=8192, right=0, decay=0.9375,
              ragged=17),
        # the last tokens of four long prompts weigh what came before, causal, grouped heads
        _case("mass", name="mass_prompt", B=4, heads=8, group=4, page=64, lo=9001, hi=12001, w_lo=50, w_hi=64, right=0,
              ragged=18),
        # one request of the 16 x 64 heads makes room where its rows lie: latency
        _case("evict", name="evict_one", B=1, heads=16, dh=64, page=16, lo=701, hi=701, budget=512, sinks=4, recent=64,
              ragged=19),
        # 16 prompts of an 8-bit cache shrink to 2048 rows in pages of their own (the prompt's pages may be shared)
        _case("evict", name="evict_batch_e4m3", B=16, heads=8, page=64, fp8=True, lo=1500, hi=12000, budget=2048, sinks=4,
              recent=128, in_place=False, move_mass=True, ragged=20),
        # the accepted tokens of 32 drafts move to the end of their requests: latency
        _case("move", name="move_accepted", B=32, heads=8, page=64, lo=70, hi=8192, w_lo=20, w_hi=64, ragged=21),
        # every head of eight requests keeps rows of its own, in place, with what they weigh
        _case("move", name="move_kept_e4m3", B=8, heads=8, page=32, fp8=True, per_head=True, with_mass=True, lo=4000, hi=8000,
              ragged=22),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "tree", "tree", "mass", "mass", "evict", "move"])
    c = _case(op, dh=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]), fp8=rng.random() < 0.5,
              heads=rng.choice([1, 2, 4, 5, 8, 16, 32]), ragged=rng.randrange(1000, 1 << 20))
    if op == "rope":
        c["group"] = rng.choice([1, 2, 3, 4, 8])
        c["rot"] = rng.choice([c["dh"], c["dh"], c["dh"] // 2, c["dh"] // 4])
        c["axes"], c["interleaved"] = rng.choice([1, 2, 3, 3, 4]), rng.random() < 0.5
        c["base"], c["far"] = rng.choice([10000.0, 500000.0, 1000000.0]), rng.choice([0, 0, 100000, 10000000])
        rows = min(_log_int(rng, 1, 16000), 16000 * 16 // (c["heads"] * (2 + c["group"])))
        c["B"] = min(rows, _log_int(rng, 1, 64))
        w = max(1, rows // c["B"])
        c["w_lo"], c["w_hi"] = max(1, w // 3), w
        c["lo"], c["hi"] = w, max(w, _log_int(rng, 1, 8192))
    elif op in ("tree", "mass"):
        c["group"] = rng.choice([1, 1, 2, 3, 4, 7, 8])
        while c["heads"] * c["group"] > 64:
            c["group"] = (c["group"] + 1) // 2
        w = _log_int(rng, 1, 300 if op == "tree" else 1200)
        c["B"] = _log_int(rng, 1, 64 if w < 64 else 8)
        c["w_lo"], c["w_hi"] = max(1, w // 2), w
        hi = _log_int(rng, w, 50000)
        # no dearer than the largest listed cases: score values, and K/V values that the plain form gathers
        hi = min(hi, 500_000_000 // (c["B"] * c["heads"] * c["group"] * w), 500_000_000 // (c["B"] * c["heads"] * c["dh"]))
        c["hi"] = max(w, hi)
        c["lo"] = rng.choice([max(w, c["hi"] // 8), c["hi"]])
        if op == "mass":
            c["right"], c["decay"] = rng.choice([0, 0, -1, 16]), rng.choice([1.0, 1.0, 0.9375, 0.5])
    else:
        c["B"] = _log_int(rng, 1, 32)
        c["hi"] = max(2, min(_log_int(rng, 2, 30000), 140_000_000 // (c["B"] * c["heads"] * c["dh"])))
        c["lo"] = rng.choice([max(2, c["hi"] // 8), c["hi"]])
        if op == "evict":
            c["budget"] = _log_int(rng, 1, c["hi"])
            c["sinks"] = min(rng.choice([0, 1, 4, 100]), c["budget"] // 4)
            c["recent"] = min(rng.choice([0, 1, 32, 200]), c["budget"] // 2)
            c["in_place"] = rng.random() < 0.5
            c["move_mass"] = not c["in_place"] and rng.random() < 0.5
        else:
            c["per_head"], c["with_mass"] = rng.random() < 0.5, rng.random() < 0.5
            if not c["per_head"]:
                c["w_hi"] = _log_int(rng, 1, min(256, c["lo"]))
                c["w_lo"] = max(1, c["w_hi"] // 3)
    return c


def _lengths(case):
    """(kv_len, new rows) of every request."""
    r = random.Random(case["ragged"])
    kv = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    w = [r.randint(case["w_lo"], case["w_hi"]) for _ in range(case["B"])]
    return [max(a, b) for a, b in zip(kv, w)], w


def _axis_of(case):
    """The axis of every rotated pair of a head."""
    half, axes = case["rot"] // 2, case["axes"]
    if case["interleaved"]:
        return [j % axes for j in range(half)]
    return [min(j * axes // half, axes - 1) for j in range(half)]


def _lists(case):
    """move: for every request (first position written, [heads or 1] ascending lists of the rows that move there)."""
    kv, w = _lengths(case)
    r, rows = random.Random(case["ragged"] + 1), np.random.RandomState(case["ragged"] + 1)
    out = []
    for n, m in zip(kv, w):
        if case["per_head"]:
            k = max(1, n // 2)
            out.append((0, [np.sort(rows.permutation(n)[:k]).tolist() for _ in range(case["heads"])]))
        else:
            k = r.randint(1, min(8, m))
            out.append((n - m, [[n - m + t for t in sorted(r.sample(range(m), k))]]))
    return out


def work(case):
    kv, w = _lengths(case)
    heads, dh, hq = case["heads"], case["dh"], case["heads"] * case["group"]
    row = dh + 1 if case["fp8"] else dh * 2                       # one cached row of one head, of K or of V
    op = case["op"]
    if op == "rope":
        rows = sum(w)
        bytes_ = rows * (4 * case["axes"] + hq * dh * 4 + heads * dh * 4 + 2 * heads * row)
        if case["fp8"]:
            bytes_ += rows * 2 * heads * (row + 2 * dh)           # read back
        return {"bytes": bytes_, "flops": rows * (hq + heads) * case["rot"] * 3}
    if op == "tree":
        pairs, bytes_ = 0, 0
        for n, m, par in zip(kv, w, _parents(case)):
            depth = []
            for p in par:
                depth.append(1 if p < 0 else depth[p] + 1)
            pairs += m * (n - m) + sum(depth)
            bytes_ += n * heads * 2 * row + m * (hq * (dh * 4 + 4) + 4)
        return {"bytes": bytes_, "flops": 4 * dh * hq * pairs}
    if op == "mass":
        pairs, bytes_ = 0, 0
        for n, m in zip(kv, w):
            pairs += sum(n if case["right"] < 0 else min(n, n - m + t + case["right"] + 1) for t in range(m))
            bytes_ += n * heads * (row + 8) + m * hq * (dh * 2 + 4)
        return {"bytes": bytes_, "flops": 2 * dh * hq * pairs}
    if op == "evict":
        kept = [min(n, case["budget"]) for n in kv]
        moved = sum(k for k, n in zip(kept, kv) if k < n or not case["in_place"])
        return {"bytes": heads * (4 * sum(kv) + 4 * sum(kept) + moved * (4 * row + (8 if case["move_mass"] else 0))), "flops": 0}
    moved = sum(len(x) for _, lists in _lists(case) for x in lists) * (1 if case["per_head"] else heads)
    return {"bytes": moved * (4 * row + (8 if case["with_mass"] else 0)), "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _parents(case):
    """tree: the parent of every drafted token (its number in the request, less than the token's own; -1: the last
    accepted token), level by level with a few continuations each, as a draft model's best guesses grow."""
    r = random.Random(case["ragged"] + 2)
    out = []
    for m in _lengths(case)[1]:
        par = []
        for t in range(m):
            if t < 3:
                par.append(-1 if r.random() < 0.7 or t == 0 else r.randrange(t))
            else:
                par.append(r.randrange(max(0, t - 12), t) if r.random() < 0.95 else -1)
        out.append(par)
    return out


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


def _pool(gen, pages, case):
    """One page pool [pages][heads][page][dh] and its scales: normal rows, channels of several sizes."""
    h, ps, dh = case["heads"], case["page"], case["dh"]
    out = torch.empty((pages, h, ps, dh), dtype=torch.float8_e4m3fn if case["fp8"] else torch.bfloat16, device=DEV)
    sc = torch.empty((pages, h, ps), dtype=torch.uint8, device=DEV) if case["fp8"] else None
    size = torch.exp(0.5 * torch.randn((h, 1, dh), generator=gen, device=DEV))
    step = max(1, (1 << 27) // (h * ps * dh))
    for a in range(0, pages, step):
        b = min(pages, a + step)
        x = torch.randn((b - a, h, ps, dh), generator=gen, device=DEV) * size
        if case["fp8"]:
            out[a:b], sc[a:b] = _quantise(x)
        else:
            out[a:b] = x
    return out, sc


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _table(need, order):
    """Page tables [requests][most pages] of the pages in `order`."""
    table, at = torch.zeros((len(need), max(need)), dtype=torch.int32), 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table.to(DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op, ps, B, h, g, dh = case["op"], case["page"], case["B"], case["heads"], case["group"], case["dh"]
    kv, w = _lengths(case)
    need = [-(-n // ps) for n in kv]
    new = [0] * B
    if op == "evict" and not case["in_place"]:
        new = [-(-min(n, case["budget"]) // ps) for n in kv]
    pages = sum(need) + sum(new) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32).cpu()
    off = [0]
    for n in w:
        off.append(off[-1] + n)
    rows = off[-1]
    s = dict(case=dict(case), table=_table(need, order), off=_int32(off), rows=rows, kv_len=_int32(kv),
             pos0=_int32([a - b for a, b in zip(kv, w)]), max_q=max(w), max_kv=max(kv))
    s["k_pages"], s["k_scale"] = _pool(gen, pages, case)
    s["v_pages"], s["v_scale"] = _pool(gen, pages, case)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    if op == "rope":
        # q, k and v lie side by side in one projection's output
        both = normal(rows, (g + 2) * h, dh)
        both *= torch.exp(0.5 * normal(1, (g + 2) * h, dh))
        both = both.to(torch.bfloat16)
        s["q"], s["k"], s["v"] = both[:, :g * h], both[:, g * h:(g + 1) * h], both[:, (g + 1) * h:]
        # where the rows are on every axis: the first counts tokens or frames, the others rows and columns of a picture
        at = torch.cat([torch.arange(n - m, n, device=DEV) for n, m in zip(kv, w)])
        grid = [at + case["far"], at // 28 % 25, at % 28, at % 700]
        s["pos"] = torch.stack(grid[:case["axes"]]).to(torch.int32)
        s["axis"] = _axis_of(case)
        s["freq"] = [case["base"] ** (-2.0 * j / case["rot"]) for j in range(case["rot"] // 2)]
        s["axis_t"] = torch.tensor(s["axis"], device=DEV)
        s["freq_t"] = torch.tensor(s["freq"], dtype=torch.float64, device=DEV)
    elif op == "tree":
        s["q"] = (1.5 * normal(rows, h * g, dh)).to(torch.bfloat16)
        s["parent"] = _int32(sum(_parents(case), []))
    elif op == "mass":
        s["q"] = (1.5 * normal(rows, h * g, dh)).to(torch.bfloat16)
        s["lse"] = _lse(s, off, kv)
        s["mass"] = normal(pages, h, ps).exp()
    elif op == "evict":
        # a few rows weigh much, many little, some nothing at all
        x = (3 * normal(pages, h, ps)).exp()
        s["mass"] = torch.where(torch.rand(x.shape, generator=gen, device=DEV) < 0.1, 0.0, x)
        s["dst"] = s["table"] if case["in_place"] else _table(new, order[sum(need):])
    else:
        lists = _lists(case)
        n = max(len(x[0]) for _, x in lists)
        s["src"] = _int32([[r + [0] * (n - len(r)) for r in x] for _, x in lists])
        s["count"] = _int32([len(x[0]) for _, x in lists])
        s["first"] = _int32([p for p, _ in lists])
        s["mass"] = normal(pages, h, ps).exp() if case["with_mass"] else None
    return s


def _lse(s, off, kv):
    """log of the sum that divides every query row's weights, as attention returned it."""
    c = s["case"]
    out = torch.empty((s["rows"], c["heads"] * c["group"]), device=DEV)
    for i, n in enumerate(kv):
        k = _cached(s, "k", i, n).float()
        q = s["q"][off[i]:off[i + 1]].float().view(-1, c["heads"], c["group"], c["dh"])
        x = torch.matmul(q.permute(1, 2, 0, 3).reshape(c["heads"], -1, c["dh"]), k.permute(1, 2, 0)) / math.sqrt(c["dh"])
        x = x.view(c["heads"], c["group"], -1, n)
        if c["right"] >= 0:
            p = torch.arange(n - x.shape[2], n, device=DEV)
            x = x.masked_fill(torch.arange(n, device=DEV) > p[:, None] + c["right"], float("-inf"))
        out[off[i]:off[i + 1]] = torch.logsumexp(x, -1).permute(2, 0, 1).reshape(-1, c["heads"] * c["group"])
    return out


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    return {"rope": _rope, "tree": _tree, "mass": _mass, "evict": _evict, "move": _move}[s["case"]["op"]](s)


def _pools(s, *more):
    """The cache as it is now, and what else a pass changed."""
    return [t for t in (s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], *more) if t is not None]


def _own(s):
    import block_decoding_gb300 as bd
    c = s["case"]
    op = c["op"]
    cache = bd.KVPages(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
    if op == "rope":
        rope = bd.Rope(c["dh"], s["axis"], s["freq"])
        q = bd.rope_kv_write(cache, rope, s["pos"], s["q"], s["k"], s["v"], s["off"], s["pos0"], s["table"])
        if c["fp8"]:
            return [q, *bd.kv_read(cache, s["off"], s["pos0"], s["table"], s["rows"])]
        return [q, s["k_pages"], s["v_pages"]]
    if op == "tree":
        mask, depth = bd.tree_mask(s["parent"], s["off"], s["max_q"])
        return [depth, *bd.tree_attn(s["q"], cache, s["off"], s["kv_len"], s["table"], mask, s["max_q"], s["max_kv"],
                                     return_lse=True)]
    if op == "mass":
        bd.attn_mass(s["q"], s["lse"], cache, s["mass"], s["off"], s["kv_len"], s["table"], s["max_q"], s["max_kv"],
                     right=c["right"], decay=c["decay"])
        return [s["mass"]]
    if op == "evict":
        n, keep = bd.kv_evict(cache, s["mass"], s["kv_len"], s["table"], c["budget"], s["max_kv"], sinks=c["sinks"],
                              recent=c["recent"], dst_table=s["dst"], move_mass=c["move_mass"])
        return _pools(s, s["mass"], n, keep)
    bd.kv_move(cache, s["src"], s["count"], s["first"], s["table"], mass=s["mass"])
    return _pools(s, s["mass"])


def _places(s):
    """Page and slot of every row of the ragged batch."""
    r = torch.arange(s["rows"], device=DEV)
    i = torch.searchsorted(s["off"][1:], r.to(torch.int32), right=True)
    pos = s["pos0"][i] + r - s["off"][i]
    ps = s["case"]["page"]
    return s["table"][i, pos // ps].long(), pos % ps


def _rope(s):
    c = s["case"]
    half = c["rot"] // 2
    # angles in 64 bits: far positions turn many times
    angle = s["pos"].to(torch.float64)[s["axis_t"]].T * s["freq_t"]                # [rows][half]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turn(x):
        x = x.float()
        a, b = x[..., :half], x[..., half:2 * half]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * half:]], -1)

    q, k, v = turn(s["q"]).to(torch.bfloat16), turn(s["k"]), s["v"].float()
    page, slot = _places(s)
    if not c["fp8"]:
        s["k_pages"][page, :, slot] = k.to(torch.bfloat16)
        s["v_pages"][page, :, slot] = s["v"]
        return [q, s["k_pages"], s["v_pages"]]
    (kc, ke), (vc, ve) = _quantise(k), _quantise(v)
    s["k_pages"].view(torch.uint8)[page, :, slot], s["k_scale"][page, :, slot] = kc.view(torch.uint8), ke
    s["v_pages"].view(torch.uint8)[page, :, slot], s["v_scale"][page, :, slot] = vc.view(torch.uint8), ve
    return [q, _gather(s, "k", page, slot).to(torch.bfloat16), _gather(s, "v", page, slot).to(torch.bfloat16)]


def _gather(s, name, page, slot):
    """Cached rows as float32 [..., heads, dh]."""
    if not s["case"]["fp8"]:
        return s[name + "_pages"][page, :, slot].float()
    codes = s[name + "_pages"].view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn)
    return codes.float() * _pow2(s[name + "_scale"][page, :, slot].to(torch.int32) - 127)[..., None]


def _batch(s):
    """The ragged batch with every request at full length: (positions [L], page and slot [B][L], rows [B][W], which of
    them there are, q [B][h][g * W][dh])."""
    c = s["case"]
    B, h, g, dh, W, L = c["B"], c["heads"], c["group"], c["dh"], s["max_q"], s["max_kv"]
    u = torch.arange(L, device=DEV)
    page = s["table"][:, u // c["page"]].long()
    slot = (u % c["page"]).expand(B, L)
    t = torch.arange(W, device=DEV)
    live = t < (s["off"][1:] - s["off"][:-1])[:, None]
    row = torch.where(live, s["off"][:-1, None] + t, 0).long()
    q = s["q"][row].float().view(B, W, h, g, dh).permute(0, 2, 3, 1, 4).reshape(B, h, g * W, dh)
    return u, page, slot, row, live, q


def _tree(s):
    c = s["case"]
    B, h, g, dh, W, L = c["B"], c["heads"], c["group"], c["dh"], s["max_q"], s["max_kv"]
    u, page, slot, row, live, q = _batch(s)
    # ancestors: the closure of "my parent", by squaring; the root is a token of its own, W
    parent = torch.where(live, s["parent"][row], -1).long()
    up = torch.where(parent < 0, W, parent)
    up = torch.cat([up, torch.full((B, 1), W, device=DEV)], 1)
    reach = torch.zeros((B, W + 1, W + 1), device=DEV).scatter_(2, up[:, :, None], 1.0)
    reach = ((reach + torch.eye(W + 1, device=DEV)) > 0).float()
    for _ in range(max(1, (W - 1).bit_length())):
        reach = (torch.matmul(reach, reach) > 0).float()
    above = reach[:, :W, :W] > 0                                                   # [B][W][W], the token itself among them
    depth = above.sum(-1, dtype=torch.int32) - 1
    k = _gather(s, "k", page, slot).permute(0, 2, 3, 1)                            # [B][h][dh][L]
    v = _gather(s, "v", page, slot).permute(0, 2, 1, 3)                            # [B][h][L][dh]
    node = u - s["pos0"][:, None]                                                  # [B][L]
    see = torch.gather(above, 2, node.clamp(0, W - 1)[:, None].expand(B, W, L)) | (node < 0)[:, None]
    see = see & (u < s["kv_len"][:, None])[:, None] & live[:, :, None]
    x = torch.matmul(q, k).view(B, h, g, W, L)
    x = (x * (1.0 / math.sqrt(dh))).masked_fill_(~see[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    none = m == float("-inf")
    x = x.sub_(torch.where(none, 0.0, m)).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, h, g * W, L), v).view(B, h, g, W, dh) / torch.where(none, 1.0, l)
    lse = (m + l.log()).squeeze(-1)
    i = torch.searchsorted(s["off"][1:], torch.arange(s["rows"], device=DEV, dtype=torch.int32), right=True)
    at = torch.arange(s["rows"], device=DEV) - s["off"][i]
    out = o.permute(0, 3, 1, 2, 4).reshape(B, W, h * g, dh)[i, at].to(torch.bfloat16)
    return [depth[i, at], out, lse.permute(0, 3, 1, 2).reshape(B, W, h * g)[i, at]]


def _mass(s):
    c = s["case"]
    B, h, g, W, L = c["B"], c["heads"], c["group"], s["max_q"], s["max_kv"]
    u, page, slot, row, live, q = _batch(s)
    k = _gather(s, "k", page, slot).permute(0, 2, 3, 1)
    lse = s["lse"][row].view(B, W, h, g).permute(0, 2, 3, 1)                       # [B][h][g][W]
    see = (u < s["kv_len"][:, None])[:, None] & live[:, :, None]
    if c["right"] >= 0:
        see = see & (u <= (s["pos0"][:, None] + torch.arange(W, device=DEV) + c["right"])[:, :, None])
    x = torch.matmul(q, k).view(B, h, g, W, L)
    x = (x * (1.0 / math.sqrt(c["dh"]))).sub_(lse[..., None]).masked_fill_(~see[:, None, None], float("-inf")).exp_()
    x = x.sum(2).sum(2)                                                            # [B][h][L]
    here = (u < s["kv_len"][:, None]).reshape(-1)
    page, slot = page.reshape(-1)[here], slot.reshape(-1)[here]
    x = x.permute(0, 2, 1).reshape(B * L, h)[here]
    s["mass"][page, :, slot] = s["mass"][page, :, slot] * c["decay"] + x
    return [s["mass"]]


def _evict(s):
    c = s["case"]
    B, h, L, ps = c["B"], c["heads"], s["max_kv"], c["page"]
    u = torch.arange(L, device=DEV)
    page, slot = s["table"][:, u // ps].long(), (u % ps).expand(B, L)
    x = s["mass"][page, :, slot].permute(0, 2, 1)                                  # [B][h][L]
    n = s["kv_len"][:, None, None]
    x = torch.where((u < c["sinks"]) | (u >= n - c["recent"]), float("inf"), x)
    x = torch.where(u < n, x, -1.0)
    best = torch.sort(x, dim=-1, descending=True, stable=True)[1][..., :c["budget"]]
    new_len = torch.minimum(s["kv_len"], torch.full_like(s["kv_len"], c["budget"]))
    j = torch.arange(best.shape[-1], device=DEV)
    live = j < new_len[:, None, None]
    keep = torch.sort(torch.where(live, best, L), dim=-1)[0]
    keep = torch.where(live, keep, -1)
    keep = torch.cat([keep, keep.new_full((B, h, c["budget"] - best.shape[-1]), -1)], -1).to(torch.int32)
    _shift(s, keep, new_len, torch.zeros_like(new_len), s["dst"], s["mass"] if c["move_mass"] else None)
    return _pools(s, s["mass"], new_len, keep)


def _move(s):
    _shift(s, s["src"].expand(-1, s["case"]["heads"], -1), s["count"], s["first"], s["table"], s["mass"])
    return _pools(s, s["mass"])


def _shift(s, src, count, first, dst, mass):
    """Rows src [B][heads][n] of the cache to positions first + 0, 1, .. of the tables `dst`."""
    ps = s["case"]["page"]
    B, h, n = src.shape
    j = torch.arange(n, device=DEV)
    live = (j < count[:, None, None]).expand(B, h, n)
    i = torch.arange(B, device=DEV)[:, None, None].expand(B, h, n)[live]
    head = torch.arange(h, device=DEV)[None, :, None].expand(B, h, n)[live]
    a = src[live].long()
    b = (first[:, None, None] + j).expand(B, h, n)[live].long()
    a, a_slot = s["table"][i, a // ps].long(), a % ps
    b, b_slot = dst[i, b // ps].long(), b % ps
    pools = [s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], mass]
    pools = [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in pools if t is not None]
    rows = [t[a, head, a_slot] for t in pools]
    [t.index_put_((b, head, b_slot), r) for t, r in zip(pools, rows)]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _two(e):
    """2^e in float64, exactly, for whole e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _e4m3_row(x):
    """float64 rows x [..., dh] as the 8-bit rows stand for them: the least power of two that brings a row under 448, and
    the nearest e4m3 value (ties to even)."""
    top = x.abs().amax(-1, keepdim=True)
    e = torch.round(torch.log2(torch.where(top > 0, top / 448, 2.0 ** E_MIN)))
    e = e + (top > 448 * _two(e)).double()
    e = e - (top <= 448 * _two(e - 1)).double()
    e = e.clamp(E_MIN, E_MAX)
    y = x / _two(e)
    step = _two((torch.frexp(y)[1] - 1).clamp(min=-6) - 3)
    return torch.round(y / step) * step * _two(e)


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
    return {"rope": _exact_rope, "tree": _exact_tree, "mass": _exact_mass, "evict": _exact_moves, "move": _exact_moves}[
        case["op"]](s, case, kv, w, off)


def _exact_rope(s, case, kv, w, off):
    def turned(x):
        z = x.to(torch.float64)
        y = z.clone()
        for j, (a, f) in enumerate(zip(_axis_of(case), s["freq"])):
            angle = s["pos"][a].to(torch.float64) * f
            turn = torch.complex(torch.cos(angle), torch.sin(angle))[:, None]
            p = torch.complex(z[..., j], z[..., j + case["rot"] // 2]) * turn
            y[..., j], y[..., j + case["rot"] // 2] = p.real, p.imag
        return y

    q, k, v = turned(s["q"]), turned(s["k"]), s["v"].to(torch.float64)
    if case["fp8"]:
        return [q, _e4m3_row(k), _e4m3_row(v)]
    outs = [q]
    for name, x in (("k", k), ("v", v)):
        pool = s[name + "_pages"].to(torch.float64)
        for i, (n, m) in enumerate(zip(kv, w)):
            at = torch.arange(n - m, n, device=DEV)
            pool[s["table"][i, at // case["page"]].long(), :, at % case["page"]] = x[off[i]:off[i + 1]]
        outs.append(pool)
    return outs


def _exact_tree(s, case, kv, w, off):
    h, g, dh = case["heads"], case["group"], case["dh"]
    out = torch.zeros((s["rows"], h * g, dh), dtype=torch.float64, device=DEV)
    lse = torch.zeros((s["rows"], h * g), dtype=torch.float64, device=DEV)
    for i, par in enumerate(_parents(case)):
        n, m = kv[i], w[i]
        hidden = torch.zeros((m, n), dtype=torch.bool)
        hidden[:, n - m:] = True
        for t in range(m):
            a = t
            while a >= 0:
                hidden[t, n - m + a] = False
                a = par[a]
        hidden = hidden.to(DEV)[:, None]
        k, v = _cached(s, "k", i, n), _cached(s, "v", i, n)
        for j in range(h):
            x = s["q"][off[i]:off[i + 1], j * g:(j + 1) * g].to(torch.float64) @ k[:, j].T / math.sqrt(dh)
            x = x.masked_fill(hidden, float("-inf"))
            z = torch.logsumexp(x, -1)
            out[off[i]:off[i + 1], j * g:(j + 1) * g] = torch.exp(x - z[..., None]) @ v[:, j]
            lse[off[i]:off[i + 1], j * g:(j + 1) * g] = z
    return [None, out, lse]


def _exact_mass(s, case, kv, w, off):
    h, g, dh = case["heads"], case["group"], case["dh"]
    mass = s["mass"].to(torch.float64)
    for i, (n, m) in enumerate(zip(kv, w)):
        k = _cached(s, "k", i, n)
        u = torch.arange(n, device=DEV)
        hidden = torch.zeros((m, n), dtype=torch.bool, device=DEV)
        if case["right"] >= 0:
            hidden = u > torch.arange(n - m, n, device=DEV)[:, None] + case["right"]
        page, slot = s["table"][i, u // case["page"]].long(), u % case["page"]
        for j in range(h):
            x = s["q"][off[i]:off[i + 1], j * g:(j + 1) * g].to(torch.float64) @ k[:, j].T / math.sqrt(dh)
            x = torch.exp(x - s["lse"][off[i]:off[i + 1], j * g:(j + 1) * g].to(torch.float64)[..., None])
            mass[page, j, slot] = mass[page, j, slot] * case["decay"] + x.masked_fill(hidden[:, None], 0.0).sum((0, 1))
    return [mass]


def _exact_moves(s, case, kv, w, off):
    B, h, ps = case["B"], case["heads"], case["page"]
    if case["op"] == "evict":
        first, lists, dst = [0] * B, [], s["dst"]
        mass = s["mass"] if case["move_mass"] else None
        for i, n in enumerate(kv):
            u = torch.arange(n, device=DEV)
            x = s["mass"][s["table"][i, u // ps].long(), :, u % ps].T.to(torch.float64).cpu()       # [h][n]
            u = u.cpu()
            chosen = (u < case["sinks"]) | (u >= n - case["recent"])
            free = max(0, min(n, case["budget"]) - int(chosen.sum()))
            per = []
            for j in range(h):
                others = [a for a in range(n) if not chosen[a]] if n > case["budget"] else u.tolist()
                row = x[j].tolist()
                if n > case["budget"]:
                    others = sorted(others, key=lambda a: (-row[a], a))[:free] + u[chosen].tolist()
                per.append(sorted(others))
            lists.append(per)
    else:
        first, dst, mass = [p for p, _ in _lists(case)], s["table"], s["mass"]
        lists = [x * (1 if case["per_head"] else h) for _, x in _lists(case)]
    names = ["k_pages", "v_pages"]
    outs = [s[x].to(torch.float64) for x in names]
    pools = list(outs)
    if case["fp8"]:
        pools += [s["k_scale"], s["v_scale"]]
    if mass is not None:
        moved = s["mass"].to(torch.float64)
        pools.append(moved)
    for i in range(B):
        for j in range(h):
            a = torch.tensor(lists[i][j], device=DEV)
            b = torch.arange(first[i], first[i] + len(lists[i][j]), device=DEV)
            for t in pools:
                t[dst[i, b // ps].long(), j, b % ps] = t[s["table"][i, a // ps].long(), j, a % ps]
    outs += [None, None] if case["fp8"] else []
    if case["op"] == "evict":
        return outs + [moved if mass is not None else s["mass"].to(torch.float64), None, None]
    return outs + ([moved] if mass is not None else [])
