"""The paged-cache operators on real sizes: block tables and slot maps built
from request lengths (grow, shrink), new keys and values written to their
slots (append), and the attention of one new token per request over the
cached ones (attend). Each has a plain form in elementary torch operations
and the call a user makes of the library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
          "f8": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "f8": 1}


def listed():
    return [
        # one chat request a few pages long: nothing but latency
        dict(name="attend_one_short", op="attend", dtype="bf16", R=1, idle=0, Hq=32, Hkv=8, D=128,
             page=16, lo=513, hi=513, window=0, sinks=0, heads_first=False),
        # a decoding batch of mixed ages, three of its rows empty
        dict(name="attend_batch", op="attend", dtype="bf16", R=64, idle=3, Hq=32, Hkv=8, D=128,
             page=16, lo=16, hi=4096, window=0, sinks=0, heads_first=False),
        # the largest: a full server, long prompts, eight query heads a key head
        dict(name="attend_large", op="attend", dtype="bf16", R=128, idle=0, Hq=64, Hkv=8, D=128,
             page=64, lo=2048, hi=8192, window=0, sinks=0, heads_first=False),
        # two very long documents: the split over the cache's length is all there is to share out
        dict(name="attend_long", op="attend", dtype="bf16", R=2, idle=0, Hq=48, Hkv=2, D=128,
             page=256, lo=70001, hi=262143, window=0, sinks=0, heads_first=True),
        # a sliding window with its first tokens kept, lengths far past the window
        dict(name="attend_window", op="attend", dtype="f16", R=48, idle=1, Hq=24, Hkv=8, D=64,
             page=32, lo=500, hi=20000, window=1000, sinks=4, heads_first=True),
        # an 8-bit cache read by 16-bit queries, five query heads a key head
        dict(name="attend_8bit", op="attend", dtype="f8", R=96, idle=0, Hq=40, Hkv=8, D=128,
             page=32, lo=256, hi=6000, window=0, sinks=0, heads_first=False),
        # full precision, one query head a key head, odd head size and page
        dict(name="attend_f32", op="attend", dtype="f32", R=17, idle=1, Hq=12, Hkv=12, D=80,
             page=24, lo=1, hi=1500, window=0, sinks=0, heads_first=False),
        # one token of each request of a batch, a few rows of the batch unused
        dict(name="append_step", op="append", dtype="bf16", T=64, pad=5, Hkv=8, D=128, page=16,
             heads_first=False),
        # the prompts of several requests at once
        dict(name="append_prompts", op="append", dtype="f16", T=16387, pad=0, Hkv=8, D=128, page=64,
             heads_first=True),
        # one token more for each request: pages are taken by the few that need one
        dict(name="grow_step", op="grow", R=256, page=16, lo=1, hi=8000, new_lo=1, new_hi=1, pad=0,
             room=True),
        # prompts enter beside decoding requests
        dict(name="grow_prompts", op="grow", R=500, page=16, lo=0, hi=4000, new_lo=1, new_hi=2000,
             pad=100, room=True),
        # a quarter of the requests end and give their pages back
        dict(name="shrink_ended", op="shrink", R=512, page=16, lo=100, hi=8000),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "grow", "shrink"])
    if op == "attend":
        biggest = work(listed()[2])["bytes"]
        while True:
            c = dict(op="attend", dtype=rng.choice(["bf16", "bf16", "f16", "f32", "f8"]),
                     R=_log(rng, 1, 192), idle=0, Hkv=rng.choice([1, 2, 3, 4, 5, 8, 12, 16]),
                     D=rng.choice([64, 64, 80, 96, 112, 128, 128, 128, 192, 256]),
                     page=rng.choice([8, 16, 16, 24, 32, 64, 100, 128, 256]),
                     hi=_log(rng, 16, 200000), window=0, sinks=0,
                     heads_first=rng.random() < 0.5)
            c["lo"] = max(1, int(c["hi"] * rng.choice([1.0, 0.5, 0.1, 0.01])))
            c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8, 12, 16, 24])
            c["idle"] = rng.choice([0, 0, 1]) if c["R"] > 2 else 0
            if rng.random() < 0.3:
                c["window"], c["sinks"] = _log(rng, 16, 8192), rng.choice([0, 1, 4, 17, 64])
            # the plain form pads every request to the longest one
            padded = c["R"] * c["hi"] * c["Hkv"] * c["D"]
            if c["Hq"] <= 128 and padded <= 2 ** 30 and work(c)["bytes"] <= biggest:
                return c
    if op == "append":
        T = _log(rng, 1, 16000)
        return dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), T=T,
                    pad=rng.choice([0, T // 10]), Hkv=rng.choice([1, 2, 3, 4, 5, 8]),
                    D=rng.choice([64, 80, 96, 112, 128, 192, 256]),
                    page=rng.choice([8, 16, 24, 32, 64, 100, 128]),
                    heads_first=rng.random() < 0.5)
    R, page = _log(rng, 1, 4000), rng.choice([8, 16, 24, 32, 64, 100, 128])
    if op == "shrink":
        hi = _log(rng, 16, 8000)
        return dict(op=op, R=R, page=page, lo=rng.randrange(0, hi), hi=hi)
    hi = _log(rng, 16, 8000)
    new_hi = rng.choice([1, 1, _log(rng, 1, max(1, 200000 // R))])
    return dict(op=op, R=R, page=page, lo=rng.randrange(0, hi), hi=hi,
                new_lo=rng.choice([1, new_hi]), new_hi=new_hi, pad=rng.choice([0, 64]),
                room=rng.random() < 0.9)


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, evenly over the logarithm of value + 1."""
    a, b = math.log(lo + 1), math.log(hi + 1)
    if n == 1:
        return [hi]
    return [int(round(math.exp(a + (b - a) * (i + 0.5) / n))) - 1 for i in range(n)]


def _lengths(case):
    """The requests' lengths, before the seed puts them in an order."""
    idle = case.get("idle", 0)
    return [0] * idle + _spread(case["R"] - idle, case["lo"], case["hi"])


def _new(case):
    return _spread(case["R"], case["new_lo"], case["new_hi"])


def _kept(case):
    """What each request keeps: a quarter nothing, a quarter a few tokens less, half all."""
    return [0 if i % 4 == 1 else max(0, n - 3) if i % 4 == 3 else n
            for i, n in enumerate(_lengths(case))]


def _pages(n, page):
    return (n + page - 1) // page


def _width(case):
    longest = max(_lengths(case)) + (max(_new(case)) if case["op"] == "grow" else 0)
    return max(1, _pages(longest, case["page"])) + 1


def _visible(case, n):
    if not case["window"]:
        return n
    return min(n, case["window"]) + min(case["sinks"], max(0, n - case["window"]))


def work(case):
    if case["op"] == "attend":
        seen = sum(_visible(case, n) for n in _lengths(case))
        q = case["R"] * case["Hq"] * case["D"] * (2 if case["dtype"] == "f8" else BYTES[case["dtype"]])
        return {"bytes": 2 * seen * case["Hkv"] * case["D"] * BYTES[case["dtype"]] + 2 * q
                + 4 * _pages(seen, case["page"]) + 4 * case["R"],
                "flops": 4 * seen * case["Hq"] * case["D"]}
    if case["op"] == "append":
        n = (case["T"] - case["pad"]) * case["Hkv"] * case["D"] * BYTES[case["dtype"]]
        return {"bytes": 4 * n + 4 * case["T"], "flops": 0}
    R, page = case["R"], case["page"]
    if case["op"] == "grow":
        held, new = _lengths(case), _new(case)
        tokens = sum(new) + case["pad"]
        took = sum(new) // page
        return {"bytes": 8 * R + 8 * took + 4 * (R + 1) + 4 * R + 8 * tokens,
                "flops": 4 * R + 2 * tokens + len(held)}
    gone = sum(_pages(n, page) - _pages(k, page) for n, k in zip(_lengths(case), _kept(case)))
    return {"bytes": 12 * R + 8 * gone, "flops": 4 * R}


def _order(n, g):
    return torch.randperm(n, generator=g, device="cuda")


def _paged(lengths, width, page, g):
    """A pool in which each request holds the pages of its length, dealt at random: its block
    table, the pages in the order the pool hands them out, and how many are out."""
    need = (lengths + page - 1) // page
    ptr = torch.cumsum(need, 0)
    used = int(ptr[-1])
    pool = _order(used + max(8, used // 4), g).to(torch.int32)
    col = torch.arange(width, device="cuda")
    at = (ptr - need)[:, None] + col
    held = col < need[:, None]
    table = torch.where(held, pool[torch.where(held, at, 0)], -1).to(torch.int32)
    return table, pool, used


def _normal(shape, dtype, g):
    """Standard normal values; those of an 8-bit cache spread over its range."""
    if dtype == torch.float8_e4m3fn:
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
        return x.mul_(16).clamp_(-448, 448).to(dtype)
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _pool(case, n_pages, g):
    """Pages of keys or values, [page, token, head, element]; heads_first: stored with each
    head's tokens together."""
    P, H, D, dt = case["page"], case["Hkv"], case["D"], DTYPES[case["dtype"]]
    if case["heads_first"]:
        return _normal((n_pages, H, P, D), dt, g).transpose(1, 2)
    return _normal((n_pages, P, H, D), dt, g)


def _attend_inputs(case, g):
    R, H, D = case["R"], case["Hkv"], case["D"]
    lengths = torch.tensor(_lengths(case), device="cuda")[_order(R, g)]
    table, pool, _ = _paged(lengths, _width(case), case["page"], g)
    s = {"k": _pool(case, pool.numel(), g), "v": _pool(case, pool.numel(), g), "table": table,
         "lengths": lengths.to(torch.int32), "k_scale": None, "v_scale": None}
    q = torch.bfloat16 if case["dtype"] == "f8" else DTYPES[case["dtype"]]
    s["q"] = _normal((R, case["Hq"], D), q, g)
    if case["dtype"] == "f8":
        s["k_scale"] = 0.05 + 0.05 * torch.rand(H, generator=g, device="cuda")
        s["v_scale"] = 0.05 + 0.05 * torch.rand(H, generator=g, device="cuda")
    return s


def _append_inputs(case, g):
    T, P, H, D, dt = case["T"], case["page"], case["Hkv"], case["D"], DTYPES[case["dtype"]]
    n_pages = _pages(max(T + T // 8, 4096), P)
    slots = _order(n_pages * P, g)[:T].to(torch.int32)
    slots[T - case["pad"]:] = -1
    # one page more than the cache has: where the plain form puts the rows of the padding
    return {"k_all": _pool(case, n_pages + 1, g), "v_all": _pool(case, n_pages + 1, g),
            "k_new": _normal((T, H, D), dt, g), "v_new": _normal((T, H, D), dt, g),
            "slots": slots, "n_pages": n_pages}


def _tables_inputs(case, g):
    R, page = case["R"], case["page"]
    order = _order(R, g)
    lengths = torch.tensor(_lengths(case), device="cuda")[order]
    table, pool, used = _paged(lengths, _width(case), page, g)
    s = {"lengths": lengths.to(torch.int32), "table": table,
         "cursor": torch.tensor([used], dtype=torch.int32, device="cuda"),
         "lengths_out": torch.zeros(R, dtype=torch.int32, device="cuda"),
         "cursor_out": torch.zeros(1, dtype=torch.int32, device="cuda"),
         "status": torch.zeros(2, dtype=torch.int32, device="cuda")}
    if case["op"] == "shrink":
        s["keep"] = torch.tensor(_kept(case), dtype=torch.int32, device="cuda")[order]
        s["free_pages"] = pool
        return s
    new = _new(case)
    extra = _pages(sum(new), page) + R if case["room"] else 0
    more = pool.numel() + _order(extra, g).to(torch.int32)
    s["free_pages"] = torch.cat([pool, more]) if case["room"] else pool[:used].clone()
    s["n_new"] = torch.tensor(new, dtype=torch.int32, device="cuda")[_order(R, g)]
    s["token_ptr"] = torch.zeros(R + 1, dtype=torch.int32, device="cuda")
    tokens = sum(new) + case["pad"]
    s["slots"] = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    s["positions"] = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    inputs = {"attend": _attend_inputs, "append": _append_inputs}.get(case["op"], _tables_inputs)
    s = inputs(case, g)
    s["case"] = case
    if case["op"] == "append":
        s["k"], s["v"] = s["k_all"][:-1], s["v_all"][:-1]
    if case["op"] == "attend":
        s["out"] = torch.empty_like(s["q"])
        s["longest"] = max(1, max(_lengths(case)))
        s["most"] = max(1, max(_visible(case, n) for n in _lengths(case)))
    if own and case["op"] in ("attend", "append"):
        # the handle a serving program makes once for a layer's cache
        import load_balanced_csr_amd as lb
        s["cache"] = lb.KvCache(s["k"], s["v"], s.get("k_scale"), s.get("v_scale"))
    return s


def _attend_plain(s):
    case, q, table, lengths = s["case"], s["q"], s["table"], s["lengths"]
    R, Hq, D = q.shape
    H, P = case["Hkv"], case["page"]
    # the tokens each request sees: its first ones, then those of its window
    n, window = lengths[:, None].long(), case["window"] or s["longest"]
    first = (n - window).clamp(0, case["sinks"])
    seen = first + n.clamp(max=window)
    j = torch.arange(s["most"], device=q.device)
    t = torch.where(j < first, j, n - seen + j).clamp(min=0)
    t = torch.where(j < seen, t, 0)
    pages = torch.gather(table, 1, t // P).clamp(min=0).long()

    def rows(cache, scale):
        raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
        x = raw[pages, t % P].permute(0, 2, 1, 3).contiguous()     # [R, H, most, D]
        x = x.view(cache.dtype).to(torch.float32)
        return x if scale is None else x * scale[None, :, None, None]

    qf = q.float().view(R, H, Hq // H, D)
    score = torch.matmul(qf, rows(s["k"], s["k_scale"]).transpose(2, 3)) * D ** -0.5
    score = torch.where((j < seen)[:, None, None, :], score, -math.inf)
    top = score.amax(dim=3, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(dim=3, keepdim=True)
    out = torch.matmul(p, rows(s["v"], s["v_scale"])) / torch.where(total == 0, 1.0, total)
    return out.view(R, Hq, D).to(q.dtype)


def _append_plain(s):
    P, slots = s["case"]["page"], s["slots"].long()
    page = torch.where(slots < 0, s["n_pages"], slots // P)
    at = torch.where(slots < 0, 0, slots % P)
    s["k_all"][page, at] = s["k_new"]
    s["v_all"][page, at] = s["v_new"]
    return s["k"], s["v"]


def _grow_plain(s):
    page, old, new = s["case"]["page"], s["lengths"].long(), s["n_new"].long()
    table, free = s["table"], s["free_pages"]
    R, width = table.shape
    held = (old + page - 1) // page
    need = (old + new + page - 1) // page - held
    taken, token_end = torch.cumsum(need, 0), torch.cumsum(new, 0)
    short = taken[-1] - (free.numel() - s["cursor"][0])
    code = torch.where(short > 0, 1, 0)
    ok = code == 0
    col = torch.arange(width, device=old.device)
    j = col - held[:, None]
    fresh = (j >= 0) & (j < need[:, None]) & ok
    at = s["cursor"][0] + (taken - need)[:, None] + j
    table.copy_(torch.where(fresh, free[torch.where(fresh, at, 0)], table))
    t = torch.arange(s["slots"].numel(), device=old.device)
    row = torch.searchsorted(token_end, t, right=True).clamp(max=R - 1)
    pos = old[row] + t - (token_end - new)[row]
    real = (t < token_end[-1]) & ok
    slot = table[row, (pos // page).clamp(max=width - 1)].long() * page + pos % page
    zero = torch.zeros(1, dtype=torch.long, device=old.device)
    return (table, torch.where(ok, old + new, old).int(),
            torch.where(ok, s["cursor"] + taken[-1], s["cursor"]).int(),
            torch.cat([zero, token_end]).int(), torch.where(real, slot, -1).int(),
            torch.where(real, pos, -1).int(),
            torch.stack([code, torch.where(ok, 0, short)]).int())


def _shrink_plain(s):
    page, old, keep = s["case"]["page"], s["lengths"].long(), s["keep"].long()
    free, table = s["free_pages"], s["table"]
    n = free.numel()
    col = torch.arange(table.shape[1], device=old.device)
    gone = (col >= ((keep + page - 1) // page)[:, None]) & (col < ((old + page - 1) // page)[:, None])
    rank = torch.cumsum(gone.view(-1).long(), 0)
    start = s["cursor"][0] - rank[-1]
    spare = torch.cat([free, free[:1]])     # one entry more: where those that stay are put
    spare.scatter_(0, torch.where(gone.view(-1), start + rank - 1, n), table.view(-1))
    free.copy_(spare[:n])
    zero = torch.zeros(2, dtype=torch.int32, device=old.device)
    return free, keep.int(), (s["cursor"] - rank[-1]).int(), zero


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"attend": _attend_plain, "append": _append_plain, "grow": _grow_plain,
                "shrink": _shrink_plain}[op](s)
    if op == "attend":
        return s["cache"].attend(s["q"], s["table"], s["lengths"], s["out"],
                                 window=s["case"]["window"], sinks=s["case"]["sinks"])
    if op == "append":
        s["cache"].append(s["k_new"], s["v_new"], s["slots"])
        return s["k"], s["v"]
    import load_balanced_csr_amd as lb
    page = s["case"]["page"]
    if op == "grow":
        lb.spmv_kv_grow(s["lengths"], s["n_new"], page, s["free_pages"], s["cursor"], s["table"],
                        s["lengths_out"], s["cursor_out"], s["token_ptr"], s["slots"],
                        s["positions"], s["status"])
        return (s["table"], s["lengths_out"], s["cursor_out"], s["token_ptr"], s["slots"],
                s["positions"], s["status"])
    lb.spmv_kv_shrink(s["lengths"], s["keep"], page, s["free_pages"], s["cursor"], s["table"],
                      s["lengths_out"], s["cursor_out"], s["status"])
    return s["free_pages"], s["lengths_out"], s["cursor_out"], s["status"]


def exact(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "append":
        s = _append_inputs(case, g)
        got = []
        for cache, new in ((s["k_all"], s["k_new"]), (s["v_all"], s["v_new"])):
            full = cache.double().cpu()
            rows, slots = new.double().cpu(), s["slots"].tolist()
            for i, slot in enumerate(slots):
                if slot >= 0:
                    full[slot // case["page"], slot % case["page"]] = rows[i]
            got.append(full[:-1])
        return tuple(got)
    if case["op"] != "attend":
        return None
    s = _attend_inputs(case, g)
    R, Hq, D = s["q"].shape
    H, P = case["Hkv"], case["page"]
    out = torch.zeros(R, Hq, D, dtype=torch.float64, device="cuda")
    for r, n in enumerate(s["lengths"].tolist()):
        t = torch.arange(n, device="cuda")
        if case["window"] and n > case["window"]:
            t = torch.cat([t[:min(case["sinks"], n - case["window"])], t[n - case["window"]:]])
        if not t.numel():
            continue
        page = s["table"][r].long()[t // P]

        def tokens(cache, scale):
            raw = cache.view(torch.uint8) if case["dtype"] == "f8" else cache
            x = raw[page, t % P].contiguous().view(cache.dtype).double()       # [n, H, D]
            return x if scale is None else x * scale.double()[None, :, None]

        k, v = tokens(s["k"], s["k_scale"]), tokens(s["v"], s["v_scale"])
        for h in range(H):
            rows = slice(h * (Hq // H), (h + 1) * (Hq // H))
            x = s["q"][r, rows].double() @ k[:, h].t().contiguous() / math.sqrt(D)
            w = torch.exp(x - x.max(dim=1, keepdim=True).values)
            out[r, rows] = (w @ v[:, h].contiguous()) / w.sum(dim=1, keepdim=True)
    return out
