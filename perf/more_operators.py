"""The resident pages' operators as they are called: block tables and slot maps
from request lengths, KV rows normalised and stored at those slots (and read
back), and the attention of a whole batch over a prefix that it shares.

Rows have one of three formats, 512 latent values and 64 rope values each:
  416 bytes   e2m1 codes (value 2b in the low half of byte b), 32 e4m3 scales
              (one per 16 values), rope values in 16 bits
  656 bytes   e4m3 codes, 4 float scales (one per 128 values), rope values in
              16 bits
  1152 bytes  everything in 16 bits
"""

import math

import numpy as np
import torch

own = False

LATENT, ROPE = 512, 64
ROW_VALUES = LATENT + ROPE
ROW4, ROW8, ROW16 = 416, 656, 1152
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
CAPACITY_BIT = 1 << 7
EPS = 1e-6


# -- cases ------------------------------------------------------------------

def _tables(name, R, mode, bs, lo, hi, draft=1, shared=0, idle=0.0, pool=1.0):
    return {"name": name, "op": "tables", "R": R, "mode": mode, "bs": bs, "lo": lo, "hi": hi, "draft": draft,
            "shared": shared, "idle": idle, "pool": pool}


def _rows(name, n, row, dtype="bf16", skip=0.0, norm=True):
    return {"name": name, "op": "rows", "n": n, "row": row, "dtype": dtype, "skip": skip, "norm": norm}


def _prefix(name, R, H, n, row, bs=64, dtype="bf16", part=True, holes=0.0):
    return {"name": name, "op": "prefix", "R": R, "H": H, "n": n, "row": row, "bs": bs, "dtype": dtype,
            "part": part, "holes": holes}


def listed():
    return [
        # 32 requests (the decode setting's batch), up to 4 drafted tokens each,
        # all taken back after verification
        _tables("tables_verify", 32, "verify", 64, 2048, 40000, draft=4),
        # a busy batch: some admitted, some grown, some finished, some idle,
        # behind a shared prefix, and too few free pages for all
        _tables("tables_mixed", 256, "mixed", 16, 2048, 32768, draft=3, shared=97, idle=0.1, pool=0.9),
        # 128 requests of mixed lengths admitted at once, and finished
        _tables("tables_admit", 128, "admit", 64, 2048, 81920),
        # the new rows of one decode step of 32 requests
        _rows("rows_step", 32, ROW8),
        # a few requests' prompts, an odd count, some padding behind them; 4-bit rows
        _rows("rows_prompts", 70001, ROW4, "f16", skip=0.05),
        # a batch of long prompts
        _rows("rows_batch", 32 * 8192, ROW8),
        # four requests with one GPU's share of the heads, a short system prompt: latency
        _prefix("prefix_small", 4, 16, 2048, ROW4),
        # odd sizes, small odd pages, pages that are not there, nothing to join
        _prefix("prefix_ragged", 37, 40, 5003, ROW8, bs=17, dtype="f16", part=False, holes=0.1),
        # the decode setting with few heads a GPU
        _prefix("prefix_heads16", 32, 16, 8192, ROW4),
        # the same with every head, 8-bit rows
        _prefix("prefix_heads128", 32, 128, 8192, ROW8),
        # the large batch over a long shared document, 16-bit rows
        _prefix("prefix_long", 256, 16, 40000, ROW16),
    ]


def _log(rng, a, b):
    return min(b, max(a, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["tables", "rows", "prefix", "prefix", "prefix"])
    if op == "tables":
        R = _log(rng, 1, 1024)
        mode = rng.choice(["verify", "mixed", "admit"])
        hi = _log(rng, 2, min(81920, 128 * 81920 // R))
        bs = rng.choice([1, 16, 32, 64, 64, 128, rng.randint(2, 100)])
        if hi * R // bs > 1 << 21:
            bs = 64
        c = _tables("", R, mode, bs, max(1, hi // rng.choice([1, 4, 40])), hi, rng.randint(1, 8),
                    rng.choice([0, 0, _log(rng, 1, max(1, hi // bs))]), rng.choice([0.0, 0.0, 0.2]),
                    rng.choice([1.0, 1.0, 0.8]))
    elif op == "rows":
        c = _rows("", _log(rng, 1, 32 * 8192), rng.choice([ROW4, ROW8, ROW8, ROW16]), rng.choice(["bf16", "f16"]),
                  rng.choice([0.0, 0.0, 0.3]), rng.random() < 0.8)
    else:
        H = rng.choice([1, 8, 16, 16, 32, 64, 128, rng.randint(2, 127)])
        R = _log(rng, 1, max(1, min(256, 4096 // H)))
        n = _log(rng, 1, 40000)
        c = _prefix("", R, H, n, rng.choice([ROW4, ROW8, ROW16]), rng.choice([1, 16, 64, 64, rng.randint(2, 200)]),
                    rng.choice(["bf16", "f16"]), rng.random() < 0.7, rng.choice([0.0, 0.0, 0.2]))
    del c["name"]
    return c


# -- inputs -----------------------------------------------------------------

def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _latents(n, dtype, g):
    """Rows of a latent with unequal channels, and a rope part."""
    x = torch.randn((n, ROW_VALUES), generator=g, device="cuda")
    channel = torch.exp(0.5 * torch.randn((ROW_VALUES,), generator=g, device="cuda"))
    return (x * channel).to(dtype)


def _lengths(case):
    """R lengths spread over [lo, hi] evenly by their logarithm."""
    u = (np.arange(case["R"]) + 0.5) / case["R"]
    return np.clip(np.round(case["lo"] * (case["hi"] / case["lo"]) ** u), case["lo"], case["hi"]).astype(np.int64)


def _buffers(case):
    """What a server sizes once: tokens of a step, and pages for all requests at
    their longest."""
    R, bs, draft = case["R"], case["bs"], case["draft"]
    n = _lengths(case)
    longest = {"verify": 0, "mixed": R * 15 // 100, "admit": R}[case["mode"]]
    tokens = int(n[R - longest:].sum()) + (0 if case["mode"] == "admit" else R * draft)
    return (tokens + 63) // 64 * 64, int((-(-(n + draft) // bs)).sum()) + 16


def _prepare_tables(case, g):
    R, bs, mode = case["R"], case["bs"], case["mode"]
    order = lambda n: torch.rand((n,), generator=g, device="cuda").argsort()  # noqa: E731
    lens0 = torch.from_numpy(_lengths(case)).cuda()[order(R)]
    extra = torch.randint(1, case["draft"] + 1, (R,), generator=g, device="cuda")
    width = (case["hi"] + case["draft"] + bs - 1) // bs
    shared = min(case["shared"], width)
    if mode == "verify":
        lens1, new = lens0 + extra, extra
    elif mode == "admit":
        lens1, lens0 = lens0, torch.zeros_like(lens0)
        new = (lens1 - shared * bs).clamp(min=0)
    else:
        rank = order(R)
        admitted = rank < R * 15 // 100
        finished = (rank >= R * 15 // 100) & (rank < R * 30 // 100)
        lens1 = torch.where(finished, 0, torch.where(admitted, lens0, lens0 + extra))
        new = torch.where(finished, 0, torch.where(admitted, (lens0 - shared * bs).clamp(min=0), extra))
        lens0 = torch.where(admitted, 0, lens0)
    idle = torch.rand((R,), generator=g, device="cuda") < case["idle"]
    lens1, new = torch.where(idle, -1, lens1), torch.where(idle, 0, new)
    tokens, pages = _buffers(case)
    held = (lens0 + bs - 1) // bs
    used = int((held - shared).clamp(min=0).sum())
    after = torch.where(idle, held, (lens1 + bs - 1) // bs)
    more = (after - shared).clamp(min=0) - (held - shared).clamp(min=0)
    grown, released = int(more.clamp(min=0).sum()), int((-more).clamp(min=0).sum())
    # free pages for all that grows, or, with those released, for a part of it
    free = pages - used if case["pool"] >= 1 else max(0, int(grown * case["pool"]) - released)
    ids = order(shared + pages).to(torch.int32)
    col = torch.arange(width, device="cuda")
    has = (col >= shared) & (col < held[:, None])
    at = (has.flatten().long().cumsum(0) - 1).clamp(min=0).view(R, width)
    tables = torch.where(has, ids[shared + at], -1)
    if shared:
        tables = torch.where((col < shared) & (col < held[:, None]), ids[col.clamp(max=shared - 1)], tables)
    free_list = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free_list[:free] = ids[shared + used:shared + used + free]
    ints = lambda n: torch.empty((n,), dtype=torch.int32, device="cuda")  # noqa: E731
    return {"op": "tables", "bs": bs, "lens0": lens0.to(torch.int32), "lens1": lens1.to(torch.int32),
            "new": new.to(torch.int32), "tables": tables.to(torch.int32).contiguous(),
            "held": held.to(torch.int32), "free_list": free_list,
            "free_count": torch.tensor([free], dtype=torch.int32, device="cuda"),
            "shared": ids[:shared].clone() if shared else None, "offsets": ints(R + 1), "slots": ints(tokens),
            "positions": ints(tokens), "status": torch.zeros((R,), dtype=torch.int32, device="cuda")}


def _prepare_rows(case, g):
    n, dtype = case["n"], DTYPES[case["dtype"]]
    count = n + n // 4 + 1
    slots = torch.rand((count,), generator=g, device="cuda").argsort()[:n].to(torch.int32)
    slots = torch.where(torch.rand((n,), generator=g, device="cuda") < case["skip"], -1, slots)
    weight = (1 + 0.2 * torch.randn((LATENT,), generator=g, device="cuda")).to(dtype) if case["norm"] else None
    # (before the norm the latent's size differs from row to row)
    size = torch.exp(0.5 * torch.randn((n, 1), generator=g, device="cuda"))
    x = (_latents(n, torch.float32, g) * size).to(dtype)
    return {"op": "rows", "x": x, "weight": weight, "slots": slots,
            "rows": torch.zeros((count, case["row"]), dtype=torch.uint8, device="cuda"),
            "values": torch.zeros((n, ROW_VALUES), dtype=dtype, device="cuda")}


def _prepare_prefix(case, g):
    R, H, n, bs, dtype = case["R"], case["H"], case["n"], case["bs"], DTYPES[case["dtype"]]
    used = (n + bs - 1) // bs
    blocks = used + used // 8 + 1
    x = _latents(blocks * bs, dtype, g)
    table = torch.rand((blocks,), generator=g, device="cuda").argsort()[:used].to(torch.int32)
    if case["holes"]:
        table = torch.where(torch.rand((used,), generator=g, device="cuda") < case["holes"], -1, table)
    # scores of a few units between the most and the least attended rows
    q = (2 * torch.randn((R, H, ROW_VALUES), generator=g, device="cuda")).to(dtype)
    s = {"op": "prefix", "q": q, "rows": _encode(x[:, :LATENT].float(), x[:, LATENT:], case["row"], dtype),
         "table": table, "bs": bs, "n": n, "scale": ROW_VALUES ** -0.5, "part": None, "part_lse": None,
         "out": torch.empty((R, H, LATENT), dtype=dtype, device="cuda"),
         "lse": torch.empty((R, H), dtype=torch.float32, device="cuda")}
    if case["part"]:
        # what each request's own top-k rows gave; one request had none
        part = 0.1 * torch.randn((R, H, LATENT), generator=g, device="cuda")
        lse = 3.3 + math.log(2048) + torch.randn((R, H), generator=g, device="cuda")
        if R > 2:
            part[R // 2], lse[R // 2] = 0, -math.inf
        s["part"], s["part_lse"] = part.to(dtype), lse
    return s


def prepare(case, seed):
    g = _rng(seed)
    return {"tables": _prepare_tables, "rows": _prepare_rows, "prefix": _prepare_prefix}[case["op"]](case, g)


# -- plain forms ------------------------------------------------------------

def _plain_tables(s, lens, new):
    """One call: release what lengths no longer cover, then grow in the order of
    the requests as far as the free list goes, then place the new tokens."""
    tables, held, free_list, bs = s["tables"], s["held"].long(), s["free_list"], s["bs"]
    R, width = tables.shape
    shared = 0 if s["shared"] is None else s["shared"].numel()
    col = torch.arange(width, device=tables.device)
    need = torch.where(lens < 0, held, (lens.long() + bs - 1) // bs)
    mine = lambda n: (n - shared).clamp(min=0)  # noqa: E731
    # released pages: the next to be taken, in order
    going = (col < held[:, None]) & (col >= need[:, None])
    freed = going & (col >= shared)
    rank = freed.flatten().long().cumsum(0).view(R, width) - 1
    count = s["free_count"].long() + freed.sum()
    place = torch.where(freed, count - 1 - rank, free_list.numel())
    padded = torch.cat([free_list, free_list[:1]])
    padded.scatter_(0, place.flatten(), tables.flatten())
    free_list.copy_(padded[:-1])
    # growth, if it and all before it fit
    grow = (mine(need) - mine(held)).clamp(min=0)
    ok = (grow.cumsum(0) <= count) | (grow == 0)
    taking = ok[:, None] & (col >= held[:, None]) & (col < need[:, None])
    taken = taking & (col >= shared)
    rank = taken.flatten().long().cumsum(0).view(R, width) - 1
    got = free_list[(count - 1 - rank).clamp(min=0, max=free_list.numel() - 1)]
    if shared:
        got = torch.where(col < shared, s["shared"][col.clamp(max=shared - 1)], got)
    tables.copy_(torch.where(taking, got, torch.where(going, -1, tables)))
    s["held"].copy_(torch.where(ok, need, held))
    s["free_count"].copy_(count - taken.sum())
    s["status"].bitwise_or_(torch.where(ok, 0, CAPACITY_BIT).to(torch.int32))
    if new is None:
        return
    first = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0).to(torch.int32)])
    i = torch.arange(s["slots"].numel(), device=new.device, dtype=torch.int32)
    r = torch.searchsorted(first[1:], i, right=True).clamp(max=R - 1)
    pos = lens[r] - new[r] + (i - first[r])
    page = tables[r, (pos.clamp(min=0) // bs).long().clamp(max=width - 1)]
    there = (i < first[R]) & ok[r] & (lens[r] >= 0) & (page >= 0)
    s["offsets"].copy_(first)
    s["slots"].copy_(torch.where(there, page * bs + pos % bs, -1))
    s["positions"].copy_(torch.where(there, pos, -1))


def _encode(latent, rope, row, dtype):
    """uint8 [n][row] of float latents and 16-bit rope values."""
    n = latent.shape[0]
    rope = rope.contiguous().view(torch.uint8)
    if row == ROW16:
        return torch.cat([latent.to(dtype).view(torch.uint8), rope], 1)
    if row == ROW8:
        x = latent.view(n, 4, 128)
        top = x.abs().amax(2)
        # the least power of two that brings the largest magnitude to 448 or less
        m, e = torch.frexp(top / 448)
        scale = torch.ldexp(torch.ones_like(m), (e - (m == 0.5).int()).clamp(min=-126))
        scale = torch.where(top == 0, 2.0 ** -126, scale)
        codes = (x.double() / scale.unsqueeze(2).double()).float().to(torch.float8_e4m3fn)
        return torch.cat([codes.view(n, LATENT).view(torch.uint8), scale.view(torch.uint8), rope], 1)
    x = latent.view(n, LATENT // 16, 16)
    scale8 = (x.abs().amax(2) / 6).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale8.float().unsqueeze(2)
    m = x.abs()
    # the nearest code, ties to the even one: borders lie half way between two
    # magnitudes
    code = ((m > 0.25 * s).to(torch.uint8) + (m >= 0.75 * s) + (m > 1.25 * s) + (m >= 1.75 * s)
            + (m > 2.5 * s) + (m >= 3.5 * s) + (m > 5.0 * s))
    code = (torch.where(s > 0, code, 0) | (torch.signbit(x).to(torch.uint8) << 3)).view(n, LATENT)
    return torch.cat([code[:, 0::2] | (code[:, 1::2] << 4), scale8.view(torch.uint8), rope], 1)


def _decode(rows, dtype):
    """float [n][512] and [n][64] of uint8 rows."""
    n, row = rows.shape
    rope = rows[:, row - 2 * ROPE:].contiguous().view(dtype).float()
    if row == ROW16:
        return rows[:, :2 * LATENT].contiguous().view(dtype).float(), rope
    if row == ROW8:
        scale = rows[:, LATENT:LATENT + 16].contiguous().view(torch.float32)
        codes = rows[:, :LATENT].contiguous().view(torch.float8_e4m3fn).float()
        return (codes.view(n, 4, 128) * scale.unsqueeze(2)).view(n, LATENT), rope
    table = torch.tensor(MAGNITUDES + tuple(-v for v in MAGNITUDES), device=rows.device)
    code = torch.stack([rows[:, :256] & 15, rows[:, :256] >> 4], -1)
    scale = rows[:, 256:288].contiguous().view(torch.float8_e4m3fn).float()
    return (table[code.int()].view(n, 32, 16) * scale.unsqueeze(2)).view(n, LATENT), rope


def _plain_rows(s):
    x, slots, dtype = s["x"], s["slots"].long(), s["x"].dtype
    y = x[:, :LATENT].float()
    if s["weight"] is not None:
        y = y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    there = (slots >= 0).unsqueeze(1)
    # (rows without a slot go behind the last)
    count = s["rows"].shape[0]
    padded = torch.cat([s["rows"], s["rows"][:1]])
    at = torch.where(slots >= 0, slots, count)
    padded[at] = _encode(y, x[:, LATENT:], s["rows"].shape[1], dtype)
    s["rows"].copy_(padded[:count])
    got = torch.cat(_decode(s["rows"][slots.clamp(min=0)], dtype), 1).to(dtype)
    s["values"].copy_(torch.where(there, got, s["values"]))


def _prefix_rows(s):
    """The prefix's rows that are there, and which (bool [n])."""
    t = torch.arange(s["n"], device=s["table"].device)
    page = s["table"][t // s["bs"]].long()
    return s["rows"][(page.clamp(min=0) * s["bs"] + t % s["bs"])], page >= 0


def _plain_prefix(s):
    q = s["q"]
    R, H, _ = q.shape
    rows, there = _prefix_rows(s)
    latent, rope = _decode(rows, q.dtype)
    x = q.float().view(R * H, ROW_VALUES)
    score = (x[:, :LATENT] @ latent.T + x[:, LATENT:] @ rope.T) * s["scale"]
    score = torch.where(there, score, -math.inf)
    top = score.amax(1, keepdim=True)
    if s["part"] is not None:
        other = s["part_lse"].view(-1, 1)
        top = torch.maximum(top, other)
    base = torch.where(top == -math.inf, 0, top)
    p = torch.exp(score - base)
    total, o = p.sum(1, keepdim=True), p @ latent
    if s["part"] is not None:
        w = torch.exp(other - base)
        total, o = total + w, o + w * s["part"].float().view(R * H, LATENT)
    s["out"].copy_((o / torch.where(total == 0, 1, total)).view(R, H, LATENT))
    s["lse"].copy_((top + total.log()).view(R, H))


# -- one pass ---------------------------------------------------------------

def run(state):
    s = state
    if own:
        from hierarchical_sparse_kv_request_gb300 import hisparse as hs
    if s["op"] == "tables":
        # a step's tokens placed, then the lengths taken back to what they were
        if own:
            hs.page_tables(s["lens1"], s["tables"], s["held"], s["free_list"], s["free_count"], s["bs"],
                           shared=s["shared"], new_tokens=s["new"], offsets=s["offsets"], slots=s["slots"],
                           positions=s["positions"], status=s["status"])
            hs.page_tables(s["lens0"], s["tables"], s["held"], s["free_list"], s["free_count"], s["bs"],
                           shared=s["shared"], status=s["status"])
        else:
            _plain_tables(s, s["lens1"], s["new"])
            _plain_tables(s, s["lens0"], None)
        return {k: s[k] for k in ("offsets", "slots", "positions", "tables", "held", "free_list", "free_count",
                                  "status")}
    if s["op"] == "rows":
        if own:
            hs.norm_rows(s["x"], s["rows"], slots=s["slots"], weight=s["weight"], eps=EPS)
            hs.gather_rows(s["rows"], s["values"], slots=s["slots"])
        else:
            _plain_rows(s)
        return {"values": s["values"]}
    if own:
        if "workspace" not in s:        # kept by a decode loop from step to step
            R, H, _ = s["q"].shape
            size = hs.attend_prefix_workspace_bytes(R, H, s["n"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        hs.attend_prefix(s["q"], s["rows"], s["table"], s["bs"], s["n"], s["out"], s["scale"], lse=s["lse"],
                         part=s["part"], part_lse=s["part_lse"], workspace=s["workspace"])
    else:
        _plain_prefix(s)
    return {"out": s["out"], "lse": s["lse"]}


# -- the work that a pass cannot do without ------------------------------------

def _mean_length(case):
    lo, hi = case["lo"], case["hi"]
    return (hi - lo) / math.log(hi / lo) if hi > lo else float(hi)


def work(case):
    if case["op"] == "tables":
        R, bs, n = case["R"], case["bs"], _mean_length(case)
        moved = {"verify": 0.0, "admit": n, "mixed": 0.3 * n}[case["mode"]]
        tokens = {"verify": (1 + case["draft"]) / 2, "admit": n, "mixed": 0.15 * n + 2}[case["mode"]]
        # lengths, counts, tokens and status in and out; an id from the list to
        # the table and back; a slot and a position a token
        return {"bytes": R * (40 + 16 * (moved / bs + 1) + 8 * tokens), "flops": 0}
    if case["op"] == "rows":
        n = case["n"]
        there = n * (1 - case["skip"])
        return {"bytes": 2 * n * 4 + 2 * there * (2 * ROW_VALUES + case["row"]), "flops": 0}
    R, H = case["R"], case["H"]
    n = case["n"] * (1 - case["holes"])
    b = n * case["row"] + 4 * n / case["bs"] + R * H * (2 * ROW_VALUES + 2 * LATENT + 4)
    if case["part"]:
        b += R * H * (2 * LATENT + 4)
    return {"bytes": b, "flops": 2 * n * R * H * (ROW_VALUES + LATENT)}


# -- the definitions in 64 bits ---------------------------------------------------

def _exact_tables(s):
    """The same, request by request, with a list."""
    bs = s["bs"]
    shared = [] if s["shared"] is None else s["shared"].tolist()
    tables, held = s["tables"].cpu().numpy().copy(), s["held"].tolist()
    listed_ = s["free_list"].cpu().numpy().copy()
    free = listed_[:int(s["free_count"])].tolist()
    R, status = len(held), np.zeros(len(held), dtype=np.int32)
    offsets = slots = positions = None
    for lens, new in ((s["lens1"].tolist(), s["new"].tolist()), (s["lens0"].tolist(), None)):
        need = [held[r] if lens[r] < 0 else -(-lens[r] // bs) for r in range(R)]
        back = []
        for r in range(R):
            if need[r] < held[r]:
                back += tables[r, max(need[r], len(shared)):held[r]].tolist()
                tables[r, need[r]:held[r]] = -1
                held[r] = need[r]
        free += back[::-1]
        listed_[len(free) - len(back):len(free)] = free[len(free) - len(back):]
        want, ok = 0, [True] * R
        room = len(free)
        for r in range(R):
            more = max(need[r] - max(held[r], len(shared)), 0)
            want += more
            if more and want > room:
                ok[r], status[r] = False, CAPACITY_BIT
                continue
            for b in range(held[r], need[r]):
                tables[r, b] = shared[b] if b < len(shared) else free.pop()
            held[r] = need[r]
        if new is not None:
            offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
            slots = np.full(s["slots"].numel(), -1, dtype=np.int32)
            positions = slots.copy()
            for r in range(R):
                if lens[r] >= 0 and ok[r] and new[r]:
                    p = np.arange(lens[r] - new[r], lens[r])
                    at = slice(offsets[r], offsets[r + 1])
                    slots[at], positions[at] = tables[r, p // bs] * bs + p % bs, p
    return {"offsets": offsets, "slots": slots, "positions": positions, "tables": tables,
            "held": np.array(held, dtype=np.int32), "free_list": listed_,
            "free_count": np.array([len(free)], dtype=np.int32), "status": status}


def _nearest(v, table):
    """Index of the entry nearest to v; of two, the even index."""
    hi = torch.searchsorted(table, v).clamp(1, table.numel() - 1)
    lo = hi - 1
    a, b = v - table[lo], table[hi] - v
    return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def _e4m3(device):
    return torch.tensor([(8 + f) * 2.0 ** (e - 10) if e else f * 2.0 ** -9 for e in range(16) for f in range(8)][:127],
                        dtype=torch.float64, device=device)


def _exact_rows(case, s):
    x = s["x"].double()
    n, y = x.shape[0], x[:, :LATENT]
    if s["weight"] is not None:
        y = y / torch.sqrt((y * y).sum(1, keepdim=True) / LATENT + EPS) * s["weight"].double()
    if case["row"] != ROW16:
        g = y.reshape(n, -1, 128 if case["row"] == ROW8 else 16)
        top = g.abs().amax(2, keepdim=True)
        if case["row"] == ROW8:
            levels = _e4m3(x.device)
            scale = torch.exp2(torch.ceil(torch.log2(top / 448).clamp(min=-126)))
            scale = torch.where(top > 448 * scale, 2 * scale, torch.where(top <= 224 * scale, scale / 2, scale))
        else:
            levels = torch.tensor(MAGNITUDES, dtype=torch.float64, device=x.device)
            grid = _e4m3(x.device)
            scale = grid[_nearest((top / 6).clamp(max=448.0), grid)]
        m = (g.abs() / torch.where(scale > 0, scale, 1)).clamp(max=levels[-1])
        y = torch.where(scale > 0, torch.sign(g) * levels[_nearest(m, levels)] * scale, 0).reshape(n, LATENT)
    got = torch.cat([y, x[:, LATENT:]], 1)
    return {"values": torch.where((s["slots"] >= 0).unsqueeze(1), got, 0)}


def _exact_values(rows, dtype):
    """float64 [n][512], [n][64] of uint8 rows."""
    n, row = rows.shape
    rope = rows[:, row - 2 * ROPE:].contiguous().view(dtype).double()
    if row == ROW16:
        return rows[:, :2 * LATENT].contiguous().view(dtype).double(), rope
    grid = _e4m3(rows.device)
    byte = lambda b: torch.where(b >= 128, -1.0, 1.0) * grid[b & 127]  # noqa: E731
    if row == ROW8:
        scale = rows[:, LATENT:LATENT + 16].contiguous().view(torch.float32).double()
        return byte(rows[:, :LATENT].long()) * scale.repeat_interleave(128, 1), rope
    codes = torch.empty((n, LATENT), dtype=torch.int64, device=rows.device)
    codes[:, 0::2], codes[:, 1::2] = rows[:, :256] % 16, rows[:, :256] // 16
    levels = torch.tensor(MAGNITUDES, dtype=torch.float64, device=rows.device)
    value = torch.where(codes >= 8, -1.0, 1.0) * levels[codes % 8]
    return value * byte(rows[:, 256:288].long()).repeat_interleave(16, 1), rope


def _exact_prefix(case, s):
    R, H, bs, dtype = case["R"], case["H"], case["bs"], s["q"].dtype
    at = [(p, b) for b, p in enumerate(s["table"].tolist()) if p >= 0]
    rows = [s["rows"][p * bs:p * bs + min(bs, case["n"] - b * bs)] for p, b in at]
    q = s["q"].double().view(R * H, ROW_VALUES)
    out = torch.zeros((R * H, LATENT), dtype=torch.float64, device=q.device)
    lse = torch.full((R * H,), -math.inf, dtype=torch.float64, device=q.device)
    if rows:
        latent, rope = _exact_values(torch.cat(rows), dtype)
        k = torch.cat([latent, rope], 1)
        for a in range(0, R * H, 1024):         # (the scores of 1,024 heads at a time)
            e = q[a:a + 1024] @ k.T * s["scale"]
            lse[a:a + 1024] = torch.logsumexp(e, 1)
            out[a:a + 1024] = torch.exp(e - lse[a:a + 1024, None]) @ latent
    out, lse = out.view(R, H, LATENT), lse.view(R, H)
    if s["part"] is not None:
        other = s["part_lse"].double()
        both = torch.logaddexp(lse, other)
        some = both > -math.inf
        share = lambda a: torch.where(some, torch.exp(a - torch.where(some, both, 0)), 0).unsqueeze(2)  # noqa: E731
        out, lse = share(lse) * out + share(other) * s["part"].double(), both
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return _exact_tables(s)
    return _exact_rows(case, s) if case["op"] == "rows" else _exact_prefix(case, s)
