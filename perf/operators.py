"""The 4-bit cache's operators as they are called: rows packed to 4 bits and
read back, attention over the rows that the slot ids of a swap-in name, and
the choice of the hot rows with the least accumulated attention weight.

A 4-bit row is 416 bytes: 512 latent values as e2m1 codes (value 2b in the low
half of byte b), 32 e4m3 scales (one per 16 latent values) and 64 rope values
of the model's 16-bit type.
"""

import math

import numpy as np
import torch

own = False

LATENT, ROPE, GROUP = 512, 64, 16
ROW_VALUES = LATENT + ROPE
SCALE_AT, ROPE_AT, ROW_BYTES = 256, 288, 416
RESIDENT_FLAG = 1 << 30
POOL_ROWS = 8192        # distinct rows that an attention case's cache is drawn from
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# -- cases ------------------------------------------------------------------

def _rows4(name, n, dtype="bf16"):
    return {"name": name, "op": "rows4", "n": n, "dtype": dtype}


def _attend(name, R, H, k, D, dtype="bf16", weights=False, pad=0.0, resident=0.0, cap=40000):
    return {"name": name, "op": "attend", "R": R, "H": H, "k": k, "D": D, "dtype": dtype,
            "weights": weights, "pad": pad, "resident": resident, "cap": cap}


def _evict(name, R, D, n, cap, recent):
    return {"name": name, "op": "evict", "R": R, "D": D, "n": n, "cap": cap, "recent": recent}


def listed():
    return [
        # the new rows of one decode step of 32 requests, before their backup
        _rows4("rows4_step", 32),
        # the prefix rows of a few requests, before prefill; an odd count
        _rows4("rows4_prefix", 70001, "f16"),
        # a batch of long prefixes at once
        _rows4("rows4_batch", 32 * 8192),
        # one request, one GPU's share of the heads: latency
        _attend("attend_single", 1, 16, 2048, 6144),
        # the decode setting (32 requests, k 2048, D 6144) with few heads a GPU
        _attend("attend_heads16", 32, 16, 2048, 6144),
        # the same with every head on the GPU
        _attend("attend_heads128", 32, 128, 2048, 6144),
        # the same with each token's weight accumulated for eviction
        _attend("attend_weights", 32, 128, 2048, 6144, weights=True),
        # odd sizes, padded rows, an empty request, resident pages beside the hot rows
        _attend("attend_ragged", 37, 40, 1001, 1500, "f16", True, 0.3, 0.25, 3001),
        # the large batch (256 requests, D 4096), weights accumulated
        _attend("attend_batch", 256, 64, 2048, 4096, "bf16", True, 0.0, 0.0, 32768),
        # the tiny setting: a fifth of 512 hot rows of 4 requests
        _evict("evict_tiny", 4, 512, 102, 8000, 16),
        # a decode step's misses (a fifth of k 2048) freed in 32 requests
        _evict("evict_step", 32, 6144, 410, 40000, 128),
        # the large batch on the largest hot buffer
        _evict("evict_batch", 256, 32768, 6144, 81920, 512),
    ]


def _log(rng, a, b):
    return min(b, max(a, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["rows4", "attend", "attend", "attend", "evict"])
    if op == "rows4":
        c = _rows4("", _log(rng, 1, 32 * 8192), rng.choice(["bf16", "f16"]))
    elif op == "attend":
        k = _log(rng, 1, 4096)
        H = rng.choice([1, 8, 16, 16, 32, 64, 64, 128, 128, rng.randint(2, 127)])
        most = 256 * 64 * 2048 / (k * max(H, 16))
        R = _log(rng, 1, max(1, min(256, int(most))))
        D = k + _log(rng, 1, 4096)
        c = _attend("", R, H, k, D, rng.choice(["bf16", "f16"]), rng.random() < 0.5,
                    rng.choice([0.0, 0.0, round(rng.uniform(0.01, 0.9), 2)]),
                    rng.choice([0.0, 0.0, round(rng.uniform(0.01, 0.9), 2)]),
                    D + _log(rng, 1, 40000))
    else:
        D = _log(rng, 2, 32768)
        c = _evict("", _log(rng, 1, 256), D, _log(rng, 1, max(1, D // 2)),
                   D + _log(rng, 1, 81920 - 32768), _log(rng, 1, 512))
    del c["name"]
    return c


# -- inputs -----------------------------------------------------------------

def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _latents(n, dtype, g):
    """Rows of a normalised latent (unequal channels) and a rope part."""
    x = torch.randn((n, ROW_VALUES), generator=g, device="cuda")
    channel = torch.exp(0.5 * torch.randn((ROW_VALUES,), generator=g, device="cuda"))
    return (x * channel).to(dtype)


def _choose(R, n, of, g):
    """int32 [R][n]: n distinct numbers below `of`, in random order."""
    return torch.rand((R, of), generator=g, device="cuda").argsort(1)[:, :n].to(torch.int32)


def prepare(case, seed):
    g = _rng(seed)
    table = torch.tensor(MAGNITUDES + tuple(-v for v in MAGNITUDES), device="cuda")
    if case["op"] == "rows4":
        n, dtype = case["n"], DTYPES[case["dtype"]]
        return {"op": "rows4", "x": _latents(n, dtype, g), "table": table,
                "rows": torch.empty((n, ROW_BYTES), dtype=torch.uint8, device="cuda"),
                "values": torch.empty((n, ROW_VALUES), dtype=dtype, device="cuda")}
    if case["op"] == "attend":
        R, H, k, D, cap = (case[x] for x in ("R", "H", "k", "D", "cap"))
        dtype = DTYPES[case["dtype"]]
        pool = _pack(_latents(POOL_ROWS, dtype, g))
        pick = torch.randint(0, POOL_ROWS, (R * D,), generator=g, device="cuda")
        ids = _choose(R, k, D, g)
        resident = None
        if case["resident"]:
            flagged = torch.rand((R, k), generator=g, device="cuda") < case["resident"]
            ids = torch.where(flagged, torch.randint(0, POOL_ROWS, (R, k), generator=g, device="cuda",
                                                     dtype=torch.int32) | RESIDENT_FLAG, ids)
            resident = pool.clone()
        positions = _choose(R, k, cap, g)
        if case["pad"]:
            empty = torch.rand((R, k), generator=g, device="cuda") < case["pad"]
            if R > 2:
                empty[R // 2] = True
            ids = torch.where(empty, -1, ids)
            positions = torch.where(empty, -1, positions)
        # scores of a few units between the most and the least attended rows
        q = (2 * torch.randn((R, H, ROW_VALUES), generator=g, device="cuda")).to(dtype)
        s = {"op": "attend", "q": q, "rows": pool[pick].view(R, D, ROW_BYTES), "ids": ids,
             "resident": resident, "scale": ROW_VALUES ** -0.5, "table": table,
             "out": torch.empty((R, H, LATENT), dtype=dtype, device="cuda"),
             "lse": torch.empty((R, H), dtype=torch.float32, device="cuda"),
             "positions": None, "weights": None}
        if case["weights"]:
            s["positions"] = positions
            # what a few earlier steps left
            s["weights"] = 0.1 * torch.rand((R, cap), generator=g, device="cuda")
        return s
    R, D, n, cap, recent = (case[x] for x in ("R", "D", "n", "cap", "recent"))
    slot2tok = _choose(R, D, cap, g)
    slot2tok = torch.where(torch.rand((R, D), generator=g, device="cuda") < 0.02, -1, slot2tok)
    # lengths above D (one request in sixteen is short and keeps all its rows)
    seq = torch.randint(D, cap, (R,), generator=g, device="cuda", dtype=torch.int32) + 1
    seq = torch.where(torch.rand((R,), generator=g, device="cuda") < 1 / 16, D, seq)
    slot2tok = torch.where(slot2tok < seq[:, None], slot2tok, -1)
    # accumulated weight falls off as a power; tokens never attended tie at 0
    w = torch.rand((R, cap), generator=g, device="cuda").pow(6) * 40
    w = torch.where(torch.rand((R, cap), generator=g, device="cuda") < 0.1, 0, w)
    return {"op": "evict", "weights": w, "slot2tok": slot2tok.contiguous(), "seq": seq.to(torch.int32),
            "recent": recent, "n": n,
            "slots": torch.empty((R, n), dtype=torch.int32, device="cuda"),
            "counts": torch.empty((R,), dtype=torch.int32, device="cuda")}


# -- plain forms ------------------------------------------------------------

def _pack(x):
    """uint8 [n][416] of values [n][576]."""
    n = x.shape[0]
    lat = x[:, :LATENT].float().view(n, LATENT // GROUP, GROUP)
    scale8 = (lat.abs().amax(2).double() / 6).clamp(max=448.0).float().to(torch.float8_e4m3fn)
    s = scale8.float().unsqueeze(2)
    m = lat.abs()
    # the nearest code, ties to the even one: the borders lie half way between
    # two magnitudes, and border * scale is exact in 32 bits
    code = ((m > 0.25 * s).to(torch.uint8) + (m >= 0.75 * s) + (m > 1.25 * s) + (m >= 1.75 * s)
            + (m > 2.5 * s) + (m >= 3.5 * s) + (m > 5.0 * s))
    code = torch.where(s > 0, code, 0) | (torch.signbit(lat).to(torch.uint8) << 3)
    code = code.view(n, LATENT)
    return torch.cat([code[:, 0::2] | (code[:, 1::2] << 4), scale8.view(torch.uint8),
                      x[:, LATENT:].contiguous().view(torch.uint8)], 1)


def _unpack(rows, dtype, table):
    """float32 [...][512] and [...][64] of uint8 [...][416]; table: the 16 codes' values."""
    lead = rows.shape[:-1]
    code = torch.stack([rows[..., :SCALE_AT] & 15, rows[..., :SCALE_AT] >> 4], -1)
    scale = rows[..., SCALE_AT:ROPE_AT].contiguous().view(torch.float8_e4m3fn).float()
    lat = table.index_select(0, code.flatten().int()).view(*lead, LATENT // GROUP, GROUP) * scale.unsqueeze(-1)
    return lat.view(*lead, LATENT), rows[..., ROPE_AT:].contiguous().view(dtype).float()


def _plain_attend(s):
    q, rows, ids = s["q"], s["rows"], s["ids"]
    R, H, _ = q.shape
    D = rows.shape[1]
    first = torch.arange(R, device=ids.device, dtype=torch.int64).unsqueeze(1) * D
    hot = first + (ids & (RESIDENT_FLAG - 1)).long().clamp(max=D - 1)
    got = rows.view(-1, ROW_BYTES)[hot]
    if s["resident"] is not None:
        flagged = (ids >= 0) & ((ids & RESIDENT_FLAG) != 0)
        pool = s["resident"]
        row = (ids & (RESIDENT_FLAG - 1)).long().clamp(max=pool.shape[0] - 1)
        got = torch.where(flagged.unsqueeze(2), pool[row], got)
    lat, rope = _unpack(got, q.dtype, s["table"])
    x = q.float()
    score = x[..., :LATENT] @ lat.transpose(1, 2) + x[..., LATENT:] @ rope.transpose(1, 2)
    score = torch.where((ids >= 0).unsqueeze(1), score * s["scale"], -math.inf)
    top = score.amax(2, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0, top))
    total = p.sum(2, keepdim=True)
    p = p / torch.where(total == 0, 1, total)
    s["out"].copy_(p @ lat)
    s["lse"].copy_((top + total.log()).squeeze(2))
    if s["weights"] is not None:
        at = s["positions"].clamp(min=0).long()
        s["weights"].scatter_add_(1, at, torch.where(s["positions"] >= 0, p.sum(1), 0))


def _plain_evict(s):
    tok, n = s["slot2tok"], s["n"]
    D = tok.shape[1]
    seq = s["seq"].unsqueeze(1)
    free = (tok >= 0) & (tok < seq - s["recent"]) & (seq > D)
    w = torch.where(free, s["weights"].gather(1, tok.clamp(min=0).long()), math.inf)
    slot = w.sort(dim=1, stable=True).indices[:, :n]
    count = free.sum(1).clamp(max=n)
    taken = torch.arange(n, device=tok.device) < count.unsqueeze(1)
    slot = torch.where(taken, slot, D).sort(1).values
    s["slots"].copy_(torch.where(taken, slot, -1))
    s["counts"].copy_(count)


# -- one pass ---------------------------------------------------------------

def run(state):
    s = state
    if own:
        from hierarchical_sparse_kv_request_gb300 import hisparse as hs
    if s["op"] == "rows4":
        if own:
            hs.pack_rows(s["x"], s["rows"])
            hs.unpack_rows(s["rows"], s["values"])
        else:
            s["rows"].copy_(_pack(s["x"]))
            s["values"].copy_(torch.cat(_unpack(s["rows"], s["x"].dtype, s["table"]), 1))
        return {"values": s["values"]}
    if s["op"] == "attend":
        if own:
            if "workspace" not in s:        # kept by a decode loop from step to step
                R, H, _ = s["q"].shape
                size = hs.attend_workspace_bytes(R, H, s["ids"].shape[1], s["weights"] is not None)
                s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
            hs.attend(s["q"], s["rows"], s["ids"], s["out"], s["scale"], lse=s["lse"],
                      positions=s["positions"], weights=s["weights"], resident_rows=s["resident"],
                      workspace=s["workspace"])
        else:
            _plain_attend(s)
        got = {"out": s["out"], "lse": s["lse"]}
        if s["weights"] is not None:
            got["weights"] = s["weights"]
        return got
    if own:
        hs.evict_select(s["weights"], s["slot2tok"], s["seq"], s["slots"], s["counts"],
                        keep_recent=s["recent"])
    else:
        _plain_evict(s)
    return {"slots": s["slots"], "counts": s["counts"]}


# -- the work that a pass cannot do without ------------------------------------

def work(case):
    if case["op"] == "rows4":
        # values read, rows written; rows read, values written
        return {"bytes": 2 * case["n"] * (2 * ROW_VALUES + ROW_BYTES), "flops": 0}
    if case["op"] == "attend":
        R, H, k = case["R"], case["H"], case["k"]
        valid = R * k * (1 - case["pad"])
        b = valid * ROW_BYTES + 4 * R * k + R * H * (2 * ROW_VALUES + 2 * LATENT + 4)
        if case["weights"]:
            b += 4 * R * k + 8 * valid
        return {"bytes": b, "flops": 2 * valid * H * (ROW_VALUES + LATENT)}
    R, D, n = case["R"], case["D"], case["n"]
    return {"bytes": R * (8 * D + 4 * n + 8), "flops": 0}


# -- the definitions in 64 bits ---------------------------------------------------

def _exact_values(rows, dtype):
    b = rows.cpu().numpy()
    code = np.empty((b.shape[0], LATENT), dtype=np.int64)
    code[:, 0::2], code[:, 1::2] = b[:, :256] % 16, b[:, :256] // 16
    e8 = b[:, 256:288].astype(np.int64)
    exponent, fraction = e8 // 8, e8 % 8
    scale = np.where(exponent == 0, fraction * 2.0 ** -9, (8 + fraction) * 2.0 ** (exponent - 10.0))
    magnitude = np.array(MAGNITUDES)[code % 8]
    lat = np.where(code >= 8, -magnitude, magnitude) * np.repeat(scale, GROUP, axis=1)
    return lat, rows[:, 288:].contiguous().view(dtype).double().cpu().numpy()


def _exact_rows4(s):
    x = s["x"].double()
    n = x.shape[0]
    lat = x[:, :LATENT].reshape(n, -1, GROUP)
    grid = torch.tensor([(8 + f) * 2.0 ** (e - 10) if e else f * 2.0 ** -9 for e in range(16) for f in range(8)][:127],
                        dtype=torch.float64, device=x.device)
    levels = torch.tensor(MAGNITUDES, dtype=torch.float64, device=x.device)

    def nearest(v, table):
        """Index of the entry nearest to v; of two, the even index."""
        hi = torch.searchsorted(table, v).clamp(1, table.numel() - 1)
        lo = hi - 1
        a, b = v - table[lo], table[hi] - v
        return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)

    s8 = grid[nearest(lat.abs().amax(2) / 6, grid)].unsqueeze(2)
    m = levels[nearest(lat.abs() / torch.where(s8 > 0, s8, 1), levels)] * s8
    return torch.cat([(torch.sign(lat) * m).reshape(n, LATENT), x[:, LATENT:]], 1)


def _exact_attend(case, s):
    R, H, k, D = case["R"], case["H"], case["k"], case["D"]
    dtype = s["q"].dtype
    out = torch.zeros((R, H, LATENT), dtype=torch.float64, device="cuda")
    lse = torch.full((R, H), -math.inf, dtype=torch.float64, device="cuda")
    weights = None if s["weights"] is None else s["weights"].double()
    ids = s["ids"].cpu().numpy().astype(np.int64)
    for r in range(R):
        use = np.nonzero(ids[r] >= 0)[0]
        if not use.size:
            continue
        hot = torch.from_numpy(ids[r, use] % RESIDENT_FLAG).cuda()
        rows = s["rows"][r][hot.clamp(max=D - 1)]
        if s["resident"] is not None:
            res = torch.from_numpy(ids[r, use] >= RESIDENT_FLAG).cuda()
            rows[res] = s["resident"][hot[res]]
        lat, rope = (torch.from_numpy(v).cuda() for v in _exact_values(rows, dtype))
        q = s["q"][r].double()
        e = (q[:, :LATENT] @ lat.T + q[:, LATENT:] @ rope.T) * s["scale"]
        lse[r] = torch.logsumexp(e, 1)
        p = torch.exp(e - lse[r].unsqueeze(1))
        out[r] = p @ lat
        if weights is not None:
            weights[r, s["positions"][r][torch.from_numpy(use).cuda()].long()] += p.sum(0)
    got = {"out": out, "lse": lse}
    if weights is not None:
        got["weights"] = weights
    return got


def _exact_evict(case, s):
    R, n, D = case["R"], case["n"], case["D"]
    tok, seq, w = (s[x].cpu().numpy() for x in ("slot2tok", "seq", "weights"))
    slots = np.full((R, n), -1, dtype=np.int32)
    counts = np.zeros(R, dtype=np.int32)
    for r in range(R):
        if seq[r] <= D:
            continue
        at = np.nonzero((tok[r] >= 0) & (tok[r] < seq[r] - s["recent"]))[0]
        at = np.sort(at[np.lexsort((at, w[r, tok[r, at]]))][:n])
        slots[r, :at.size], counts[r] = at, at.size
    return {"slots": slots, "counts": counts}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rows4":
        return {"values": _exact_rows4(s)}
    return _exact_attend(case, s) if case["op"] == "attend" else _exact_evict(case, s)
