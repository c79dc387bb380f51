"""Cases of the 4-bit paged cache: page tables and slot maps, rows to pages and back, decode attention.

A unit is one KV head of one sequence. Its rows live in pages of 32 rows; page `table[n][j]` holds rows 32 j .. 32 j + 31
of unit n. For every 32 channels of a row a page keeps one half-precision scale, the smallest one that is at least
max|x| / 7, and the codes c + 8 with c = x / scale rounded to the nearest whole number (ties to even). With nb = d / 32
the bytes of a page are, one after the other:

  K codes   [nb][32 rows][16]         two channels a byte, the even one in the low four bits
  V codes   [nb][16 row pairs][8 channel quads][2 rows][2]   the same two bytes of a quad for each of the two rows
  K scales  [32 rows][nb] half
  V scales  [nb][32 rows] half
  log-counts [32] float
"""
import math

import torch

own = False   # True: run() calls the framework's operators; False: the plain forms below

PAGE = 32
QMAX = 7.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step over the 2048-row budget of the chunked prefill, with the new token's row appended
        dict(name="decode budget 2048", kind="decode", B=1, H=8, G=4, d=128, lo=2048, hi=2048, append=True, dtype="bf16"),
        # one decode step of one layer after 32K tokens merged to half
        dict(name="decode 32K merged 2x", kind="decode", B=1, H=8, G=4, d=128, lo=16384, hi=16384, append=False, dtype="bf16"),
        # one decode step of one layer after 128K tokens merged to a quarter
        dict(name="decode 128K merged 4x", kind="decode", B=1, H=8, G=4, d=128, lo=32768, hi=32768, append=True, dtype="bf16"),
        # a batch of eight whose heads share one budget per sequence, so that each head has a length of its own
        dict(name="decode batch 8 pooled", kind="decode", B=8, H=8, G=4, d=128, lo=11003, hi=21765, append=False, dtype="bf16"),
        # sixteen sequences of 8K to 64K tokens merged to an eighth
        dict(name="decode serving mix", kind="decode", B=16, H=8, G=4, d=128, lo=1024, hi=8192, append=True, dtype="bf16"),
        # the small fp32 shape that is checked on the CPU
        dict(name="decode tiny fp32", kind="decode", B=1, H=2, G=2, d=64, lo=256, hi=256, append=True, dtype="f32"),
        # a merged layer moved into pages, and all of it read back
        dict(name="store layer", kind="store", B=1, H=8, G=4, d=128, lo=32768, hi=32768, dtype="bf16"),
        # the newest 64 rows of every head of the serving mix, written back after a re-merge
        dict(name="store segments", kind="store", B=16, H=8, G=4, d=128, lo=8, hi=64, dtype="bf16"),
        # the same layer read back into a cache that is to be merged again
        dict(name="load layer", kind="load", B=1, H=8, G=4, d=128, lo=32768, hi=32768, dtype="bf16"),
        # fp32 rows of ragged heads read back
        dict(name="load ragged fp32", kind="load", B=4, H=8, G=2, d=64, lo=33, hi=2001, dtype="f32"),
        # the serving batch leaves and another one of its kind is admitted
        dict(name="tables turnover", kind="tables", B=16, H=8, lo=1024, hi=8192, add=0),
        # each unit gives back the rows of drafted tokens that were not taken and reserves eight new ones
        dict(name="tables reserve 8", kind="tables", B=16, H=8, lo=1024, hi=8192, add=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "decode", "store", "load", "tables"])
    B, H = rng.choice([1, 1, 2, 3, 5, 8, 16]), rng.choice([1, 2, 4, 8])
    hi = _log(rng, 1, min(65536, 1048576 // (B * H)))
    lo = rng.choice([0, hi // 8, hi // 2, hi])
    if kind == "tables":
        return dict(kind=kind, B=B, H=H, lo=lo, hi=hi, add=rng.choice([0, 1, 2, 7, 33]))
    d, dtype = rng.choice([64, 128, 128]), rng.choice(["bf16", "bf16", "f32"])
    if kind != "decode" or dtype == "f32":
        hi = max(1, hi // 4)
        lo = min(lo, hi)
    case = dict(kind=kind, B=B, H=H, G=rng.choice([1, 2, 4, 4, 8]), d=d, lo=lo, hi=hi, dtype=dtype)
    if kind == "decode":
        case["append"] = rng.random() < 0.5
    return case


def _lengths(case, gen):
    """Rows of each unit, between lo and hi, the first one hi."""
    n = case["B"] * case["H"]
    rows = torch.randint(case["lo"], case["hi"] + 1, (n,), generator=gen, dtype=torch.int32)
    rows[0] = case["hi"]
    return rows


def _page_bytes(d):
    return 36 * d + 4 * PAGE


def _row_bytes(case):
    """Bytes of a row's keys and values and its log-count as the cache's type holds them."""
    return 2 * case["d"] * DTYPES[case["dtype"]].itemsize + 4


def work(case):
    n = case["B"] * case["H"]
    rows = n * (case["lo"] + case["hi"]) / 2           # the mean of the lengths that are drawn
    if case["kind"] == "tables":
        pages, add = rows / PAGE, case["add"]
        # a release and a growth: page numbers read and written once each way, lengths and counts, the slots of the map
        moved = pages if not add else n * min(1.0, add / PAGE)
        slots = n * (case["hi"] if not add else add)
        return {"bytes": 4 * (4 * moved + 8 * n + slots), "flops": 0}
    d = case["d"]
    page = rows * _page_bytes(d) / PAGE
    if case["kind"] == "decode":
        io = 2 * n * case["G"] * d * DTYPES[case["dtype"]].itemsize + 4 * n + 4 * rows / PAGE
        return {"bytes": page + io, "flops": 4 * rows * case["G"] * d}
    one = rows * (_row_bytes(case) + 4) + page
    return {"bytes": one * (2 if case["kind"] == "store" else 1), "flops": 0}


# ----------------------------------------------------------------------------------------------------------------------
# The format in elementary operations
# ----------------------------------------------------------------------------------------------------------------------

def _quantise(x):
    """Codes (uint8) and half scales of rows x [..., d]; in 64 bits, so that no value next to a border goes astray."""
    blocks = x.double().unflatten(-1, (-1, 32))
    top = blocks.abs().amax(-1)
    s = (top / QMAX).half()
    s = torch.where(s.double() * QMAX < top, (s.view(torch.int16) + 1).view(torch.half), s)    # the next half up
    c = torch.round(blocks / torch.where(s == 0, 1, s.double()).unsqueeze(-1))
    return (c + 8).to(torch.uint8).flatten(-2), s


def _dequantise(code, s):
    return ((code.float() - 8).unflatten(-1, (-1, 32)) * s.float().unsqueeze(-1)).flatten(-2)


def _bytes_of_page(kc, ks, vc, vs, logn):
    """Bytes [P, page] of pages given as [P, 32, d] codes, [P, 32, nb] scales and [P, 32] log-counts."""
    P, _, d = kc.shape
    nb = d // 32
    pair = lambda c: c[..., 0::2] | (c[..., 1::2] << 4)                                            # noqa: E731
    k = pair(kc).view(P, PAGE, nb, 16).permute(0, 2, 1, 3)
    v = pair(vc).view(P, PAGE // 2, 2, nb, 8, 2).permute(0, 3, 1, 4, 2, 5)
    parts = [k, v, ks.contiguous().view(torch.uint8), vs.transpose(1, 2).contiguous().view(torch.uint8),
             logn.contiguous().view(torch.uint8)]
    return torch.cat([p.reshape(P, -1) for p in parts], 1)


def _of_page_bytes(page, d):
    """The codes, scales and log-counts of pages [..., page]."""
    lead, nb = page.shape[:-1], d // 32
    k, v, ks, vs, ln = page.split([16 * d, 16 * d, 2 * d, 2 * d, 4 * PAGE], -1)
    wide = lambda b: torch.stack((b & 15, b >> 4), -1).flatten(-2)                                 # noqa: E731
    k = wide(k.reshape(-1, nb, PAGE, 16).transpose(1, 2)).reshape(*lead, PAGE, d)
    v = wide(v.reshape(-1, nb, PAGE // 2, 8, 2, 2).permute(0, 2, 4, 1, 3, 5)).reshape(*lead, PAGE, d)
    ks = ks.contiguous().view(torch.half).unflatten(-1, (PAGE, nb))
    vs = vs.contiguous().view(torch.half).unflatten(-1, (nb, PAGE)).transpose(-1, -2)
    return k, ks, v, vs, ln.contiguous().view(torch.float32)


def _put_rows(pages, slots, k, v, logn):
    """Writes rows k, v [R, d] and log-counts [R] at slots [R]; a slot below zero is left out."""
    d, nb = k.shape[-1], k.shape[-1] // 32
    keep = slots >= 0
    at = slots[keep].long()
    page, r = at // PAGE, at % PAGE
    pair = lambda c: c[..., 0::2] | (c[..., 1::2] << 4)                                            # noqa: E731
    (kc, ks), (vc, vs) = _quantise(k[keep]), _quantise(v[keep])
    n, b = page.numel(), torch.arange(nb, device=at.device)
    K, V, S, T, L = (16 * d, 16 * d, 2 * d, 2 * d, 4 * PAGE)
    col = lambda *shape: torch.arange(math.prod(shape), device=at.device).view(shape)              # noqa: E731
    off = (b[:, None] * 512 + col(16)) + r[:, None, None] * 16
    pages[page[:, None], off.view(n, -1)] = pair(kc)
    off = K + b[:, None, None] * 512 + col(8, 1) * 4 + col(2) + ((r // 2) * 32 + (r % 2) * 2)[:, None, None, None]
    pages[page[:, None], off.view(n, -1)] = pair(vc)
    off = K + V + r[:, None] * 2 * nb + col(2 * nb)
    pages[page[:, None], off] = ks.contiguous().view(torch.uint8)
    off = K + V + S + b[:, None] * 64 + col(2) + r[:, None, None] * 2
    pages[page[:, None], off.view(n, -1)] = vs.contiguous().view(torch.uint8)
    off = K + V + S + T + r[:, None] * 4 + col(4)
    pages[page[:, None], off] = logn[keep].contiguous().view(n, 1).view(torch.uint8)


def _get_rows(pages, slots, d, dtype, k, v, logn):
    """Reads the rows at slots [N, T] into k, v [N, T, d] and logn [N, T]; where a slot is below zero they stay."""
    nb = d // 32
    keep = slots >= 0
    at = slots[keep].long()
    page, r = at // PAGE, at % PAGE
    n, b = page.numel(), torch.arange(nb, device=at.device)
    col = lambda *shape: torch.arange(math.prod(shape), device=at.device).view(shape)              # noqa: E731
    wide = lambda x: torch.stack((x & 15, x >> 4), -1).flatten(-2)                                 # noqa: E731
    off = (b[:, None] * 512 + col(16)) + r[:, None, None] * 16
    kc = wide(pages[page[:, None], off.view(n, -1)])
    off = 16 * d + b[:, None, None] * 512 + col(8, 1) * 4 + col(2) + ((r // 2) * 32 + (r % 2) * 2)[:, None, None, None]
    vc = wide(pages[page[:, None], off.view(n, -1)])
    ks = pages[page[:, None], 32 * d + r[:, None] * 2 * nb + col(2 * nb)].view(torch.half)
    off = 34 * d + b[:, None] * 64 + col(2) + r[:, None, None] * 2
    vs = pages[page[:, None], off.view(n, -1)].view(torch.half)
    k[keep] = _dequantise(kc, ks).to(dtype)
    v[keep] = _dequantise(vc, vs).to(dtype)
    logn[keep] = pages[page[:, None], 36 * d + r[:, None] * 4 + col(4)].view(torch.float32)[:, 0]


# ----------------------------------------------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------------------------------------------

def _rows(gen, n, d, keys):
    """Rows as the cache meets them: keys whose channels differ much in size, values whose channels do not."""
    x = torch.randn(n, d, generator=gen, device="cuda")
    if keys:
        x *= torch.exp(0.7 * torch.randn(d, generator=gen, device="cuda"))
    return x


def _log_counts(gen, *shape):
    return torch.log(torch.randint(1, 9, shape, generator=gen, device="cuda").float())


def prepare(case, seed):
    host, gen = torch.Generator().manual_seed(seed), torch.Generator(device="cuda").manual_seed(seed)
    n, rows = case["B"] * case["H"], _lengths(case, host)
    if case["kind"] == "tables":
        return _prepare_tables(case, host, n, rows)
    d, dtype, append = case["d"], DTYPES[case["dtype"]], case.get("append", False)
    cap = case["hi"] + 2 + case["hi"] % 2                          # rows that a unit may come to hold, an even number
    maxp = -(-cap // PAGE)
    held = torch.where(rows > 0, (rows + int(append) + PAGE - 1) // PAGE, int(append))
    total = int(held.sum()) + 3                                    # the pool has a few pages that no unit holds
    order = torch.randperm(total, generator=host, dtype=torch.int32)
    table = torch.full((n, maxp), -1, dtype=torch.int32)
    mask = torch.arange(maxp) < held[:, None]
    table[mask] = order[:int(held.sum())]
    s = dict(kind=case["kind"], d=d, dtype=dtype, table=table.cuda(), rows=rows.cuda())
    if case["kind"] == "store":
        s["pages"] = torch.zeros(total, _page_bytes(d), dtype=torch.uint8, device="cuda")
    else:
        (kc, ks), (vc, vs) = (_quantise(_rows(gen, total * PAGE, d, key)) for key in (True, False))
        s["pages"] = _bytes_of_page(*(x.view(total, PAGE, -1) for x in (kc, ks, vc, vs)), _log_counts(gen, total, PAGE))
    t = torch.arange(cap)
    slots = torch.where(t < rows[:, None], table.repeat_interleave(PAGE, 1)[:, :cap] * PAGE + t % PAGE, -1)
    if case["kind"] != "decode":
        s["slots"] = slots.to(torch.int32).view(case["B"], case["H"], cap).cuda()
        shape = (case["B"], case["H"], cap, d)
        for name in ("K", "V"):
            if case["kind"] == "store":
                s[name] = _rows(gen, n * cap, d, name == "K").to(dtype).view(shape)
            s[name + "_out"] = torch.zeros(shape, dtype=dtype, device="cuda")
        s["logn"], s["logn_out"] = _log_counts(gen, *shape[:3]), torch.zeros(shape[:3], device="cuda")
    else:
        q = torch.randn(case["B"], case["H"] * case["G"], d, generator=gen, device="cuda")
        s.update(q=(1.5 * q).to(dtype), out=torch.empty_like(q, dtype=dtype), lens=rows.cuda(), append=append)
        if append:
            new = torch.full((n, 2), -1, dtype=torch.int32)
            new[:, 0] = table[torch.arange(n), rows.long() // PAGE] * PAGE + rows % PAGE
            s["new_slots"] = new.cuda()
            s["k_new"], s["v_new"] = (_rows(gen, n, d, key).to(dtype).view(case["B"], case["H"], d) for key in (True, False))
            s["K_row"], s["V_row"] = (torch.zeros(case["B"], case["H"], 2, d, dtype=dtype, device="cuda") for _ in range(2))
            s["logn_row"] = torch.zeros(case["B"], case["H"], 2, device="cuda")
    if own:                                                        # the handles that a user's program keeps
        from asymmetric_kv_merging_b200 import kvs
        H_q = case["H"] * case["G"]
        s["kvs"], s["pool"] = kvs, kvs.page_pool(s["pages"], s["table"])
        s["desc"] = kvs.make_desc(case["B"], case["H"], H_q, d, cap, dtype)
        s["row_desc"] = kvs.make_desc(case["B"], case["H"], H_q, d, 2, dtype)
        s["ws"] = kvs.workspace(s["desc"], ops=(kvs.OP_PAGES,))
    return s


def _prepare_tables(case, host, n, rows):
    """Units that hold the pages of `base` rows and are to hold those of `rows`."""
    base = rows if case["add"] else torch.zeros_like(rows)
    rows = rows + case["add"]
    stride = case["add"] or case["hi"]
    maxp = -(-(case["hi"] + case["add"]) // PAGE)
    held = (base + PAGE - 1) // PAGE
    total = int(((rows + PAGE - 1) // PAGE).sum()) + 17
    order = torch.randperm(total, generator=host, dtype=torch.int32)
    table = torch.full((n, maxp), -1, dtype=torch.int32)
    first = total - int(held.sum())
    table[torch.arange(maxp) < held[:, None]] = order[first:]
    s = dict(kind="tables", table=table, base=base, rows=rows, held=held, free=order,
             n_free=torch.tensor([first], dtype=torch.int32), slots=torch.full((n, stride), -1, dtype=torch.int32))
    s = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    if own:
        from asymmetric_kv_merging_b200 import kvs
        s["pages"] = torch.zeros(total, _page_bytes(64), dtype=torch.uint8, device="cuda")
        s["kvs"], s["pool"] = kvs, kvs.page_pool(s["pages"], s["table"])
        s["ws"] = kvs.workspace(kvs.make_desc(case["B"], case["H"], case["H"], 64, 2, kvs.BF16), ops=(kvs.OP_PAGES,))
    return s


# ----------------------------------------------------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------------------------------------------------

def run(s):
    return {"decode": _decode, "store": _store, "load": _load, "tables": _tables}[s["kind"]](s)


def _decode(s):
    if s["append"]:
        s["lens"].copy_(s["rows"])                                 # the step starts from the same lengths every time
    if own:
        kvs = s["kvs"]
        kvs.page_decode_attn(s["desc"], s["q"], s["pool"], s["lens"], s["out"], s["ws"], s.get("k_new"), s.get("v_new"))
        if s["append"]:
            kvs.page_load(s["row_desc"], s["pool"], s["new_slots"], s["K_row"], s["V_row"], s["logn_row"], s["ws"])
    else:
        _decode_plain(s)
    if not s["append"]:
        return {"out": s["out"]}
    return {"out": s["out"], "lens": s["lens"], "K": s["K_row"], "V": s["V_row"], "logn": s["logn_row"]}


def _decode_plain(s):
    table, d = s["table"], s["d"]
    n, maxp = table.shape
    kc, ks, vc, vs, ln = _of_page_bytes(s["pages"][table.clamp(min=0)], d)
    k, v = _dequantise(kc, ks).view(n, -1, d), _dequantise(vc, vs).view(n, -1, d)
    q = s["q"].float().view(n, -1, d) / math.sqrt(d)
    live = torch.arange(maxp * PAGE, device="cuda") < s["lens"][:, None]
    x = torch.where(live[:, None], q @ k.transpose(1, 2) + ln.view(n, 1, -1), -math.inf)
    if s["append"]:
        kn, vn = s["k_new"].float().view(n, 1, d), s["v_new"].float().view(n, 1, d)
        x, v = torch.cat((x, q @ kn.transpose(1, 2)), 2), torch.cat((v, vn), 1)
        live = torch.cat((live, torch.ones_like(live[:, :1])), 1)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0, top))
    total = p.sum(-1, keepdim=True)
    o = (p @ torch.where(live[..., None], v, 0)) / torch.where(total == 0, 1, total)
    s["out"].copy_(o.view(s["out"].shape))
    if s["append"]:
        new = s["new_slots"]
        _put_rows(s["pages"], new[:, 0], s["k_new"].view(n, d), s["v_new"].view(n, d), torch.zeros(n, device="cuda"))
        _get_rows(s["pages"], new, d, s["dtype"], s["K_row"].view(n, 2, d), s["V_row"].view(n, 2, d), s["logn_row"].view(n, 2))
        s["lens"] += 1


def _store(s):
    """Rows into pages and back: what the pages hold is returned as the values that it stands for."""
    if own:
        s["kvs"].page_store(s["desc"], s["K"], s["V"], s["logn"], s["slots"], s["pool"], s["ws"])
    else:
        d = s["d"]
        _put_rows(s["pages"], s["slots"].view(-1), s["K"].view(-1, d), s["V"].view(-1, d), s["logn"].view(-1))
    return _load(s)


def _load(s):
    if own:
        s["kvs"].page_load(s["desc"], s["pool"], s["slots"], s["K_out"], s["V_out"], s["logn_out"], s["ws"])
    else:
        _get_rows(s["pages"], s["slots"], s["d"], s["dtype"], s["K_out"], s["V_out"], s["logn_out"])
    return {"K": s["K_out"], "V": s["V_out"], "logn": s["logn_out"]}


def _tables(s):
    """The units go back to their base rows (which frees pages), then take their new ones, with the slots of the new rows."""
    if own:
        kvs = s["kvs"]
        kvs.page_assign(s["pool"], s["base"], s["held"], s["free"], s["n_free"], s["ws"])
        kvs.page_assign(s["pool"], s["rows"], s["held"], s["free"], s["n_free"], s["ws"], s["slots"], s["base"])
    else:
        _assign_plain(s, s["base"])
        _assign_plain(s, s["rows"])
        t = s["base"][:, None] + torch.arange(s["slots"].shape[1], device="cuda")
        page = s["table"].gather(1, (t // PAGE).clamp(max=s["table"].shape[1] - 1).long())
        s["slots"].copy_(torch.where(t < s["rows"][:, None], page * PAGE + t % PAGE, -1))
    return {"table": s["table"], "held": s["held"], "n_free": s["n_free"], "slots": s["slots"]}


def _assign_plain(s, rows):
    table, held, free, n_free = s["table"], s["held"], s["free"], s["n_free"]
    want = (rows + PAGE - 1) // PAGE
    grow, give = (want - held).clamp(min=0), (held - want).clamp(min=0)
    taken = grow.sum()
    j = torch.arange(table.shape[1], device="cuda")
    # pages given back go on top of the stack, unit after unit
    leaving = (j >= want[:, None]) & (j < held[:, None])
    to = torch.where(leaving, (n_free + give.cumsum(0) - give)[:, None] + j - want[:, None], free.numel())
    free.copy_(torch.cat((free, free[:1])).scatter(0, to.view(-1), table.view(-1))[:-1])
    n_free += give.sum() - taken
    # the topmost `taken` ones are taken, the lowest of them first
    new = (j >= held[:, None]) & (j < want[:, None])
    at = torch.where(new, (n_free + grow.cumsum(0) - grow)[:, None] + j - held[:, None], 0)
    table.copy_(torch.where(new, free[at], torch.where(leaving, -1, table)))
    held.copy_(want)


# ----------------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ----------------------------------------------------------------------------------------------------------------------

def _row_values(pages, page, r, d):
    """Rows r of pages `page` (both [R]) as doubles, block by block: keys, values, log-counts."""
    raw, blocks = pages.to(torch.int64), ([], [])
    half = lambda at: (raw[page, at] + 256 * raw[page, at + 1]).to(torch.int16).view(torch.half).double()  # noqa: E731
    for b in range(d // 32):
        for c in range(0, 32, 2):
            byte = raw[page, 512 * b + 16 * r + c // 2]
            s = half(32 * d + (r * (d // 32) + b) * 2)
            blocks[0].extend(((byte % 16 - 8) * s, (byte // 16 - 8) * s))
            byte = raw[page, 16 * d + 512 * b + (r // 2) * 32 + (c // 4) * 4 + (r % 2) * 2 + (c // 2) % 2]
            s = half(34 * d + (b * 32 + r) * 2)
            blocks[1].extend(((byte % 16 - 8) * s, (byte // 16 - 8) * s))
    logn = pages[page[:, None], 36 * d + 4 * r[:, None] + torch.arange(4, device="cuda")].view(torch.float32)[:, 0].double()
    return torch.stack(blocks[0], 1), torch.stack(blocks[1], 1), logn


def _held_values(x):
    """The values that rows x stand for once they are held in 4 bits."""
    out, x = torch.empty_like(x, dtype=torch.float64), x.double()
    every = torch.arange(31744, dtype=torch.int16, device="cuda").view(torch.half).double()        # the finite halves from 0 up
    for b in range(0, x.shape[-1], 32):
        y = x[..., b:b + 32]
        s = every[torch.searchsorted(every * 7, y.abs().amax(-1).contiguous())][..., None]
        whole = torch.floor(y / torch.where(s == 0, 1, s))
        rest = y - whole * s
        up = (rest * 2 > s) | ((rest * 2 == s) & (whole % 2 != 0))
        out[..., b:b + 32] = (whole + up) * s
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "tables":
        return None
    n, d = s["table"].shape[0], s["d"]
    if case["kind"] == "decode":
        out = torch.zeros(n, case["G"], d, dtype=torch.float64, device="cuda")
        for u in range(n):
            rows = int(s["rows"][u])
            t = torch.arange(rows, device="cuda")
            k, v, ln = [], [], []
            for part in t.split(16384):
                page = s["table"][u, part // PAGE].long()
                here, at = torch.unique(page, return_inverse=True)
                a, b, c = _row_values(s["pages"][here], at, part % PAGE, d)
                k.append(a), v.append(b), ln.append(c)
            if case["append"]:
                k.append(s["k_new"].view(n, 1, d)[u].double()), v.append(s["v_new"].view(n, 1, d)[u].double())
                ln.append(torch.zeros(1, dtype=torch.float64, device="cuda"))
            if k:
                q = s["q"].view(n, -1, d)[u].double()
                w = torch.softmax(q @ torch.cat(k).T / d ** 0.5 + torch.cat(ln), -1)
                out[u] = w @ torch.cat(v)
        result = {"out": out.view(s["out"].shape)}
        if case["append"]:
            pad = lambda x: torch.stack((x, torch.zeros_like(x)), 2)                               # noqa: E731
            result.update(lens=s["rows"] + 1, K=pad(_held_values(s["k_new"])), V=pad(_held_values(s["v_new"])),
                          logn=torch.zeros(case["B"], case["H"], 2, dtype=torch.float64, device="cuda"))
        return result
    shape = s["K_out"].shape
    live = s["slots"] >= 0
    if case["kind"] == "store":
        K, V = (torch.where(live[..., None], _held_values(s[x]), 0) for x in "KV")
        ln = torch.where(live, s["logn"].double(), 0)
    else:
        K, V = (torch.zeros(shape, dtype=torch.float64, device="cuda") for _ in range(2))
        ln = torch.zeros(shape[:3], dtype=torch.float64, device="cuda")
        at = s["slots"][live].long()
        got = [[], [], []]
        for part in at.split(16384):
            here, i = torch.unique(part // PAGE, return_inverse=True)
            for g, x in zip(got, _row_values(s["pages"][here], i, part % PAGE, d)):
                g.append(x)
        for to, g in zip((K, V, ln), got):
            if g:
                to[live] = torch.cat(g)
    return {"K": K, "V": V, "logn": ln}
