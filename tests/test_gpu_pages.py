"""The 4-bit paged cache on the GPU against the plain 64-bit oracle in tests/pages_ref.py.

Page tables, slot maps, page bytes and rows read back are exact. Decode outputs carry a bound
that is derived, with A = sum_t p_t |v_t| and n rows:
  fp32  d + 6 roundings of a logit's products and sums, each half a last place of at most
        X = sum |q k| / sqrt(d) (+ |logn|), make the weights off by 2 (d + 6) 2^-24 X relative;
        n + 16 roundings of the sums and the exponential's 2^-22 add to that.
  bf16  in addition, with s the scale of a value's block and S = sum_t p_t s_t:
        the weight is rounded to half, h(p), which both sums of  sum u w - 8 sum s h(p)  see, and so
        does the sum of the weights that divides them: 2^-11 (A + |out|);
        w = half(s h(p)) is seen by the first one only, where the code u is at most 15: 15 2^-11 S;
        weights (and w) below the half range are off by at most 2^-25 each, the largest p being at
        least 2^7 over the largest scale above 1: n 2^-32 max(1, s) (2 |v| + 15 s), and the logit's
        offset sum is held to 2^-33 of it; and the output is rounded to bf16, 2^-8 |out|.
"""

import gc

import numpy as np
import pytest
import torch

import pages_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
PAGE = 32


@pytest.fixture(scope="module")
def kvs():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from asymmetric_kv_merging_b200 import build
    build.build()
    from asymmetric_kv_merging_b200 import kvs as mod
    yield mod
    gc.collect()
    torch.cuda.empty_cache()             # later tests watch the device's free memory


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV).contiguous()


def workspace(kvs, B, H, G=1, d=64):
    return kvs.workspace(kvs.make_desc(B, H, H * G, d, 2, kvs.BF16), ops=(kvs.OP_PAGES,))


# ---------------------------------------------------------------------------
# Page tables and slot maps
# ---------------------------------------------------------------------------

class DeviceTables:
    def __init__(self, kvs, units, max_pages, free, n_pages=None):
        self.kvs, n_pages = kvs, n_pages or len(free)
        self.table = torch.full((units, max_pages), -1, dtype=torch.int32, device=DEV)
        self.pages = torch.zeros(n_pages, kvs.page_bytes(64), dtype=torch.uint8, device=DEV)
        self.pool = kvs.page_pool(self.pages, self.table)
        self.held = torch.zeros(units, dtype=torch.int32, device=DEV)
        self.free = i32(list(free) + [-7] * (n_pages - len(free)))
        self.n_free = i32([len(free)])
        self.ws = workspace(kvs, 1, units)

    def assign(self, rows, slots=None, begin=None):
        self.kvs.page_assign(self.pool, i32(rows), self.held, self.free, self.n_free, self.ws, slots,
                             None if begin is None else i32(begin))

    def check(self, want):
        assert self.held.tolist() == want.held
        assert np.array_equal(self.table.cpu().numpy(), want.table)
        n = int(self.n_free)
        assert self.free[:n].tolist() == want.free


@pytest.mark.parametrize("units,max_pages", [(1, 1), (3, 5), (33, 9), (1025, 3), (5000, 2)])
def test_tables_follow_random_lengths(kvs, units, max_pages):
    rng = np.random.default_rng(units)
    order = rng.permutation(units * max_pages)
    dev, want = DeviceTables(kvs, units, max_pages, order), ref.Tables(units, max_pages, order.tolist())
    for step in range(6):
        rows = rng.integers(0, max_pages * PAGE + 1, units)
        if step == 2:
            rows[:] = 0                                     # everything goes back
        begin = rng.integers(0, max_pages * PAGE, units) if step % 2 else np.zeros(units, int)
        stride = [1, 7, 40][step % 3]
        slots = torch.full((units, stride), -5, dtype=torch.int32, device=DEV)
        dev.assign(rows, slots, begin if step % 2 else None)
        assert want.assign(rows.tolist())
        dev.check(want)
        assert np.array_equal(slots.cpu().numpy(), want.slots(rows, begin, stride))
    assert kvs.device_flags(dev.ws) == 0


def test_one_unit_with_a_long_table(kvs):
    order = list(range(4999, -1, -1))
    dev, want = DeviceTables(kvs, 2, 5000, order), ref.Tables(2, 5000, order)
    for rows in ([5000 * PAGE, 0], [31, 4998 * PAGE + 1], [0, 0]):
        slots = torch.empty(2, 300, dtype=torch.int32, device=DEV)
        dev.assign(rows, slots, [max(0, r - 300) for r in rows])
        assert want.assign(rows)
        dev.check(want)
        assert np.array_equal(slots.cpu().numpy(), want.slots(rows, [max(0, r - 300) for r in rows], 300))


def test_a_shortage_changes_nothing(kvs):
    dev, want = DeviceTables(kvs, 3, 4, [5, 1, 4, 2], n_pages=6), ref.Tables(3, 4, [5, 1, 4, 2])
    dev.assign([40, 0, 33])
    assert want.assign([40, 0, 33])
    dev.check(want)
    slots = torch.empty(3, 70, dtype=torch.int32, device=DEV)
    dev.assign([100, 40, 32], slots)       # four more pages wanted, one given back, none free
    assert not want.assign([100, 40, 32])
    dev.check(want)
    assert np.array_equal(slots.cpu().numpy(), want.slots([100, 40, 32], [0, 0, 0], 70))
    assert kvs.device_flags(dev.ws, clear=True) == kvs.FLAG_NO_PAGES
    dev.assign([128, 0, 0])                # two more, and the two that are given back
    assert want.assign([128, 0, 0])
    dev.check(want)
    dev.n_free.fill_(7)                    # more free pages than the pool has
    dev.assign([0, 0, 0])
    assert dev.held.tolist() == want.held and int(dev.n_free) == 7
    assert kvs.device_flags(dev.ws, clear=True) == kvs.FLAG_NO_PAGES


def test_lengths_out_of_range_leave_the_unit_alone(kvs):
    dev, want = DeviceTables(kvs, 3, 4, range(12)), ref.Tables(3, 4, range(12))
    for rows in ([50, 60, 70], [-1, 129, 10], [-2 ** 31, 2 ** 31 - 1, 128]):
        slots = torch.empty(3, 4, dtype=torch.int32, device=DEV)
        dev.assign(rows, slots)
        assert want.assign(rows)
        dev.check(want)
        assert kvs.device_flags(dev.ws, clear=True) == (0 if rows[0] == 50 else kvs.FLAG_BAD_LENGTH)
        if rows[0] < 0:
            assert slots[0].tolist() == [-1] * 4


# ---------------------------------------------------------------------------
# Rows to pages and back
# ---------------------------------------------------------------------------

def hard_rows(rng, n, d, dtype):
    """Rows with every kind of block: ordinary, on rounding borders, zero, tiny, huge, one large
    element, infinite, NaN."""
    x = rng.standard_normal((n, d))
    x[n // 8] = 0
    x[n // 8 + 1] *= 1e-7                                   # subnormal half scales
    x[n // 8 + 2] *= 1e-9                                   # below the smallest scale's half step
    x[n // 8 + 3] *= 6e4
    x[n // 8 + 4, 1] = 1e4
    for i in range(min(8, n - n // 8 - 5)):                 # multiples of half a scale: ties
        half = 2.0 ** (i - 4)
        x[n // 8 + 5 + i] = rng.integers(-14, 15, d) * half
        x[n // 8 + 5 + i, ::32] = 14 * half
    t = torch.tensor(x, dtype=torch.float32).to(dtype)
    t[-1, 3], t[-2, 5], t[-3, d - 1] = float("inf"), float("nan"), 3e38
    t[-4, 0] = 7 * 65504.0
    return t


def row_case(rng, B, H, T, d, dtype, shuffle):
    n = B * H * T
    K = torch.stack([hard_rows(rng, T, d, dtype) for _ in range(B * H)]).view(B, H, T, d)
    V = torch.stack([hard_rows(rng, T, d, dtype).flip(0) for _ in range(B * H)]).view(B, H, T, d)
    logn = torch.tensor(rng.standard_normal((B, H, T)), dtype=torch.float32)
    n_pages = -(-n // PAGE) + 3
    slots = np.arange(n) + PAGE
    if shuffle:
        slots = rng.permutation(n_pages * PAGE)[:n]
    slots = np.where(rng.random(n) < 0.2, -rng.integers(1, 9, n), slots)
    return K, V, logn, slots.reshape(B, H, T), n_pages


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shuffle", [False, True])
@pytest.mark.parametrize("shape", [(1, 1, 24), (2, 3, 70)])
def test_store_and_load_are_exact(kvs, dtype, d, shuffle, shape):
    rng = np.random.default_rng(d + shuffle)
    B, H, T = shape
    K, V, logn, slots, n_pages = row_case(rng, B, H, T, d, dtype, shuffle)
    before = rng.integers(0, 256, (n_pages, ref.page_bytes(d)), dtype=np.uint8)
    pages = torch.tensor(before, device=DEV)
    pool = kvs.page_pool(pages, torch.zeros(1, 1, dtype=torch.int32, device=DEV))
    desc, ws = kvs.make_desc(B, H, H, d, T, dtype), workspace(kvs, B, H)
    kvs.page_store(desc, K.to(DEV), V.to(DEV), logn.to(DEV), i32(slots), pool, ws)
    want = before.copy()
    Kn, Vn = K.double().numpy(), V.double().numpy()
    for i in np.ndindex(B, H, T):
        if slots[i] >= 0:
            ref.put_row(want, slots[i], Kn[i], Vn[i], logn[i])
    assert np.array_equal(pages.cpu().numpy(), want)        # rows left out, and other rows, as they were
    # and back
    Ko = torch.full_like(K, 77.0, device=DEV)
    Vo, lo = torch.full_like(Ko, -77.0), torch.full((B, H, T), 5.0, device=DEV)
    kvs.page_load(desc, pool, i32(slots), Ko, Vo, lo, ws)
    live = slots >= 0
    for got, x, fill in ((Ko, Kn, 77.0), (Vo, Vn, -77.0)):
        back = torch.tensor(np.where(live[..., None], ref.held(x), fill)).to(torch.float32).to(dtype)
        assert torch.equal(torch.nan_to_num(got.cpu(), nan=1e30), torch.nan_to_num(back, nan=1e30))
    assert torch.equal(lo.cpu(), torch.where(torch.tensor(live), logn, torch.tensor(5.0)))
    assert kvs.device_flags(ws) == 0


def test_every_bf16_against_every_kind_of_scale(kvs):
    """Blocks of all bf16 magnitudes below a maximum, for maxima of all mantissas: every code of
    every scale, borders included."""
    d = 64
    bits = torch.arange(0x3f80 - 5 * 128, 0x3f80, dtype=torch.int16)
    small = bits.view(torch.bfloat16)                       # 2^-5 .. 1
    top = torch.arange(0x3f80, 0x3f80 + 128, dtype=torch.int16).view(torch.bfloat16)
    rows = []
    for m in top:
        x = small.view(-1, 20)
        rows.append(torch.cat([m.expand(x.shape[0], 1), x, -x[:, :11]], 1))
    x = torch.cat(rows)
    x = x[:x.shape[0] // 2 * 2].view(1, 1, -1, d).contiguous()
    T = x.shape[2] // 2 * 2
    x = x[:, :, :T].contiguous()
    pages = torch.zeros(-(-T // PAGE), kvs.page_bytes(d), dtype=torch.uint8, device=DEV)
    pool = kvs.page_pool(pages, torch.zeros(1, 1, dtype=torch.int32, device=DEV))
    for dtype in (torch.bfloat16, torch.float32):
        desc, ws = kvs.make_desc(1, 1, 1, d, T, dtype), workspace(kvs, 1, 1)
        X, slots = x.to(dtype).to(DEV), i32(np.arange(T).reshape(1, 1, T))
        kvs.page_store(desc, X, X, None, slots, pool, ws)
        f32 = kvs.make_desc(1, 1, 1, d, T, torch.float32)
        K, V = torch.empty(1, 1, T, d, device=DEV), torch.empty(1, 1, T, d, device=DEV)
        kvs.page_load(f32, pool, slots, K, V, None, ws)
        want = torch.tensor(ref.held(x.double().numpy())).float()
        assert torch.equal(K.cpu(), want) and torch.equal(V.cpu(), want)


def test_slots_past_the_pool_are_skipped(kvs):
    d, T = 64, 4
    pages = torch.zeros(2, kvs.page_bytes(d), dtype=torch.uint8, device=DEV)
    pool = kvs.page_pool(pages, torch.zeros(1, 1, dtype=torch.int32, device=DEV))
    desc, ws = kvs.make_desc(1, 1, 1, d, T, torch.bfloat16), workspace(kvs, 1, 1)
    K = torch.ones(1, 1, T, d, dtype=torch.bfloat16, device=DEV)
    slots = i32([[[64, 63, 2 ** 31 - 1, -1]]])
    kvs.page_store(desc, K, K, None, slots, pool, ws)
    assert kvs.device_flags(ws, clear=True) == kvs.FLAG_BAD_PAGE
    Ko, Vo = torch.zeros_like(K), torch.zeros_like(K)
    kvs.page_load(desc, pool, slots, Ko, Vo, None, ws)
    assert kvs.device_flags(ws, clear=True) == kvs.FLAG_BAD_PAGE
    assert torch.equal(Ko[0, 0, 1], K[0, 0, 1]) and float(Ko.float().abs().sum()) == d


# ---------------------------------------------------------------------------
# Decode attention
# ---------------------------------------------------------------------------

@pytest.fixture(params=[0, 5000], ids=["short-tables", "wide-tables"])
def wide(request):
    """Columns added to the page tables: few units with short tables are decoded by a cluster of
    CTAs each (one or two units with longer tables by several), long tables (and many units) by the
    kernel that splits the pages evenly."""
    return request.param


class Cache:
    """A paged cache of given lengths with random pages; unused rows and pages hold garbage."""

    def __init__(self, kvs, B, H, G, d, lens, dtype, seed=0, room=1, logn_scale=1.0, v_scale=1.0,
                 k_scale=1.0, wide=0):
        self.kvs, self.B, self.H, self.G, self.d, self.dtype = kvs, B, H, G, d, dtype
        rng = self.rng = np.random.default_rng(seed)
        lens = self.lens_np = np.asarray(lens, np.int64)
        units = B * H
        held = -(-(lens + room) // PAGE)
        maxp = int(held.max()) + 1 + wide
        total = int(held.sum()) + 2
        order = rng.permutation(total)
        self.table_np = -np.ones((units, maxp), np.int64)
        at = 0
        for u in range(units):
            self.table_np[u, :held[u]] = order[at:at + held[u]]
            at += held[u]
        self.pages_np = rng.integers(0, 256, (total, ref.page_bytes(d)), dtype=np.uint8)
        self.pages_np[:, 32 * d:36 * d] = 255                # NaN scales where no row is
        for u in range(units):
            for t in range(lens[u]):
                ref.put_row(self.pages_np, self.slot(u, t), rng.standard_normal(d) * k_scale,
                            rng.standard_normal(d) * v_scale, rng.random() * logn_scale)
        self.to_device()

    def slot(self, u, t):
        return int(self.table_np[u, t // PAGE]) * PAGE + t % PAGE

    def to_device(self):
        self.pages, self.table = torch.tensor(self.pages_np, device=DEV), i32(self.table_np)
        self.lens = i32(self.lens_np)
        self.pool = self.kvs.page_pool(self.pages, self.table)
        self.desc = self.kvs.make_desc(self.B, self.H, self.H * self.G, self.d, 2, self.dtype)
        self.ws = self.kvs.workspace(self.desc, ops=(self.kvs.OP_PAGES,))

    def random(self, *shape, scale=1.0):
        x = torch.tensor(self.rng.standard_normal(shape) * scale, dtype=torch.float32)
        return x.to(self.dtype).to(DEV)

    def step(self, q, k_new=None, v_new=None):
        out = torch.full_like(q, 99.0)
        self.kvs.page_decode_attn(self.desc, q, self.pool, self.lens, out, self.ws, k_new, v_new)
        return out

    def check(self, q, out, k_new=None, v_new=None, fits=None):
        """`out` against attention over the rows as they were before the step."""
        units, G, d = self.B * self.H, self.G, self.d
        q, got = q.double().cpu().numpy().reshape(units, G, d), out.double().cpu().numpy().reshape(units, G, d)
        worst = 0.0
        for u in range(units):
            k, v, ln = ref.rows_of(self.pages_np, self.table_np[u], int(self.lens_np[u]), d)
            if k_new is not None and (fits is None or fits[u]):
                k = np.concatenate([k, k_new.double().cpu().numpy().reshape(units, 1, d)[u]])
                v = np.concatenate([v, v_new.double().cpu().numpy().reshape(units, 1, d)[u]])
                ln = np.append(ln, 0.0)
            want, size = ref.attend(q[u], k, v, ln)
            scales = ref.value_scales(self.pages_np, self.table_np[u], int(self.lens_np[u]), d)
            bound = tolerance(self.dtype, q[u], k, v, ln, want, size, scales)
            err = np.abs(got[u] - want)
            assert np.all(err <= bound), (u, len(k), float((err / bound).max()))
            worst = max(worst, float((err / np.maximum(bound, 1e-300)).max()))
        return worst

    def append(self, k_new, v_new, fits=None):
        """The step's effect on the oracle's pages and lengths; the device's must be the same."""
        for u in range(self.B * self.H):
            if fits is None or fits[u]:
                ref.put_row(self.pages_np, self.slot(u, int(self.lens_np[u])),
                            k_new.double().cpu().numpy().reshape(-1, self.d)[u],
                            v_new.double().cpu().numpy().reshape(-1, self.d)[u], 0.0)
                self.lens_np[u] += 1
        assert np.array_equal(self.pages.cpu().numpy(), self.pages_np)
        assert self.lens.tolist() == self.lens_np.tolist()


def tolerance(dtype, q, k, v, logn, want, size, scales=None):
    n, d = max(1, len(k)), q.shape[1]
    if len(k) == 0:
        return np.zeros_like(want)
    x = float((np.abs(q) @ np.abs(k).T).max()) / np.sqrt(d) + float(np.abs(logn[np.isfinite(logn)]).max(initial=0.0))
    rel = 2 * (d + 6) * 2.0 ** -24 * x + (n + 16) * 2.0 ** -24 + 2.0 ** -21
    if dtype == torch.float32:
        return rel * size + 2.0 ** -24 * np.abs(want) + 1e-30
    s = np.zeros_like(v)                            # the new row, if there is one, is not rounded
    s[:len(scales)] = np.repeat(scales, 32, 1)
    p = ref.weights(q, k, logn)
    low = n * 2.0 ** -32 * max(1.0, float(s.max())) * (2 * np.abs(v) + 15 * s).max(0)
    return rel * size + 2.0 ** -11 * (size + np.abs(want)) + 15 * 2.0 ** -11 * (p @ s) + low + 2.0 ** -8 * np.abs(want)


EDGE = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 255, 256, 257]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_decode_at_the_edges_of_pages(kvs, dtype, d, G, wide):
    c = Cache(kvs, 2, 8, G, d, EDGE, dtype, seed=G + d, wide=wide)
    q, kn, vn = c.random(2, 8 * G, d, scale=1.5), c.random(2, 8, d), c.random(2, 8, d)
    c.check(q, c.step(q))
    assert c.lens.tolist() == EDGE and np.array_equal(c.pages.cpu().numpy(), c.pages_np)
    out = c.step(q, kn, vn)
    c.check(q, out, kn, vn)
    c.append(kn, vn)
    c.check(q, c.step(q))
    assert kvs.device_flags(c.ws) == 0


@pytest.mark.parametrize("dtype,d,G,lens", [
    (torch.bfloat16, 128, 4, [5000]),                        # one unit over many CTAs
    (torch.float32, 128, 2, [3001]),
    (torch.bfloat16, 64, 8, [2500, 3, 0, 1777]),
    (torch.bfloat16, 128, 8, [1, 4097, 1, 31]),
    (torch.float32, 64, 1, [900, 0, 901, 77]),
    (torch.bfloat16, 128, 4, [1200, 0, 1, 333, 64] * 6),     # some units whole in a CTA, some split
    (torch.float32, 128, 4, [260, 0, 1, 333, 64] * 6)])
def test_decode_of_long_and_ragged_units(kvs, dtype, d, G, lens, wide):
    c = Cache(kvs, 1, len(lens), G, d, lens, dtype, seed=3, logn_scale=3.0, wide=wide)
    q = c.random(1, len(lens) * G, d, scale=2.0)
    c.check(q, c.step(q))
    kn, vn = c.random(1, len(lens), d), c.random(1, len(lens), d)
    c.check(q, c.step(q, kn, vn), kn, vn)
    c.append(kn, vn)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_of_many_short_units(kvs, dtype):
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 40, 700)
    lens[::50] = 0
    c = Cache(kvs, 100, 7, 2, 64, lens, dtype, seed=2)
    q, kn, vn = c.random(100, 14, 64), c.random(100, 7, 64), c.random(100, 7, 64)
    c.check(q, c.step(q, kn, vn), kn, vn)
    c.append(kn, vn)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens", [[6000] + [k % 40 for k in range(63)],          # one long among 64
                                  [k * 37 % 90 for k in range(149)] + [1900],    # more units than half the CTAs
                                  [0, 0, 3, 0, 1200, 0] * 60])
def test_decode_of_units_that_differ_much(kvs, dtype, lens):
    c = Cache(kvs, 1, len(lens), 2, 64, lens, dtype, seed=4, wide=2000)
    q, kn, vn = c.random(1, 2 * len(lens), 64), c.random(1, len(lens), 64), c.random(1, len(lens), 64)
    c.check(q, c.step(q))
    c.check(q, c.step(q, kn, vn), kn, vn)
    c.append(kn, vn)
    assert kvs.device_flags(c.ws) == 0


def long_cache(kvs, dtype, d, G, rows, n_pages, first, wide=0):
    """One unit of `rows` rows in pages from `first` on, stored from random rows; and its rows as
    the pages hold them."""
    g = torch.Generator(device=DEV).manual_seed(rows)
    n = -(-rows // PAGE)
    pages = torch.empty(n_pages, kvs.page_bytes(d), dtype=torch.uint8, device=DEV)
    table = torch.full((1, n + 1 + wide), -1, dtype=torch.int32, device=DEV)
    table[0, :n] = first + torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    pool = kvs.page_pool(pages, table)
    desc = kvs.make_desc(1, 1, G, d, rows + rows % 2, dtype)
    ws = kvs.workspace(desc, ops=(kvs.OP_PAGES,))
    t = torch.arange(desc.T_cap, device=DEV)
    slots = torch.where(t < rows, table[0].repeat_interleave(PAGE)[:desc.T_cap] * PAGE + t % PAGE, -1)
    slots = slots.to(torch.int32).view(1, 1, -1)
    K, V = (torch.randn(1, 1, desc.T_cap, d, generator=g, device=DEV).to(dtype) for _ in range(2))
    logn = torch.rand(1, 1, desc.T_cap, generator=g, device=DEV)
    kvs.page_store(desc, K, V, logn, slots, pool, ws)
    f32 = kvs.make_desc(1, 1, G, d, desc.T_cap, torch.float32)
    K, V = torch.zeros(1, 1, desc.T_cap, d, device=DEV), torch.zeros(1, 1, desc.T_cap, d, device=DEV)
    kvs.page_load(f32, pool, slots, K, V, None, ws)
    q = (2 * torch.randn(1, G, d, generator=g, device=DEV)).to(dtype)
    lens = torch.tensor([rows], dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    kvs.page_decode_attn(desc, q, pool, lens, out, ws)
    k, v = K[0, 0, :rows].double(), V[0, 0, :rows].double()
    w = torch.softmax(q[0].double() @ k.T / d ** 0.5 + logn[0, 0, :rows].double(), -1)
    s = v.abs().view(rows, -1, 32).amax(-1).repeat_interleave(32, 1) / 7      # (no scale is subnormal here)
    x = float((q[0].double().abs() @ k.abs().T).max()) / d ** 0.5 + 1
    size, want = w @ v.abs(), w @ v
    bound = (2 * (d + 6) * 2.0 ** -24 * x + (rows + 16) * 2.0 ** -24 + 2.0 ** -21) * size + 2.0 ** -24 * want.abs()
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -11 * (size + want.abs() + 15 * (w @ s)) + 2.0 ** -8 * want.abs() + rows * 2.0 ** -27
    err = (out[0].double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    assert kvs.device_flags(ws) == 0


@pytest.mark.parametrize("dtype,d,G,rows,wide", [
    (torch.bfloat16, 64, 4, 300001, 0),             # more pages per warp than one list holds
    (torch.bfloat16, 128, 1, 40000, 0),
    (torch.float32, 64, 2, 90017, 0),
    (torch.bfloat16, 64, 1, 2600011, 0),            # the same for the split kernel
    (torch.bfloat16, 128, 4, 100003, 9000)])
def test_decode_of_very_long_units(kvs, dtype, d, G, rows, wide):
    n = -(-rows // PAGE)
    long_cache(kvs, dtype, d, G, rows, n + 5, 3, wide)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,G", [(64, 1), (64, 8), (128, 2), (128, 4)])
@pytest.mark.parametrize("lens", [[0], [1], [9001], [4100, 33], [0, 2560], [31, 0]])
def test_decode_of_one_or_two_units_with_wide_tables(kvs, dtype, d, G, lens):
    """Several clusters a unit."""
    c = Cache(kvs, 1, len(lens), G, d, lens, dtype, seed=20, room=3, logn_scale=3.0, wide=1100)
    q = c.random(1, len(lens) * G, d, scale=2.0)
    c.check(q, c.step(q))
    assert c.lens.tolist() == lens and np.array_equal(c.pages.cpu().numpy(), c.pages_np)
    for _ in range(3):
        kn, vn = c.random(1, len(lens), d), c.random(1, len(lens), d)
        first = c.step(q)
        assert all(torch.equal(c.step(q), first) for _ in range(5))
        c.check(q, c.step(q, kn, vn), kn, vn)
        c.append(kn, vn)
    assert kvs.device_flags(c.ws) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens", [[1500], [1500, 40]])
def test_table_widths_take_turns_on_one_workspace(kvs, dtype, lens):
    """The same pages through tables of every width, each with its own way to decode, one after
    another: eager steps against the oracle, captured ones against them."""
    def pools(c):
        tables = [i32(np.concatenate([c.table_np, -np.ones((len(lens), n), np.int64)], 1))
                  for n in (0, 1024 - c.table_np.shape[1], 1025 - c.table_np.shape[1], 30000)]
        return [kvs.page_pool(c.pages, t) for t in tables]

    eager, graph = (Cache(kvs, 1, len(lens), 4, 128, lens, dtype, seed=21, room=17) for _ in range(2))
    q, kn, vn = eager.random(1, 4 * len(lens), 128), eager.random(1, len(lens), 128), eager.random(1, len(lens), 128)
    lens0, pages0, at = graph.lens.clone(), graph.pages.clone(), pools(graph)
    outs = [torch.empty_like(q) for _ in at]

    def calls():
        for pool, out in zip(at, outs):
            kvs.page_decode_attn(graph.desc, q, pool, graph.lens, out, graph.ws, kn, vn)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    graph.lens.copy_(lens0)
    graph.pages.copy_(pages0)
    for _ in range(3):
        g.replay()
        for eager.pool, out in zip(pools(eager), outs):
            want = eager.step(q, kn, vn)
            eager.check(q, want, kn, vn)
            eager.append(kn, vn)
            assert torch.equal(out, want)
        assert torch.equal(graph.lens, eager.lens) and torch.equal(graph.pages, eager.pages)
    assert kvs.device_flags(eager.ws) == kvs.device_flags(graph.ws) == 0


def test_pages_past_four_gigabytes(kvs):
    n = 2 ** 32 // kvs.page_bytes(128) + 100
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB of device memory")
    long_cache(kvs, torch.bfloat16, 128, 4, 3001, n, n - 97)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_steps_cross_a_page(kvs, dtype, wide):
    c = Cache(kvs, 1, 4, 4, 128, [0, 30, 31, 61], dtype, seed=5, room=5, wide=wide)
    for _ in range(5):
        q, kn, vn = c.random(1, 16, 128), c.random(1, 4, 128), c.random(1, 4, 128)
        c.check(q, c.step(q, kn, vn), kn, vn)
        c.append(kn, vn)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("qs,ks,vs,ls", [(1, 1, 1e-4, 1), (1, 1, 1e-6, 1), (1, 1, 300., 1), (1, 1, 6e4, 1),
                                         (1e-5, 1, 1, 1), (1e4, 1e-3, 1, 1), (8, 4, 1, 1), (1, 1e-6, 1, 1),
                                         (1e-3, 2e3, 1, 40.)])
def test_decode_over_the_range_of_values(kvs, dtype, qs, ks, vs, ls, wide):
    c = Cache(kvs, 1, 3, 4, 128, [300, 33, 1], dtype, seed=8, k_scale=ks, v_scale=vs, logn_scale=ls, wide=wide)
    q = c.random(1, 12, 128, scale=qs)
    q[0, 5] = 0
    q[0, 6, 1:] = 0
    c.check(q, c.step(q))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,lens", [(128, [3000, 33, 700]), (64, [31, 2049, 64]), (128, [300, 0, 200, 40] * 30)])
@pytest.mark.parametrize("low", [-1e9, -1e30, -1e38, float(np.finfo(np.float32).min) / 2, 1e9])
def test_log_counts_far_from_zero(kvs, dtype, d, lens, low, wide):
    """Units whose rows all have the same one. Logits are within X (log2) of one another, so weights
    relative to equal ones are within 2^(+-2 X), also where X is lost against the log-count; the
    oracle's too: off by at most (2^(4 X) - 1) sum p |v|, and the roundings."""
    c = Cache(kvs, 1, len(lens), 4, d, lens, dtype, seed=22, wide=wide)
    for u, n in enumerate(lens):
        for t in range(n):
            ref.put_logn(c.pages_np, c.slot(u, t), low)
    c.to_device()
    q = c.random(1, 4 * len(lens), d, scale=2.0 ** -14)
    got = c.step(q).double().cpu().numpy().reshape(len(lens), 4, d)
    for u, n in enumerate(lens):
        k, v, _ = ref.rows_of(c.pages_np, c.table_np[u], n, d)
        qu = q.double().cpu().numpy().reshape(len(lens), 4, d)[u]
        want, size = ref.attend(qu, k, v, np.zeros(n))
        x = np.log2(np.e) * (np.abs(qu) @ np.abs(k).T).max(initial=0.0) / np.sqrt(d)
        scales = ref.value_scales(c.pages_np, c.table_np[u], n, d)
        bound = tolerance(dtype, qu, k, v, np.zeros(n), want, size, scales) + (2 ** (4 * x) - 1) * size
        assert np.all(np.abs(got[u] - want) <= bound), (u, float((np.abs(got[u] - want) / bound).max()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_log_counts_of_the_lowest_value_leave_rows_out(kvs, dtype, wide):
    low = float(np.finfo(np.float32).min)
    c = Cache(kvs, 1, 3, 4, 128, [100, 100, 100], dtype, seed=23, wide=wide)
    for u, t in [(0, t) for t in range(100)] + [(1, t) for t in range(99)]:
        ref.put_logn(c.pages_np, c.slot(u, t), low)
    c.to_device()
    q, kn, vn = c.random(1, 12, 128), c.random(1, 3, 128), c.random(1, 3, 128)
    out = c.step(q)
    assert not out[0, :4].any()
    _, v, _ = ref.rows_of(c.pages_np, c.table_np[1], 100, 128)
    assert np.allclose(out[0, 4:8].double().cpu().numpy(), v[99], rtol=2.0 ** -6, atol=1e-30)
    out = c.step(q, kn, vn)                               # nothing but the new row
    assert torch.equal(out[0, :4], vn[0, 0].expand(4, -1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_with_masked_rows(kvs, dtype, wide):
    """Log-counts of -inf or near the type's lowest value take rows out; a unit of nothing but
    -inf is zeros."""
    c = Cache(kvs, 1, 4, 4, 64, [70, 40, 65, 64], dtype, seed=9, wide=wide)
    low = float(np.finfo(np.float32).min)
    for u, t, x in [(0, t, -np.inf) for t in range(0, 70, 3)] + [(1, t, -np.inf) for t in range(40)] + \
            [(2, t, low / 2) for t in range(64)] + [(3, t, -np.inf) for t in range(32)]:
        pg = c.pages_np[c.slot(u, t) // PAGE]
        pg[36 * 64 + 4 * (t % PAGE):][:4] = np.frombuffer(np.float32(x).tobytes(), np.uint8)
    c.to_device()
    q = c.random(1, 16, 64)
    out = c.step(q)
    assert not out[0, 4:8].any()
    got = out.double().cpu().numpy().reshape(4, 4, 64)
    for u in (0, 2, 3):
        k, v, ln = ref.rows_of(c.pages_np, c.table_np[u], int(c.lens_np[u]), 64)
        keep = ln > low / 4
        want, size = ref.attend(q.double().cpu().numpy().reshape(4, 4, 64)[u], k[keep], v[keep], ln[keep])
        scales = ref.value_scales(c.pages_np, c.table_np[u], int(c.lens_np[u]), 64)[keep]
        bound = tolerance(dtype, q.double().cpu().numpy().reshape(4, 4, 64)[u], k[keep], v[keep], ln[keep], want,
                          size, scales)
        assert np.all(np.abs(got[u] - want) <= bound)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nan_stays_in_its_unit_or_query(kvs, dtype, wide):
    c = Cache(kvs, 1, 4, 2, 64, [50, 50, 50, 50], dtype, seed=10, wide=wide)
    pg = c.pages_np[c.slot(1, 40) // PAGE]
    pg[34 * 64 + (1 * 32 + 40 % PAGE) * 2:][:2] = 255                 # value block 1 of one row of unit 1
    pg = c.pages_np[c.slot(3, 7) // PAGE]
    pg[32 * 64 + (7 * 2 + 0) * 2:][:2] = 255                          # a key block of unit 3
    c.to_device()
    q = c.random(1, 8, 64)
    q[0, 0, 9] = float("nan")                                         # query head 0 (unit 0)
    out = c.step(q).float().cpu()
    nan = torch.isnan(out[0])
    assert nan[0].all() and not nan[1].any()
    assert nan[2:4, 32:].all() and not nan[2:4, :32].any()
    assert not nan[4:6].any() and nan[6:8].all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_full_units_and_bad_pages(kvs, dtype, wide):
    c = Cache(kvs, 1, 5, 2, 64, [64, 10, 32, 40, 40], dtype, seed=11, room=0, wide=wide)
    c.table_np[0, 2:] = -1                                   # full: no page for row 64
    c.table_np[2, 1:] = -1
    c.table_np[4, 1] = len(c.pages_np)                       # past the pool: rows 32.. are skipped
    c.lens_np[4] = 32                                        # what the oracle sees of unit 4
    c.to_device()
    c.lens[4] = 40
    q, kn, vn = c.random(1, 10, 64), c.random(1, 5, 64), c.random(1, 5, 64)
    fits = [False, True, False, True, False]
    c.check(q, c.step(q, kn, vn), kn, vn, fits)
    assert kvs.device_flags(c.ws, clear=True) == kvs.FLAG_OUT_CAPACITY | kvs.FLAG_BAD_PAGE
    assert c.lens.tolist() == [64, 11, 32, 41, 40]
    # lengths out of range: zeros, and the length stays
    c.lens.copy_(i32([-3, 11, 32 * c.table.shape[1] + 1, 41, 0]))
    out = c.step(q, kn, vn)
    assert not out[0, :2].any() and not out[0, 4:6].any() and out[0, 2:4].any()
    assert kvs.device_flags(c.ws, clear=True) == kvs.FLAG_BAD_LENGTH
    assert c.lens.tolist() == [-3, 12, 32 * c.table.shape[1] + 1, 42, 1]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_units_share_pages_that_none_appends_to(kvs, dtype, wide):
    c = Cache(kvs, 1, 2, 2, 128, [64, 70], dtype, seed=12, wide=wide)
    c.table_np[0, :2] = c.table_np[1, :2]
    c.to_device()
    q, kn, vn = c.random(1, 4, 128), c.random(1, 2, 128), c.random(1, 2, 128)
    c.check(q, c.step(q, kn, vn), kn, vn)
    c.append(kn, vn)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_same_call_gives_the_same_bits(kvs, dtype, wide):
    c = Cache(kvs, 1, 3, 4, 128, [4000, 1, 333], dtype, seed=13, wide=wide)
    q = c.random(1, 12, 128)
    first = c.step(q)
    for _ in range(20):
        assert torch.equal(c.step(q), first)


def test_captured_steps_replay_like_eager_ones(kvs, wide):
    eager = Cache(kvs, 1, 4, 4, 128, [500, 0, 31, 64], torch.bfloat16, seed=14, room=8, wide=wide)
    graph = Cache(kvs, 1, 4, 4, 128, [500, 0, 31, 64], torch.bfloat16, seed=14, room=8, wide=wide)
    q, kn, vn = eager.random(1, 16, 128), eager.random(1, 4, 128), eager.random(1, 4, 128)
    lens0, pages0 = graph.lens.clone(), graph.pages.clone()
    out = torch.empty_like(q)
    call = lambda: kvs.page_decode_attn(graph.desc, q, graph.pool, graph.lens, out, graph.ws, kn, vn)   # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()
    graph.lens.copy_(lens0)
    graph.pages.copy_(pages0)
    for _ in range(3):
        g.replay()
        eager.step(q, kn, vn)
        want = eager.step(q, kn, vn)
        assert torch.equal(out, want) and torch.equal(graph.lens, eager.lens)
        assert torch.equal(graph.pages, eager.pages)


def test_one_workspace_for_batches_of_any_size(kvs):
    """A workspace of the largest batch serves the smaller ones in between."""
    big = Cache(kvs, 100, 1, 4, 128, [2500 if k % 10 == 9 else k % 40 for k in range(100)], torch.bfloat16,
                seed=24)
    small = Cache(kvs, 4, 5, 4, 128, [90 * k % 1100 for k in range(20)], torch.bfloat16, seed=25, wide=5000)
    one = Cache(kvs, 1, 1, 4, 128, [3000], torch.bfloat16, seed=26, wide=1100)
    qs = [c.random(c.B, 4 * c.H, 128) for c in (big, small, one)]
    wants = [c.step(q) for c, q in zip((big, small, one), qs)]
    small.ws = one.ws = big.ws
    for _ in range(3):
        for c, q, want in zip((small, big, one, big), [qs[i] for i in (1, 0, 2, 0)], [wants[i] for i in (1, 0, 2, 0)]):
            assert torch.equal(c.step(q), want)
    assert kvs.device_flags(big.ws) == 0


def test_tables_of_fewer_units_than_the_workspace_has(kvs):
    units, few, d = 6000, 4500, 64
    g = torch.Generator(device=DEV).manual_seed(27)
    pages = torch.randint(0, 256, (7 * units, kvs.page_bytes(d)), generator=g, device=DEV, dtype=torch.uint8)
    pages[:, 32 * d:36 * d].view(torch.float16)[:] = 1.0
    pages[:, 36 * d:] = 0
    table = torch.arange(7 * units, dtype=torch.int32, device=DEV).view(units, 7)
    pool = kvs.page_pool(pages, table)
    desc = kvs.make_desc(1, units, units, d, 2, torch.bfloat16)
    ws = kvs.workspace(desc, ops=(kvs.OP_PAGES,))
    q = torch.randn(1, units, d, generator=g, device=DEV).to(torch.bfloat16)
    lens, outs = torch.full((units,), 200, dtype=torch.int32, device=DEV), []
    for _ in range(2):
        out = torch.full_like(q, 99.0)
        kvs.page_decode_attn(desc, q, pool, lens, out, ws)
        outs.append(out)
        table2 = torch.full((few, 2), -1, dtype=torch.int32, device=DEV)
        held, free = torch.zeros(few, dtype=torch.int32, device=DEV), torch.arange(9000, dtype=torch.int32, device=DEV)
        n_free = torch.tensor([9000], dtype=torch.int32, device=DEV)
        rows = (torch.arange(few, device=DEV) % 60).to(torch.int32)
        kvs.page_assign(kvs.page_pool(torch.zeros(9000, kvs.page_bytes(d), dtype=torch.uint8, device=DEV), table2),
                        rows, held, free, n_free, ws)
        assert torch.equal(held, (rows + 31) // 32)
    assert torch.equal(*outs) and kvs.device_flags(ws) == 0


def test_two_streams_with_a_workspace_each(kvs):
    a = Cache(kvs, 1, 4, 4, 128, [3000, 5, 70, 1000], torch.bfloat16, seed=15)
    b = Cache(kvs, 2, 2, 4, 128, [10, 2900, 0, 64], torch.bfloat16, seed=16, wide=5000)
    qa, qb = a.random(1, 16, 128), b.random(2, 8, 128)
    want_a, want_b = a.step(qa), b.step(qb)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(30):
        with torch.cuda.stream(sa):
            outs.append((a.step(qa), want_a))
        with torch.cuda.stream(sb):
            outs.append((b.step(qb), want_b))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in outs)


def test_tensors_that_do_not_fit_are_refused(kvs):
    c = Cache(kvs, 1, 2, 2, 64, [10, 20], torch.bfloat16, seed=17)
    q, out = c.random(1, 4, 64), torch.empty(1, 4, 64, dtype=torch.bfloat16, device=DEV)
    bad = [dict(q=q.float()), dict(q=q[:, :2]), dict(lens=c.lens.long()), dict(lens=c.lens.cpu()),
           dict(out=torch.empty(1, 64, 4, dtype=torch.bfloat16, device=DEV).transpose(1, 2)),
           dict(k_new=c.random(1, 2, 64).float()), dict(desc=kvs.make_desc(1, 2, 4, 128, 2, kvs.BF16)),
           dict(desc=kvs.make_desc(1, 3, 6, 64, 2, kvs.BF16))]
    for over in bad:
        a = dict(desc=c.desc, q=q, pool=c.pool, lens=c.lens, out=out, ws=c.ws)
        a.update(over)
        with pytest.raises(ValueError):
            kvs.page_decode_attn(**a)
    for over, status in [(dict(k_new=c.random(1, 2, 64)), 1), (dict(out=q), 5), (dict(ws=c.ws[:256]), 4)]:
        a = dict(desc=c.desc, q=q, pool=c.pool, lens=c.lens, out=out, ws=c.ws)
        a.update(over)
        with pytest.raises(kvs.KvsError) as e:
            kvs.page_decode_attn(**a)
        assert e.value.status == status


# ---------------------------------------------------------------------------
# As they are used together
# ---------------------------------------------------------------------------

def test_merge_store_decode_and_remerge(kvs):
    """A merged cache goes into pages, decode appends to it, the newest segment is read back,
    merged again in place and stored again, and decode goes on over the shorter cache."""
    B, H, G, d, T, W = 2, 2, 4, 128, 512, 16
    rng = np.random.default_rng(20)
    bf = torch.bfloat16
    rand = lambda *s: torch.tensor(rng.standard_normal(s), dtype=torch.float32).to(bf).to(DEV)    # noqa: E731
    desc, units = kvs.make_desc(B, H, H * G, d, T, bf), B * H
    ws = kvs.workspace(desc, W, ops=(kvs.OP_SCORE, kvs.OP_MERGE, kvs.OP_PAGES))
    K, V, Q = rand(B, H, T, d), rand(B, H, T, d), rand(B, H * G, W, d)
    logn, lens = torch.zeros(B, H, T, device=DEV), torch.full((units,), T, dtype=torch.int32, device=DEV)
    cand = torch.full((units,), 8, dtype=torch.int32, device=DEV)
    score, w_b = torch.zeros(B, H, T // 2, device=DEV), torch.zeros(B, H, T // 2, device=DEV)
    Km, Vm, lm, nm = torch.zeros_like(K), torch.zeros_like(V), torch.zeros_like(logn), torch.zeros_like(lens)
    kvs.score_pairs(desc, K, V, logn, lens, cand, W, Q, W, score, w_b, ws)
    kvs.merge_compact(desc, K, V, logn, lens, cand, W, score, w_b,
                      torch.full((B,), H * 300, dtype=torch.int32, device=DEV), kvs.SCOPE_POOLED, T, Km, Vm,
                      lm, nm, ws)
    rows = nm.tolist()                                       # pooled: every head has its own length
    assert sum(rows) == B * H * 300

    # into pages, with room for eight decoded rows
    maxp, n_pages = T // PAGE, units * T // PAGE
    pages = torch.full((n_pages, kvs.page_bytes(d)), 255, dtype=torch.uint8, device=DEV)
    table = torch.full((units, maxp), -1, dtype=torch.int32, device=DEV)
    pool = kvs.page_pool(pages, table)
    held, n_free = torch.zeros(units, dtype=torch.int32, device=DEV), i32([n_pages])
    free = i32(np.arange(n_pages))
    slots = torch.empty(units, T, dtype=torch.int32, device=DEV)
    kvs.page_assign(pool, nm, held, free, n_free, ws, slots)
    kvs.page_store(desc, Km, Vm, lm, slots, pool, ws)
    kvs.page_assign(pool, nm + 8, held, free, n_free, ws)
    c = Cache.__new__(Cache)
    c.kvs, c.B, c.H, c.G, c.d, c.dtype, c.rng = kvs, B, H, G, d, bf, rng
    c.pages, c.table, c.pool, c.lens, c.ws, c.desc = pages, table, pool, nm, ws, desc

    def decode(steps):
        for _ in range(steps):
            c.pages_np, c.table_np = pages.cpu().numpy(), table.cpu().numpy()
            c.lens_np = np.array(nm.tolist())
            q, kn, vn = rand(B, H * G, d), rand(B, H, d), rand(B, H, d)
            c.check(q, c.step(q, kn, vn), kn, vn)
            c.append(kn, vn)

    decode(8)
    # what the pages hold is the merged rows in 4 bits
    for u in range(units):
        k, v, ln = ref.rows_of(c.pages_np, c.table_np[u], rows[u], d)
        at = (u // H, u % H)
        assert np.array_equal(k, ref.held(Km[at][:rows[u]].double().cpu().numpy()))
        assert np.array_equal(v, ref.held(Vm[at][:rows[u]].double().cpu().numpy()))
        assert np.array_equal(ln, lm[at][:rows[u]].double().cpu().numpy())
    # the newest 64 rows of every head: read back, merged to 32 in place, stored again
    S = 64
    start = nm - S
    seg = torch.empty(units, S, dtype=torch.int32, device=DEV)
    kvs.page_assign(pool, nm, held, free, n_free, ws, seg, start)
    sdesc = kvs.make_desc(B, H, H * G, d, S, bf)
    Ks, Vs, ls = torch.zeros(B, H, S, d, dtype=bf, device=DEV), torch.zeros(B, H, S, d, dtype=bf, device=DEV), \
        torch.zeros(B, H, S, device=DEV)
    kvs.page_load(sdesc, pool, seg, Ks, Vs, ls, ws)
    sl = torch.full((units,), S, dtype=torch.int32, device=DEV)
    zero = torch.zeros(units, dtype=torch.int32, device=DEV)
    total = torch.exp(ls.double()).sum()
    kvs.score_pairs(sdesc, Ks, Vs, ls, sl, zero, 0, Q, W, score, w_b, ws)
    kvs.merge_compact(sdesc, Ks, Vs, ls, sl, zero, 0, score, w_b,
                      torch.full((units,), 32, dtype=torch.int32, device=DEV), kvs.SCOPE_HEAD, S, Ks, Vs,
                      ls, sl, ws)
    assert sl.tolist() == [32] * units
    assert torch.allclose(torch.exp(ls[:, :, :32].double()).sum(), total, rtol=1e-5)
    nm.copy_(start + 32)
    kvs.page_assign(pool, nm, held, free, n_free, ws, seg, start)
    kvs.page_store(sdesc, Ks, Vs, ls, seg, pool, ws)
    kvs.page_assign(pool, nm + 3, held, free, n_free, ws)
    decode(3)
    kvs.page_assign(pool, zero, held, free, n_free, ws)      # the batch ends: every page is free again
    assert int(n_free) == n_pages and sorted(free.tolist()) == list(range(n_pages))
    assert kvs.device_flags(ws) == 0
