"""The paged decode over long units whose log-counts or values lie far apart, against softmax
attention in 64 bits.

The rows go into the pages by kvs_page_store and come back by kvs_page_load in fp32, where both are
exact (tests/test_gpu_pages.py), so the oracle sees what the pages hold. Everything is batched over
the units on the device: these units are too long for the row-by-row oracle.

Bounds, with A = sum_t p_t |v_t|, n rows, X = max |q k| / sqrt(d) plus the largest log-count that a
row with a weight has:
  both   2 (d + 6) 2^-24 X for the roundings of a logit, n + 16 roundings of the sums and 2^-21 for
         the exponentials, relative to A;
  bf16   2^-11 (A + |out|) for the weights, rounded to half; 15 2^-11 S, S = sum_t p_t s_t, for weight
         times scale, whose error counts on a code u <= 15; below the half range both are off by half
         a subnormal step, 2^-25, the largest weight being at least 2^7: n 2^-32 2 |v| for the
         weights, and n 2^-32 15 U for their products with the scales, which a warp holds in units of
         at most U for each block of channels: 1 for a largest scale of the block in [2^-6, 1), else
         the power of two above that scale (at most twice it); scales far below that unit may leave
         the half range: 7 2^-25 U; and 2^-8 |out| for the output.
"""

import gc
import random

import pytest
import torch

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


class Units:
    """`units` KV heads of T rows each (T even) in shuffled pages, made from fp32 rows."""

    def __init__(self, kvs, units, T, G, d, dtype, seed, k_scale=1.0, v_scale=1.0, wide=0):
        self.kvs, self.units, self.T, self.G, self.d, self.dtype = kvs, units, T, G, d, dtype
        self.gen = torch.Generator(device=DEV).manual_seed(seed)
        self.K = k_scale * self.randn(1, units, T, d)
        self.V = v_scale * self.randn(1, units, T, d)
        self.logn = torch.zeros(1, units, T, device=DEV)
        self.wide = wide

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.gen, device=DEV)

    def store(self):
        kvs, units, T = self.kvs, self.units, self.T
        per = T // PAGE + 1                                   # room for one row more
        self.pages = torch.full((units * per + 3, kvs.page_bytes(self.d)), 255, dtype=torch.uint8, device=DEV)
        order = torch.randperm(units * per, generator=self.gen, device=DEV).to(torch.int32).view(units, per) + 3
        self.table = torch.full((units, per + self.wide), -1, dtype=torch.int32, device=DEV)
        self.table[:, :per] = order
        self.pool = kvs.page_pool(self.pages, self.table)
        t = torch.arange(T, device=DEV)
        slots = (order[:, t // PAGE] * PAGE + t % PAGE).to(torch.int32).view(1, units, T)
        f32 = kvs.make_desc(1, units, units, self.d, T, torch.float32)
        self.desc = kvs.make_desc(1, units, units * self.G, self.d, 2, self.dtype)
        self.ws = kvs.workspace(self.desc, ops=(kvs.OP_PAGES,))
        kvs.page_store(f32, self.K, self.V, self.logn, slots, self.pool, self.ws)
        kvs.page_load(f32, self.pool, slots, self.K, self.V, None, self.ws)
        if not hasattr(self, "lens"):
            self.lens = torch.full((units,), T, dtype=torch.int32, device=DEV)
        return self

    def queries(self, scale):
        return (scale * self.randn(1, self.units * self.G, self.d)).to(self.dtype)

    def decode(self, q, k_new=None, v_new=None):
        out = torch.full_like(q, 99.0)
        self.kvs.page_decode_attn(self.desc, q, self.pool, self.lens, out, self.ws, k_new, v_new)
        assert self.kvs.device_flags(self.ws) == 0
        return out

    def scales(self, u):
        """The scales [T, d / 32] of a unit's values."""
        at = self.table[u, :-(-self.T // PAGE)].long()
        s = self.pages[at, 34 * self.d:36 * self.d].view(torch.float16).view(len(at), -1, PAGE)
        return s.transpose(1, 2).reshape(-1, self.d // 32)[:self.T].double()

    def check(self, q, out, extra=0.0, but=None, lens=None, new=None):
        """`extra`: what log-counts of rows without a weight add to X. `but`: a unit to leave out.
        `lens`: rows of each unit, if not T. `new`: keys and values [units, d] of a row appended."""
        d, worst = self.d, 0.0
        q, out = (x.view(self.units, self.G, d).double() for x in (q, out))
        for u in [u for u in range(self.units) if u != but]:
            T = self.T if lens is None else lens[u]
            keep = self.logn[0, u, :T] * 1.44269504 > -float("inf")
            k, v, ln = (x[0, u, :T][keep].double() for x in (self.K, self.V, self.logn))
            s = self.scales(u)[:T][keep].repeat_interleave(32, 1)
            if new is not None:
                k, v = (torch.cat([x, y[u, None].double()]) for x, y in zip((k, v), new))
                ln, s = torch.cat([ln, ln.new_zeros(1)]), torch.cat([s, s.new_zeros(1, d)])
            if len(k) == 0:
                assert not out[u].any()
                continue
            ln = ln - ln.max()                               # the same softmax, and exact
            w = torch.softmax(q[u] @ k.T / d ** 0.5 + ln, -1)
            want, size = w @ v, w @ v.abs()
            live = w.amax(0) > 0
            x = float((q[u].abs() @ k[live].abs().T).max()) / d ** 0.5 + float(ln[live].abs().max()) + extra
            bound = (2 * (d + 6) * 2.0 ** -24 * x + (T + 16) * 2.0 ** -24 + 2.0 ** -21) * size
            bound += 2.0 ** -24 * want.abs()
            if self.dtype == torch.bfloat16:
                top = s.max(0).values
                unit = torch.where((top >= 2.0 ** -6) & (top < 1), 1.0, 2 * top)
                bound += 2.0 ** -11 * (size + want.abs()) + 15 * 2.0 ** -11 * (w @ s) + 2.0 ** -8 * want.abs()
                bound += T * 2.0 ** -32 * (2 * v.abs().max(0).values + 15 * unit) + 7 * 2.0 ** -25 * unit
            err = (out[u] - want).abs()
            worst = max(worst, float((err / bound).max()))
            assert bool((err <= bound).all()), (u, worst, float((err / want.abs().clamp(min=1e-30)).median()))
        return worst


@pytest.fixture(params=[(8, 0), (8, 5000), (2, 1100), (80, 0)], ids=["cluster", "split", "clusters", "many"])
def shape(request):
    """Units, and columns added to their page tables: each way that a call may be decoded."""
    return request.param


LOW = [-1e4, -1e6, -1e9, -1e30, -1e38]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("low", LOW)
@pytest.mark.parametrize("masked", ["first half", "every other page", "all but the last page", "last half"])
def test_rows_masked_by_a_large_negative_log_count(kvs, dtype, shape, low, masked):
    """Pages of masked rows before, between and after pages of rows that count."""
    units, wide = shape
    T = 16384 + 64 if units * (1 + wide) == 8 else 4096 + 64         # (several pages a warp)
    c = Units(kvs, units, T, 4, 128, dtype, seed=1, wide=wide)
    t = torch.arange(T, device=DEV)
    off = {"first half": t < T // 2, "every other page": t // PAGE % 2 == 0, "all but the last page": t < T - PAGE,
           "last half": t >= T // 2}[masked]
    c.logn[:] = torch.rand(units, T, generator=c.gen, device=DEV)
    c.logn[:, :, off] = low
    c.store()
    q = c.queries(2.0)
    c.check(q, c.decode(q))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_log_counts_that_climb(kvs, dtype, shape):
    """Every page's log-counts above the last one's, by steps that the reference follows and by
    steps that it would be lost against; rows of the last two pages count."""
    units, wide = shape
    T = 64 * PAGE
    for step in (15.0, 600.0, 1000.0, 3e4, 1e7):
        c = Units(kvs, units, T, 2, 64, dtype, seed=2, wide=wide)
        page = torch.arange(T, device=DEV) // PAGE
        c.logn[:] = torch.where(page >= 62, 0.0, (page - 62) * step)
        c.store()
        q = c.queries(2.0)
        # what counts may be up to 1024 log 2 above the log-count that a warp's logits are relative to
        c.check(q, c.decode(q), extra=720.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16])
@pytest.mark.parametrize("low", LOW + [1e6, 1e9, 1e30])
def test_logits_count_beside_a_far_log_count_that_all_rows_have(kvs, dtype, shape, low):
    """Logits of tens: neither lost beside the log-count, nor cut off."""
    units, wide = shape
    c = Units(kvs, units, 4096, 4, 64, dtype, seed=3, wide=wide)
    c.logn[:] = low
    c.store()
    q = c.queries(8.0)
    c.check(q, c.decode(q))


LONG = [(160, 8192, 0), (8, 16384 + 64, 0), (8, 8192, 5000), (2, 30000, 1100)]


def heavy(c, nats):
    """One row in 2048 that many nats above the others."""
    c.logn[:] = torch.where(torch.arange(c.T, device=DEV) % 2048 == 5, nats, 0.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("units,T,wide", LONG, ids=["many", "cluster", "split", "clusters"])
@pytest.mark.parametrize("v_scale", [1e-6, 1e-5, 3e-5, 1e-4, 1e-3, 1e-2, 30.0, 1e3, 6e4])
def test_values_of_every_size(kvs, dtype, units, T, wide, v_scale):
    c = Units(kvs, units, T, 2, 64, dtype, seed=4, v_scale=v_scale, wide=wide)
    heavy(c, 10.0)
    c.store()
    q = c.queries(1.0)
    c.check(q, c.decode(q))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("units,T,wide", LONG, ids=["many", "cluster", "split", "clusters"])
@pytest.mark.parametrize("down", [False, True])
def test_values_whose_size_changes(kvs, dtype, units, T, wide, down):
    """Blocks of channels of their own sizes, two of them growing (or shrinking) along the rows and
    one zero for the first half."""
    c = Units(kvs, units, T, 4, 128, dtype, seed=5, wide=wide)
    ramp = torch.linspace(-20, 14, T, device=DEV)
    ramp = torch.exp2(ramp.flip(0) if down else ramp)[:, None]
    c.V[..., :32] *= ramp
    c.V[..., 32:64] *= 3e-6
    c.V[..., 64:96] *= 2.0 ** -10 * ramp
    c.V[:, :, :T // 2, 96:] = 0
    heavy(c, 10.0)
    c.store()
    q = c.queries(1.0)
    c.check(q, c.decode(q))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("units,T,wide", LONG, ids=["many", "cluster", "split", "clusters"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("low", [-float("inf"), torch.finfo(torch.float32).min])
def test_rows_left_out_may_hold_nan(kvs, dtype, units, T, wide, d, low):
    """Rows with a log-count of -inf (or one whose product with log2 e is) hold NaN or infinite keys
    or values, alone, by pages and, in unit 1, throughout."""
    c = Units(kvs, units, T, 2, d, dtype, seed=6, wide=wide)
    t = torch.arange(T, device=DEV)
    off = [t % 7 == 3, t % 11 == 5, t // PAGE % 5 == 4]
    c.K[:, :, off[0], 1] = float("nan")
    c.V[:, :, off[1], d - 1] = -float("inf")
    c.K[:, :, off[2]] = float("inf")
    c.V[:, :, off[2]] = float("nan")
    gone = off[0] | off[1] | off[2]
    c.K[0, 1, :, 40], c.V[0, 1, :, 3] = float("nan"), float("nan")
    c.logn[:, :, gone] = low
    c.logn[0, 1] = low
    c.store()
    for x in (c.K, c.V):
        x[:, :, gone] = 0                                    # (for the oracle)
    q = c.queries(1.0)
    out = c.decode(q).view(units, 2, d)
    assert not out[1].any()
    c.check(q, out, but=1)


@pytest.mark.parametrize("low", LOW + [1e6, 1e9, 1e30])
def test_fp32_logits_count_beside_a_far_log_count_that_all_rows_have(kvs, shape, low):
    units, wide = shape
    c = Units(kvs, units, 4096, 4, 128, torch.float32, seed=7, wide=wide)
    c.logn[:] = low
    c.store()
    q = c.queries(4.0)
    c.check(q, c.decode(q))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("low", [-3e5, 2e4, -5e6])
def test_far_log_counts_that_differ(kvs, dtype, shape, low):
    """Counts of 1 to 20 beside a common offset: their differences are exact in fp32 and count."""
    units, wide = shape
    c = Units(kvs, units, 4096, 2, 64, dtype, seed=8, wide=wide)
    n = torch.randint(1, 21, c.logn.shape, generator=c.gen, device=DEV)
    c.logn[:] = low + torch.log(n.float())
    c.store()
    q = c.queries(1.0)
    c.check(q, c.decode(q))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("low", [0.0, -1e9, -1e30, 1e30])
def test_large_logits_beside_far_log_counts(kvs, dtype, shape, low):
    """Logits of up to about 80, with masked rows in between and a row appended."""
    units, wide = shape
    c = Units(kvs, units, 4096, 2, 64, dtype, seed=9, wide=wide)
    c.logn[:] = low
    c.logn[:, :, torch.arange(4096, device=DEV) // 64 % 3 == 1] = -2e30
    c.store()
    q = c.queries(18.0)
    c.check(q, c.decode(q))
    kn, vn = c.randn(1, units, 64).to(dtype), c.randn(1, units, 64).to(dtype)
    out = c.decode(q, kn, vn)
    if low < 0:                                              # nothing but the new row
        assert torch.equal(out.view(units, 2, 64), vn[0, :, None].expand(-1, 2, -1))
    elif low > 0:                                            # everything but it
        c.check(q, out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("seed", range(12))
def test_everything_at_once(kvs, dtype, seed):
    """Ragged units, values of a size of their own in every block, far log-counts, masks of several
    kinds with NaN where nothing counts, and a row appended."""
    rng = random.Random(seed)
    units, wide = rng.choice([(1, 1100), (2, 0), (8, 0), (8, 6000), (64, 0), (150, 1100), (310, 0)])
    G, d, T = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), 2 * rng.randint(1, 300000 // units // 2 // 15)
    c = Units(kvs, units, T, G, d, dtype, seed, wide=wide)
    gen, t = c.gen, torch.arange(T, device=DEV)
    for b in range(0, d, 32):
        c.V[..., b:b + 32] *= 10.0 ** rng.uniform(-7, 4.5)
    c.logn[:] = rng.choice([0, 0, -3e5, -1e9, 2e4]) + torch.rand(c.logn.shape, generator=gen, device=DEV)
    for low in rng.sample([-1e4, -1e9, -1e30, -float("inf"), torch.finfo(torch.float32).min], 2):
        off = {"pages": torch.rand(units, T // PAGE + 1, generator=gen, device=DEV).repeat_interleave(PAGE, 1)[:, :T] < .6,
               "rows": torch.rand(units, T, generator=gen, device=DEV) < .5, "head": (t < T // 2).expand(units, T),
               "units": (torch.rand(units, 1, generator=gen, device=DEV) < .3).expand(units, T)}
        c.logn[0][off[rng.choice(list(off))]] = low
    gone = c.logn[0] * 1.44269504 == -float("inf")
    c.K[0][gone & (torch.rand(units, T, generator=gen, device=DEV) < .3)] = float("nan")
    c.V[0][gone & (torch.rand(units, T, generator=gen, device=DEV) < .3)] = float("inf")
    c.lens = torch.randint(0, T + 1, (units,), generator=gen, device=DEV).to(torch.int32)
    lens = c.lens.tolist()
    c.store()
    q = c.queries(rng.choice([0.3, 2.0, 8.0]))
    c.check(q, c.decode(q), lens=lens)
    new = [c.randn(units, d).to(dtype) for _ in range(2)]
    c.check(q, c.decode(q, *new), lens=lens, new=new)
    assert c.lens.tolist() == [n + 1 for n in lens]
