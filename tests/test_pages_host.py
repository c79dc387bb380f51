"""Host-side checks of the 4-bit paged cache's entry points (no GPU needed: nothing here
launches), and of the oracle the GPU tests use."""

import ctypes

import numpy as np
import pytest

import pages_ref as ref

FAKE = 1 << 40          # aligned fake device addresses: validation never dereferences


def _fake(i, off=0):
    return ctypes.c_void_p(FAKE + i * (1 << 36) + off)


@pytest.fixture(scope="module")
def kvs():
    from asymmetric_kv_merging_b200 import build
    build.build()
    from asymmetric_kv_merging_b200 import kvs as mod
    return mod


def _pool(kvs, **over):
    a = dict(pages=_fake(1), table=_fake(2), n_pages=1000, max_pages=64)
    a.update(over)
    return kvs.PagePool(a["pages"], a["table"], a["n_pages"], a["max_pages"])


def test_page_sizes(kvs):
    assert [kvs.page_bytes(d) for d in (64, 128, 96, 0, -1)] == [2432, 4736, 0, 0, 0]
    assert kvs.PAGE_ROWS == ref.PAGE and ref.page_bytes(128) == 4736
    d = kvs.make_desc(4, 8, 32, 128, 64, kvs.BF16)
    assert kvs.workspace_size(d, 0, kvs.OP_PAGES) % 256 == 0
    assert kvs.workspace_size(d, 0, kvs.OP_PAGES) >= 2 * 256 + 32 * 8
    assert kvs.workspace_size(kvs.make_desc(4, 8, 32, 96, 64, kvs.BF16), 0, kvs.OP_PAGES) == 0


BAD_POOLS = [dict(pages=None), dict(table=None), dict(n_pages=0), dict(max_pages=0), dict(n_pages=-1),
             dict(n_pages=1 << 26), dict(max_pages=1 << 26), dict(pages=_fake(1, 8)),
             dict(table=_fake(2, 2))]


def test_assign_refusals(kvs):
    def call(pool=None, **o):
        a = dict(units=32, rows=_fake(3), held=_fake(4), free=_fake(5), n_free=_fake(6), begin=None,
                 slots=None, stride=0, ws=_fake(9), ws_bytes=1 << 30)
        a.update(o)
        return kvs._lib.kvs_page_assign(ctypes.byref(pool or _pool(kvs)), a["units"], a["rows"], a["held"],
                                        a["free"], a["n_free"], a["begin"], a["slots"], a["stride"],
                                        a["ws"], a["ws_bytes"], None)
    for p in BAD_POOLS:
        assert call(_pool(kvs, **p)) == 1, p
    for o in (dict(units=0), dict(rows=None), dict(held=None), dict(free=None), dict(n_free=None),
              dict(slots=_fake(7), stride=0), dict(slots=_fake(7), stride=-1), dict(rows=_fake(3, 2)),
              dict(slots=_fake(7, 1), stride=4)):
        assert call(**o) == 1, o
    assert kvs._lib.kvs_page_assign(None, 1, _fake(3), _fake(4), _fake(5), _fake(6), None, None, 0, _fake(9),
                                    1 << 30, None) == 1
    for o in (dict(held=_fake(3)), dict(free=_fake(2, 64)), dict(slots=_fake(5), stride=2),
              dict(begin=_fake(7), slots=_fake(7), stride=2), dict(n_free=_fake(4, 4))):
        assert call(**o) == 5, o
    for o in (dict(ws=None), dict(ws=_fake(9, 128)), dict(ws_bytes=512)):
        assert call(**o) == 4, o


@pytest.mark.parametrize("load", [False, True])
def test_store_and_load_refusals(kvs, load):
    def call(desc=None, pool=None, **o):
        a = dict(K=_fake(3), V=_fake(4), logn=_fake(5), slots=_fake(6), ws=_fake(9), ws_bytes=256)
        a.update(o)
        d = ctypes.byref(desc or kvs.make_desc(1, 8, 32, 128, 64, kvs.BF16))
        p = ctypes.byref(pool or _pool(kvs))
        if load:
            return kvs._lib.kvs_page_load(d, p, a["slots"], a["K"], a["V"], a["logn"], a["ws"], a["ws_bytes"], None)
        return kvs._lib.kvs_page_store(d, a["K"], a["V"], a["logn"], a["slots"], p, a["ws"], a["ws_bytes"], None)
    for p in BAD_POOLS:
        assert call(pool=_pool(kvs, **p)) == 1, p
    for o in (dict(K=None), dict(V=None), dict(slots=None), dict(K=_fake(3, 8)), dict(logn=_fake(5, 2))):
        assert call(**o) == 1, o
    assert call(kvs.make_desc(1, 8, 32, 96, 64, kvs.BF16)) == 2
    assert call(kvs.make_desc(1, 8, 32, 128, 64, 3)) == 2
    assert call(kvs.make_desc(1, 8, 32, 128, 63, kvs.BF16)) == 1
    assert call(K=_fake(1)) == 5 and call(slots=_fake(1, 1024)) == 5
    if load:                                    # two outputs may not overlap; two inputs may
        assert call(V=_fake(3)) == 5 and call(logn=_fake(4)) == 5
    assert call(ws=None) == 4 and call(ws_bytes=128) == 4


def test_decode_refusals(kvs):
    def call(desc=None, pool=None, **o):
        a = dict(q=_fake(3), len=_fake(4), kn=None, vn=None, out=_fake(5), ws=_fake(9), ws_bytes=1 << 30)
        a.update(o)
        return kvs._lib.kvs_page_decode_attn(
            ctypes.byref(desc or kvs.make_desc(1, 8, 32, 128, 2, kvs.BF16)), a["q"],
            ctypes.byref(pool or _pool(kvs)), a["len"], a["kn"], a["vn"], a["out"], a["ws"], a["ws_bytes"], None)
    for p in BAD_POOLS:
        assert call(pool=_pool(kvs, **p)) == 1, p
    for o in (dict(q=None), dict(len=None), dict(out=None), dict(kn=_fake(6)), dict(vn=_fake(6)),
              dict(q=_fake(3, 4)), dict(out=_fake(5, 8)), dict(len=_fake(4, 1)),
              dict(kn=_fake(6, 1), vn=_fake(7))):
        assert call(**o) == 1, o
    assert call(kvs.make_desc(1, 8, 24, 128, 2, kvs.BF16)) == 2            # three query heads per KV head
    assert call(kvs.make_desc(1, 8, 32, 32, 2, kvs.BF16)) == 2
    for o in (dict(out=_fake(3)), dict(out=_fake(1)), dict(q=_fake(1)), dict(len=_fake(2)),
              dict(kn=_fake(5), vn=_fake(6)), dict(out=_fake(4, -16))):
        assert call(**o) == 5, o
    assert call(ws=None) == 4 and call(ws_bytes=4096) == 4


def test_oracle_rounds_to_nearest_even_and_bounds_the_error():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 64)) * np.exp(rng.uniform(-12, 12, (200, 1)))
    code, s = ref.quantise(x)
    assert code.min() >= 1 and code.max() <= 15
    step = np.repeat(s.astype(np.float64), 32, 1)
    assert np.all(np.abs(ref.held(x) - x) <= step / 2 * (1 + 1e-12))
    top = np.abs(x).reshape(200, 2, 32).max(-1)
    assert np.all(7 * s.astype(np.float64) >= top)
    lower = np.nextafter(s, np.float16(0)).astype(np.float64)
    assert np.all(7 * lower < top)
    y = np.zeros((1, 64))
    y[0, :8] = [7, .5, 1.5, 2.5, -.5, -1.5, -2.5, 6.5]
    assert ref.held(y)[0, :8].tolist() == [7, 0, 2, 2, 0, -2, -2, 6]
    assert np.isnan(ref.held(np.array([[np.inf] + [1.0] * 31]))).all()


def test_oracle_pages_round_trip():
    rng = np.random.default_rng(1)
    for d in (64, 128):
        pages = np.zeros((2, ref.page_bytes(d)), np.uint8)
        k, v = rng.standard_normal((64, d)), rng.standard_normal((64, d))
        for t in range(64):
            ref.put_row(pages, t, k[t], v[t], t / 3)
        got = ref.rows_of(pages, [0, 1], 64, d)
        assert np.array_equal(got[0], ref.held(k)) and np.array_equal(got[1], ref.held(v))
        assert np.allclose(got[2], np.arange(64) / 3, rtol=1e-7)
        # every byte of a page belongs to exactly one row
        seen = np.zeros(ref.page_bytes(d), int)
        for r in range(32):
            ko, vo, ks, vs, ln = ref._offsets(d, r)
            for o in ko + vo:
                seen[o] += 1
            for o in ks + vs:
                seen[[o, o + 1]] += 1
            seen[ln:ln + 4] += 1
        assert np.all(seen == 1)


def test_accounting_of_pages(kvs):
    from asymmetric_kv_merging_b200 import accounting
    for d in (64, 128):
        assert accounting.page_bytes(d) == kvs.page_bytes(d) == ref.page_bytes(d)
    # 148 bytes a row against 516 at d = 128 in bf16
    assert accounting.page_bytes(128) / 32 == 148
    assert accounting.decode_bytes_per_token(128, 2) == 516
    assert accounting.page_decode_bytes(320, 2, 4, 128, 2) == 320 * 148 + 40 + 2 * (4 + 2048)
    assert accounting.page_store_bytes(64, 64, 4) == 64 * (520 + 76)
