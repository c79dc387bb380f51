"""Page tables on the GPU: what the free stack should not hold."""

import gc

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")


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
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("bad", [6, 7, 1 << 26, (1 << 27) + 3, 2 ** 31 - 1, -1, -2 ** 31])
def test_slots_of_a_page_outside_the_pool(kvs, bad):
    """Such a page has no slots: 32 times its number may be another page's."""
    pages = torch.zeros(6, kvs.page_bytes(64), dtype=torch.uint8, device=DEV)
    table = torch.full((2, 4), -1, dtype=torch.int32, device=DEV)
    pool, held, n_free = kvs.page_pool(pages, table), i32([0, 0]), i32([6])
    free, slots = i32([0, 1, 2, bad, 4, 5]), torch.empty(2, 70, dtype=torch.int32, device=DEV)
    ws = kvs.workspace(kvs.make_desc(1, 2, 2, 64, 2, kvs.BF16), ops=(kvs.OP_PAGES,))
    rows = [70, 40]                          # three pages and two: 1, 2, bad and 4, 5
    kvs.page_assign(pool, i32(rows), held, free, n_free, ws, slots)
    want = [[32 * p + r for p in (1, 2) for r in range(32)] + [-1] * 6,
            [32 * p + r for p in (4, 5) for r in range(32)][:40] + [-1] * 30]
    assert slots.tolist() == want and held.tolist() == [3, 2] and int(n_free) == 1
    assert kvs.device_flags(ws, clear=True) == (kvs.FLAG_BAD_PAGE if bad >= 0 else 0)
    # the same page held from an earlier call
    slots.fill_(7)
    kvs.page_assign(pool, i32(rows), held, free, n_free, ws, slots)
    assert slots.tolist() == want
    assert kvs.device_flags(ws) == (kvs.FLAG_BAD_PAGE if bad >= 0 else 0)
