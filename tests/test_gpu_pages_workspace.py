"""One workspace for the paged calls of a batch and for every other call of a single sequence, as a
server has them: a new sequence is scored, merged, prefilled or decoded while the batch decodes."""

import gc

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


class Batch:
    """Units of T rows in pages with finite random contents, and a step that appends."""

    def __init__(self, kvs, units, T, G, d, dtype, wide, seed=0):
        self.kvs = kvs
        gen = torch.Generator(device=DEV).manual_seed(seed)
        per = T // PAGE + 1
        self.pages = torch.randint(0, 256, (units * per, kvs.page_bytes(d)), generator=gen, device=DEV, dtype=torch.uint8)
        self.pages[:, 32 * d:36 * d].view(torch.float16)[:] = 0.25
        self.pages[:, 36 * d:] = 0
        self.table = torch.full((units, per + wide), -1, dtype=torch.int32, device=DEV)
        self.table[:, :per] = torch.randperm(units * per, generator=gen, device=DEV).to(torch.int32).view(units, per)
        self.pool = kvs.page_pool(self.pages, self.table)
        self.desc = kvs.make_desc(1, units, units * G, d, 2, dtype)
        self.q = torch.randn(1, units * G, d, generator=gen, device=DEV).to(dtype)
        self.kn, self.vn = (torch.randn(1, units, d, generator=gen, device=DEV).to(dtype) for _ in range(2))
        self.lens0 = torch.full((units,), T, dtype=torch.int32, device=DEV)
        self.lens0[::7] -= T // 3

    def step(self, ws):
        """Output, lengths and pages of a step from the same state every time."""
        lens, pages = self.lens0.clone(), self.pages.clone()
        pool, out = self.kvs.page_pool(pages, self.table), torch.full_like(self.q, 99.0)
        self.kvs.page_decode_attn(self.desc, self.q, pool, lens, out, ws, self.kn, self.vn)
        return out, lens, pages


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("units,T,wide", [(128, 3000, 0), (400, 900, 0), (8, 9000, 6000), (2, 20000, 1100), (1, 20000, 1100)])
def test_calls_of_other_shapes_in_between(kvs, dtype, units, T, wide):
    H, G, d, W, Tc = 8 if units >= 8 else 1, 4, 128, 32, 1024
    batch = Batch(kvs, units, T, G, d, dtype, wide)
    one = kvs.make_desc(1, H, H * G, d, Tc, dtype)
    big = kvs.make_desc(1, units, units * G, d, Tc, dtype)
    ops = (kvs.OP_SCORE, kvs.OP_MERGE, kvs.OP_DECODE, kvs.OP_PREFILL, kvs.OP_PAGES)
    size = max(kvs.workspace_size(big, W, op) for op in (kvs.OP_DECODE, kvs.OP_PAGES))
    size = max([size] + [kvs.workspace_size(one, W, op) for op in ops])
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    want = batch.step(torch.zeros_like(ws))

    g = torch.Generator(device=DEV).manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV).to(dtype)                        # noqa: E731
    K, V, Q, q = rand(1, H, Tc, d), rand(1, H, Tc, d), rand(1, H * G, W, d), rand(1, H * G, d)
    logn, lens = torch.zeros(1, H, Tc, device=DEV), torch.full((H,), Tc - W, dtype=torch.int32, device=DEV)
    cand, target = torch.full((H,), 8, dtype=torch.int32, device=DEV), torch.full((H,), 700, dtype=torch.int32, device=DEV)
    score, w_b = torch.zeros(1, H, Tc // 2, device=DEV), torch.zeros(1, H, Tc // 2, device=DEV)
    Ko, Vo, lo, no = torch.zeros_like(K), torch.zeros_like(V), torch.zeros_like(logn), torch.zeros_like(lens)

    def scored(ws):
        kvs.score_pairs(one, K, V, logn, lens, cand, W, Q, W, score, w_b, ws)
        return score, w_b

    def merged(ws):
        kvs.merge_compact(one, K, V, logn, lens, cand, W, score, w_b, target, kvs.SCOPE_HEAD, Tc, Ko, Vo, lo, no, ws)
        return Ko, Vo, lo, no

    def decoded(ws):
        out = torch.empty_like(q)
        kvs.decode_attn(one, q, K, V, logn, lens, out, ws)
        return (out,)

    def prefilled(ws):
        k, v, ln, n = K.clone(), V.clone(), logn.clone(), lens.clone()
        kvs.prefill_chunk(one, k, v, ln, n, Tc - W, K[:, :, :W].clone(), V[:, :, :W].clone(), Q, W, 900, 32, ws)
        return k[:, :, :900], v[:, :, :900], ln[:, :, :900], n

    for call in (scored, merged, decoded, prefilled):
        fresh = [x.clone() for x in call(torch.zeros_like(ws))]
        for _ in range(2):
            assert all(torch.equal(x, y) for x, y in zip(call(ws), fresh)), call.__name__
            assert all(torch.equal(x, y) for x, y in zip(batch.step(ws), want)), call.__name__
    assert kvs.device_flags(ws) == 0
