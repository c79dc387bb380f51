"""The README's Python example as it stands there, block by block."""

import gc
import os
import re

import numpy as np
import pytest
import torch

import pages_ref as ref

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_the_example_runs_and_keeps_every_row():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from asymmetric_kv_merging_b200 import build
    build.build()
    from asymmetric_kv_merging_b200 import kvs
    blocks = re.findall(r"```python\n(.*?)```", open(README, encoding="utf-8").read(), re.S)
    assert len(blocks) == 2
    # what the example takes as given
    g = torch.Generator(device="cuda").manual_seed(0)
    B, H, d, T_cap, W, T = 1, 8, 128, 32896, 32, 1200
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)            # noqa: E731
    full = lambda x, *s: torch.full(s, x, dtype=torch.int32, device="cuda")                     # noqa: E731
    env = dict(K=rand(B, H, T_cap, d), V=rand(B, H, T_cap, d), logn=torch.zeros(B, H, T_cap, device="cuda"),
               lens=full(T, H), cand_begin=full(32, H), Q_win=rand(B, 4 * H, W, d), target=full(700, H), T_cap_out=768,
               score=torch.zeros(B, H, T_cap // 2, device="cuda"), w_b=torch.zeros(B, H, T_cap // 2, device="cuda"),
               K2=rand(B, H, 768, d), V2=rand(B, H, 768, d), logn2=torch.ones(B, H, 768, device="cuda"), lens2=full(0, H),
               q=rand(B, 4 * H, d), k_new=rand(B, H, d), v_new=rand(B, H, d), out=rand(B, 4 * H, d),
               desc_out=kvs.make_desc(B, H, 4 * H, d, 768, torch.bfloat16))
    exec(blocks[0], env)
    assert env["lens2"].tolist() == [701] * H                   # merged to 700, and one row appended
    K, V = env["K2"].clone(), env["V2"].clone()
    env.update(units=H, n_pages=H * 26, max_pages=26)
    env["K2"].fill_(99), env["V2"].fill_(99)
    exec(blocks[1].replace("kvs.page_store(desc_out, K2, V2", "kvs.page_store(desc_out, K2_, V2_"), env | dict(K2_=K, V2_=V))
    assert env["lens2"].tolist() == [702] * H
    for got, x, new in ((env["K2"], K, env["k_new"]), (env["V2"], V, env["v_new"])):
        x[:, :, 701] = new
        want = torch.tensor(ref.held(x[:, :, :702].double().cpu().numpy())).float().to(torch.bfloat16)
        assert torch.equal(got[:, :, :702].cpu(), want)
    assert np.all(env["logn2"][:, :, 701].cpu().numpy() == 0) and kvs.device_flags(env["ws"]) == 0
    env.clear()
    gc.collect()
    torch.cuda.empty_cache()             # later tests watch the device's free memory
