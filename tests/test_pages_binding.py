"""Errors of the paged calls' Python binding that need no device."""

import pytest


@pytest.fixture(scope="module")
def kvs():
    from asymmetric_kv_merging_b200 import build
    build.build()
    from asymmetric_kv_merging_b200 import kvs as mod
    return mod


@pytest.mark.parametrize("code", [-1, 2, 99])
def test_a_descriptor_of_a_type_that_is_not_built_is_refused(kvs, code):
    desc = kvs.make_desc(1, 2, 4, 64, 64, code)
    for call in (lambda: kvs.page_store(desc, None, None, None, None, None, None),
                 lambda: kvs.page_load(desc, None, None, None, None, None, None),
                 lambda: kvs.page_decode_attn(desc, None, None, None, None, None)):
        with pytest.raises(kvs.KvsError) as e:
            call()
        assert e.value.status == 2
