"""The binding's own checks of the paged cache's tensors, which come before the
library is asked (so without a GPU)."""
import pytest
import torch

import tensor_transformer_layer_cube_gb300 as t

BF16 = torch.bfloat16


def cache(pages=2, page=16, kv_heads=2, d=64):
    k, v = (torch.zeros(pages, page, kv_heads, d, dtype=BF16) for _ in range(2))
    return t.kv_cache(k, v)


def batch(tokens=3):
    i32 = {"dtype": torch.int32}
    return t.paged_batch(torch.zeros(2, **i32), torch.zeros(1, **i32), torch.zeros(1, 1, **i32), tokens)


@pytest.mark.parametrize("slots", [torch.zeros(3), torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.float64),
                                   torch.zeros(3, dtype=torch.complex64), torch.zeros(2, dtype=torch.int64),
                                   torch.zeros(6, dtype=torch.int64)[::2]])
def test_slots_are_int64_one_for_each_token(slots):
    k = torch.zeros(3, 2, 64, dtype=BF16)
    with pytest.raises(ValueError):
        t.tp3d_paged_store(None, cache(), k, k, slots)


@pytest.mark.parametrize("lse", [torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, 4, dtype=torch.float64),
                                 torch.zeros(3, 4, dtype=BF16), torch.zeros(4, 4), torch.zeros(4, 3).t()])
def test_lse_is_dense_float32(lse):
    q = torch.zeros(3, 4, 64, dtype=BF16)
    with pytest.raises(ValueError):
        t.tp3d_paged_attn(None, cache(), batch(), q, torch.empty_like(q), lse, 1.0, None)


def test_pools_of_integers_are_no_cache_type():
    k = torch.zeros(2, 16, 2, 64, dtype=torch.int64)
    assert t.kv_cache(k, k).dtype not in (t.TP3D_F32, t.TP3D_BF16)
