"""The binding's checks of the rotation's tables: where they lie, and that they hold what is written to them."""
import pytest
import torch

import tensor_transformer_layer_cube_gb300 as t

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    t.build()


@pytest.mark.parametrize("bad", [torch.zeros(31, dtype=torch.int64), torch.zeros(32, dtype=torch.int32), torch.zeros(32),
                                 torch.zeros(64, dtype=torch.int64)[::2],
                                 torch.empty(32, dtype=torch.int64, device="meta")])
def test_turns_are_written_to_words_that_hold_them(bad):
    with pytest.raises(ValueError):
        t.tp3d_rope_turns(64, 10000.0, t.TP3D_ROPE_PLAIN, 1.0, 1.0, bad)


def test_turns_of_a_longer_tensor_and_refusals_of_the_library():
    words = torch.full((40,), -5, dtype=torch.int64)
    assert t.tp3d_rope_turns(64, 10000.0, t.TP3D_ROPE_PLAIN, 1.0, 1.0, words) == (0, 1.0)
    assert bool((words[:32] > 0).all()) and bool((words[32:] == -5).all())
    assert t.tp3d_rope_turns(64, 10000.0, t.TP3D_ROPE_PLAIN, 1.0, 1.0, None)[0] == 1
    assert t.tp3d_rope_turns(-2, 10000.0, t.TP3D_ROPE_PLAIN, 1.0, 1.0, words)[0] == 2


class OnDevice(torch.Tensor):
    """A host tensor that says it lies on the device, for what is looked at before anything is launched."""

    @property
    def is_cuda(self):
        return True


def calls(rope):
    q, k, pos = torch.zeros(3, 4, 64, dtype=BF16), torch.zeros(3, 2, 64, dtype=BF16), torch.zeros(3, dtype=torch.int32)
    pool = torch.zeros(2, 16, 2, 64, dtype=BF16)
    cache, slots = t.kv_cache(pool, torch.zeros_like(pool)), torch.zeros(3, dtype=torch.int64)
    # (no context: the library would refuse the call with a status)
    yield lambda: t.tp3d_qk_rope(None, rope, q, k, pos, q, k, stream=0)
    yield lambda: t.tp3d_qk_rope_bwd(None, rope, q, k, pos, q, k, q, k, None, None, None, stream=0)
    yield lambda: t.tp3d_paged_rope_store(None, rope, cache, q, k, k, pos, slots, q, stream=0)


def test_tables_on_the_host_are_refused():
    turns, _ = t.rope_turns(64)
    there, w = turns.as_subclass(OnDevice), torch.ones(64, dtype=BF16)
    on_device = w.as_subclass(OnDevice)
    for rope in (t.rope(turns, BF16, 64, 64), t.rope(there, BF16, 64, 64, norm=True, q_weight=w),
                 t.rope(there, BF16, 64, 64, norm=True, q_weight=on_device, k_weight=w)):
        for call in calls(rope):
            with pytest.raises(TypeError):
                call()


def test_tables_that_are_not_used_may_lie_anywhere():
    turns, _ = t.rope_turns(64)
    there, w = turns.as_subclass(OnDevice), torch.ones(64, dtype=BF16)
    on_device = w.as_subclass(OnDevice)
    for rope in (t.rope(turns, BF16, 64, 0, norm=True, q_weight=on_device), t.rope(None, BF16, 64, 0),
                 t.rope(there, BF16, 64, 64, q_weight=w, k_weight=w), t.tp3d_rope()):
        assert not rope.on_host
    for call in calls(t.rope(there, BF16, 64, 64)):
        assert call() == 1
