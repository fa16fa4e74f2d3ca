"""Positions behind shared prefixes belong to one step of the cache (on the host: torch alone)."""
import types

import pytest
import torch

from speculative_decoding_draft_04_gb300 import _lib, engine


def cache_of():
    """Three requests and two holders of 7 and 4 tokens; 2, 0 and 3 new rows, room for seven."""
    i32 = torch.int32
    return types.SimpleNamespace(steps=1, row_ptr=torch.tensor([0, 2, 2, 5, 5, 5], dtype=i32),
                                 kv_len=torch.tensor([2, 5, 9, 7, 4], dtype=i32),
                                 positions=torch.tensor([0, 1, 6, 7, 8, -1, -1], dtype=i32))


def prefixes_of():
    return engine.Prefixes(requests=3, group_ptr=torch.tensor([0, 1, 3], dtype=torch.int32),
                           group=torch.tensor([0, 1, 1]), positions=torch.zeros(7, dtype=torch.int32), workspace=None)


def attend(c, s, rotary=True):
    x = torch.zeros((5, 2, 64))
    engine.attend(c, 0, x, x, x, x, rotary=engine.Rotary(rope=None) if rotary else None, prefixes=s)


def test_positions_count_the_prefix():
    c, s = cache_of(), prefixes_of()
    engine.place_after(c, s)
    assert s.positions.tolist() == [7, 8, 10, 11, 12, -1, -1] and s.placed == 1


def test_positions_of_another_step_are_refused(monkeypatch):
    c, s = cache_of(), prefixes_of()
    calls = []
    c.slots, c.layers, c.k_scale, c.v_scale, c.status = torch.zeros(7), [None], [1.0], [1.0], None
    c.block_table, c.softmax_scale = torch.zeros((5, 1)), 1.0
    for name in ("spec_rotary_append", "spec_cache_append", "spec_prefix_attention"):
        monkeypatch.setattr(_lib, name, lambda *a, name=name, **kw: calls.append(name))
    with pytest.raises(_lib.SpecError, match="place_after"):
        attend(c, s)                                         # never placed
    engine.place_after(c, s)
    attend(c, s)
    c.steps += 1                                             # as make_room does
    with pytest.raises(_lib.SpecError, match="place_after"):
        attend(c, s)
    assert calls == ["spec_rotary_append", "spec_prefix_attention"]
    attend(c, s, rotary=False)                               # needs no positions
    assert calls[2:] == ["spec_cache_append", "spec_prefix_attention"]


def test_every_step_counts(monkeypatch):
    c = types.SimpleNamespace(newest=0, steps=0, seq_len=[0, 0], num_blocks=[0, 0], ring_pos=[0, 0], free_ring=0,
                              block_table=0, kv_len=0, row_ptr=0, slots=0, positions=0, status=0, page_size=16)
    monkeypatch.setattr(_lib, "spec_block_tables", lambda *a, **kw: None)
    for _ in range(3):
        engine.make_room(c, None)
    assert (c.steps, c.newest) == (3, 1)
