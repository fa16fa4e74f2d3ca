"""What engine.Prefixes refuses before anything is on a device."""
import types

import pytest
import torch

from speculative_decoding_draft_04_gb300 import _lib, engine


@pytest.mark.parametrize("requests,sizes", [(4, [2, 1]), (2, [0, 0]), (0, []), (3, [3, -1])])
def test_groups_that_do_not_fit_the_cache(requests, sizes):
    c = types.SimpleNamespace(kv_len=torch.zeros(requests, dtype=torch.int32))
    with pytest.raises(_lib.SpecError):
        engine.Prefixes.allocate(c, sizes, 8)
