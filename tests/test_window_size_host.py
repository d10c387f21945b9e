"""CPU: the workspace-size queries refuse a window or sinks that a C int would
wrap (2^32 would read as no window)."""
import types

import pytest
import torch

from medusa_head_speculative_02_b200 import api

TREE = types.SimpleNamespace(handle=None)


@pytest.mark.parametrize("query", [api.attention_packed_workspace_size,
                                   api.attention_window_workspace_size])
def test_sizes_refuse_what_would_wrap(query):
    for window, sinks in ((2 ** 32, 0), (2 ** 31, 0), (-1, 0), (8, 2 ** 32), (8, -1)):
        with pytest.raises(ValueError, match="window"):
            query(TREE, 1, 4, 4, 128, 64, torch.bfloat16, window, sinks)
    # within range the C query answers (0 for no tree)
    assert query(TREE, 1, 4, 4, 128, 64, torch.bfloat16, 2 ** 31 - 1, 2 ** 31 - 1) == 0
