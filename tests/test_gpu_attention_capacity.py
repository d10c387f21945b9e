"""Capacities whose slots would not fit 31 bits once rounded up to whole tiles
are refused by the windowed and the 4-bit attention on the host; no launch is
made (the arrays behind these calls are small)."""
import pytest
import torch

from medusa_head_speculative_02_b200 import _lib as L
from medusa_head_speculative_02_b200 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dh,dtype", [(64, L.BF16), (128, L.BF16), (64, L.F32)])
@pytest.mark.parametrize("lcap", [2 ** 31 - 4, 2 ** 31 - 1024])
def test_capacities_past_31_bits_are_refused(lcap, dh, dtype):
    tree, lib = api.Tree(1, 1, 1), L.lib()
    buf = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    p = buf.data_ptr()
    shape = (1, 2, 1, dh, lcap)
    for rc in (lib.medusa_tree_attention_packed(p, p, p, p, p, p, tree.handle, *shape, 0.1, dtype,
                                                0, 0, p, p, buf.numel(), None),
               lib.medusa_tree_attention_window(p, p, p, p, tree.handle, *shape, 0.1, dtype, 8, 0,
                                                p, p, buf.numel(), None)):
        assert rc == L.ERR_UNSUPPORTED and b"2^31" in lib.medusa_last_error()
    tdt = torch.float32 if dtype == L.F32 else torch.bfloat16
    assert api.attention_packed_workspace_size(tree, *shape, tdt) == 0
    # the last one that fits has a plan
    assert api.attention_packed_workspace_size(tree, *shape[:4], 2 ** 31 - 1028, tdt) > 0
    torch.cuda.synchronize()
    assert api.device_status() == 0
