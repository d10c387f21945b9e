"""B200-native Medusa draft-and-verify step: CUDA kernels (sm_100a) behind a
C ABI (include/medusa.h), with a thin PyTorch binding in ``api``."""
from .api import (PackedCache, Tree, device_status, medusa_accept_greedy,  # noqa: F401
                  medusa_accept_typical, medusa_build_tree, medusa_heads_forward,
                  medusa_kv_compact, medusa_kv_compact_packed, medusa_kv_pack, medusa_kv_unpack,
                  medusa_topk, medusa_tree_attention, medusa_tree_attention_packed,
                  medusa_tree_attention_window, tree_plan_host, version)
