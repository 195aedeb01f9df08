"""GB300 (sm_103a) fused mixture-of-experts layer forward.

NaN-safe top-k routing, atomic-free permutation by expert, tcgen05/TMEM
grouped GEMMs (TF32, BF16, FP8 e4m3 with [128,128] block scales) with SiLU
and the top-k weighted combine fused into their epilogues, behind the C ABI
in ``include/moe_route.h``; and the decode step around it: block tables, a
paged key-value cache, attention of one new token per request or of a tree of
drafted ones, shared pages, adjusted logits, sampling.
"""
from ._binding import MoeError, MoePlan, lib, moe_plan  # noqa: F401
from .decode import (KVFork, KVStep, TreeAccept, TreeMasks, adjust_logits,  # noqa: F401
                     attn_decode, attn_tree, attn_tree_workspace, attn_workspace, check_word,
                     kv_append, kv_compact, kv_copy_pages, kv_fork, kv_release, kv_step, kv_trim,
                     sample_tokens, tree_accept, tree_masks)
from .ep import ep_forward  # noqa: F401
from .layer import BF16, F32, FP8, SIGMOID, SOFTMAX, MoELayer, route_topk  # noqa: F401

__all__ = ["MoELayer", "MoePlan", "MoeError", "route_topk", "ep_forward", "moe_plan", "lib",
           "KVStep", "kv_step", "kv_release", "kv_append", "attn_decode", "attn_workspace",
           "sample_tokens", "check_word", "TreeMasks", "TreeAccept", "KVFork", "tree_masks",
           "attn_tree", "attn_tree_workspace", "tree_accept", "kv_compact", "kv_copy_pages",
           "kv_fork", "kv_trim", "adjust_logits", "F32", "BF16", "FP8", "SOFTMAX", "SIGMOID"]
