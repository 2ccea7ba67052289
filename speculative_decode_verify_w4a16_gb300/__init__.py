"""GB300-native W4A16 speculative-verify hot path.

Exposes the C-ABI library libw4a16sv (CUDA kernels for sm_103a) through a thin
torch-tensor binding:
  quantize, prepack, PackedWeight, linear      -- the W4A16 verify linear
  linear_logits                                -- the lm_head with fused softmax statistics
  spec_accept, spec_accept_prestat,
  spec_accept_node                             -- the speculative accept step
  tree_attention, kv_compact                   -- tree-masked verify attention, accepted-path KV compaction
  KV8Cache, kv8_cache, BlockPlan, kv_block_plan,
  kv8_append, kv8_tree_attention               -- paged 8-bit KV cache: block tables, append, verify attention
  Rope, rope_angles, rope_frequencies, rope    -- rotary positions
  KV16Cache, kv16_cache, kv16_append,
  kv16_attention                               -- paged 16-bit KV cache: append with rotation, causal attention of a
                                                  step's rows (decoding rows, drafts, chunks of prompts)
  token_logprobs, TokenLogprobs                -- log probabilities, entropy and top tokens of logit rows
  check_device_status                          -- device error word
"""
from .api import (KV_BLOCK, BlockPlan, KV16Cache, KV8Cache, PackedWeight, Rope, TokenLogprobs, accept_workspace_bytes,
                  check_device_status, kv16_append, kv16_attention, kv16_attention_workspace_bytes, kv16_cache,
                  kv8_append, kv8_cache, kv8_tree_attention, kv8_tree_attention_workspace_bytes, kv_block_plan,
                  kv_compact, linear, linear_logits, linear_logits_workspace_bytes, linear_noalloc,
                  linear_workspace_bytes, packed_scale_bytes, packed_weight_bytes, prepack, quantize, rope, rope_angles,
                  rope_frequencies, spec_accept, spec_accept_node, spec_accept_prestat, token_logprobs,
                  token_logprobs_workspace_bytes, tree_attention, tree_attention_workspace_bytes, workspace)
from ._lib import LIB_PATH, W4A16Error, lib, status_string

__all__ = [
    "KV_BLOCK", "BlockPlan", "KV16Cache", "KV8Cache", "PackedWeight", "Rope", "TokenLogprobs", "accept_workspace_bytes",
    "check_device_status", "kv16_append", "kv16_attention", "kv16_attention_workspace_bytes", "kv16_cache",
    "kv8_append", "kv8_cache", "kv8_tree_attention", "kv8_tree_attention_workspace_bytes", "kv_block_plan",
    "kv_compact", "linear", "linear_logits", "linear_logits_workspace_bytes", "linear_noalloc",
    "linear_workspace_bytes", "packed_scale_bytes", "packed_weight_bytes", "prepack", "quantize", "rope", "rope_angles",
    "rope_frequencies", "spec_accept", "spec_accept_node", "spec_accept_prestat", "token_logprobs",
    "token_logprobs_workspace_bytes", "tree_attention", "tree_attention_workspace_bytes", "workspace",
    "LIB_PATH", "W4A16Error", "lib", "status_string",
]
