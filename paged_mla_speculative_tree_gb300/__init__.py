"""GB300 (sm_103a) MLA tree-verify attention over a paged bf16 latent KV pool.

The compute path is the CUDA library built from ``csrc/`` behind the C ABI in
``include/mla_tree_verify.h`` (verify attention), ``include/mla_tree_ops.h``
(the tree steps around it), ``include/mla_step_ops.h`` (page tables, slot maps,
rotary positions, log probabilities) and ``include/mla_layer_ops.h`` (norms with
the rotation, the per-head products, attention over expanded keys);
``binding`` is its ctypes binding and ``workloads`` draws seeded synthetic
inputs.
"""
from .binding import (MlaPrefill, MlaTreeVerify, MtvError, MtvPlan, RopeScaling, choose_nsplit,  # noqa: F401
                      clear_device_error, head_product, kv_defrag, load, norm_rope_write, page_table_update, plan,
                      prefill_run, prefill_workspace, read_device_error, read_static_device_error, rope_freqs,
                      rope_write, run, run_static, slot_map_build, strerror, token_logprobs, ROPE_HALF,
                      ROPE_INTERLEAVED)
