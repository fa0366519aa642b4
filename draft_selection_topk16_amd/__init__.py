"""MI355X (gfx950) DFlash 2 path selector.

The compute path is the HIP library libdflash2.so (C ABI: include/dflash2.h);
`binding` marshals torch tensors into it, `target` those of the target's side
(paged cache, attention over it, verification of drafts).  `synth` draws seeded synthetic
inputs.  Importing the package does not load the library: the first call
does, and raises if it has not been built.
"""
from .binding import (PreparedSelect, SelectorError, conv2, device_error, draft_rows, lmhead_topk, load,
                      pair_scores, philox_uniforms, philox_uniforms_next, plan,
                      plan_override, project, release, sample_walk, select, select_sample, topk, version,
                      viterbi, walk)
from .target import (PreparedAppend, PreparedAttention, PreparedVerify, kv_append, paged_attention, rope_freqs,
                     verify)

__all__ = ["PreparedAppend", "PreparedAttention", "PreparedSelect", "PreparedVerify", "SelectorError", "conv2",
           "device_error", "draft_rows", "kv_append", "lmhead_topk", "load", "paged_attention", "rope_freqs", "verify",
           "pair_scores", "philox_uniforms", "philox_uniforms_next", "plan",
           "plan_override", "project", "release", "sample_walk", "select", "select_sample", "topk", "version",
           "viterbi", "walk"]
