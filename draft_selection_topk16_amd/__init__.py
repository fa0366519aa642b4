"""MI355X (gfx950) DFlash 2 path selector.

The compute path is the HIP library libdflash2.so (C ABI: include/dflash2.h);
`binding` marshals torch tensors into it, `target` those of the target's side
(paged cache, attention over it, verification of drafts), `fp4` a cache of 4-bit values, `steps` what stands between
its steps (pages of the next one, penalties and masks on rows).  `synth` draws seeded synthetic
inputs.  Importing the package does not load the library: the first call
does, and raises if it has not been built.
"""
from .binding import (PreparedSelect, SelectorError, conv2, device_error, draft_rows, lmhead_topk, load,
                      pair_scores, philox_uniforms, philox_uniforms_next, plan,
                      plan_override, project, release, sample_walk, select, select_sample, topk, version,
                      viterbi, walk)
from .fp4 import (PreparedAppendFp4, PreparedAttentionFp4, PreparedUnpackFp4, fp4_cache, fp4_page_bytes,
                  kv_append_fp4, kv_unpack_fp4, paged_attention_fp4)
from .steps import PreparedAdjust, PreparedPages, adjust_logits, plan_pages
from .target import (PreparedAppend, PreparedAttention, PreparedVerify, kv_append, paged_attention, rope_freqs,
                     verify)

__all__ = ["PreparedAdjust", "PreparedAppend", "PreparedAppendFp4", "PreparedAttention", "PreparedAttentionFp4", "PreparedPages",
           "PreparedSelect", "PreparedUnpackFp4", "PreparedVerify", "SelectorError", "adjust_logits", "conv2",
           "device_error", "draft_rows", "fp4_cache", "fp4_page_bytes", "kv_append", "kv_append_fp4", "kv_unpack_fp4",
           "lmhead_topk", "load", "paged_attention", "paged_attention_fp4", "rope_freqs", "verify",
           "pair_scores", "philox_uniforms", "philox_uniforms_next", "plan",
           "plan_override", "plan_pages", "project", "release", "sample_walk", "select", "select_sample", "topk", "version",
           "viterbi", "walk"]
