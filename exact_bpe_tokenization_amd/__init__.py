"""MI355X-native exact byte-level BPE tokenization (gfx950 HIP kernels behind a C ABI).

The public entry points mirror include/toktier.h; see ``binding`` for the argument conventions.
"""
from .binding import (EXPORTS, FAMILIES, KERNELS, TOKTIER_CL100K, TOKTIER_DEEPSEEK, TOKTIER_GPT2, TOKTIER_IGNORE_MERGES,
                      TOKTIER_O200K,
                      BucketPlan, HipEvents, Plan, RepairSession, Tokenizer, ToktierError, Vocab, lib, toktier_encode_batch, toktier_encode_batch_spans,
                      toktier_encode_batch_static,
                      toktier_encode_batch_timed, toktier_free_vocab, toktier_last_status, toktier_load_vocab,
                      toktier_load_vocab_ex, toktier_pretokenize_batch, toktier_repair_append,
                      toktier_repair_scratch_bytes, toktier_unicode_table_sha256,
                      toktier_vocab_info, toktier_workspace_bytes, toktier_workspace_bytes_ex)
from .binding import (TOKTIER_BF16, TOKTIER_F16, TOKTIER_F32, TOKTIER_MAX_VOCAB, toktier_cross_entropy,
                      toktier_cross_entropy_backward, toktier_cross_entropy_workspace_bytes, toktier_embed,
                      toktier_embed_backward, toktier_embed_backward_workspace_bytes, toktier_linear_cross_entropy,
                      toktier_linear_cross_entropy_backward, toktier_linear_cross_entropy_workspace_bytes, toktier_sample,
                      toktier_sample_workspace_bytes)
from .binding import (TOKTIER_MAX_LINEAR_DIM, TOKTIER_MAX_LINEAR_ROWS, TOKTIER_MAX_TOP, toktier_distill,
                      toktier_distill_backward, toktier_distill_workspace_bytes, toktier_top_logits,
                      toktier_top_logits_workspace_bytes)

__all__ = ["EXPORTS", "FAMILIES", "KERNELS", "TOKTIER_CL100K", "TOKTIER_DEEPSEEK", "TOKTIER_GPT2", "TOKTIER_IGNORE_MERGES",
           "TOKTIER_O200K",
           "BucketPlan", "HipEvents", "Plan", "RepairSession", "Tokenizer", "ToktierError", "Vocab", "lib", "toktier_encode_batch",
           "toktier_encode_batch_spans", "toktier_encode_batch_static", "toktier_encode_batch_timed", "toktier_free_vocab", "toktier_last_status",
           "toktier_load_vocab", "toktier_load_vocab_ex", "toktier_pretokenize_batch", "toktier_repair_append",
           "toktier_repair_scratch_bytes", "toktier_unicode_table_sha256",
           "toktier_vocab_info", "toktier_workspace_bytes", "toktier_workspace_bytes_ex",
           "TOKTIER_BF16", "TOKTIER_F16", "TOKTIER_F32", "TOKTIER_MAX_VOCAB", "toktier_cross_entropy",
           "toktier_cross_entropy_backward", "toktier_cross_entropy_workspace_bytes", "toktier_embed",
           "toktier_embed_backward", "toktier_embed_backward_workspace_bytes", "toktier_linear_cross_entropy",
           "toktier_linear_cross_entropy_backward", "toktier_linear_cross_entropy_workspace_bytes", "toktier_sample",
           "toktier_sample_workspace_bytes",
           "TOKTIER_MAX_LINEAR_DIM", "TOKTIER_MAX_LINEAR_ROWS", "TOKTIER_MAX_TOP", "toktier_distill",
           "toktier_distill_backward", "toktier_distill_workspace_bytes", "toktier_top_logits",
           "toktier_top_logits_workspace_bytes"]
