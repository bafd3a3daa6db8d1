"""MI355X-native Kimi Delta Attention (KDA) multi-token recurrent prefill.

``prefill`` runs the chunked KDA recurrence in libkda's HIP kernels for gfx950
(the library's C ABI is declared in include/kda.h); ``decode`` advances
requests held in a state pool by a few tokens, and ``decode_verify`` then
``decode_commit`` or ``decode_advance`` do the same for speculative drafts,
keeping the state of the accepted prefix.  Around a recurrent-state layer
(include/kda_ssm.h): ``conv_prefill`` and ``conv_decode``, the short causal
convolution; ``ssm_prefill`` and ``ssm_decode``, the selective state space
scan; ``add_rmsnorm``, the residual RMS norm with an optional 8-bit output.
The submodule ``attn`` (include/kda_attn.h) has the softmax attention of the
layers between recurrent ones: ``attn.prefill`` over prompts, ``attn.decode``
over a paged cache, ``attn.store`` and ``attn.assign_pages``, which fill it.
``synth`` draws the
seeded synthetic workloads used by the tests and the benchmark.
"""
from . import attn
from .ops import (DecodeProblem, KDAError, Problem, decode, decode_advance, decode_advance_raw,
                  decode_commit, decode_commit_raw, decode_raw, decode_validate_raw, decode_verify,
                  decode_verify_raw,
                  load_library, library_path, make_decode_problem, make_problem, periodic_offsets,
                  plan, prefill, prefill_noalloc_raw, prefill_raw, validate_raw,
                  workspace_size)
from .ssm_ops import (ConvDecodeProblem, ConvProblem, NormProblem, SsmDecodeProblem, SsmProblem, add_rmsnorm,
                      conv_decode, conv_prefill, ssm_decode, ssm_plan, ssm_prefill, ssm_workspace_size)

__all__ = ["DecodeProblem", "KDAError", "Problem", "decode", "decode_advance", "decode_advance_raw",
           "decode_commit", "decode_commit_raw", "decode_raw", "decode_validate_raw", "decode_verify",
           "decode_verify_raw",
           "load_library", "library_path", "make_decode_problem", "make_problem",
           "periodic_offsets", "plan", "prefill", "prefill_noalloc_raw", "prefill_raw",
           "validate_raw", "workspace_size",
           "ConvDecodeProblem", "ConvProblem", "NormProblem", "SsmDecodeProblem", "SsmProblem",
           "add_rmsnorm", "conv_decode", "conv_prefill", "ssm_decode", "ssm_plan", "ssm_prefill",
           "ssm_workspace_size", "attn"]
