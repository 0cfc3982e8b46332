"""GB300-native (sm_103a) Compressed Sparse Attention hot path.

The library is the C ABI in include/csa.h, include/csa_serve.h and
include/csa_rows.h, built as libcsa.so next to this file.  ``csa``, ``serve``
(the quantised cache and the single-token calls) and ``rows`` (norms, rotary
positions, the compressor of new tokens) are its Python binding (same function names);
``inputs`` holds the seeded synthetic workloads.  Importing the package does not load the
library; the first call does, and raises if it is missing.
"""
from .csa import (csa_attn_bwd, csa_attn_fwd, csa_compress, csa_compress_bwd,  # noqa: F401
                  csa_compress_overlap, csa_compress_overlap_bwd,
                  csa_get_device_status, csa_indexer_loss, csa_indexer_teacher, csa_indexer_topk,
                  csa_indexer_topk_fp8, csa_indexer_topk_workspace_size, csa_quantize_e4m3, load_library, CSAError)
from .serve import (csa_attn_decode, csa_attn_decode_workspace_size, csa_cache_page_bytes,  # noqa: F401
                    csa_cache_read, csa_cache_write, csa_indexer_topk_decode,
                    csa_indexer_topk_decode_workspace_size)
from .rows import (CSA_NORM_LAYER, CSA_NORM_RMS, CsaRope, csa_compress_decode, csa_norm,  # noqa: F401
                   csa_norm_bwd, csa_norm_bwd_workspace_size, csa_norm_rope, csa_norm_rope_bwd,
                   csa_rope, csa_rope_bwd, csa_rope_freqs, csa_rope_turns)
