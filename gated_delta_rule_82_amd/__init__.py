"""MI355X (gfx950) Kimi Delta Attention core: chunkwise forward, decode step and
segment composition, and the softmax attention of the stack's other layers (rotary
positions, forward, backward, the 8-bit cache and its decode step), as hand-written
HIP kernels behind a C ABI (include/kda.h).

`kda` is the ctypes binding; `inputs` draws the seeded synthetic workloads.
The shared library is loaded on first use and never replaced by a fallback.
"""

from . import inputs  # noqa: F401
from .kda import (  # noqa: F401
    FLAGS_DEFAULT, KDAError, attn_bwd, attn_fwd, attn_step, cache_append, chunk_fwd, load,
    new_cache, rotary, rotary_freqs, safe_chunk_size, segment_compose, segment_fixup, step,
    workspace_bytes,
)
