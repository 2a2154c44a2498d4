"""MI355X (gfx950) Kimi Delta Attention core: chunkwise forward, decode step and
segment composition, and the softmax attention of the stack's other layers (rotary
positions, forward, backward, the 8-bit cache and its decode step), as hand-written
HIP kernels behind a C ABI (include/kda.h).  Prompts continued several times (beams,
samples) share cache pages, attend over them once and follow a selection's parents.

`kda` is the ctypes binding; `inputs` draws the seeded synthetic workloads.
The shared library is loaded on first use and never replaced by a fallback.
"""

from . import inputs  # noqa: F401
from .kda import (  # noqa: F401
    FLAGS_DEFAULT, KDAError, attn_bwd, attn_fwd, attn_shared, attn_step, beam_select, cache_append,
    cache_compact, cache_copy, cache_fork, cache_free, cache_reserve, chunk_fwd, load, new_cache,
    rotary, rotary_freqs, safe_chunk_size, segment_compose, segment_fixup, state_reorder, step,
    workspace_bytes,
)
