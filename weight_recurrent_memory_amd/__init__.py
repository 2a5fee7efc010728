"""Falcon fast-weight attention on MI355X (gfx950): HIP kernels behind a C ABI.

The compute lives in ``libfalcon.so`` and ``libfalcon_block.so`` (built from
``csrc/``); this package only marshals torch tensors into their C entry points.
Importing the package does not load a library; the first call does, and fails loudly
if it is missing.
"""
from .binding import (  # noqa: F401
    FALCON_1, FALCON_2, FALCON_3, FALCON_1A, FALCON_2A, FALCON_3A,
    VARIANT_NAMES, FalconError, bwd_chunk, bwd_chunk_noalloc, decode_step, fwd_chunk,
    fwd_masked, fwd_recurrent, library_path, load_library,
)
from .delta import (  # noqa: F401
    gated_delta_bwd_chunk, gated_delta_decode_step, gated_delta_fwd_chunk,
)
from .gated import gated_bwd_chunk, gated_decode_step, gated_fwd_chunk  # noqa: F401
from .norms import norm_in, norm_in_bwd, norm_out, norm_out_bwd  # noqa: F401
from .rotary import rotary_frequencies, rotary_in, rotary_in_bwd  # noqa: F401
