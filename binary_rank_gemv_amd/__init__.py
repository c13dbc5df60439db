"""MI355X (gfx950) implementation of the LittleBit factored binary linear layer.

The compute path lives in ``csrc/`` (HIP kernels behind a C ABI, built into
``_lib/liblittlebit.so``); ``littlebit`` is the thin ctypes binding over that
ABI.  ``head`` binds the dense operators around the layers (the residual norm,
the 8-bit product, the token log probabilities; ``_lib/liblittlebit_head.so``),
``attn`` what lies between a block's projections (head norm and rotation, a
paged cache, the attention over it; ``_lib/liblittlebit_attn.so``).
``synth`` draws seeded synthetic inputs.  Importing the package does not load
the shared libraries; ``binary_rank_gemv_amd.littlebit``, ``.head`` and
``.attn`` do, and raise if theirs has not been built.
"""

__all__ = ["attn", "head", "littlebit", "synth"]
