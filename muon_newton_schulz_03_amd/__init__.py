"""MI355X (gfx950) Muon optimizer step: HIP kernels behind a C ABI, and a thin binding.

``MuonStep`` runs the whole step (momentum, short-side-first Frobenius
normalisation, quintic Newton-Schulz iterations, weight update) in the HIP
library ``libmuon_mi355x.so``; build it with
``python -m muon_newton_schulz_03_amd.build``.  ``embedding_*``,
``layer_norm_*``, ``qk_norm_*`` (with a ``Rotation``) and
``packed_attention_*`` are the forward and backward calls of the operators
that the block around those matrices needs.
"""
from .block import (layer_norm_backward, layer_norm_forward, packed_attention_backward,  # noqa: F401
                    packed_attention_forward)
from .embedding import embedding_backward, embedding_forward  # noqa: F401
from .muon import DEFAULT_COEFFS, MuonStep, describe, version  # noqa: F401
from .qk_norm import Rotation, qk_norm_backward, qk_norm_forward  # noqa: F401
