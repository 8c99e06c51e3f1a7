"""MI355X (gfx950) Muon optimizer step: HIP kernels behind a C ABI, and a thin binding.

``MuonStep`` runs the whole step (momentum, short-side-first Frobenius
normalisation, quintic Newton-Schulz iterations, weight update) in the HIP
library ``libmuon_mi355x.so``; build it with
``python -m muon_newton_schulz_03_amd.build``.  ``layer_norm_*`` and
``packed_attention_*`` are the forward and backward calls of the operators
that the block around those matrices needs.
"""
from .block import (layer_norm_backward, layer_norm_forward, packed_attention_backward,  # noqa: F401
                    packed_attention_forward)
from .muon import DEFAULT_COEFFS, MuonStep, describe, version  # noqa: F401
