"""GB300-native fused linear cross entropy (FLCE): forward and backward of a language-model
head without materialising the [BT, V] logits, and the operators beside it (token embedding,
residual RMS norm, 8-bit activation checkpoints) with their gradients.

The compute path is the C-ABI library ``libflce.so`` (hand-written sm_103a CUDA); this
package holds its thin ctypes binding (``flce``), the build step (``build``) and the seeded
input generators (``inputs``). Importing the package does not load the library; the first
call into ``flce`` does, and fails loudly if it has not been built.
"""

__all__ = ["flce", "inputs", "build"]
