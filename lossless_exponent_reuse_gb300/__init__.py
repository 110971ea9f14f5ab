"""GB300-native lossless cross-iteration exponent reuse for sharded bf16 weights.

The compute path is libciera (``include/ciera.h``): hand-written sm_103a
kernels behind a C ABI.  ``ciera`` is its thin Python binding,
``allgather.SimulatedAllgather`` drives one plan's device state,
and ``workloads`` makes the seeded synthetic inputs.  ``experts`` holds the
operators of the mixture-of-experts layer whose weights are rebuilt,
``attention`` those of the attention half before it, and ``moe_layer`` runs
them together.  Importing the package does
not load the CUDA library; the first call does, and fails loudly if it cannot.
"""
__all__ = ["ciera", "allgather", "workloads", "experts", "attention",
           "moe_layer"]
