"""libtpmlp: the tensor-parallel Transformer MLP block (forward and backward)
as hand-written sm_103a CUDA behind a C ABI (include/tpmlp.h).

Modules:
  build    compiles csrc/*.cu into _build/libtpmlp.so with nvcc
  binding  ctypes binding with the C ABI's names (marshalling only)
  block    device buffers for one block and the calls that run it
  linear   the same for one tensor-parallel linear layer (attention projections)
  sp       the sequence-parallel LayerNorm / Dropout sublayer around the block
  fp8      8-bit quantisation with scales per 128, and linear layers on 8-bit operands
  norm     the norms before and after a block with its gate and residual scale
  inputs   seeded synthetic workloads (shared with the tests)

Importing the package does not load the library; importing ``binding`` does,
and fails loudly if it has not been built.
"""
