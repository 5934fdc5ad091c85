"""GB300-native single-GPU MoE layer (router, deterministic dispatch,
tcgen05 grouped-GEMM SwiGLU experts, fixed-order combine, backward, forward
MegaKernel) and its generation-step form (up to 64 tokens in one launch, bf16 or
4-bit weights, with the linear layers beside it) and the ends of a training step (cross
entropy, balance loss, orthogonalised updates) behind a C ABI.  ``moe`` is the ctypes binding; importing this
package does not load the CUDA library."""
from .configs import MoEConfig, ALL, BY_NAME  # noqa: F401
