"""libtwell: activation-sparse ReLU-gated FFN with TwELL-packed activations on MI355X (gfx950).

The compute lives in libtwell.so (hand-written HIP kernels behind a C ABI,
declared in include/twell.h); `twell` is its thin ctypes binding and
`autograd` a torch.autograd / nn.Module wrapper of the whole path.
"""
from . import twell  # noqa: F401
from .twell import (BF16, F32, TwellError, TwellFFN, TwellServe, add_rms_norm, add_rms_norm_bwd,  # noqa: F401
                    alloc_hybrid, alloc_pack, alloc_workspace, dequantize_mx4, ffn_bwd, ffn_fwd, gate_pack,
                    gate_pack_fp8, linear_mx4, make_dims, matmul_mx4, n_tiles, pack_preact, quantize_e4m3,
                    quantize_mx4, query_sizes, route_hybrid)
