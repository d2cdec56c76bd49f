"""Fused rotate + quantize (FlatQuantV2-style) for B200, sm_100a.

For each token of x[K, M, N]: x'' = P1 . (x . P2), quantized per token to INT4 or per
32-group to FP4 E2M1 with E8M0 scales, by hand-written CUDA kernels behind the C ABI of
include/fq.h (libfq.so, built in-tree). The Python layer marshals arguments only.

Beside it, the 8-bit serving path of a rotated layer: INT8 codes per token and their product
with INT8 weights (int8_matmul), and a paged key / value cache in E4M3 with rotary appending
and attention over it (KVCache).
"""

from .api import (FlatQuant, HostPipeline, KVCache, debug_rotate, int8_device_status, int8_matmul,  # noqa: F401
                  quantize_mx, quantize_mx_static, quantize_per_token)
from ._lib import FQError, load as load_library  # noqa: F401
