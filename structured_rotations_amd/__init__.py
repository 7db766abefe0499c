"""HARP / randomized-Hadamard apply path for MI355X (gfx950).

The compute lives in libharp.so (C ABI: include/harp.h); `api` is its Python
binding, `q8` that of the 8-bit operators (coded rows and weights, the norm
with 8-bit output and its backward pass, products of coded matrices), `kv4`
that of attention over a 4-bit cache (norm, position and rotation of heads with
their backward pass, the cache, attention over it).  `inputs` and `workloads`
draw seeded synthetic inputs.
"""
from .api import (  # noqa: F401
    harp_apply, harp_apply_decode, harp_apply_decode_workspace, harp_apply_inverse, harp_apply_vjp,
    harp_apply_vjp_workspace, harp_theta_vjp, harp_block_count, harp_gauss_count, harp_group_count,
    harp_materialize_blocks, harp_materialize_blocks_q8, harp_quantize_theta, harp_rotate_weight, harp_rotate_weight_workspace, harp_theta_count,
    rht_compose,
)
from .q8 import (  # noqa: F401
    RmsnormQ8, harp_matmul_q8, harp_matmul_q8_wgrad, harp_matmul_q8_wgrad_workspace, harp_matmul_q8_workspace,
    harp_quantize_q8, harp_rmsnorm_q8, harp_rmsnorm_q8_vjp, harp_rmsnorm_q8_vjp_workspace,
)
from .kv4 import (  # noqa: F401
    Cache4, QkGrads, harp_kv4_attention, harp_kv4_attention_workspace, harp_kv4_cache, harp_kv4_read, harp_kv4_write,
    harp_qk_norm_rope, harp_qk_norm_rope_vjp, harp_qk_norm_rope_vjp_workspace,
)

__version__ = "0.1.0"
