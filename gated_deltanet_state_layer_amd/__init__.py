"""MI355X-native Gated DeltaNet state layer: a slot pool with multi-slot
decode, speculative verify (one call, or over a ring of committed tokens)
and chunked prefill, the norms around the layer and projections with 4-bit
weights, run by the HIP kernels of
libgdn.so (see include/gdn.h) through a thin ctypes binding."""
from .binding import (  # noqa: F401
    GDN_BF16, GDN_F32, GDN_GROUP_KERNEL, GDN_VALIDATE, GdnError, Pool, PoolDesc, block_norm, load_library,
    make_desc, mx_dequantize, mx_proj, mx_proj_workspace_bytes, mx_quantize, pool_bytes, ring_layout,
    status_string,
)
