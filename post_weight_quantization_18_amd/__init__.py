"""MI355X (gfx950) GPTQ layer-quantization hot path.

The kernels live in libgptq_mi355x.so (C ABI in include/gptq.h); this package
holds the in-tree build script, a ctypes binding with the same entry-point
names, and the seeded synthetic layer generator.
"""

from . import synthetic  # noqa: F401
from .gptq import (accumulate_hessian, kv_append, kv_evict, load_library, pack_codes,  # noqa: F401
                   paged_attention, paged_prefill, prepare_hinv, quantize, quantize_layer, workspace_bytes)
