"""B200 (sm_100a) HSTU layer forward, M-FALCON scoring and a paged history cache
behind a C ABI.

The CUDA library (libhstu.so, built by `build.py`) does all the arithmetic;
`hstu` is its ctypes binding.
"""
from . import hstu  # noqa: F401
from .hstu import (HSTUError, Jagged, LayerConfig, LayerWeights, PagedCache,  # noqa: F401
                   attn_fwd, extend, forward, layer_fwd, mfalcon_score, paged_attn_fwd)
