"""GB300-native (sm_103a) routed-MoE feed-forward block of a DiffusionGemma
layer: router + top-k, token->expert grouping, grouped tcgen05 GEMMs with
fused GEGLU and weighted combine, dense branch, norm sandwich and residual.

Beside it the attention half: rotary positions, a paged key/value cache with
its page operations, and attention of a chunk of new tokens over that cache.

The compute runs in ``lib/libdgmoe.so`` (built by :func:`build`) behind the C
ABI of ``include/dg_moe.h`` and ``include/dg_attn.h``; this package is its
Python binding.
"""

from .build import build, LIB  # noqa: F401
from . import binding  # noqa: F401
from .binding import DgError, load_library  # noqa: F401


def __getattr__(name):
    # the torch-level holder imports torch lazily
    if name in ("MoEBlock", "ScMlp", "params_to_device"):
        from . import block
        return getattr(block, name)
    if name in ("Rope", "KvBatch", "KvCache", "KvFork", "KvPager", "PagedAttention"):
        from . import attention
        return getattr(attention, name)
    raise AttributeError(name)
