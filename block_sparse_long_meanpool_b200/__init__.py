"""B200-native MoBA (Mixture of Block Attention): the causal prefill forward and its backward
pass, the decode step with the mean or the min/max block gate, and a paged KV cache in 4 bits.

The compute path is the C-ABI library ``libmoba.so`` (CUDA for sm_100a, headers in
``include/moba.h``); ``moba`` and ``cache`` are its thin ctypes binding and ``workloads`` makes
seeded synthetic inputs.  Build the library with ``python -m block_sparse_long_meanpool_b200.build``.
"""

from .cache import (  # noqa: F401
    KVCache,
    cache_append,
    cache_compact,
    cache_decode,
    cache_fork,
    cache_free,
    cache_reserve,
    cache_status,
)
from .moba import (  # noqa: F401
    MobaError,
    attn_bwd,
    attn_fwd,
    decode_fwd,
    decode_minmax_fwd,
    gate_topk,
    load_library,
    make_params,
    meanpool,
    minmaxpool,
    num_blocks,
    workspace_size,
)
