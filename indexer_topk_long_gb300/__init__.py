"""GB300-native fused Indexer-TopK (LiteTopK-style sample / filter / select).

The compute path lives in the CUDA library ``libltk.so`` (sources in ``csrc/``,
C ABI in ``include/ltk.h``); ``ltk`` is a thin ctypes binding over it and
``kv`` the same for the paged 8-bit key/value cache and its attention, ``sampling``
for the draw of tokens from logits.
"""
from .ltk import IndexerTopK, LtkError, litedsa_pack, load_library, library_path  # noqa: F401
from .kv import PagedKVCache  # noqa: F401
from .sampling import sample  # noqa: F401
