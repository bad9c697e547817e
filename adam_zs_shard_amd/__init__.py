"""libzshard: the per-shard ZeRO optimizer step on MI355X (gfx950).

The product is the C-ABI shared library built from csrc/ (declared in
include/zshard.h, zsadamw.h and zslayer.h); `zshard`, `zsadamw` and `zslayer`
are its ctypes bindings.
"""

from . import zshard  # noqa: F401
