"""FP64 CPU oracle of the decode MoE-layer tail and of the expert operators
before it (test infrastructure only).

Only ``tests/``, ``__graft_entry__.smoke()`` and ``bench.py``'s CPU-baseline
legs import this package.  It shares no code with the CUDA library.
"""
from .oracle import *  # noqa: F401,F403
from .oracle import __all__ as _tail
from .experts import *  # noqa: F401,F403
from .experts import __all__ as _experts

__all__ = [*_tail, *_experts]
