"""CPU oracle for the affine group-quantized W4A16 projection ``y = x · dequant(Wq)ᵀ``.

TEST INFRASTRUCTURE, NOT PART OF THE PRODUCT.  Only ``tests/``,
``__graft_entry__.smoke()`` and the ``cpu_baseline`` leg of ``bench.py`` may
import, call or execute anything in this package.  The HIP library and its
Python binding never import it, and this package imports nothing from them.

Everything here is plain NumPy (fp32 where the format fixes fp32, fp64 for
accumulation) or pure-Python loops for tiny cases; see ``w4a16_oracle`` for
the definitions and the passages of the pages each function follows.

``mxfp4_oracle`` has the MXFP4 operators, pinned by ``tests/test_mxfp4_cpu.py``, ``experts_oracle`` the int8
products and the experts' operators, pinned by ``tests/test_w8a8_cpu.py``.

Pinning status: every function in ``w4a16_oracle`` is pinned by
``tests/test_oracle.py`` against closed forms, exact brute force, library
routines or mathematical bounds.  No function is "parity unpinned".
"""

from .w4a16_oracle import *  # noqa: F401,F403
from .w4a16_oracle import __all__  # noqa: F401
from .mxfp4_oracle import *  # noqa: E402,F401,F403
from . import mxfp4_oracle as _mxfp4_oracle  # noqa: E402
from .experts_oracle import *  # noqa: E402,F401,F403
from . import experts_oracle as _experts_oracle  # noqa: E402

__all__ = [*__all__, *_mxfp4_oracle.__all__, *_experts_oracle.__all__]
