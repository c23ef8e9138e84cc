"""HiSparse RESOLVE hot path for GB300 (sm_103a).

``hisparse`` is the ctypes binding of ``include/hisparse.h``; ``runtime``
wraps it with torch-managed device memory and streams.  ``cache8`` (rotary positions,
packing into 8-bit records, sparse attention) and ``pages`` (the pages of the resident
tier) are the operators on either side of RESOLVE.
"""
from . import hisparse  # noqa: F401
