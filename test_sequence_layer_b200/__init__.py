"""B200-native (sm_100a) Mesa layer: chunkwise-parallel forward and recurrent decode,
and the mixers that stand beside it in a hybrid stack (a gated linear recurrence and
sliding-window attention with sinks).

The computation lives in the CUDA library ``libmesa_b200.so`` (C ABI in
``include/mesa.h``, ``include/mesa_mixers.h``); ``mesa`` is a thin ctypes binding that only marshals
torch tensors (device memory, streams) into that ABI.
"""
from . import mesa  # noqa: F401
from .mesa import (forward, forward_host, get_error, library_path, lru_backward, lru_forward,  # noqa: F401
                   lru_step, step, swa_backward, swa_cache_fill, swa_forward, swa_step, timing_enable,
                   timing_read, workspace_size, MesaError)
