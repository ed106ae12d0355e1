"""GB300-native (sm_103a) Mamba2 SSD selective scan over packed varlen sequences.

The compute lives in ``libssd_scan.so`` (hand-written CUDA, C ABI in
``include/ssd_scan.h``); :mod:`.binding` marshals torch tensors into it.
:mod:`.mixer` binds the operators around the scan (``include/ssd_mixer.h``):
packed convolution, single-token step, gated norm and the 8-bit state cache.
"""
from .binding import (ReplayParams, SSDError, ScanParams, call, call_noalloc,  # noqa: F401
                      call_replay, kernel_path, load, make_params, make_replay_params,
                      num_launches, ssd_scan_varlen, workspace_size)
from .mixer import conv_varlen, gated_rms_norm, state_load, state_store  # noqa: F401
from .mixer import step as ssd_step  # noqa: F401
from ._build import build  # noqa: F401
