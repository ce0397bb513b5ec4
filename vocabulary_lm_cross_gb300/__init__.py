"""GB300-native (sm_103a) fused large-vocabulary LM cross-entropy, and the
decoder-layer operators around it (RMS norm, linear and gated layers).

The compute lives in ``lib/libvlmce.so`` (hand-written CUDA kernels behind the
C ABI in ``include/vlmce.h``); this package holds the build script, a thin
ctypes/PyTorch binding and the seeded synthetic workloads.
"""
from .ce import (CEResult, ce_fwd_bwd, ce_fwd_bwd_host, describe_plan, host_workspace_bytes,  # noqa: F401
                 max_vocab, workspace_bytes)
from .errors import check_device_errors, take_device_errors  # noqa: F401
from .flce import FLCEResult, flce_fwd_bwd  # noqa: F401
from .linear import (LinearGrads, LinearPlan, LinearResult, describe_linear_plan,  # noqa: F401
                     glu_bwd, glu_fwd, linear_bwd, linear_fwd)
from .rmsnorm import RMSNormGrads, RMSNormResult, rmsnorm_bwd, rmsnorm_fwd  # noqa: F401
