"""GB300-native (sm_103a) FP32 matrix multiply C = A x B, row-major.

The compute path is the CUDA library ``libt2s_gemm.so`` (C ABI in
``include/t2s_gemm.h``); ``binding`` is its ctypes binding. ``roofline`` holds the
performance model used for reporting and ``inputs`` the seeded synthetic inputs. ``feed_forward``
holds the operators of a transformer's feed-forward block on 16-bit tensors.
"""
from . import binding, feed_forward, inputs, roofline  # noqa: F401
from .binding import gemm, gemm_bf16, gemm_f16, gemm_f64, device_status, plan  # noqa: F401
from .feed_forward import (gated_linear, gated_linear_backward, linear,  # noqa: F401
                           linear_backward)

__all__ = ["binding", "feed_forward", "inputs", "roofline", "gemm", "gemm_bf16", "gemm_f16", "gemm_f64",
           "device_status", "plan", "linear", "linear_backward", "gated_linear",
           "gated_linear_backward"]
