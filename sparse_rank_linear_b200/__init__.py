"""SALR sparse + low-rank linear layer for NVIDIA B200 (sm_100a).

``Y = X (M (.) W)^T + (X A_cat) B_cat`` with W magnitude-pruned per row and stored as a
bitmap plus compact values, or held as 4-bit codes with group scales; its gradients and an
AdamW step for the adapters; all in hand-written CUDA kernels.  The Python layer is
a ctypes binding of the C ABI in ``include/salr.h``; importing it does not load the
library, the first call does (and fails loudly if it has not been built).
"""
from .binding import (SIGNATURES, SalrError, SalrPlan, Weight, encode, encode_q4, linear,
                      linear_backward, linear_host, load, load_library, pack_q4, plan, residual_adapter,
                      status_string)
from .optim import AdamW

__all__ = ["AdamW", "SIGNATURES", "SalrError", "SalrPlan", "Weight", "encode", "encode_q4", "linear",
           "linear_backward", "linear_host", "load", "load_library", "pack_q4", "plan", "residual_adapter", "status_string"]
