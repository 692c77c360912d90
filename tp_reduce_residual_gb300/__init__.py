"""libbeamnorm: the arithmetic epilogue of a fused tensor-parallel all-reduce
(rank-ordered FP32 sum of R BF16 shards, optional per-shard MoE top-k
finalize, post-RMSNorm, residual add, next-layer RMSNorm) on one GB300.

The compute runs in hand-written sm_103a CUDA kernels behind a C ABI
(``include/beamnorm.h``); ``beamnorm`` is the Python binding and ``inputs``
draws the seeded synthetic workloads.  ``experts`` binds the operators around
a mixture-of-experts layer's experts: routing and its gradient, the plan that
groups token slots by expert, 4-bit microscaled quantisation, and the experts'
product.
"""
from . import experts  # noqa: F401
from .beamnorm import (BeamNormError, Debug, check_device_error, finalize_only,  # noqa: F401
                       finalize_reduce_norm, finalize_reduce_only,
                       finalize_reduce_residual_norm, norm_only, reduce_norm, reduce_only,
                       reduce_residual_norm, set_tuning, supports, version)
