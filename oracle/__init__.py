"""CPU oracle for the sparse MoE layer forward pass (test infrastructure only).

Only the test suite, the smoke check and the CPU-baseline leg of the benchmark
may import this package; the HIP library never does, and this package never
imports the HIP library or its binding.
"""
from . import fp8_oracle, moe_oracle, training_oracle
from .fp8_oracle import *  # noqa: F401,F403
from .moe_oracle import *  # noqa: F401,F403
from .training_oracle import *  # noqa: F401,F403

__all__ = moe_oracle.__all__ + training_oracle.__all__ + fp8_oracle.__all__
