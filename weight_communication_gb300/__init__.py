"""GB300-native quantized gradient communication kernels.

ZeRO++ quantized gradient reduction (qgZ) with LoCo error feedback, qwZ int8
weight quantization and ZeRO-2 stochastic-rounding accumulation, as sm_103a
CUDA kernels behind the C ABI of include/wc.h.  `binding` is the Python face
of that ABI; `workloads` draws the seeded synthetic inputs; `qgz` composes the
calls into whole reduce steps.  Next to them, for the training step around
the exchange: `fp8` (8-bit block-scaled linear layers), `embedding` (lookup
and gradient) and `gradnorm` (global norm and clipping); `train_step` runs all
of it together.
"""
from . import workloads  # noqa: F401  (no CUDA needed to import)

_LAZY = ("binding", "qgz", "fp8", "embedding", "gradnorm", "train_step")
__all__ = ["workloads", *_LAZY]


def __getattr__(name):
    # The binding and the composed steps load libwc.so lazily, so importing
    # the package works on a machine without the library or a GPU.
    if name in _LAZY:
        import importlib
        return importlib.import_module(f".{name}", __name__)
    raise AttributeError(name)
