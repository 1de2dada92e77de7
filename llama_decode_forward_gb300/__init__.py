"""Batch-1 Llama decode forward pass on one GB300 (sm_103a).

The computation lives in the CUDA library libllmdecode (csrc/, C ABI in
include/llm.h); ``binding`` marshals arguments to it.  Importing the package
builds the library if needed and fails if it cannot be built or loaded.
"""
from .binding import *  # noqa: F401,F403
from .binding import Decoder, DeviceWeights, LlmError, LIBRARY_PATH, declared_symbols  # noqa: F401

_BATCH = ("AdjustLogits", "AttendBatch", "BatchDecoder", "KvAppend", "KvRead", "LogProbs", "PagePool", "PagedBatch", "PagedBatchQ4",
          "PagesCompact", "PagesUpdate", "q4_pages", "rope_table")


def __getattr__(name):
    # the batched operators take CUDA tensors: torch is imported with the first of them
    if name in _BATCH:
        from . import batch
        return getattr(batch, name)
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
