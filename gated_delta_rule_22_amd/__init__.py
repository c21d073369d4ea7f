"""Complex KDA (CKDA) recurrence on AMD Instinct MI355X (gfx950).

``forward``, ``kda_forward``, ``backward`` and ``decode_step`` are thin wrappers over the C-ABI library
``libckda.so`` (see ``include/ckda.h``); they marshal torch tensors and the
current HIP stream and nothing else.  The library is loaded on first use; if it
is missing the call raises instead of falling back to any other code.
"""
from . import workloads  # noqa: F401  (seeded input generators; no GPU needed)

_BINDING = ("forward", "kda_forward", "backward", "decode_step", "forward_workspace_bytes",
            "backward_workspace_bytes", "gdr_forward", "gdr_backward", "gdr_decode_step",
            "gdr_forward_workspace_bytes", "gdr_backward_workspace_bytes", "qk_norm_rotary",
            "qk_norm_rotary_backward", "rotary", "rotary_frequencies", "library", "CkdaError")

__all__ = [*_BINDING, "workloads"]


def __getattr__(name):
    if name in _BINDING:
        from . import _lib
        value = globals()[name] = getattr(_lib, name)
        return value
    raise AttributeError(name)
