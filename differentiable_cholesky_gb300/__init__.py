"""GB300-native differentiable Cholesky: batched/blocked potrf and its adjoint.

The compute path is the C-ABI library ``libchol_gb300.so`` (CUDA for sm_103a,
declared in ``include/chol.h``); :mod:`differentiable_cholesky_gb300.binding`
marshals torch device tensors into it, and :mod:`.learn` does so for the
operators for learning with the factor (``include/chol_learn.h``).  The library
is loaded on first use, so importing this package (e.g. for :mod:`.workloads`)
needs no GPU.
"""
from __future__ import annotations

_BINDING = ["chol_fwd", "chol_adj", "cholesky", "load_library"]
_LEARN = ["rms_norm", "linrec", "AdamW"]
__all__ = _BINDING + _LEARN


def __getattr__(name):
    if name in _BINDING:
        from . import binding
        return getattr(binding, name)
    if name in _LEARN:
        from . import learn
        return getattr(learn, name)
    raise AttributeError(name)
