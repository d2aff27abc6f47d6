"""MI355X-native Clebsch-Gordan tensor-product (CGTP) convolution.

The compute path is libcgtp.so (HIP kernels for gfx950 behind the C ABI in
include/cgtp.h); ``Plan`` in ``ops`` is its thin torch-facing binding.  The
node-side operators of a training step (include/cgtp_train.h) are the functions
of ``train``.  The library is loaded on first use and its absence raises.
"""
_TRAIN = ("embed_fwd", "embed_bwd", "embed_bwd_workspace_size", "norm_act_fwd", "norm_act_bwd",
          "norm_act_workspace_size", "orthogonalize", "orthogonalize_workspace_size")


def __getattr__(name):
    if name in ("Plan",):
        from .ops import Plan
        return Plan
    if name in _TRAIN:
        from . import train
        return getattr(train, name)
    raise AttributeError(name)
