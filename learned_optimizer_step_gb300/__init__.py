"""GB300-native learned-optimizer step (small_fc_lopt kind).

The compute lives in liblopt.so (C ABI in include/lopt.h, CUDA kernels for
sm_103a); this package holds the in-tree build and the ctypes binding."""
from .lopt import (LearnedOptimizer, LoptError, PreparedList, TensorState,  # noqa: F401
                   load_library, schedule_info, weight_set_size, zeros_state, MLP_FP32, MLP_TC)

_TRAIN_OPS = ("check_indices", "distill_forward", "distill_forward_backward", "embedding_backward",
              "embedding_forward", "layernorm_backward", "layernorm_forward", "release_workspaces")


def __getattr__(name):
    """The training operators, whose module imports torch, on first use."""
    if name in _TRAIN_OPS:
        from . import train_ops
        globals().update({n: getattr(train_ops, n) for n in _TRAIN_OPS})
        return globals()[name]
    raise AttributeError("module %r has no attribute %r" % (__name__, name))
