"""GB300-native WTConv layer (forward + backward) behind a C ABI, with a thin Python binding.

The compute path is ``libwtconv.so`` (CUDA kernels for sm_103a, built in-tree by ``_build``);
``wtconv`` marshals PyTorch tensors into it.  ``scan`` (a gated scan over the layer's pixels or over
tokens) and ``optim`` (AdamW over many tensors, gradient norm) do the same for the operators that
train and serve beside the layer.  ``inputs`` makes the seeded synthetic workloads.
"""
from . import inputs  # noqa: F401
from .optim import AdamW  # noqa: F401
from .scan import (  # noqa: F401
    WTConvScanFunction,
    gated_scan,
    wtconv_scan_backward,
    wtconv_scan_forward,
    wtconv_scan_status,
    wtconv_scan_step,
    wtconv_scan_workspace_size,
)
from .wtconv import (  # noqa: F401
    WTConvError,
    WTConvFunction,
    wtconv_backward,
    wtconv_backward_input,
    wtconv_backward_weights,
    wtconv_forward,
    wtconv_strerror,
    wtconv_version,
    wtconv_workspace_size,
)
