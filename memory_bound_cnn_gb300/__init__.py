"""GB300-native WTConv layer (forward + backward) behind a C ABI, with a thin Python binding.

The compute path is ``libwtconv.so`` (CUDA kernels for sm_103a, built in-tree by ``_build``);
``wtconv`` marshals PyTorch tensors into it.  ``scan`` (a gated scan over the layer's pixels or over
tokens), ``ssm`` (a selective scan with many states a channel, and the short causal convolution before it),
``norm`` (root-mean-square norm with the residual's addition) and ``optim`` (AdamW over many tensors,
gradient norm) do the same for the operators that train and serve beside the layer.  ``inputs`` makes the
seeded synthetic workloads.
"""
from . import inputs  # noqa: F401
from .norm import (  # noqa: F401
    WTConvRmsFunction,
    rms_norm,
    wtconv_rms_backward,
    wtconv_rms_forward,
    wtconv_rms_forward_e4m3,
)
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
from .ssm import (  # noqa: F401
    WTConvCausalFunction,
    WTConvSelectiveFunction,
    causal_conv,
    selective_scan,
    wtconv_causal_backward,
    wtconv_causal_forward,
    wtconv_causal_step,
    wtconv_selective_backward,
    wtconv_selective_forward,
    wtconv_selective_step,
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
