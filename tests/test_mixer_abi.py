"""Every function of the mixers' and the norm's headers is exported and bound, and the headers are C."""
import ctypes
import os
import re
import subprocess

import pytest

from memory_bound_cnn_gb300 import norm as N
from memory_bound_cnn_gb300 import ssm as M
from memory_bound_cnn_gb300 import wtconv as W

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("header,bound", [("wtconv_ssm.h", M.EXPORTED), ("wtconv_norm.h", N.EXPORTED)])
def test_declared_functions_are_bound(header, bound):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    declared = set(re.findall(r"^(?:int|size_t)\s+(wtconv_\w+)\s*\(", text, flags=re.M))
    assert declared == set(bound)
    for name in declared:
        assert hasattr(W.load(), name)


def test_headers_compile_as_c(tmp_path):
    """Also that the binding's structures have the header's sizes."""
    src = tmp_path / "t.c"
    src.write_text('#include "wtconv_ssm.h"\n#include "wtconv_norm.h"\n#include <stdio.h>\n'
                   'int main(void) { printf("%zu %zu %zu %zu %zu %zu %zu %d %d %d", sizeof(wtconv_ssm_tensor), sizeof(wtconv_selective_shape),'
                   ' sizeof(wtconv_selective_inputs), sizeof(wtconv_selective_grads), sizeof(wtconv_causal_shape), sizeof(wtconv_rms_shape),'
                   ' sizeof(wtconv_rms_tensor), WTCONV_SELECTIVE_KEEP, WTCONV_SELECTIVE_MAX_STATES, WTCONV_RMS_MAX_CHANNELS); return 0; }\n')
    exe = str(tmp_path / "t")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I" + os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = [int(v) for v in subprocess.check_output([exe]).split()]
    structures = (M.SsmTensor, M.SelectiveShape, M.SelectiveInputs, M.SelectiveGrads, M.CausalShape, N.RmsShape, N.RmsTensor)
    assert got == [ctypes.sizeof(s) for s in structures] + [M.SELECTIVE_KEEP, M.SELECTIVE_MAX_STATES, N.RMS_MAX_CHANNELS]
