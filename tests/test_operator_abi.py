"""Every function of the operators' headers is exported and bound, and the headers are C."""
import os
import re
import subprocess

import pytest

from memory_bound_cnn_gb300 import optim as O
from memory_bound_cnn_gb300 import scan as S
from memory_bound_cnn_gb300 import wtconv as W

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("header,bound", [("wtconv_scan.h", S.EXPORTED), ("wtconv_optim.h", O.EXPORTED)])
def test_declared_functions_are_bound(header, bound):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    declared = set(re.findall(r"^(?:int|size_t)\s+(wtconv_\w+)\s*\(", text, flags=re.M))
    assert declared == set(bound)
    for name in declared:
        assert hasattr(W.load(), name)


def test_headers_compile_as_c(tmp_path):
    """Also that the binding's structures have the header's sizes."""
    src = tmp_path / "t.c"
    src.write_text('#include "wtconv_scan.h"\n#include "wtconv_optim.h"\n#include <stdio.h>\n'
                   'int main(void) { printf("%zu %zu %d %d", sizeof(wtconv_optim_tensor), sizeof(wtconv_adamw_config),'
                   ' WTCONV_SCAN_KEEP, WTCONV_ADAMW_BLOCK); return 0; }\n')
    exe = str(tmp_path / "t")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I" + os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    import ctypes
    got = [int(v) for v in subprocess.check_output([exe]).split()]
    assert got == [ctypes.sizeof(O.OptimTensor), ctypes.sizeof(O.AdamWConfig), S.SCAN_KEEP, O.ADAMW_BLOCK]
