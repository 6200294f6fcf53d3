"""The package loads on a torch that lacks the 8-bit types of the paged caches: what does not use them works,
and codes and scales may come as uint8 everywhere."""

from __future__ import annotations

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("missing", [["float8_e8m0fnu"], ["float8_e8m0fnu", "float8_e4m3fn"]])
def test_import_without_8_bit_types(missing):
    code = "import torch\n" + "".join(f"del torch.{name}\n" for name in missing) + (
        "import exact_attention_116_b200 as fa\n"
        "from exact_attention_116_b200 import binding\n"
        "assert torch.uint8 in binding._E4M3 and torch.uint8 in binding._E8M0\n"
        f"assert len(binding._E8M0) == 1 and len(binding._E4M3) == {2 - missing.count('float8_e4m3fn')}\n")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT, timeout=300)
