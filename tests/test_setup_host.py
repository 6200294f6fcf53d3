"""What a first call pays for: the set-up of a device touches the kernels of the calls that share it, and the
paged chunk calls bring their own (setting an attribute loads a kernel). Seen in the source; no GPU."""

from __future__ import annotations

import os
import re

API = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_116_b200", "csrc", "fa_api.cu")


def body(text, name):
    start = re.search(r"^\w[\w ]* " + name + r"\([^;{]*\) \{", text, re.M).end()
    return text[start:text.index("\n}\n", start)]


def test_the_device_set_up_leaves_the_chunk_kernels_alone():
    with open(API) as f:
        text = f.read()
    assert "chunk" not in body(text, "device_setup")
    for kernels in ("fa_chunk_few_kernel", "chunk_attributes<64>", "chunk_attributes<128>"):
        assert body(text, "chunk_setup").count(kernels) == 1
    for call in ("fa_chunk_workspace_bytes", "fa_chunk_paged"):
        assert "chunk_setup(&dev, &sms)" in body(text, call)
