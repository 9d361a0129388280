"""The attention kernels' headers define nothing that no kernel uses."""
import glob
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "matmul_quantize_q8_amd", "csrc")


@pytest.mark.parametrize("header", ["kv_layout.h", "attn_chunk.h"])
def test_every_definition_is_used(header):
    text = re.sub(r"//[^\n]*", "", "\n".join(
        open(f).read() for f in glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.hip"))))
    own = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, header)).read())
    names = re.findall(r"^(?:__device__ __forceinline__|constexpr|template <[^>]*> constexpr|typedef)[^;={]*?\b(\w+)"
                       r"(?=\(| =|\{| __attribute__)", own, re.M)
    names += re.findall(r"^__device__ __forceinline__[^(]*?\b(\w+)\(", own, re.M)
    assert len(set(names)) > 20
    unused = sorted(n for n in set(names) if len(re.findall(rf"\b{n}\b", text)) < 2)
    assert unused == []
