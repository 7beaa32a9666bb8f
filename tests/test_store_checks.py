"""Every store of the expert-layer kernels to a caller's buffer goes through the check that debug builds make, from the
sources (no GPU needed): a store past it would go unseen there."""
import os
import re

import pytest

from newton_schulz_quintic_gb300 import build

FILES = ["ns_route.cu", "ns_blocks.cu", "ns_blocks_mm.cu", "ns_block_norm.cu", "ns_block_norm.cuh", "ns_block_norm_back.cu", "ns_dropout.cu"]


@pytest.mark.parametrize("name", FILES)
def test_stores_are_checked(name):
    with open(os.path.join(build.CSRC, name)) as f:
        lines = [re.sub(r"//.*", "", line) for line in f]
    text = "".join(lines)
    text = text[:text.find('extern "C"')] if 'extern "C"' in text else text  # the kernels
    # what points into a buffer: the parameters' pointers, and those formed from them
    pointers = set(re.findall(r"\*\s*(?:const\s+)?(\w+) = (?:static_cast<[^;]*>\()?p\.\w+", text)) - {"x", "mine"}
    bad = []
    for line in text.splitlines():
        stores = re.findall(r"(?<![=\w.])(p\.\w+|static_cast<[^;=]*\*>\(p\.\w+\)|\w+)\[[^=;]*\] (?:\+|\|)?= |(\*p\.\w+) = ", line)
        for indexed, plain in stores:
            name_of = indexed or plain
            if (name_of.startswith(("p.", "*p.", "static_cast")) or name_of in pointers) and "in_bounds" not in line:
                bad.append(line.strip())
    assert not bad, bad
