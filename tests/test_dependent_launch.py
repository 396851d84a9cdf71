"""Kernels that are launched to overlap the tail of the one before (programmatic dependent launch): those of the cache
and chunk entry points touch no memory of a call, not even their inputs, before they have waited for what came before.
CPU only: read from the sources."""
from __future__ import annotations

import os
import re

import pytest

from sparse_attention_decode_sd_b200 import build as sdbuild

POINTERS = ("q", "K", "V", "scales", "page_table", "lens", "first", "row_start", "idx", "out", "status", "part", "ml", "tail",
            "few_part", "few_ml", "few_tail", "k_in", "v_in", "k_out", "v_out", "boxes")
FILES = {"cache_io.cu": 2, "cache_sparse.cu": 2, "cache_decode.cu": 2, "chunk_attention.cu": 2}


def _kernels(text):
    """(name, body) of every __global__ function."""
    for m in re.finditer(r"__global__[^{;]*?(\w+_kernel)\s*\(", text):
        i = text.index("{", text.index(")", m.end()))
        depth, j = 1, i + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[j], 0)
            j += 1
        yield m.group(1), text[i:j]


@pytest.mark.parametrize("name", FILES)
def test_kernels_wait_before_they_touch_memory(name):
    with open(os.path.join(sdbuild.CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found = list(_kernels(text))
    assert len(found) == FILES[name]
    for kernel, body in found:
        waits = re.findall(r"^(.*)\b(?:pdl_enter|pdl_wait)\(\);", body, re.M)
        assert len(waits) == 1 and not waits[0].strip(), (kernel, waits)          # one, in no branch
        before = body[:re.search(r"\b(?:pdl_enter|pdl_wait)\(\);", body).start()]
        depth = before.count("{") - before.count("}")
        assert depth == 1, kernel                                                   # in no block either
        assert not re.search(r"\ba\.(%s)\b" % "|".join(POINTERS), before), (kernel, before)
