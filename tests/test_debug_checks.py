"""The self-checking build, read as text: every TMA load of every kernel stands behind a check of what it loads
(ptx::dbg_check, compiled away in release builds)."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "structured_sparse_attention_cowa_b200",
                    "csrc")
SOURCES = sorted(p for p in glob.glob(os.path.join(CSRC, "*.cu")) if "tma_load_4d(" in open(p).read())
REACH = 45  # lines between a producer's check and the loads it stands for


def test_there_are_sources_with_loads():
    assert {os.path.basename(p) for p in SOURCES} >= {"cowa_fwd.cu", "cowa_bwd.cu", "cowa_decode.cu", "cowa_paged.cu"}


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_every_load_is_checked(path):
    lines = open(path).read().splitlines()
    checks = [i for i, x in enumerate(lines) if "ptx::dbg_check(" in x]
    for i, x in enumerate(lines):
        if "tma_load_4d(" in x:
            assert any(0 < i - c <= REACH for c in checks), f"{os.path.basename(path)}:{i + 1}"


def test_codes_are_distinct():
    codes = []
    for path in SOURCES:
        text = open(path).read()
        for m in re.finditer(r"ptx::dbg_check\(", text):
            codes.append(re.search(r"0x[0-9a-f]{3}\b", text[m.start():m.start() + 700]).group())
    assert len(codes) == len(set(codes)) and len(codes) >= 12
