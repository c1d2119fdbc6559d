"""Static checks of the feed-forward block's copies into LDS (no GPU needed),
in the code that the compiler generates for gfx950.

The copies are asm statements, of which the compiler knows only what they
declare."""

import concurrent.futures as cf
import os
import re

import pytest

from test_gemm_barrier_counts import CSRC, HIPCC, _assembly

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")

SOURCES = ("wq_block_fwd.hip", "wq_block_small.hip", "wq_block_bwd.hip")


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    """{source: generated code}"""
    where = tmp_path_factory.mktemp("asm")
    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        return dict(zip(SOURCES, ex.map(lambda s: _assembly(os.path.join(CSRC, s), where), SOURCES)))


def test_copies_write_only_what_they_declare(code):
    """m0 holds a copy's target: it comes as the statement's operand, so that
    the compiler, which puts values of its own there, knows of it.  A write
    inside the statement would be none that it knows of."""
    copies = 0
    for src, asm in code.items():
        for text in re.findall(r";;#ASMSTART\n(.*?);;#ASMEND", asm, re.S):
            lines = [line.split(";")[0].strip() for line in text.splitlines()]
            copies += sum(line.endswith(" lds") for line in lines)
            bad = [line for line in lines if re.match(r"\S+\s+m0\b", line)]
            assert not bad, (src, bad)
    assert copies > 1000
