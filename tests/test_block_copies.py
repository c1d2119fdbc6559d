"""Static checks of the feed-forward block's copies into LDS (no GPU needed),
in the code that the compiler generates for gfx950.

The copies are asm statements, of which the compiler knows only what they
declare, and the forward tile kernel ends a stage with a wait that leaves the
newest copies in flight."""

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


def kernels(asm, pattern):
    for name in re.findall(r"^(_ZN\S*" + pattern + r"\S*):", asm, re.M):
        yield name, asm.split(name + ":", 1)[1].split(".Lfunc_end", 1)[0]


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


def test_a_stage_leaves_only_the_newest_rows_in_flight(code):
    """At the barriers of the forward tile kernel's loop the copies still in
    flight are those of one stage's rows of x, as many as a wavefront issues:
    the packed words, scales and zero-points that the next stage reads, and
    its rows, were copied before them."""
    seen = 0
    for name, body in kernels(code["wq_block_fwd.hip"], "16block_fwd_kernel"):
        seen += 1
        rows = int(re.search(r"ELi(\d+)EEEv", name).group(1))
        flight, barriers = [], []
        for line in body.splitlines():
            line = line.split(";")[0].strip()
            if re.match(r"(global|buffer|flat|scratch)_", line):
                src = re.search(r"s\[\d+:\d+\]", line)
                flight.append((src and src.group(0), line.endswith(" lds")))
                continue
            wait = re.match(r"s_waitcnt\s.*vmcnt\((\d+)\)", line)
            if wait:
                flight = flight[max(0, len(flight) - int(wait.group(1))):]
            elif line.startswith("s_barrier"):
                barriers.append(list(flight))
        # the first stage's, the loop's; those behind the loop leave none
        first, loop, rest = barriers[0], barriers[1], barriers[2:]
        assert len(first) == len(loop) == rows // 32, (name, first, loop)
        assert all(f == loop[0] and f[1] for f in first + loop), (name, first, loop)
        assert rest and not rest[0], (name, rest)
    assert seen == 24


def _sgprs(operand):
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    return {int(operand[1:])} if re.fullmatch(r"s\d+", operand) else set()


def _written(op, operands):
    """Scalar registers that an instruction writes (a few vector ones have a
    second result, a carry)."""
    regs = set(_sgprs(operands[0])) if operands else set()
    if re.match(r"v_(mad_[iu]64|add_co|sub_co|subrev_co|addc|subb|div_scale)", op) and len(operands) > 1:
        regs |= _sgprs(operands[1])
    return regs


def _too_early(body):
    """Copies whose resource the vector ALU wrote fewer than five wait states
    before, in code order: the compiler adds those waits before loads of its
    own, not inside an asm statement."""
    at, last, bad = 0, {}, []
    for line in body.splitlines():
        line = line.split(";")[0].strip()
        if not line or line.startswith(".") or line.endswith(":"):
            continue
        op, *operands = re.split(r"[\s,]+", line)
        if op == "s_nop":
            at += int(operands[0], 0) + 1
            continue
        if line.endswith(" lds"):
            read = set().union(*(_sgprs(o) for o in operands))
            bad += [(line, last[r][1]) for r in read if r in last and at - last[r][0] - 1 < 5]
        for r in _written(op, operands):
            if op.startswith("v_"):
                last[r] = (at, line)
            else:
                last.pop(r, None)
        at += 1
    return bad


def test_the_walk_sees_an_early_copy():
    copy = "\ts_nop 0\n\tbuffer_load_dwordx4 v1, s[8:11], 0 offen lds\n"
    write = "\tv_readfirstlane_b32 s9, v0\n"
    assert _too_early(write + copy)
    assert _too_early(write + "\ts_mov_b32 m0, s3\n\tv_mov_b32 v2, v3\n\tv_mov_b32 v2, v3\n" + copy)
    assert not _too_early(write + "\ts_nop 3\n" + copy)
    assert not _too_early(write + "\ts_mov_b32 s9, s4\n" + copy)
    assert _too_early("\tv_mad_u64_u32 v[2:3], s[10:11], v2, s1, 0\n" + copy)


def test_resources_are_ready_when_a_copy_reads_them(code):
    for src, asm in code.items():
        for name, body in kernels(asm, r"block_\w+_kernel"):
            assert not _too_early(body), (src, name, _too_early(body)[:3])
