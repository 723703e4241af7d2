"""tcgen05.ld is asynchronous: its registers hold nothing defined until tcgen05.wait::ld. A read of one before
the wait is right only while the assembler makes no instruction of it, so the sources are held to the rule."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_lora_fine_b200", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))


def asm_blocks(text):
    """The PTX of every asm statement: its string literals, joined."""
    for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(", text):
        lits, at = [], m.end()
        while True:
            lit = re.compile(r'\s*"((?:[^"\\]|\\.)*)"').match(text, at)
            if not lit:
                break
            lits.append(lit.group(1))
            at = lit.end()
        yield "".join(lits).replace("\\n", "\n").replace("\\t", "\t")


def early_reads(ptx):
    """Instructions between a tcgen05.ld and its wait that name one of the load's registers."""
    pending, early = set(), []
    for ins in re.split(r";", ptx):
        ins = ins.strip().lstrip("{").strip()
        if ins.startswith("tcgen05.wait::ld"):
            pending = set()
        elif ins.startswith("tcgen05.ld"):
            dst = re.search(r"\{([^}]*)\}", ins).group(1)
            pending |= {r.strip() for r in dst.split(",")}
        elif pending & set(re.findall(r"%?\w+", ins)):
            early.append(ins)
    return early


def test_the_rule_sees_an_early_read():
    ld = "{.reg .b32 t<2>; tcgen05.ld.sync.aligned.32x32b.x2.b32 {t0, t1}, [%1]; "
    assert early_reads(ld + "mov.b64 %0, {t0, t1}; tcgen05.wait::ld.sync.aligned; }") == ["mov.b64 %0, {t0, t1}"]
    assert not early_reads(ld + "tcgen05.wait::ld.sync.aligned; mov.b64 %0, {t0, t1}; }")


@pytest.mark.parametrize("path", FILES, ids=[os.path.basename(f) for f in FILES])
def test_no_register_of_a_tmem_load_is_read_before_the_wait(path):
    with open(path) as f:
        blocks = list(asm_blocks(f.read()))
    if path.endswith("ptx.cuh"):
        assert sum("tcgen05.ld" in b for b in blocks) >= 2      # (that they are found at all)
    for b in blocks:
        early = early_reads(b)
        assert not early, f"{len(early)} reads before the wait, first: {early[0]}"
