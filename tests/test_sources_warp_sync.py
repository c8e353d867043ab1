"""Inline PTX that all lanes of a warp execute together stays where it is
written: without `volatile` a compiler may move it, as a pure function of its
operands, under a condition that only some lanes take."""
import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "ring_allreduce_reduction_gb300" / "csrc"
# asm, whether volatile, and the instruction's text (string literals may follow one another)
STATEMENT = re.compile(r'\basm\b\s*(volatile|__volatile__)?\s*\(\s*((?:"(?:[^"\\]|\\.)*"\s*)+)')
TOGETHER = re.compile(r"\.sync\b|\bbar(rier)?\.|\.aligned\b|\bactivemask\b|\belect\.|\bmbarrier\.|\bgriddepcontrol\.|\bfence\.")


def _plain(text):
    return [m[2] for m in STATEMENT.finditer(text) if not m[1] and TOGETHER.search(m[2])]


def test_the_search_finds_what_it_is_for():
    assert _plain('asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));')
    assert _plain('asm (\n  "bar.sync %0,"\n " %1;" ::"r"(a));')
    assert not _plain('asm volatile("bar.sync %0, %1;" ::"r"(a));') and not _plain('asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r));')


@pytest.mark.parametrize("path", sorted(p for p in CSRC.iterdir() if p.suffix in (".cu", ".cuh", ".h", ".cc")), ids=lambda p: p.name)
def test_synchronising_instructions_are_volatile(path):
    assert not _plain(path.read_text())
