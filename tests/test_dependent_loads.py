"""Every kernel may start while the one before it in its stream still runs, and waits
for it before it reads memory.  A load by __ldg is of memory that nothing writes while
the kernel lasts, which the compiler may take before that wait: what a preceding kernel
can have written (parents, block tables, lengths, pools) is read by load_after_wait."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_cache_283_gb300", "csrc")
FILES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


def code(name):
    """The file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", FILES)
def test_no_load_is_taken_as_constant(name):
    text = code(name)
    assert re.findall(r"\b__ldg\s*\(|ld\.global\.nc", text) == []


def test_loads_after_the_wait_stay_there():
    """Each is volatile, as the wait is, so that neither passes the other."""
    text = code("device.cuh")
    bodies = re.findall(r"load_after_wait\(const \w+\* p\) \{(.*?)\n\}", text, flags=re.S)
    assert len(bodies) >= 6
    for body in bodies:
        assert re.search(r"asm volatile\(\"ld\.global\.\w", body) and ".nc" not in body
        assert '"memory"' in body
    assert 'asm volatile("griddepcontrol.wait;" ::: "memory")' in text
