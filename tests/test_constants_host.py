"""Numbers that several source files share: each stands for one thing (CPU only)."""
import os
import re

from attention_fa2_forward_03_gb300 import build


def read(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return f.read()


def test_kernel_slots_that_are_named_are_those_that_there_are():
    """The ranges in the comment at kKernelSlots are all of the array's entries, each once."""
    text = read("fa2_fwd_sm103.cu")
    m = re.search(r"// Kernel slots:(.*?)constexpr int kKernelSlots = (\d+);", text, re.S)
    named = [range(int(a), int(b) + 1) for a, b in re.findall(r"(?<![\d-])(\d+)-(\d+)", m[1])]
    assert sorted(s for r in named for s in r) == list(range(int(m[2])))


def test_no_two_places_have_the_same_site():
    """A site in the status word says where a kernel gave up: one number, one name, one file."""
    found = {}
    for name in sorted(os.listdir(build.CSRC)):
        for site, number in re.findall(r"\b(k(?:Site|Dbg)\w+) = (\d+)\b", re.sub(r"//.*", "", read(name))):
            found.setdefault(int(number), set()).add((name, site))
    assert len(found) > 20 and max(found) < 256   # bits 8 to 15
    assert {n: s for n, s in found.items() if len(s) > 1} == {}
