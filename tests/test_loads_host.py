"""Loads of tensors in the kernels, from the sources.  A kernel starts while the one before it still
writes (programmatic launches), so what it reads is not constant for its lifetime: the read-only path
(__ldg, ld.global.nc) is not for it, and an asm load has to be volatile to stay behind the wait."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "rmsnorm_modulate_gb300", "csrc")


def sources():
    for f in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, f)) as fh:
            text = re.sub(r"/\*.*?\*/", "", fh.read(), flags=re.S)
        yield f, re.sub(r"//[^\n]*", "", text)


def faults(text):
    """Loads by the read-only path, and global loads whose asm is not volatile."""
    bad = re.findall(r"__ldg\w*", text)
    for m in re.finditer(r"\basm\b(\s+volatile)?\s*\(\s*((?:\"(?:[^\"\\]|\\.)*\"\s*)+)", text):
        if "ld.global.nc" in m.group(2) or ("ld.global" in m.group(2) and not m.group(1)):
            bad.append(m.group(2).strip())
    return bad


def test_the_pattern_sees_each_kind():
    load = '("{}.v4.u32 {{%0}}, [%1];" : "=r"(v) : "l"(p));'
    assert faults("asm" + load.format("ld.global.nc")) and faults("x = __ldg(p);")
    assert faults("asm volatile" + load.format("ld.global.nc"))
    assert faults("asm" + load.format("ld.global"))
    assert not faults("asm volatile" + load.format("ld.global"))


def test_no_load_by_the_read_only_path():
    bad = {f: b for f, b in ((f, faults(t)) for f, t in sources()) if b}
    assert not bad, bad
