"""Rules that the CUDA sources keep, checked on their text (no GPU)."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dsa_sparse_mla_prefill_gb300", "csrc")


def sources():
    """{file name: text without comments, string literals that follow each other joined}."""
    out = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        text = open(path).read()
        text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
        text = re.sub(r"//[^\n]*", "", text)
        out[os.path.basename(path)] = re.sub(r'"\s*"', "", text)
    return out


def test_no_copy_is_multicast_to_a_cluster():
    """Every load and copy names the shared memory of one CTA.  (A tcgen05.commit that signals the barriers of
    several CTAs moves no data.)"""
    found = {name: re.findall(r"cp\.(?:async|reduce)[^\s\[]*multicast[^\s\[]*", text) for name, text in sources().items()}
    assert not {name: f for name, f in found.items() if f}


def test_kernels_that_start_early_read_through_coherent_loads():
    """A kernel that is put on the GPU while the one before it still writes may not read what that one writes through
    the read-only path: its memory has to stay as it is for the kernel's whole duration, and the compiler may move
    such a load above the wait."""
    early = {name: text for name, text in sources().items() if "wait_for_previous()" in text}
    assert len(early) >= 3
    found = {name: re.findall(r"__ldg\w*\s*\(|\.nc\b|__restrict__", text) for name, text in early.items()}
    assert not {name: f for name, f in found.items() if f}
