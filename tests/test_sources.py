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


def test_signals_between_ctas_are_of_cluster_scope():
    """An arrival on another CTA's barrier that releases at CTA scope, or a wait for one that acquires there, orders
    nothing between the two."""
    found = {name: re.findall(r"mbarrier\.arrive\S*\.cta\.shared::cluster\S*", text) for name, text in sources().items()}
    assert not {name: f for name, f in found.items() if f}
    assert "acquire.cta" not in sources()["tree_pair.cu"]     # (its waits are for both CTAs' arrivals)


def test_what_a_call_keeps_may_be_set_by_several_threads():
    """Local variables that outlive a call are constants or atomic: calls run without the interpreter's lock, so the
    first ones of a process may come from several threads at once."""
    plain = re.compile(r"^\s+static\s+(?!const\b|constexpr\b|__device__|(?:dsa::)?PerDevice\b)[\w:<>]+\s+\w+\s*[\[=;{].*", re.M)
    found = {name: plain.findall(text) for name, text in sources().items()}
    assert not {name: f for name, f in found.items() if f}
    assert "using PerDevice = std::atomic<int>[64];" in sources()["dsa_launch.cuh"]
    info = re.search(r"struct DevInfo \{(.*?)\n\};", sources()["dsa_api.cu"], re.S).group(1)
    assert info.count("std::atomic<") == info.count(";") == 3
