"""The source of the latent attention kernel: a softmax warp's accesses to
tensor memory are fenced (tcgen05.fence::before_thread_sync) ahead of every
barrier or arrival that hands them over to other threads.  What lacks the
fence is a race that no run need show -- no GPU needed."""
import os
import re

import pytest

from draft_sampling_verification_gb300 import build

ACCESS, FENCE = "access", "fence"
# in the source: loads and stores; the fence; barriers that the softmax warps meet at, arrivals
TOKENS = re.compile(r"\b(tmem_load\d+|tmem_store\d+)\(|\b(tc_before_sync)\(|"
                    r"\b(any_of_256|lost|pair_arrive|mbar_arrive|__syncthreads|cluster_sync)\(")


def unfenced(source):
    """The lines of barriers and arrivals behind an access without a fence between them, in the
    order of the text."""
    source = re.sub(r"//[^\n]*", "", source)
    open_access, found = None, []
    for m in TOKENS.finditer(source):
        line = source.count("\n", 0, m.start()) + 1
        if m.group(1):
            open_access = line
        elif m.group(2):
            open_access = None
        elif open_access is not None:
            found.append((open_access, line, m.group(3)))
    return found


def softmax_part():
    with open(os.path.join(build.CSRC, "latent_attention.cuh")) as f:
        text = f.read()
    begin = text.index("softmax and results")
    end = text.index("keys and values\n", begin)
    part = text[begin:end]
    assert len(re.findall(r"\btmem_(load|store)\d+\(", part)) == 4    # scores, rescaling, results
    return part


def test_accesses_are_fenced_before_they_are_handed_over():
    assert unfenced(softmax_part()) == []


@pytest.mark.parametrize("text,lines", [
    ("tmem_load32(v, a);\ntc_before_sync();\nany_of_256(false);", []),
    ("tmem_store16(a, v);\n// tc_before_sync();\nany_of_256(false);", [(1, 3, "any_of_256")]),
    ("any_of_256(true);\ntmem_load16(v, a);\nif (lost()) break;\ntc_before_sync();\npair_arrive(b);",
     [(2, 3, "lost")]),
])
def test_the_search(text, lines):
    assert unfenced(text) == lines
