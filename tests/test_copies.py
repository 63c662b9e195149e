"""Tensor copies into shared memory, by their source (CPU only)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "attention_forward_blackwell_gb300", "csrc")


def instructions():
    """Every inline instruction of the sources, its string pieces joined."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            text = f.read()
        for piece in re.findall(r'asm volatile\(\s*((?:"[^"]*"\s*)+)', text):
            yield os.path.basename(path), "".join(re.findall(r'"([^"]*)"', piece))


def test_copies_and_commits_stay_in_their_cta():
    """The library is loaded by every rank of a job, and its tensors may be any
    memory that the device maps: a copy brings its tile to the CTA that asked
    for it and to no other, and a commit arrives on that CTA's own barrier.
    So what completes is followed by its operands, not by a further qualifier."""
    loads = commits = 0
    for where, text in instructions():
        if "cp.async.bulk" in text and "complete_tx" in text:
            loads += 1
            assert re.search(r"complete_tx::bytes \[", text), (where, text)
        if "tcgen05.commit" in text:
            commits += 1
            assert re.search(r"arrive::one\.shared::cluster\.b64 \[", text), (where, text)
    assert loads >= 2 and commits >= 1   # the pattern above still finds them
