"""The attention over 8-bit pages, in its source: it starts beside the kernel that writes its workspace, so what that
one writes must not come by read-only loads, which are undefined for memory that changes while a kernel runs."""
import os
import re

SRC = os.path.join(os.path.dirname(__file__), "..", "speculative_decoding_verification_09_gb300", "csrc",
                   "attention.cuh")


def fields(struct, text):
    """Names of the pointers to what is not const in a struct."""
    body = re.search(r"struct %s \{(.*?)\n\};" % struct, text, re.S).group(1)
    return re.findall(r"^\s*(?!const\b)\w+\*\s+(\w+);", body, re.M)


def read_only_loads(text):
    text = re.sub(r"//[^\n]*", "", text)
    written = fields("Prep8", text)
    assert len(written) >= 4, written
    return [n for n in written if re.search(r"__ldg\((?:[^;]*?)\bA\.%s\b" % n, text)]


def test_what_the_first_kernel_writes_is_not_read_only():
    assert read_only_loads(open(SRC).read()) == []


def test_a_read_only_load_is_found():
    text = open(SRC).read()
    assert read_only_loads(text.replace("__ldcg(A.qf", "__ldg(A.qf")) == ["qf"]
