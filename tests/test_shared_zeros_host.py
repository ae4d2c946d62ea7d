"""Host-side check (no GPU) of the kernels' sources: what one thread of a CTA sets up in shared memory
for all is behind a barrier of the CTA before it is used."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "exact_attention_15_gb300", "csrc")
BARRIER = re.compile(r"__syncthreads(?:_or)?\(|\bcluster_wait\(|\bcluster_sync_all\(")
ZEROED = re.compile(r"if \(tid (?:==|<) \d+\) (?:\{[^}]*\}|[^;]*;)|for \(int i = tid;[^;]*;[^)]*\) sh\.\w+\[i\] = 0;")


def _body(file, kernel):
    """The kernel's text without comments, from its name to the brace in the first column."""
    with open(os.path.join(CSRC, file)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = text.index(f"\n{kernel}(const")
    return text[at:text.index("\n}\n", at)]


def _first_uses(body):
    """(field, text between its zeroing and its next use) of the shared fields that are zeroed before
    the first barrier."""
    head = body[:body.index("grid_wait()")]
    for block in ZEROED.finditer(head):
        for field in sorted(set(re.findall(r"sh\.(\w+)(?:\[\w+\])? = ", block.group()))):
            use = re.compile(rf"\bsh\.{field}\b").search(body, block.end())
            if use:
                yield field, body[block.end():use.start()]


@pytest.mark.parametrize("file,kernel,fields", [
    ("paged_select.cu", "paged_select_kernel", {"hist", "l1", "k_most", "most", "least", "sure", "unsure", "chosen"}),
    ("paged_append_pages.cu", "paged_append_rows_kernel", {"most"})])
def test_zeros_are_behind_a_barrier(file, kernel, fields):
    seen = dict(_first_uses(_body(file, kernel)))
    assert fields <= set(seen)
    for field, between in seen.items():
        assert BARRIER.search(between), f"sh.{field} of {kernel} is used without a barrier behind its zeros"
