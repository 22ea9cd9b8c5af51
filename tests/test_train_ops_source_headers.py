"""The kernels that stand in headers, looked at as the others are: shared memory of another
CTA is used only between two barriers of the whole cluster."""
import os
import re

import pytest

from test_train_ops_source import (
    CSRC, functions, test_no_kernel_touches_a_cta_of_its_cluster_before_that_one_is_known_to_run
    as check_first_use)

REMOTE = re.compile(r"map_shared_rank|mapa\.")
LEFT = re.compile(r"\bcluster\.sync\s*\(|\bcluster_wait\s*\(|barrier\.cluster\.wait")


def kernels():
    """Of all files."""
    return [(f, name, body) for f in sorted(os.listdir(CSRC)) if f.endswith((".h", ".cu", ".cuh"))
            for name, body in functions(open(os.path.join(CSRC, f)).read())
            if REMOTE.search(body)]


def label(x):
    return x if len(x) < 40 else "body"


def test_each_use_is_among_the_functions_looked_at():
    """However a function is written: no use stands outside of those found."""
    uses = 0
    for f in os.listdir(CSRC):
        if f.endswith((".h", ".cu", ".cuh", ".cpp")):
            text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read())
            uses += len(REMOTE.findall(text))
    assert uses == sum(len(REMOTE.findall(body)) for _, _, body in kernels())
    assert {"distill_kernel", "write_sums", "cluster_sort_kernel"} <= {k[1] for k in kernels()}


@pytest.mark.parametrize("file,name,body", [k for k in kernels() if not k[0].endswith(".cu")],
                         ids=label)
def test_no_kernel_in_a_header_touches_a_cta_before_that_one_is_known_to_run(file, name, body):
    check_first_use(file, name, body)


@pytest.mark.parametrize("file,name,body", kernels(), ids=label)
def test_no_cta_leaves_while_another_may_touch_its_memory(file, name, body):
    last = [m.start() for m in REMOTE.finditer(body)][-1]
    assert any(m.start() > last for m in LEFT.finditer(body)), f"{file}: {name}"
