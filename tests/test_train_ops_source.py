"""What no run of the operators' kernels can show: orders that hold by chance of
timing when they are missing.  Read from the source."""
import os
import re

import pytest

import optimizer_step_gb300

CSRC = os.path.join(os.path.dirname(os.path.abspath(optimizer_step_gb300.__file__)), "csrc")


def functions(text):
    """(name, body) of every function whose body opens at the end of a line and
    closes with a brace in the first column."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"\b(?!__)(\w+)\s*\([^;{}]*\)\s*\{\n(.*?)^\}", text, re.S | re.M):
        yield m.group(1), m.group(2)


def sources():
    return sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))


def kernels_with_remote_shared_memory():
    return [(f, name, body) for f in sources()
            for name, body in functions(open(os.path.join(CSRC, f)).read())
            if "map_shared_rank" in body or "mapa." in body]


def test_the_cluster_sort_is_among_the_kernels_looked_at():
    assert "cluster_sort_kernel" in [k[1] for k in kernels_with_remote_shared_memory()]


@pytest.mark.parametrize("file,name,body", kernels_with_remote_shared_memory(),
                         ids=lambda x: x if len(x) < 40 else "body")
def test_no_kernel_touches_a_cta_of_its_cluster_before_that_one_is_known_to_run(file, name, body):
    """Shared memory of another CTA may be used only behind a barrier of the
    whole cluster: until then that CTA need not have started."""
    first = re.search(r"map_shared_rank|mapa\.", body).start()
    wait = re.search(r"\bcluster\.sync\s*\(|\bcluster_wait\s*\(|barrier\.cluster\.wait", body)
    assert wait and wait.start() < first, f"{file}: {name}"
    if not wait.group().startswith("cluster.sync"):
        arrive = re.search(r"\bcluster_arrive\s*\(|barrier\.cluster\.arrive", body)
        assert arrive and arrive.start() < wait.start(), f"{file}: {name}"
