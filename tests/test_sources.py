"""CPU: rules that the kernels' sources keep and that no run can show to be broken."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_350_b200", "csrc")


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu"))), ids=os.path.basename)
def test_the_wait_for_tensor_memory_names_what_was_loaded(path):
    """A tensor-memory load writes its registers until the wait after it: the wait takes them as operands,
    so that the compiler cannot use one before."""
    source = re.sub(r"//[^\n]*", "", open(path).read())
    loaded = set()
    for m in re.finditer(r"tc05::(ld\w*)\s*\(.*?,\s*([\w\[\]]+)\)\s*;|tc05::wait_ld\s*\(([^;]*)\)\s*;", source):
        if m.group(1):
            loaded.add(m.group(2))
        else:
            named = {x.strip() for x in m.group(3).split(",")}
            assert loaded and loaded == named, (loaded, named, source[:m.start()].count("\n") + 1)
            loaded = set()
    assert not loaded
