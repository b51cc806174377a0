"""CPU: what needs torch and what does not, and when the step calls' module is built anew."""

import os
import subprocess
import sys

import pytest

from paged_kv_cache_350_b200 import build as bld

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)


HOST = """
import paged_kv_cache_350_b200 as pa
a = pa.Allocator(8, 4)
a.add_seq(1, 5)
a.fork(1, 2)
assert a.append_tokens(1, 9)[1] and a.num_free() == 3   # 2 shared, 1 copied, 2 fresh
assert pa.pa_attention_workspace_size(16, 2, 8, 8, 2, 64, 16, 4) > 0 and len(pa.pa_rope_frequencies(8)[0]) == 4
"""


def test_host_calls_need_neither_torch_nor_the_step_calls():
    r = run("import sys\nsys.modules['torch'] = None\n" + HOST + "assert sys.modules['torch'] is None\n")
    assert r.returncode == 0, r.stderr
    r = run(HOST + "import sys\nassert 'torch' not in sys.modules\n")
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("missing", ["torch", "paged_kv_cache_350_b200._calls"])
def test_a_step_call_that_cannot_be_loaded_says_why(missing):
    r = run(f"import sys\nsys.modules[{missing!r}] = None\n" + HOST + """
try:
    pa.pa_attention
except ImportError as e:
    assert "_calls.so" in str(e) and "paged_kv_cache_350_b200.build" in str(e) and "not built" not in str(e), e
else:
    raise SystemExit("loaded")
try:
    pa.binding.no_such_name
except AttributeError as e:
    assert "no_such_name" in str(e)
""")
    assert r.returncode == 0, r.stderr


def test_step_calls_are_the_modules_own():
    r = run("from paged_kv_cache_350_b200 import binding, pa_attention, pa_beam_topk\n"
            "from paged_kv_cache_350_b200 import _calls\n"
            "assert pa_attention is _calls.pa_attention is binding.pa_attention and pa_beam_topk is _calls.pa_beam_topk\n"
            "assert 'pa_attention' in vars(binding)\n")
    assert r.returncode == 0, r.stderr


def test_step_calls_are_built_anew_for_another_torch(monkeypatch):
    assert not bld.calls_stale()
    for other in ("0.0", None):
        monkeypatch.setattr(bld, "_calls_made_for", lambda other=other: other)
        assert bld.calls_stale()
    assert bld.build_calls() is None   # without torch: left out
    monkeypatch.undo()
    monkeypatch.setattr(bld, "CALLS_STAMP", bld.CALLS_STAMP + ".missing")
    assert bld.calls_stale()


def test_a_torch_without_package_metadata_is_known_by_its_files(monkeypatch):
    def none(name):
        raise bld.importlib.metadata.PackageNotFoundError(name)
    known = bld._calls_made_for()
    monkeypatch.setattr(bld.importlib.metadata, "version", none)
    assert bld._calls_made_for() not in (None, known)
    assert bld._calls_made_for() == bld._calls_made_for()
