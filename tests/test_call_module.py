"""The module that makes linear()'s and attend()'s calls in C belongs to one interpreter, and the package works without it
(no GPU needed)."""
import os
import subprocess
import sys
import sysconfig

import pytest

mk = pytest.importorskip("persistent_megakernel_decode_sm_gb300")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

NO_MODULE = """
import importlib.util
find = importlib.util.find_spec
importlib.util.find_spec = lambda name, *args: None if name.endswith("._mk_call") else find(name, *args)
"""


def run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout


def test_the_module_is_named_for_its_interpreter():
    # another interpreter does not find it, and builds its own
    from persistent_megakernel_decode_sm_gb300 import build
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert "cpython" in suffix and build.CALL.endswith("_mk_call" + suffix)
    assert mk._mk_call is None or mk._mk_call.__file__ == build.CALL
    assert not os.path.exists(os.path.join(os.path.dirname(build.CALL), "_mk_call.so"))


def test_the_package_works_without_it():
    out = run(NO_MODULE + """
import torch
import persistent_megakernel_decode_sm_gb300 as mk
assert mk._mk_call is None
mk.Schedule(__import__("workload").small_config(), 4)
x = torch.ones(2, 16, dtype=torch.bfloat16)
kv = type("KV", (), dict(k=torch.ones(1, 1, 1, 8, 32, dtype=torch.bfloat16), v=torch.ones(1, 1, 1, 8, 32, dtype=torch.bfloat16)))
for call in (lambda: mk.linear(x, x), lambda: mk.attend(torch.ones(1, 1, 32, dtype=torch.bfloat16), kv, [1], [8])):
    try:
        call()
    except ValueError as e:
        print(e)
""")
    assert out.count("must be a CUDA tensor") == 2


def test_the_library_is_built_without_python_headers(monkeypatch):
    from persistent_megakernel_decode_sm_gb300 import build
    assert build.up_to_date()
    monkeypatch.setattr(build, "CALL", build.CALL + ".of-another-interpreter")
    assert not build.up_to_date()
    monkeypatch.setattr(build, "_python_headers", lambda: None)
    assert build.up_to_date()
