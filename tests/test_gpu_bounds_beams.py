"""Attention over shared prefixes and the reordering of pages in the bounds-checked build (libkvq_checked.so, see
tests/test_gpu_bounds.py): no check fires, the results are those of the oracle, and with every segment's last row taken
away the checks do fire."""

import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _checked_run():
    from bit_kv_cache_04_gb300 import kvq as K
    from tests import test_gpu_prefix_attention as A
    from tests import test_gpu_reorder as R

    assert K.LIB_PATH.endswith("libkvq_checked.so"), K.LIB_PATH
    for key in A.FORMATS:
        for new in ("one", "few", "many"):
            A.test_formats(key, new)  # a bit of the status word, KVQ_DEV_BOUNDS among them, is an error in there
    for prefix in (15, 16, 127, 129, 300):
        A.test_prefix_lengths(prefix, 20)
    A.test_heads_and_beams(beams=33, g=8, H=2)
    A.test_rows_of_many_sequences_in_several_row_tiles()
    for group, groups, rows, kw in ((4, 3, 5, {}), (9, 1, 20, dict(D=256, L=3, H=1)), (32, 2, 20, {})):
        R.test_steps_of_a_search(group, groups, rows, kw)
    print("clean")


def _shrunk_run():
    from bit_kv_cache_04_gb300 import kvq as K
    from tests import test_gpu_prefix_attention as A
    from tests import test_gpu_reorder as R

    res = {}
    for key in ("rot4", "q4_0", "rot4_bf16_window", "rot4_d256", "p5_direct"):
        c = A.build([300], [[84, 90, 100]], [[1, 1, 1]], **A.FORMATS[key])
        K.kvq_test_shrink_bounds(1)
        try:
            pa = A.attend(c[0], c[2], c[3], c[4], c[5])[3]
        finally:
            K.kvq_test_shrink_bounds(0)
        res[key] = pa.device_status()
    print(json.dumps(res))


def _run(what):
    from bit_kv_cache_04_gb300 import _build

    env = dict(os.environ, KVQ_LIBRARY=_build.build(checked=True))
    r = subprocess.run([sys.executable, "-c", f"import tests.test_gpu_bounds_beams as t; t.{what}()"],
                       capture_output=True, text=True, env=env, cwd=ROOT, timeout=1800)
    assert r.returncode == 0, r.stderr[-4000:]
    return r.stdout.strip().splitlines()[-1]


def test_no_check_fires():
    assert _run("_checked_run") == "clean"


def test_checks_fire_when_segments_are_shrunk():
    from bit_kv_cache_04_gb300 import kvq as K

    for name, status in json.loads(_run("_shrunk_run")).items():
        assert status & K.DEV_BOUNDS, name
