"""The serving operators in the bounds-checked build (libkvq_checked.so, see
tests/test_gpu_bounds.py): chunk attention of every format, with windows and
without, at ragged lengths, in all forms; histories of page calls.  No check
fires, the results are those of the oracle, and with every segment's last row (or
the pool's last page) taken away the checks do fire."""

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
    """Runs in a fresh interpreter with KVQ_LIBRARY pointing at the checked build."""
    from bit_kv_cache_04_gb300 import kvq as K
    from tests import test_gpu_chunk_attention as C
    from tests import test_gpu_pages as P

    assert K.LIB_PATH.endswith("libkvq_checked.so"), K.LIB_PATH
    for key, (name, kw) in C.FORMATS.items():
        w = C.workload(name, [391, 200, 1, 160], L=1, **kw)
        for n in ([1, 1, 1, 1], [7, 3, 1, 0], [20, 9, 1, 12], [150, 64, 0, 33]):
            C.check(w, n)  # a bit of the status word, KVQ_DEV_BOUNDS among them, is an error in there
            C.check(w, n, window=45, sinks=3)
    for T in (1, 31, 33, 64, 65, 129):
        C.check(C.workload("gqa8b_hadamard4_paged", [T], heads=(1, 8)), [T])
        C.check(C.workload("ctx262k_hadamard4", [T], heads=(1, 6)), [T])
    for shape in (dict(), dict(R=20), dict(pt=1, pages=300, max_T=40), dict(pt=7, R=5, D=256, pages=60),
                  dict(fmt=K.Fmt(3, 128), vfmt=K.Fmt(4, 32), pt=5, H=1, L=1, pages=80)):
        P.test_random_histories(shape)  # ends with a clean status word
    P.test_compact_out_of_place(1025)
    P.test_last_reader_keeps_the_page()
    print("clean")


def _shrunk_run():
    from bit_kv_cache_04_gb300 import kvq as K
    from tests import test_gpu_chunk_attention as C
    from tests import test_gpu_pages as P
    from tests.gpu_cases import appended_cache

    res = {}
    for name, heads, lengths in (("gqa8b_hadamard4_paged", (2, 4), [300, 129]), ("llama2_7b_kivi4", (2, 4), [512, 64]),
                                 ("ctx262k_hadamard4", (1, 6), [512])):
        w = C.workload(name, lengths, heads=heads)
        cache, lens, _, _ = appended_cache(w, with_oracle=False)
        cu = torch.arange(0, w.cfg.batch + 1, dtype=torch.int32, device="cuda")
        q = C.queries(w.cfg, 1, w.cfg.batch)
        K.kvq_test_shrink_bounds(1)
        try:
            cache.chunk_attention(0, 1, q, cu, w.cfg.batch, 1, lens, torch.empty_like(q))
            torch.cuda.synchronize()
        finally:
            K.kvq_test_shrink_bounds(0)
        res[name] = cache.chunk_workspace[:4].view(torch.int32).item()
    # the pool's last page, moved to the first
    cache, pool, _, _ = P.make(batch=2, max_T=64, pages=8, table=[[7, -1, -1, -1], [-1, -1, -1, -1]])
    K.kvq_test_shrink_bounds(1)
    try:
        pool.compact()
        torch.cuda.synchronize()
    finally:
        K.kvq_test_shrink_bounds(0)
    res["compact"] = pool.device_status()
    print(json.dumps(res))


def _run(what):
    from bit_kv_cache_04_gb300 import _build

    env = dict(os.environ, KVQ_LIBRARY=_build.build(checked=True))
    r = subprocess.run([sys.executable, "-c", f"import tests.test_gpu_bounds_serving as t; t.{what}()"],
                       capture_output=True, text=True, env=env, cwd=ROOT, timeout=1800)
    assert r.returncode == 0, r.stderr[-4000:]
    return r.stdout.strip().splitlines()[-1]


def test_no_check_fires():
    assert _run("_checked_run") == "clean"


def test_checks_fire_when_segments_are_shrunk():
    from bit_kv_cache_04_gb300 import kvq as K

    for name, status in json.loads(_run("_shrunk_run")).items():
        assert status == K.DEV_BOUNDS, name
