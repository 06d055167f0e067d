"""The serving entries from several host threads: calls of different formats
and list lengths side by side, each on a stream and a workspace of its own."""

import ctypes
import threading
from dataclasses import replace

import pytest

from tests.gpu_cases import appended_cache

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from bit_kv_cache_04_gb300 import kvq as K  # noqa: E402
from bit_kv_cache_04_gb300 import workloads as W  # noqa: E402


def started(name="gqa8b_hadamard4_paged", lengths=(3000, 1700), new=(4, 4), **kw):
    """A filled cache, a call on it (out, which of four queries, ...) and the outputs of those queries."""
    w = W.make(name)
    w = W.Workload(w.name, replace(w.cfg, **kw), w.lengths, w.values, w.extra_tokens)
    w = w.scaled(L=1, lengths=list(lengths), extra=0)
    cache, lens, _, _ = appended_cache(w, with_oracle=False)
    cfg = w.cfg
    cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(5)
    dt = torch.float16 if cfg.in_dtype == K.DT_F16 else torch.bfloat16
    qs = torch.randn((4, 1, sum(new), cfg.H_q, cfg.D), generator=gen, device="cuda").to(dt)

    def call(out, which=0, **kw):
        cache.chunk_attention(0, 1, qs[which], cu, sum(new), max(new), lens, out, **kw)

    refs, ws = torch.empty_like(qs), cache.make_chunk_workspace()
    for i in range(4):
        call(refs[i], i, workspace=ws)
    torch.cuda.synchronize()
    call.raw = lambda out, ws, s: (ctypes.byref(cache.c_cfg), ctypes.byref(cache.c_cache), 0, 1, qs[0].data_ptr(), cu.data_ptr(),
                                   sum(new), max(new), lens.data_ptr(), 0, 0, out.data_ptr(), ws.data_ptr(), ws.numel(),
                                   s.cuda_stream)
    return cache, call, refs


def test_formats_side_by_side_from_several_threads():
    """One kernel for several formats: what a call asks of its launch must not
    change under another thread's call."""
    heads = dict(H_kv=2, H_q=8)
    kinds = [started(**heads), started("llama2_7b_kivi4", **heads), started("q8_0_mha_1k", **heads)]
    failed = []

    def work(cache, call, refs):
        s, ws = torch.cuda.Stream(), cache.make_chunk_workspace()
        out = torch.empty_like(refs[0])
        torch.cuda.synchronize()
        args, fn = call.raw(out, ws, s), K.LIB.kvq_chunk_attention
        for _ in range(40):
            statuses = [fn(*args) for _ in range(250)]
            if any(statuses):
                failed.append(K.LIB.kvq_last_error())
                break
            s.synchronize()
        s.synchronize()
        if not torch.equal(out, refs[0]):
            failed.append("other outputs")

    threads = [threading.Thread(target=work, args=k) for k in kinds]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed


def test_reservations_of_many_sequences_side_by_side():
    """Lists that ask the reserve kernel for more shared memory than a launch has without asking."""
    failed = []

    def work(batch):
        mp = 2
        cfg = K.Config(L=1, H_kv=1, H_q=1, D=128, batch=batch, max_T=32, k_fmt=K.Fmt(4, 128), v_fmt=K.Fmt(4, 128),
                       page_tokens=16, n_pages=64, max_pages_per_seq=mp)
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            cache = K.KVCache(cfg, block_table=torch.full((batch, mp), -1, dtype=torch.int32))
            pool, lens = K.PagePool(cache), torch.zeros(batch, dtype=torch.int32, device="cuda")
            seqs = torch.arange(batch, dtype=torch.int32, device="cuda")
            n_new = torch.zeros_like(seqs)
            n_new[batch - 1] = 20
            fn = K.LIB.kvq_pages_reserve
            args = (ctypes.byref(cache.c_cfg), ctypes.byref(cache.c_cache), cache.block_table.data_ptr(), pool.refs.data_ptr(),
                    lens.data_ptr(), seqs.data_ptr(), n_new.data_ptr(), batch, pool.workspace.data_ptr(), pool.ws_bytes,
                    s.cuda_stream)
            for _ in range(10):
                if any([fn(*args) for _ in range(100)]):
                    failed.append("a call")
                s.synchronize()
            want = torch.full((batch, mp), -1, dtype=torch.int32)
            want[-1] = torch.tensor([0, 1])
            if not torch.equal(cache.block_table.cpu(), want) or pool.device_status():
                failed.append("the table")

    threads = [threading.Thread(target=work, args=(b,)) for b in (12289, 20000, 32768)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
