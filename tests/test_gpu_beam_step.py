"""A beam search as one program runs it: prompts appended once and forked into their beams, then step by step norm and turn,
reservation, append, attention over the shared prompts, selection, reordering.  Every step's selection is that of its logits;
at the end every beam's cache holds what a cache of its own would hold, byte for byte, and its attention and
score are those of its history alone."""

import numpy as np
import pytest

from tests.test_gpu_beam_select import check as check_selection

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from bit_kv_cache_04_gb300 import kvq as K  # noqa: E402

V, EOS = 500, 3


def _i(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Model:
    """Tables in place of weights: a token's projection and logits do not depend on the batch that it is in."""

    def __init__(self, cfg, seed=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.cfg, L, H, Hq, D = cfg, cfg.L, cfg.H_kv, cfg.H_q, cfg.D
        self.dt = torch.float16 if cfg.in_dtype == K.DT_F16 else torch.bfloat16
        self.qkv = torch.randn((L, V, Hq + 2 * H, D), generator=g, device="cuda").to(self.dt)
        self.head = 2 * torch.randn((V, V), generator=g, device="cuda")
        self.mix = torch.randn((L * Hq * D, V), generator=g, device="cuda") / (L * Hq * D) ** 0.5
        self.plan, self.w = K.rope_plan(D), torch.ones(D, dtype=self.dt, device="cuda")

    def project(self, tokens, positions):
        cfg, H, Hq = self.cfg, self.cfg.H_kv, self.cfg.H_q
        x = self.qkv[:, tokens.long()]
        q, k = torch.empty_like(x[:, :, :Hq]), torch.empty_like(x[:, :, Hq:Hq + H])
        for l in range(cfg.L):
            K.qk_norm_rope(cfg, x[l, :, :Hq], x[l, :, Hq:Hq + H], positions, q[l], k[l], plan=self.plan, q_weight=self.w, k_weight=self.w)
        return q.contiguous(), k.contiguous(), x[:, :, Hq + H:].contiguous()

    def logits(self, tokens, out):  # out [L, n, Hq, D]
        x = out.float().transpose(0, 1).reshape(len(tokens), -1)
        return self.head[tokens.long()] + x @ self.mix


def config(batch, max_T, **kw):
    kw = dict(dict(L=2, H_kv=2, H_q=8, D=128, k_fmt=K.Fmt(4, 128), v_fmt=K.Fmt(4, 128), flags=K.ROTATE_K | K.ROTATE_V, sign_seed=5), **kw)
    mp = -(-max_T // 16)
    return K.Config(batch=batch, max_T=max_T, page_tokens=16, n_pages=batch * mp + 2, max_pages_per_seq=mp, **kw)


def own_history(cfg, model, tokens):
    """A cache of its own for one history: the last token's attention, and what the cache holds."""
    one = K.Config(**{**cfg.__dict__, "batch": 1})
    table = torch.arange(one.max_pages_per_seq, dtype=torch.int32, device="cuda").view(1, -1)
    cache, n = K.KVCache(one, "cuda", block_table=table), len(tokens)
    t, lens = _i(tokens), _i([0])
    q, k, v = model.project(t, torch.arange(n, dtype=torch.int32, device="cuda"))
    for a, b in ((0, n - 1), (n - 1, n)):
        cache.append(0, one.L, k[:, a:b].contiguous(), v[:, a:b].contiguous(), _i([0, b - a]), lens, b - a, b - a)
        cache.commit_lengths(_i([0, b - a]), lens)
    out = torch.empty_like(q[:, -1:].contiguous())
    cache.chunk_attention(0, one.L, q[:, -1:].contiguous(), _i([0, 1]), 1, 1, lens, out)
    return cache, lens, out


def held(cache, seq, lens, n):
    res = []
    for l in range(cache.cfg.L):
        k, v = (torch.empty((n, cache.cfg.H_kv, cache.cfg.D), device="cuda") for _ in range(2))
        cache.dequantize(l, seq, 0, n, lens, k, v)
        res += [k, v]
    return torch.stack(res)


@pytest.mark.parametrize("beams", [1, 4, 9])
@pytest.mark.parametrize("kw", [dict(), dict(residual_window=20), dict(in_dtype=K.DT_BF16, k_fmt=K.Fmt(8, 32), v_fmt=K.Fmt(4, 32), flags=0)])
def test_search(beams, kw):
    prompts = [150, 300, 17]
    G, B, steps = len(prompts), len(prompts) * beams, 7
    rng = np.random.default_rng(beams)
    cfg = config(B, max(prompts) + steps + 1, **kw)
    model = Model(cfg)
    table = torch.full((B, cfg.max_pages_per_seq), -1, dtype=torch.int32, device="cuda")
    cache = K.KVCache(cfg, "cuda", block_table=table)
    pool, lens = K.PagePool(cache), torch.zeros(B, dtype=torch.int32, device="cuda")
    attention, select = K.PrefixAttention(cache, G, B), K.BeamSelect(G, beams, V)
    history = [rng.integers(4, V, prompts[b // beams]).tolist() for b in range(B)]
    for b in range(B):
        history[b] = history[b // beams * beams]

    def append(seqs, tokens):  # lists of tokens of each listed sequence
        n_new = [0] * B
        for s, t in zip(seqs, tokens):
            n_new[s] = len(t)
        cu = _i(np.concatenate([[0], np.cumsum(n_new)]).tolist())
        start = lens.tolist()
        pos = _i([start[s] + j for s in range(B) for j in range(n_new[s])])
        flat = {s: t for s, t in zip(seqs, tokens)}
        pool.reserve(_i(seqs), _i([len(t) for t in tokens]), lens)
        q, k, v = model.project(_i([x for s in range(B) for x in flat.get(s, [])]), pos)
        cache.append(0, cfg.L, k, v, cu, lens, sum(n_new), max(n_new))
        cache.commit_lengths(cu, lens)
        return q, cu

    firsts = [g * beams for g in range(G)]
    append(firsts, [history[b][:-1] for b in firsts])
    if beams > 1:
        pool.fork(_i([b // beams * beams for b in range(B) if b % beams]), _i([b for b in range(B) if b % beams]), lens)
    scores = torch.full((G, beams), -float("inf"), device="cuda")
    scores[:, 0] = 0
    done = torch.zeros((G, beams), dtype=torch.int32, device="cuda")
    tokens, parents = torch.empty_like(done), torch.empty_like(done)
    cu_groups = _i([g * beams for g in range(G + 1)])
    sums = [0.0] * B  # of the histories' log-probabilities, in 64 bits
    for step in range(steps):
        q, cu = append(list(range(B)), [h[-1:] for h in history])
        out = torch.empty_like(q)
        attention.plan(cu_groups, cu, B, 1, beams, lens)
        attention.attention(0, cfg.L, q, out)
        last = _i([h[-1] for h in history])
        logits = model.logits(last, out).view(G, beams, V)
        was, was_done = scores.clone(), done.clone()
        select.select(logits, scores, scores, tokens, parents, done=done, done_out=done, eos=EOS)
        got = check_selection(logits, was, was_done, EOS)
        assert np.array_equal(got[0], scores.cpu()) and np.array_equal(got[1], tokens.cpu()) and np.array_equal(got[2], parents.cpu())
        assert np.array_equal(got[3], done.cpu())
        if step + 1 == steps:
            break
        pool.reorder(parents.view(-1), beams, lens)
        lp = torch.log_softmax(logits.double(), -1).view(B, V)
        src = [b // beams * beams + int(parents.view(-1)[b]) for b in range(B)]
        sums = [sums[s] + (0.0 if was_done.view(-1)[s] else float(lp[s, int(tokens.view(-1)[b])])) for b, s in enumerate(src)]
        history = [history[s] + [int(tokens.view(-1)[b])] for b, s in enumerate(src)]
        fin = torch.isfinite(scores).view(-1).cpu().numpy()
        # fp32 scores, rounded once a step, and the selection's own error: below 2^-21 of a score of at most some 60, a step
        assert np.all(np.abs(scores.view(-1).cpu().numpy() - np.array(sums))[fin] <= 60 * 2.0 ** -21 * (step + 1))
        refs = torch.bincount(table[table >= 0].long(), minlength=cfg.n_pages)
        assert torch.equal(refs.int(), pool.refs)
    torch.cuda.synchronize()
    assert cache.device_status() == 0 and pool.device_status() == 0 and attention.device_status() == 0
    u = 2.0 ** -11 if cfg.in_dtype == K.DT_F16 else 2.0 ** -8
    for b in range(B):
        c, l1, ref = own_history(cfg, model, history[b])
        n = len(history[b])
        assert lens[b] == n and torch.equal(held(cache, b, lens, n), held(c, 0, l1, n))
        a, r = out[:, b].float(), ref[:, 0].float()
        assert (a - r).norm() <= 8 * u * r.norm()  # two calls' roundings of keys, values, probabilities and outputs


def test_a_step_captured():
    """Reservation, append, plan, attention, selection and reordering of a step as one graph, replayed."""
    beams, G = 4, 2
    B = beams * G
    cfg = config(B, 260, residual_window=8)
    model = Model(cfg)

    def program():
        table = torch.full((B, cfg.max_pages_per_seq), -1, dtype=torch.int32, device="cuda")
        cache = K.KVCache(cfg, "cuda", block_table=table)
        pool, lens = K.PagePool(cache), torch.zeros(B, dtype=torch.int32, device="cuda")
        attention, select = K.PrefixAttention(cache, G, B), K.BeamSelect(G, beams, V)
        prompt = torch.arange(10, 210, dtype=torch.int32, device="cuda")
        n = [200 if b % beams == 0 else 0 for b in range(B)]
        pool.reserve(_i([0, beams]), _i([200, 200]), lens)
        _, k, v = model.project(prompt.repeat(G), torch.arange(200, dtype=torch.int32, device="cuda").repeat(G))
        cu = _i(np.concatenate([[0], np.cumsum(n)]).tolist())
        cache.append(0, cfg.L, k, v, cu, lens, 400, 200)
        cache.commit_lengths(cu, lens)
        pool.fork(_i([b // beams * beams for b in range(B) if b % beams]), _i([b for b in range(B) if b % beams]), lens)
        tok = torch.full((G, beams), 9, dtype=torch.int32, device="cuda")
        parents, scores = torch.zeros_like(tok), torch.full((G, beams), -float("inf"), device="cuda")
        scores[:, 0] = 0
        every, one, cu1, cu_groups = _i(list(range(B))), _i([1] * B), _i(list(range(B + 1))), _i([0, beams, B])

        def step():
            pool.reserve(every, one, lens)
            q, k, v = model.project(tok.view(-1), lens)
            cache.append(0, cfg.L, k, v, cu1, lens, B, 1)
            cache.commit_lengths(cu1, lens)
            out = torch.empty_like(q)
            attention.plan(cu_groups, cu1, B, 1, beams, lens)
            attention.attention(0, cfg.L, q, out)
            logits = model.logits(tok.view(-1), out).view(G, beams, V)
            select.select(logits, scores, scores, tok, parents)
            pool.reorder(parents.view(-1), beams, lens)

        return step, (tok, parents, scores, lens, table, pool.refs)

    eager, want = program()
    for _ in range(6):
        eager()
    step, state = program()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # warms the libraries of the toy model up
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(state, want):
        assert torch.equal(a, b)
