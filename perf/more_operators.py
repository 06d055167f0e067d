"""Cases of the operators that a beam search needs around the quantized cache, for measurement.

Three families, in the order of one step of the search:
  * prefix_attention: the newest tokens of every sequence attend to the paged
    cache; sequences of a group hold the same pages for their common prompt,
    which is read once for all of them;
  * beam_select: the best continuations of every group's beams over the whole vocabulary;
  * reorder: the beams' states (block table rows, lengths, 16-bit windows, page
    counts) follow the selection.

`own` False computes them in elementary torch operations in 32 bits (64 for
long sums and values next to a border); `own` True calls the framework.
"""

import math
import random

import torch

own = False

PAGE = 16
SIGN_SEED = 0x5EED5EED
EOS = 2
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
BLOCK = {"rot4": 128, "q4": 32}  # values of a 4-bit block; rot4 holds values of the rotated domain


# ---- the cases -----------------------------------------------------------------


def _attn(name, fmt, dtype, groups, beams, kv_heads, group, head_dim, prefix, own_tokens, new, window16, ragged):
    c = dict(op="prefix_attention", format=fmt, dtype=dtype, groups=groups, beams=beams, kv_heads=kv_heads, group=group,
             head_dim=head_dim, prefix=prefix, own_tokens=own_tokens, new=new, window16=window16, ragged=ragged)
    return dict(c, name=name) if name else c


def _select(name, dtype, groups, beams, vocab, finished):
    c = dict(op="beam_select", dtype=dtype, groups=groups, beams=beams, vocab=vocab, finished=finished)
    return dict(c, name=name) if name else c


def _reorder(name, layers, kv_heads, head_dim, groups, beams, context, window16):
    c = dict(op="reorder", layers=layers, kv_heads=kv_heads, head_dim=head_dim, groups=groups, beams=beams,
             context=context, window16=window16)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a single chat's four beams behind a prompt of 4096 tokens, one decode step: latency
        _attn("prefix_1x4", "q4", "fp16", 1, 4, 8, 4, 128, 4096, 33, 1, 0, False),
        # eight prompts searched with eight beams each, prompts and answers of mixed lengths, a 16-bit window beside the pages
        _attn("prefix_8x8", "rot4", "bf16", 8, 8, 8, 4, 128, 8192, 512, 1, 128, True),
        # 32 chats over one long system prompt, drafts of up to 4 tokens verified
        _attn("prefix_drafts_32", "rot4", "fp16", 1, 32, 8, 4, 128, 32768, 1024, 4, 0, True),
        # sixteen questions of up to 200 tokens about one document, wide heads
        _attn("prefix_questions_wide", "rot4", "bf16", 1, 16, 4, 6, 256, 12007, 200, 200, 0, True),
        # the smallest search
        _select("select_1x4", "fp16", 1, 4, 32000, False),
        # a small batch with full-precision logits, an odd vocabulary, some beams finished
        _select("select_16x5", "fp32", 16, 5, 50257, True),
        # many beams
        _select("select_8x32", "bf16", 8, 32, 32001, True),
        # a full batch over a large vocabulary
        _select("select_64x8", "bf16", 64, 8, 131072, False),
        # four beams of one chat: bookkeeping alone
        _reorder("reorder_1x4", 32, 8, 128, 1, 4, 4099, 0),
        # sixteen searches of eight beams with a 16-bit window in every layer
        _reorder("reorder_16x8_window", 16, 8, 128, 16, 8, 2048, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["prefix_attention", "prefix_attention", "beam_select", "reorder"])
    if op == "prefix_attention":
        d = rng.choice([128, 128, 256])
        h, g = rng.choice([(8, 4), (4, 2), (8, 8), (4, 1), (2, 5)])
        groups = _log(rng, 1, 8)
        beams = _log(rng, 1, max(1, 64 // groups))
        new = 1 if rng.random() < 0.4 else _log(rng, 1, 200)
        # score pairs and cached values stay below the largest listed case's
        room = min(32768, 400_000_000 // (groups * beams * new * h * g), 100_000_000 // (groups * beams * h * (d // 128)))
        own_tokens = new + _log(rng, 1, max(1, min(1024, room // 2)))
        return _attn("", rng.choice(["q4", "rot4"]), rng.choice(["fp16", "bf16"]), groups, beams, h, g, d,
                     _log(rng, 1, max(1, room)), own_tokens, new, rng.choice([0, 0, 128]), rng.random() < 0.6)
    if op == "beam_select":
        groups = _log(rng, 1, 64)
        beams = _log(rng, 1, 32)
        top = min(131072, 60_000_000 // (groups * beams))
        return _select("", rng.choice(["fp16", "bf16", "fp32"]), groups, beams, _log(rng, min(300, top), top), rng.random() < 0.5)
    layers, h = _log(rng, 1, 32), rng.choice([2, 4, 8])
    groups = _log(rng, 1, 16)
    beams = _log(rng, 2, max(2, min(32, 128 * 16 * 8 // (groups * layers * h))))
    return _reorder("", layers, h, 128, groups, beams, _log(rng, 1, 4099), rng.choice([0, 128]))


# ---- shapes that follow from a case ----------------------------------------------


def _lengths(case):
    """(prefix of every group; cached tokens and new tokens of every sequence, the new ones being the last cached)."""
    G, K = case["groups"], case["beams"]
    pre = [case["prefix"]] * G
    own_t, n = [case["own_tokens"]] * (G * K), [case["new"]] * (G * K)
    if case["ragged"]:
        pre = [max(1, p - (1237 * i) % (p // 2 + 1)) for i, p in enumerate(pre)]
        n = [max(1, x - (3 * i) % (x // 2 + 1)) for i, x in enumerate(n)]
        own_t = [max(a, t - (97 * i) % (t // 2 + 1)) for i, (t, a) in enumerate(zip(own_t, n))]
    return pre, [pre[i // K] + t for i, t in enumerate(own_t)], n


def _row_bytes(case):
    per = BLOCK[case["format"]]
    return case["head_dim"] // per * (2 + per // 2)


def work(case):
    if case["op"] == "prefix_attention":
        d, h, g, K = case["head_dim"], case["kv_heads"], case["group"], case["beams"]
        pre, t, n = _lengths(case)
        nbytes = flops = 0
        for i, p in enumerate(pre):
            shared = p // PAGE * PAGE
            nbytes += 2 * h * shared * _row_bytes(case)
            for b in range(i * K, i * K + K):
                raw = min(case["window16"], t[b] - shared)  # tokens of the 16-bit window behind the shared pages
                nbytes += 2 * h * ((t[b] - shared - raw) * _row_bytes(case) + raw * d * 2) + 2 * 2 * n[b] * h * g * d
                flops += 4 * d * h * g * sum(range(t[b] - n[b] + 1, t[b] + 1))
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "beam_select":
        x = case["groups"] * case["beams"] * case["vocab"]
        return {"bytes": x * DTYPES[case["dtype"]].itemsize + 24 * case["groups"] * case["beams"], "flops": 4 * x}
    B, K = case["groups"] * case["beams"], case["beams"]
    window = (case["window16"] + 1 if case["window16"] else 0) * case["kv_heads"] * case["head_dim"] * 2 * 2 * case["layers"]
    kept = (K + 1) // 2  # beams that live on, with two children each; about one of the slots keeps its place
    moved = case["groups"] * (K - 1 + min(kept, K - 1)) * window
    return {"bytes": moved + 2 * 4 * B * _columns(case), "flops": 0}


def _columns(case):
    return -(-(case["context"] + 1) // PAGE) + 1


# ---- inputs -----------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _pack4(x, per):
    """Blocks of `per` values along the last axis: fp16 scale, then code + 8 in nibbles, low nibble first."""
    b = x.unflatten(-1, (-1, per))
    scale = (b.abs().amax(-1) / 7).clamp(max=65504).half()
    s = scale.float().unsqueeze(-1)
    code = torch.where(s > 0, torch.round(b / torch.where(s > 0, s, 1.0)).clamp(-7, 7), 0.0).to(torch.int32) + 8
    nib = (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8)
    return torch.cat([scale.unsqueeze(-1).contiguous().view(torch.uint8), nib], -1).flatten(-2)


def _attn_inputs(case, seed):
    """Queries and a filled paged cache, one layer: a group's sequences share the whole pages of their prefix."""
    g = _gen(seed)
    G, K, h, d = case["groups"], case["beams"], case["kv_heads"], case["head_dim"]
    dt, B, R = DTYPES[case["dtype"]], G * K, case["window16"]
    pre, t, n = _lengths(case)
    per_seq = -(-max(t) // PAGE)
    shared = [p // PAGE for p in pre]
    n_shared = sum(shared)
    own_pages = [-(-t[b] // PAGE) - shared[b // K] for b in range(B)]
    pages = n_shared + sum(own_pages) + 3
    s = {"case": case}
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, per_seq), -1, dtype=torch.int32, device="cuda")
    at, first = n_shared, [sum(shared[:i]) for i in range(G)]
    for b in range(B):
        i = b // K
        table[b, : shared[i]] = perm[first[i]: first[i] + shared[i]]
        table[b, shared[i]: shared[i] + own_pages[b]] = perm[at: at + own_pages[b]]
        at += own_pages[b]
    s["table"] = table
    for name in ("k_main", "v_main"):
        x = torch.randn((pages, h, PAGE, d), generator=g, device="cuda")
        if name == "v_main":
            x *= torch.exp(0.5 * torch.randn((pages, 1, PAGE, 1), generator=g, device="cuda"))
        s[name] = _pack4(x, BLOCK[case["format"]])
        del x
    s["k_resid"] = s["v_resid"] = None
    if R:
        for name in ("k_resid", "v_resid"):
            s[name] = torch.randn((B, h, R + 1, d), generator=g, device="cuda").to(dt)
    s["seq_lens"] = torch.tensor(t, dtype=torch.int32, device="cuda")
    s["cu_q"] = torch.tensor([sum(n[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
    s["cu_groups"] = torch.arange(0, B + 1, K, dtype=torch.int32, device="cuda")
    s["total_q"], s["max_q"], s["max_t"] = sum(n), max(n), max(t)
    s["max_group_q"] = max(sum(n[i * K:i * K + K]) for i in range(G))
    s["q"] = torch.randn((1, sum(n), h * case["group"], d), generator=g, device="cuda").to(dt)
    s["out"] = torch.empty_like(s["q"])
    return s


def _select_inputs(case, seed):
    g = _gen(seed)
    G, K, V = case["groups"], case["beams"], case["vocab"]
    x = 2.5 * torch.randn((G, K, V), generator=g, device="cuda")
    x[..., V - 1 - V // 50:] = -math.inf  # tokens that may not follow
    s = {"case": case, "logits": x.to(DTYPES[case["dtype"]])}
    s["scores"] = -10 - 3 * torch.rand((G, K), generator=g, device="cuda")  # beams that a search keeps lie close together
    s["done"] = None
    if case["finished"]:
        s["done"] = (torch.rand((G, K), generator=g, device="cuda") < 0.2).to(torch.int32)
    s["out"] = (torch.empty((G, K), dtype=torch.float32, device="cuda"),
                *(torch.empty((G, K), dtype=torch.int32, device="cuda") for _ in range(3)))
    return s


def _reorder_inputs(case, seed):
    g = _gen(seed)
    G, K = case["groups"], case["beams"]
    B, cols = G * K, _columns(case)
    end = max(0, case["context"] - case["window16"])
    full = -(-end // PAGE)
    shared = full * 3 // 4  # the prompt's pages, then every beam's own
    pages = G * shared + B * (cols - shared) + 5
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
    table[:, :shared] = perm[: G * shared].view(G, 1, shared).expand(G, K, shared).reshape(B, shared)
    table[:, shared:full] = perm[G * shared: G * shared + B * (full - shared)].view(B, full - shared)
    s = {"case": case, "table": table}
    s["refs"] = torch.bincount(table[table >= 0].long(), minlength=pages).to(torch.int32)
    s["seq_lens"] = torch.full((B,), case["context"], dtype=torch.int32, device="cuda")
    behind = torch.randint(0, 2, (B,), generator=g, device="cuda", dtype=torch.int32)  # a finished beam is a token behind
    s["seq_lens"] -= behind * (end % PAGE != 1)  # in the same pages: none holds pages that it has not begun
    live = torch.rand((G, K), generator=g, device="cuda").argsort(-1)[:, : (K + 1) // 2]  # each with two children
    mix = torch.rand((G, K), generator=g, device="cuda").argsort(-1)
    s["parents"] = live.repeat(1, 2)[:, :K].gather(1, mix).to(torch.int32)
    s["k_resid"] = s["v_resid"] = None
    if case["window16"]:
        ring = (case["layers"], B, case["kv_heads"], case["window16"] + 1, case["head_dim"])
        s["k_resid"] = torch.randn(ring, generator=g, device="cuda", dtype=torch.float16)
        s["v_resid"] = torch.randn(ring, generator=g, device="cuda", dtype=torch.float16)
    return s


def prepare(case, seed):
    s = {"prefix_attention": _attn_inputs, "beam_select": _select_inputs, "reorder": _reorder_inputs}[case["op"]](case, seed)
    if own:
        s["own"] = _handle(case, s)
    return s


# ---- the framework's calls -----------------------------------------------------------


def _handle(case, s):
    """What a user's program keeps: the cache over its buffers, the page pool, workspaces."""
    from bit_kv_cache_04_gb300 import kvq as K

    if case["op"] == "beam_select":
        return K.BeamSelect(case["groups"], case["beams"], case["vocab"])
    table, h, d = s["table"], case["kv_heads"], case["head_dim"]
    rotated = case.get("format", "rot4") == "rot4"
    fmt = dict(k_fmt=K.Fmt(4, 128), v_fmt=K.Fmt(4, 128), flags=K.ROTATE_K | K.ROTATE_V, sign_seed=SIGN_SEED) if rotated else dict(
        k_fmt=K.Fmt(4, 32), v_fmt=K.Fmt(4, 32))
    pages = s["k_main"].shape[0] if "k_main" in s else s["refs"].numel()
    cfg = K.Config(L=case.get("layers", 1), H_kv=h, H_q=h * case.get("group", 1), D=d, batch=table.shape[0],
                   max_T=table.shape[1] * PAGE, in_dtype=K.DT_BF16 if case.get("dtype") == "bf16" else K.DT_F16,
                   residual_window=case["window16"], page_tokens=PAGE, n_pages=pages, max_pages_per_seq=table.shape[1], **fmt)
    buffers = {x: s[x] for x in ("k_main", "v_main", "k_resid", "v_resid") if s.get(x) is not None}
    if case["op"] == "reorder":  # the pages' bytes stay where they are
        for x in ("k_main", "v_main"):
            buffers[x] = torch.empty(K.kvq_buffer_sizes(cfg)[0], dtype=torch.uint8, device="cuda")
    cache = K.KVCache.from_buffers(cfg, buffers, block_table=table)
    if case["op"] == "reorder":
        return K.PagePool(cache, s["refs"])
    return K.PrefixAttention(cache, case["groups"], s["total_q"])


def _run_own(s):
    case, o = s["case"], s["own"]
    if case["op"] == "prefix_attention":
        o.plan(s["cu_groups"], s["cu_q"], s["total_q"], s["max_q"], s["max_group_q"], s["seq_lens"])
        o.attention(0, 1, s["q"], s["out"])
        return s["out"]
    if case["op"] == "beam_select":
        scores, tokens, parents, done = s["out"]
        o.select(s["logits"], s["scores"], scores, tokens, parents, done=s["done"], done_out=done, eos=EOS)
        return s["out"]
    o.reorder(s["parents"].view(-1), case["beams"], s["seq_lens"])
    return _reorder_state(s)


def _reorder_state(s):
    return {x: s[x] for x in ("table", "refs", "seq_lens", "k_resid", "v_resid") if s[x] is not None}


# ---- the plain forms -------------------------------------------------------------------


def _unpack4(x, per):
    b = x.unflatten(-1, (-1, 2 + per // 2))
    scale = b[..., :2].contiguous().view(torch.float16).float()
    nib = b[..., 2:]
    code = torch.stack([nib & 15, nib >> 4], -1).flatten(-2).float() - 8
    return (code * scale).flatten(-2)


def _transform(device):
    """The 128-point transform of the rotated format as a matrix, y = x @ R; its signs are SplitMix64's first four words."""
    mask, state, bits = (1 << 64) - 1, SIGN_SEED, []
    while len(bits) < 256:
        state = (state + 0x9E3779B97F4A7C15) & mask
        z = state
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & mask
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
        z ^= z >> 31
        bits += [(z >> i) & 1 for i in range(64)]
    sign = 1.0 - 2.0 * torch.tensor(bits, dtype=torch.float32, device=device)
    i = torch.arange(128, device=device)
    p = i[:, None] & i[None, :]
    p = p ^ (p >> 4)
    p = p ^ (p >> 2)
    p = (p ^ (p >> 1)) & 1
    return sign[:128, None] * (1.0 - 2.0 * p.float()) * sign[None, 128:] / math.sqrt(128.0)


def _rotate(x, r):
    return (x.unflatten(-1, (-1, 128)) @ r).flatten(-2)


def _plain_cache(s):
    """Every cached token's key and value in 32 bits, in the rotated domain where the format has one: [b][h][token][d]."""
    case, got = s["case"], []
    for name in ("k_main", "v_main"):
        x = _unpack4(s[name], BLOCK[case["format"]])[s["table"].long().clamp(min=0)].transpose(1, 2).flatten(2, 3)
        if case["window16"]:
            t = torch.arange(x.shape[2], device="cuda")
            raw = s[name[0] + "_resid"].float()[:, :, t % (case["window16"] + 1)]
            if case["format"] == "rot4":
                raw = _rotate(raw, _transform("cuda"))
            late = t[None] >= (s["seq_lens"].long() - case["window16"]).clamp(min=0)[:, None]
            x = torch.where(late[:, None, :, None], raw, x)
        got.append(x)
    return got


def _plain_attention(s):
    case = s["case"]
    B, h, g, d = case["groups"] * case["beams"], case["kv_heads"], case["group"], case["head_dim"]
    k, v = _plain_cache(s)
    cu, lens = s["cu_q"].long(), s["seq_lens"].long()
    n = cu[1:] - cu[:-1]
    row = torch.arange(s["max_q"], device="cuda")
    at = (cu[:-1, None] + row[None]).clamp(max=s["total_q"] - 1)  # [b][max_q], padded rows repeat others
    q = s["q"][0].float()[at]
    if case["format"] == "rot4":
        q = _rotate(q, _transform("cuda"))
    q = q.unflatten(2, (h, g)).permute(0, 2, 1, 3, 4).reshape(B, h, -1, d)
    score = (q @ k.transpose(2, 3)).div_(math.sqrt(d)).view(B, h, s["max_q"], g, -1)
    pos = (lens - n)[:, None] + row[None]
    seen = torch.arange(k.shape[2], device="cuda") <= pos[..., None]
    score.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    score -= score.amax(-1, keepdim=True)
    p = score.exp_()
    p /= p.sum(-1, keepdim=True)
    out = (p.view(B, h, -1, k.shape[2]) @ v).view(B, h, s["max_q"], g, d).permute(0, 2, 1, 3, 4).reshape(B, s["max_q"], h * g, d)
    if case["format"] == "rot4":
        out = _rotate(out, _transform("cuda").t())
    return out[row[None] < n[:, None]].to(s["q"].dtype)[None]


def _plain_select(s):
    G, K, V = s["logits"].shape
    x = s["logits"].double()
    m = x.amax(-1, keepdim=True)
    c = x - (m + (x - m).exp().sum(-1, keepdim=True).log()) + s["scores"].double().unsqueeze(-1)
    if s["done"] is not None:  # a finished beam goes on as it is, with the end token
        one = torch.full_like(c, -math.inf)
        one[..., EOS] = s["scores"].double()
        c = torch.where(s["done"].bool().unsqueeze(-1), one, c)
    value, at = torch.sort(c.view(G, K * V), dim=-1, descending=True, stable=True)
    value, at = value[:, :K], at[:, :K]
    tokens, parents = at % V, at // V
    done = tokens == EOS
    if s["done"] is not None:
        done |= s["done"].bool().gather(1, parents)
    return value.float(), tokens.to(torch.int32), parents.to(torch.int32), done.to(torch.int32)


def _plain_reorder(s):
    case, table, refs = s["case"], s["table"], s["refs"]
    B, K = table.shape[0], case["beams"]
    src = torch.arange(B, device="cuda") // K * K + s["parents"].view(-1).long()
    new = table[src]
    for t, sign in ((table, -1), (new, 1)):
        refs.index_add_(0, t.flatten().long().clamp(min=0), sign * (t.flatten() >= 0).to(torch.int32))
    table.copy_(new)
    s["seq_lens"].copy_(s["seq_lens"][src])
    if case["window16"]:
        s["k_resid"].copy_(s["k_resid"][:, src])
        s["v_resid"].copy_(s["v_resid"][:, src])
    return _reorder_state(s)


def run(s):
    if own:
        return _run_own(s)
    return {"prefix_attention": _plain_attention, "beam_select": _plain_select, "reorder": _plain_reorder}[s["case"]["op"]](s)


# ---- 64 bits, from the definitions ---------------------------------------------------------


def _exact_values(block, per):
    """Values of packed blocks [..][2 + per / 2], each element on its own."""
    i = torch.arange(per, device=block.device)
    byte = block[..., 2 + i // 2].to(torch.int64)
    code = torch.bitwise_and(torch.bitwise_right_shift(byte, 4 * (i % 2)), 15) - 8
    bits = block[..., 0].to(torch.int64) + 256 * block[..., 1].to(torch.int64)
    sign, e, m = bits >> 15, (bits >> 10) & 31, bits & 1023
    mag = torch.where(e > 0, (1024 + m).double() * torch.pow(2.0, e.double() - 25), m.double() * 2.0 ** -24)
    return code.double() * (torch.where(sign > 0, -mag, mag)).unsqueeze(-1)


def _exact_attention(case, seed):
    s = _attn_inputs(case, seed)
    h, g, d, R, per = case["kv_heads"], case["group"], case["head_dim"], case["window16"], BLOCK[case["format"]]
    _, t, n = _lengths(case)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    r = torch.sign(_transform("cuda").double()) / math.sqrt(128.0)
    first = 0
    for b in range(len(t)):
        page = s["table"][b][: -(-t[b] // PAGE)].long()
        kv = []
        for name in ("k_main", "v_main"):
            x = s[name][page].permute(1, 0, 2, 3).flatten(1, 2)[:, : t[b]]  # [head][token][bytes]
            x = _exact_values(x.reshape(h, t[b], d // per, 2 + per // 2), per)
            x = (x @ r.t() if case["format"] == "rot4" else x).reshape(h, t[b], d)  # back from the rotated domain
            if R:
                late = torch.arange(max(0, t[b] - R), t[b], device="cuda")
                x[:, late] = s[name[0] + "_resid"][b].double()[:, late % (R + 1)]
            kv.append(x)
        q = s["q"][0, first:first + n[b]].double().view(n[b], h, g, d)
        z = torch.einsum("ihgd,htd->hgit", q, kv[0]) / math.sqrt(d)
        hide = torch.arange(t[b], device="cuda")[None] > torch.arange(t[b] - n[b], t[b], device="cuda")[:, None]
        z = torch.softmax(z.masked_fill(hide, -math.inf), -1)
        out[0, first:first + n[b]] = torch.einsum("hgit,htd->ihgd", z, kv[1]).reshape(n[b], h * g, d)
        first += n[b]
    return out


def _exact_select(case, seed):
    s = _select_inputs(case, seed)
    G, K, V = s["logits"].shape
    best = torch.empty((G, K), dtype=torch.float64, device="cuda")
    for i in range(G):
        found = []
        for b in range(K):
            score = s["scores"][i, b].double()
            if s["done"] is not None and s["done"][i, b]:
                found.append(score[None])
                continue
            x = s["logits"][i, b].double()
            found.append(torch.topk(torch.log_softmax(x, 0), min(K, V)).values + score)
        best[i] = torch.cat(found).sort(descending=True).values[:K]
    return best, None, None, None


def exact(case, seed):
    if case["op"] == "prefix_attention":
        return _exact_attention(case, seed)
    if case["op"] == "beam_select":
        return _exact_select(case, seed)
    return None  # states are moved: whole numbers and copies, compared as they are
