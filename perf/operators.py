"""Cases of the serving operators around the quantized cache, for measurement.

Three families, as one serving step uses them:
  * qk_norm_rope: a fused projection's queries and keys get their per-head RMS
    norm and their rotary turn, ready for append and attention;
  * branch / compact: pages of a paged cache: children released, forked from
    their parents and given a private last page; used pages moved together;
  * chunk_attention: the newest tokens of every sequence (one when decoding, a
    few when verifying a draft, thousands when prefilling) attend to the packed
    cache, causally, over a sliding window plus the first `sinks` tokens.

`own` False computes them in elementary torch operations in 32 bits (64 for
angles); `own` True calls the framework.
"""

import math
import random

import torch

own = False

AXIS_TOKEN, AXIS_CHANNEL = 0, 1
KIVI_WINDOW, GROUP = 128, 32  # 16-bit window and token group of the per-channel format
PAGE = 16
SIGN_SEED = 0x5EED5EED
EPS = 1e-6
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---- the cases -----------------------------------------------------------------


def _attn(name, fmt, dtype, batch, kv_heads, group, head_dim, context, ragged, new, window, sinks):
    c = dict(op="chunk_attention", format=fmt, dtype=dtype, batch=batch, kv_heads=kv_heads, group=group,
             head_dim=head_dim, context=context, ragged=ragged, new=new, window=window, sinks=sinks)
    return dict(c, name=name) if name else c


def _rope(name, dtype, tokens, heads, kv_heads, head_dim, rot_dim, interleaved, norm, scaling, factor, reach):
    c = dict(op="qk_norm_rope", dtype=dtype, tokens=tokens, heads=heads, kv_heads=kv_heads, head_dim=head_dim,
             rot_dim=rot_dim, interleaved=interleaved, norm=norm, scaling=scaling, factor=factor, reach=reach)
    return dict(c, name=name) if name else c


def _branch(name, layers, kv_heads, head_dim, parents, width, context, window):
    c = dict(op="branch", layers=layers, kv_heads=kv_heads, head_dim=head_dim, parents=parents, width=width,
             context=context, window=window)
    return dict(c, name=name) if name else c


def _compact(name, layers, kv_heads, head_dim, pages, used, batch):
    c = dict(op="compact", layers=layers, kv_heads=kv_heads, head_dim=head_dim, pages=pages, used=used, batch=batch)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user, one new token, a long chat read through a sliding window: latency
        _attn("decode_1_window", "kivi4", "fp16", 1, 8, 4, 128, 32768, False, 1, 4096, 4),
        # a full batch decoding over a paged rotated cache of mixed lengths
        _attn("decode_64_paged_window", "rot4_paged", "fp16", 64, 8, 4, 128, 8192, True, 1, 4096, 4),
        # drafts of up to 8 tokens verified against the whole history of 16 chats
        _attn("verify_16", "kivi4", "fp16", 16, 8, 4, 128, 32768, True, 8, 0, 0),
        # an odd chunk of a prompt, wide heads, bf16, full causal attention
        _attn("chunk_1000_wide", "rot4", "bf16", 1, 4, 6, 256, 20011, False, 1000, 0, 0),
        # prefill chunks of two long prompts under a sliding window with sinks
        _attn("chunk_2x2048_window", "rot4_paged", "fp16", 2, 8, 4, 128, 32768, True, 2048, 4096, 4),
        # the one token of a decode step
        _rope("rope_1", "fp16", 1, 32, 8, 128, 128, False, False, "none", 1.0, 32768),
        # a prefill batch: norm and half-split turn in one pass
        _rope("norm_rope_8192", "bf16", 8192, 32, 8, 128, 128, False, True, "none", 1.0, 32768),
        # part of a wide head, interleaved pairs, frequencies stretched for a long context
        _rope("rope_1777_long", "bf16", 1777, 24, 4, 256, 64, True, True, "yarn", 8.0, 262144),
        # two prompts, two samples each, one layer group
        _branch("branch_2x2", 16, 4, 256, 2, 2, 4099, 0),
        # 16 prompts, 4 samples each, all layers, a 16-bit window beside the pages
        _branch("branch_16x4", 32, 8, 128, 16, 4, 1021, 128),
        # a small pool after a few chats ended
        _compact("compact_500", 4, 8, 128, 500, 0.5, 8),
        # a large pool, half empty
        _compact("compact_6000", 32, 8, 128, 6000, 0.5, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["chunk_attention", "chunk_attention", "qk_norm_rope", "branch", "compact"])
    if op == "chunk_attention":
        d = rng.choice([128, 128, 256])
        fmt = rng.choice(["kivi4", "rot4", "rot4_paged"])
        h, g = rng.choice([(8, 4), (4, 6), (8, 8), (4, 1), (2, 5)])
        batch = _log(rng, 1, 64)
        new = 1 if rng.random() < 0.3 else _log(rng, 1, 2048)
        # pairs and cached values stay below the largest listed case's
        top = max(new + 1, min(32768, 2_000_000_000 // (batch * new * h * g), 60_000_000 // (batch * h)))
        if top <= new + 1:
            batch, top = 1, max(new + 1, min(32768, 2_000_000_000 // (new * h * g)))
        context = _log(rng, new + 1, top)
        window = rng.choice([0, _log(rng, 1, 8192)])
        sinks = 0 if not window else rng.choice([0, 1, 4, 129])
        return _attn("", fmt, rng.choice(["fp16", "bf16"]), batch, h, g, d, context, rng.random() < 0.6, new, window,
                     sinks)
    if op == "qk_norm_rope":
        d = rng.choice([128, 256])
        h, g = rng.choice([(8, 4), (4, 6), (8, 8), (4, 1), (2, 5)])
        rot = rng.choice([d, d // 2, 64, 34, 2 * rng.randint(1, d // 2)])
        scaling = rng.choice(["none", "linear", "ntk", "yarn", "bands"])
        return _rope("", rng.choice(["fp16", "bf16"]), _log(rng, 1, 8192), h * g, h, d, rot, rng.random() < 0.5,
                     rng.random() < 0.5, scaling, 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
                     _log(rng, 64, 1 << 20))
    if op == "branch":
        d = rng.choice([128, 256])
        return _branch("", _log(rng, 1, 32), rng.choice([2, 4, 8]), d, _log(rng, 1, 16), _log(rng, 1, 4),
                       _log(rng, 1, 1021 if d == 256 else 2048), rng.choice([0, 128]))
    layers, h = _log(rng, 1, 32), rng.choice([2, 4, 8])
    return _compact("", layers, h, rng.choice([128, 256]), _log(rng, 3, max(3, 6000 * 128 // (layers * h))),
                    rng.uniform(0.1, 0.95), _log(rng, 1, 64))


# ---- shapes that follow from a case ----------------------------------------------


def _lengths(case):
    """(cached tokens, new tokens) of every sequence: the chunk is the last of the cached tokens."""
    new, context, b = case["new"], case["context"], case["batch"]
    if not case["ragged"]:
        return [context] * b, [new] * b
    n = [max(1, new - (5 * i) % (new // 2 + 1)) for i in range(b)]
    t = [max(n[i], context - (977 * i) % (context // 2 + 1)) for i in range(b)]
    return t, n


def _quantized_end(case, t):
    """First token still in the 16-bit window."""
    if case["format"] != "kivi4":
        return t
    return max(0, t - KIVI_WINDOW) // GROUP * GROUP


def _block_bytes(case):
    return (18, 32) if case.get("format") == "kivi4" else (66, 128)


def work(case):
    if case["op"] == "chunk_attention":
        d, h, g = case["head_dim"], case["kv_heads"], case["group"]
        bb, per = _block_bytes(case)
        nbytes = flops = 0
        for t, n in zip(*_lengths(case)):
            first, w, s = t - n, case["window"], case["sinks"]
            lo = max(0, first - w + 1) if w else 0
            seen = t - lo + min(s, lo)  # keys that some new token sees
            raw = min(seen, t - _quantized_end(case, t))
            nbytes += h * (2 * (seen - raw) * d * bb // per + 2 * raw * d * 2) + 2 * n * h * g * d * 2
            for p in range(first, t):
                low = max(0, p - w + 1) if w else 0
                flops += 4 * d * h * g * (p + 1 - low + min(s, low))
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "qk_norm_rope":
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["head_dim"]
        return {"bytes": 2 * 2 * n + 4 * case["tokens"], "flops": n * (6 if case["norm"] else 3)}
    row = case["head_dim"] // 128 * 66
    page = case["layers"] * case["kv_heads"] * PAGE * row * 2  # one page over all layers, K and V
    if case["op"] == "branch":
        kids = case["parents"] * case["width"]
        end = max(0, case["context"] - case["window"])
        ring = (case["window"] + 1 if case["window"] else 0) * case["kv_heads"] * case["head_dim"] * 2 * 2 * case["layers"]
        copied = kids * (page if end % PAGE else 0) + kids * ring
        return {"bytes": 2 * copied + kids * 3 * 4 * -(-(case["context"] + 1) // PAGE), "flops": 0}
    used, pages = _used(case), case["pages"]
    moved = round(used * (pages - used) / pages)  # used pages behind the first `used`, on average
    return {"bytes": 2 * moved * page + 2 * 4 * pages + 2 * 4 * case["batch"] * _row(case), "flops": 0}


def _used(case):
    return max(1, min(case["pages"] - 1, round(case["pages"] * case["used"])))


def _row(case):
    return -(-_used(case) // case["batch"]) + 2


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
    """Queries and a filled cache in the packed layout, one layer."""
    g = _gen(seed)
    b, h, d = case["batch"], case["kv_heads"], case["head_dim"]
    dt = DTYPES[case["dtype"]]
    t, n = _lengths(case)
    cap = -(-max(t) // 32) * 32
    k = torch.randn((b, h, cap, d), generator=g, device="cuda")
    hot = torch.randperm(d, generator=g, device="cuda")[: max(1, d // 50)]
    if case["format"] == "kivi4":
        k[..., hot] *= 15.0  # outlier channels, as keys have
    v = torch.randn((b, h, cap, d), generator=g, device="cuda")
    v *= torch.exp(0.5 * torch.randn((b, 1, cap, 1), generator=g, device="cuda"))
    k, v = k.to(dt).float(), v.to(dt).float()
    s = {"case": case}
    s["seq_lens"] = torch.tensor(t, dtype=torch.int32, device="cuda")
    s["cu_q"] = torch.tensor([sum(n[:i]) for i in range(b + 1)], dtype=torch.int32, device="cuda")
    s["total_q"], s["max_q"], s["max_t"] = sum(n), max(n), max(t)
    s["q"] = torch.randn((1, sum(n), h * case["group"], d), generator=g, device="cuda").to(dt)
    s["table"] = s["k_resid"] = s["v_resid"] = None
    if case["format"] == "kivi4":
        s["k_main"] = _pack4(k.unflatten(2, (-1, 32)).transpose(3, 4), 32).flatten(-2)  # [b][h][token group][channel blocks]
        s["v_main"] = _pack4(v, 32)
        ring = KIVI_WINDOW + GROUP
        slot = torch.arange(ring, device="cuda")
        last = s["seq_lens"].long()[:, None] - 1
        tok = (last - (last - slot) % ring).clamp(min=0)  # the newest token of each slot
        at = tok[:, None, :, None].expand(b, h, ring, d)
        s["k_resid"], s["v_resid"] = k.gather(2, at).to(dt), v.gather(2, at).to(dt)
    else:
        s["k_main"], s["v_main"] = _pack4(k, 128), _pack4(v, 128)  # values of the rotated domain
        if case["format"] == "rot4_paged":
            per_seq = -(-max(t) // PAGE)
            pages = b * per_seq + 3
            perm = torch.randperm(pages, generator=g, device="cuda")
            s["table"] = perm[: b * per_seq].view(b, per_seq).to(torch.int32)
            for name in ("k_main", "v_main"):
                rows = s[name]
                pool = torch.zeros((pages, h, PAGE, rows.shape[-1]), dtype=torch.uint8, device="cuda")
                paged = rows[:, :, : per_seq * PAGE].unflatten(2, (per_seq, PAGE)).transpose(1, 2)
                pool[s["table"].long().flatten()] = paged.flatten(0, 1)
                s[name] = pool
    s["out"] = torch.empty_like(s["q"])
    return s


def _rope_inputs(case, seed):
    g = _gen(seed)
    n, hq, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"]
    dt = DTYPES[case["dtype"]]
    qkv = torch.randn((n, (hq + 2 * hk) * d), generator=g, device="cuda").to(dt)  # a fused projection's output
    s = {"case": case, "q": qkv[:, : hq * d].unflatten(1, (hq, d)), "k": qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))}
    s["positions"] = torch.randint(0, case["reach"], (n,), generator=g, device="cuda", dtype=torch.int32)
    s["q_weight"] = s["k_weight"] = None
    if case["norm"]:
        s["q_weight"] = (1 + 0.2 * torch.randn((d,), generator=g, device="cuda")).to(dt)
        s["k_weight"] = (1 + 0.2 * torch.randn((d,), generator=g, device="cuda")).to(dt)
    s["q_out"] = torch.empty((n, hq, d), dtype=dt, device="cuda")
    s["k_out"] = torch.empty((n, hk, d), dtype=dt, device="cuda")
    return s


ROPE = dict(theta=500000.0, original=8192, low=1.0, high=4.0, slow=1.0, fast=32.0)


def _pool(case, pages, seed):
    g = _gen(seed)
    row = case["head_dim"] // 128 * 66
    shape = (case["layers"], pages, case["kv_heads"], PAGE, row)
    # scales and codes of stored keys and values; copying takes them as they are
    k = torch.randint(0, 120, shape, generator=g, device="cuda", dtype=torch.uint8)
    v = torch.randint(0, 120, shape, generator=g, device="cuda", dtype=torch.uint8)
    return g, k, v


def _branch_inputs(case, seed):
    par, kids = case["parents"], case["parents"] * case["width"]
    end = max(0, case["context"] - case["window"])
    full, cols = -(-end // PAGE), -(-(case["context"] + 1) // PAGE) + 1
    pages = par * full + kids * (cols - full + 1) + 5
    g, k, v = _pool(case, pages, seed)
    s = {"case": case, "k_main": k, "v_main": v}
    table = torch.full((par + kids, cols), -1, dtype=torch.int32, device="cuda")
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table[:par, :full] = perm[: par * full].view(par, full)
    s["table"] = table
    s["refs"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
    s["refs"][perm[: par * full].long()] = 1
    s["seq_lens"] = torch.zeros(par + kids, dtype=torch.int32, device="cuda")
    s["seq_lens"][:par] = case["context"]
    s["kids"] = torch.arange(par, par + kids, dtype=torch.int32, device="cuda")
    s["from"] = torch.arange(kids, dtype=torch.int32, device="cuda") % par
    s["n_new"] = torch.ones(kids, dtype=torch.int32, device="cuda")
    s["k_resid"] = s["v_resid"] = None
    if case["window"]:
        ring = (case["layers"], par + kids, case["kv_heads"], case["window"] + 1, case["head_dim"])
        s["k_resid"] = torch.randn(ring, generator=g, device="cuda", dtype=torch.float16)
        s["v_resid"] = torch.randn(ring, generator=g, device="cuda", dtype=torch.float16)
    return s


def _compact_inputs(case, seed):
    pages, used, b, cols = case["pages"], _used(case), case["batch"], _row(case)
    g, k, v = _pool(case, pages, seed)
    s = {"case": case, "k_main": k, "v_main": v}
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[:used]
    table = torch.full((b * (cols - 2),), -1, dtype=torch.int32, device="cuda")
    table[:used] = perm
    table = torch.nn.functional.pad(table.view(cols - 2, b).t(), (0, 2), value=-1).contiguous()
    if b > 1:  # a shared first page, as after a fork
        share = table[0, 0].clone()
        table[b - 1, cols - 2] = share
    s["table"] = table
    s["refs"] = torch.bincount(table[table >= 0].long(), minlength=pages).to(torch.int32)
    s["table_out"], s["refs_out"] = torch.empty_like(table), torch.empty_like(s["refs"])
    return s


def prepare(case, seed):
    make = {"chunk_attention": _attn_inputs, "qk_norm_rope": _rope_inputs, "branch": _branch_inputs,
            "compact": _compact_inputs}[case["op"]]
    s = make(case, seed)
    if own:
        s["own"] = _handle(case, s)
    return s


# ---- the framework's calls -----------------------------------------------------------


def _handle(case, s):
    """What a user's program keeps: the cache object over its buffers, the page pool, the rotary plan."""
    from bit_kv_cache_04_gb300 import kvq as K

    dt = K.DT_BF16 if case.get("dtype") == "bf16" else K.DT_F16
    d, h = case["head_dim"], case["kv_heads"]
    if case["op"] == "qk_norm_rope":
        cfg = K.Config(L=1, H_kv=h, H_q=case["heads"], D=d, batch=1, max_T=1, in_dtype=dt)
        scaling = {"none": K.ROPE_NONE, "linear": K.ROPE_LINEAR, "ntk": K.ROPE_NTK, "yarn": K.ROPE_YARN,
                   "bands": K.ROPE_BANDS}[case["scaling"]]
        plan = K.rope_plan(D=d, rot_dim=case["rot_dim"], interleaved=case["interleaved"], theta=ROPE["theta"],
                           scaling=scaling, factor=case["factor"], original_len=ROPE["original"],
                           low=ROPE["slow"] if case["scaling"] == "yarn" else ROPE["low"],
                           high=ROPE["fast"] if case["scaling"] == "yarn" else ROPE["high"])
        return {"K": K, "cfg": cfg, "plan": plan}
    table = s["table"]
    if case["op"] == "chunk_attention":
        kivi = case["format"] == "kivi4"
        fmt = dict(k_fmt=K.Fmt(4, 32, K.AXIS_CHANNEL), v_fmt=K.Fmt(4, 32), residual_window=KIVI_WINDOW) if kivi else dict(
            k_fmt=K.Fmt(4, 128), v_fmt=K.Fmt(4, 128), flags=K.ROTATE_K | K.ROTATE_V, sign_seed=SIGN_SEED)
        if table is not None:
            fmt |= dict(page_tokens=PAGE, n_pages=s["k_main"].shape[0], max_pages_per_seq=table.shape[1])
        cfg = K.Config(L=1, H_kv=h, H_q=h * case["group"], D=d, batch=case["batch"], max_T=s["max_t"], in_dtype=dt, **fmt)
    else:
        cfg = K.Config(L=case["layers"], H_kv=h, H_q=h, D=d, batch=table.shape[0], max_T=table.shape[1] * PAGE,
                       k_fmt=K.Fmt(4, 128), v_fmt=K.Fmt(4, 128), flags=K.ROTATE_K | K.ROTATE_V, sign_seed=SIGN_SEED,
                       residual_window=case.get("window", 0), page_tokens=PAGE, n_pages=s["k_main"].shape[1],
                       max_pages_per_seq=table.shape[1])
    names = ("k_main", "v_main", "k_resid", "v_resid")
    cache = K.KVCache.from_buffers(cfg, {x: s[x] for x in names if s.get(x) is not None}, block_table=table)
    if case["op"] == "chunk_attention":
        return {"cache": cache}
    return {"cache": cache, "pool": K.PagePool(cache, s["refs"])}


def _run_own(s):
    case, o = s["case"], s["own"]
    if case["op"] == "chunk_attention":
        o["cache"].chunk_attention(0, 1, s["q"], s["cu_q"], s["total_q"], s["max_q"], s["seq_lens"], s["out"],
                                   window=case["window"], sinks=case["sinks"])
        return s["out"]
    if case["op"] == "qk_norm_rope":
        o["K"].qk_norm_rope(o["cfg"], s["q"], s["k"], s["positions"], s["q_out"], s["k_out"], plan=o["plan"],
                            q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
        return s["q_out"], s["k_out"]
    if case["op"] == "branch":
        o["pool"].release(s["kids"], s["seq_lens"])
        o["pool"].fork(s["from"], s["kids"], s["seq_lens"])
        o["pool"].reserve(s["kids"], s["n_new"], s["seq_lens"])
        return _branch_state(s)
    o["pool"].compact(refs_out=s["refs_out"], table_out=s["table_out"])
    return s["refs_out"], s["table_out"], s["k_main"], s["v_main"]


def _branch_state(s):
    return {x: s[x] for x in ("table", "refs", "seq_lens", "k_main", "v_main", "k_resid", "v_resid") if s[x] is not None}


# ---- the plain forms -------------------------------------------------------------------


def _unpack4(x, per):
    b = x.unflatten(-1, (-1, 2 + per // 2))
    scale = b[..., :2].contiguous().view(torch.float16).float()
    nib = b[..., 2:]
    code = torch.stack([nib & 15, nib >> 4], -1).flatten(-2).float() - 8
    return (code * scale).flatten(-2)


def _signs(device):
    """Sign vectors of the randomized transform: SplitMix64's first four words."""
    mask, state, w = (1 << 64) - 1, SIGN_SEED, []
    while len(w) < 4:
        state = (state + 0x9E3779B97F4A7C15) & mask
        z = state
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & mask
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
        w.append(z ^ (z >> 31))
    bits = [(w[i // 64] >> (i % 64)) & 1 for i in range(256)]
    s = 1.0 - 2.0 * torch.tensor(bits, dtype=torch.float32, device=device)
    return s[:128], s[128:]


def _transform(device):
    """The 128-point transform of the rotated formats as a matrix: y = x @ R."""
    i = torch.arange(128, device=device)
    p = i[:, None] & i[None, :]
    p = p ^ (p >> 4)
    p = p ^ (p >> 2)
    p = (p ^ (p >> 1)) & 1
    d1, d2 = _signs(device)
    return d1[:, None] * (1.0 - 2.0 * p.float()) * d2[None, :] / math.sqrt(128.0)


def _plain_cache(s):
    """Every cached token's key and value, in 32 bits and the stored domain: [b][h][token][d]."""
    case, got = s["case"], []
    for name in ("k_main", "v_main"):
        x = s[name]
        if s["table"] is not None:
            x = x[s["table"].long()].transpose(1, 2).flatten(2, 3)
        if case["format"] != "kivi4":
            got.append(_unpack4(x, 128)[:, :, : s["max_t"]])
            continue
        if name == "k_main":
            x = _unpack4(x.unflatten(-1, (case["head_dim"], 18)), 32).transpose(3, 4).flatten(2, 3)
        else:
            x = _unpack4(x, 32)
        x = x[:, :, : s["max_t"]]
        t = torch.arange(s["max_t"], device="cuda")
        raw = s[name[0] + "_resid"].float()[:, :, t % raw_len(s)]
        end = (s["seq_lens"].long() - KIVI_WINDOW).clamp(min=0) // GROUP * GROUP
        got.append(torch.where((t[None] >= end[:, None])[:, None, :, None], raw, x))
    return got


def raw_len(s):
    return s["k_resid"].shape[2]


def _plain_attention(s):
    case = s["case"]
    b, h, g, d = case["batch"], case["kv_heads"], case["group"], case["head_dim"]
    k, v = _plain_cache(s)
    cu, lens = s["cu_q"].long(), s["seq_lens"].long()
    n = cu[1:] - cu[:-1]
    row = torch.arange(s["max_q"], device="cuda")
    at = (cu[:-1, None] + row[None]).clamp(max=s["total_q"] - 1)  # [b][max_q], padded rows repeat others
    q = s["q"][0].float()[at]  # [b][row][head][d]
    if case["format"] != "kivi4":
        q = (q.unflatten(-1, (-1, 128)) @ _transform(q.device)).flatten(-2)
    q = q.unflatten(2, (h, g)).permute(0, 2, 1, 3, 4).reshape(b, h, -1, d)
    score = (q @ k.transpose(2, 3)).div_(math.sqrt(d)).view(b, h, s["max_q"], g, -1)
    pos = (lens - n)[:, None] + row[None]  # [b][row]
    key = torch.arange(s["max_t"], device="cuda")
    seen = key <= pos[..., None]
    if case["window"]:
        seen &= (key > pos[..., None] - case["window"]) | (key < case["sinks"])
    score.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    score -= score.amax(-1, keepdim=True)
    p = score.exp_()
    p /= p.sum(-1, keepdim=True)
    out = (p.view(b, h, -1, s["max_t"]) @ v).view(b, h, s["max_q"], g, d).permute(0, 2, 1, 3, 4).reshape(b, s["max_q"], h * g, d)
    if case["format"] != "kivi4":
        out = (out.unflatten(-1, (-1, 128)) @ _transform(out.device).t()).flatten(-2)
    return out[row[None] < n[:, None]].to(s["q"].dtype)[None]


def _frequencies(case, device):
    """(radians a position of every pair, factor on cos and sin), in 64 bits."""
    rot, f = case["rot_dim"], case["factor"]
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=device)
    theta = ROPE["theta"]
    if case["scaling"] == "ntk":
        theta *= f ** (rot / (rot - 2)) if rot > 2 else 1.0
    inv = theta ** (-i / rot)
    if case["scaling"] == "linear":
        return inv / f, 1.0
    if case["scaling"] == "bands":
        turns = ROPE["original"] * inv / (2 * math.pi)  # turns within the original context
        keep = ((turns - ROPE["low"]) / (ROPE["high"] - ROPE["low"])).clamp(0, 1)
        return keep * inv + (1 - keep) * inv / f, 1.0
    if case["scaling"] == "yarn":
        pair = [rot * math.log(ROPE["original"] / (r * 2 * math.pi)) / (2 * math.log(theta)) for r in (ROPE["fast"], ROPE["slow"])]
        lo, hi = max(0, math.floor(pair[0])), min(rot - 1, math.ceil(pair[1]))
        ramp = ((i / 2 - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return ramp * inv / f + (1 - ramp) * inv, 0.1 * math.log(f) + 1.0
    return inv, 1.0


def _turn(x, case, cos, sin):
    rot = case["rot_dim"]
    a, rest = x[..., :rot], x[..., rot:]
    if case["interleaved"]:
        u, w = a[..., 0::2], a[..., 1::2]
        a = torch.stack([u * cos - w * sin, w * cos + u * sin], -1).flatten(-2)
    else:
        u, w = a[..., : rot // 2], a[..., rot // 2:]
        a = torch.cat([u * cos - w * sin, w * cos + u * sin], -1)
    return torch.cat([a, rest], -1)


def _plain_rope(s):
    case = s["case"]
    inv, m = _frequencies(case, "cuda")
    ang = s["positions"].double()[:, None] * inv
    cos, sin = (torch.cos(ang) * m).float()[:, None], (torch.sin(ang) * m).float()[:, None]
    got = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        x = x.float()
        if w is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        got.append(_turn(x, case, cos, sin).to(s["q"].dtype))
    return tuple(got)


def _plain_branch(s):
    case = s["case"]
    table, refs, lens, kids, src = s["table"], s["refs"], s["seq_lens"], s["kids"].long(), s["from"].long()
    # release: the children's pages lose a reader
    old = table[kids].flatten().long()
    refs.index_add_(0, old.clamp(min=0), -(old >= 0).to(torch.int32))
    # fork: the children share the pages that hold their parents' quantized tokens
    end = (lens[src] - case["window"]).clamp(min=0).long()
    col = torch.arange(table.shape[1], device="cuda")
    rows = torch.where(col[None] < ((end + PAGE - 1) // PAGE)[:, None], table[src], -1)
    refs.index_add_(0, rows.flatten().long().clamp(min=0), (rows.flatten() >= 0).to(torch.int32))
    lens[kids] = lens[src]
    if case["window"]:
        s["k_resid"][:, kids], s["v_resid"][:, kids] = s["k_resid"][:, src], s["v_resid"][:, src]
    # reserve: free pages, lowest first, for a shared last page and for the new token, child by child
    need = (lens[kids].long() + s["n_new"] + PAGE - 1) // PAGE
    part = (end % PAGE > 0)[:, None] & (col[None] == (end // PAGE)[:, None])  # its last reader may keep it: the parent reads on
    want = part | ((col[None] >= ((end + PAGE - 1) // PAGE)[:, None]) & (col[None] < need[:, None]))
    free = torch.nonzero(refs == 0).flatten()
    at = want.flatten().long().cumsum(0) - 1
    page = torch.where(want.flatten(), free[at.clamp(min=0)], -1).view_as(rows)
    was, now = rows[part].long(), page[part]
    refs.index_add_(0, was, torch.full_like(was, -1, dtype=torch.int32))
    refs[page[want]] = 1
    table[kids] = torch.where(want, page.to(torch.int32), rows)
    for x in (s["k_main"], s["v_main"]):
        x[:, now] = x[:, was]
    return _branch_state(s)


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    n = (refs > 0).sum()
    page = torch.arange(refs.numel(), device="cuda")
    src, dst = torch.nonzero((refs > 0) & (page >= n)).flatten(), torch.nonzero((refs == 0) & (page < n)).flatten()
    to = page.clone()
    to[src] = dst
    out = refs.clone()
    out[dst], out[src] = refs[src], 0
    s["refs_out"].copy_(out)
    s["table_out"].copy_(torch.where(table >= 0, to[table.long().clamp(min=0)].to(torch.int32), -1))
    for x in (s["k_main"], s["v_main"]):
        x[:, dst] = x[:, src]
    return s["refs_out"], s["table_out"], s["k_main"], s["v_main"]


def run(s):
    if own:
        return _run_own(s)
    return {"chunk_attention": _plain_attention, "qk_norm_rope": _plain_rope, "branch": _plain_branch,
            "compact": _plain_compact}[s["case"]["op"]](s)


# ---- 64 bits, from the definitions ---------------------------------------------------------


def _exact_row_values(block, per):
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
    h, g, d, kivi = case["kv_heads"], case["group"], case["head_dim"], case["format"] == "kivi4"
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    r = torch.sign(_transform("cuda").double()) / math.sqrt(128.0)
    first = 0
    for b, (t, n) in enumerate(zip(*_lengths(case))):
        for head in range(h):
            kv = []
            for name in ("k_main", "v_main"):
                x = s[name]
                if s["table"] is not None:
                    x = x[s["table"][b].long(), head].reshape(-1, x.shape[-1])[:t]
                elif not (kivi and name == "k_main"):
                    x = x[b, head, :t]
                else:
                    x = x[b, head]
                if not kivi:
                    x = _exact_row_values(x.reshape(x.shape[0], d // 128, 66), 128).reshape(-1, d)
                    x = (x.reshape(-1, d // 128, 128) @ r.t()).reshape(-1, d)  # back from the rotated domain
                else:
                    if name == "k_main":
                        x = _exact_row_values(x.reshape(-1, d, 18), 32).permute(0, 2, 1).reshape(-1, d)[:t].clone()
                    else:
                        x = _exact_row_values(x.reshape(-1, d // 32, 18), 32).reshape(-1, d)[:t].clone()
                    raw = s[name[0] + "_resid"][b, head].double()
                    late = torch.arange(_quantized_end(case, t), t, device="cuda")
                    x[late] = raw[late % raw.shape[0]]
                kv.append(x)
            k, v = kv
            for a in range(0, n, 1024):
                e = min(n, a + 1024)
                q = s["q"][0, first + a:first + e, head * g:(head + 1) * g].double()
                z = torch.einsum("igd,td->igt", q, k) / math.sqrt(d)
                p = torch.arange(t - n + a, t - n + e, device="cuda")[:, None]
                j = torch.arange(t, device="cuda")[None]
                hide = j > p
                if case["window"]:
                    hide = hide | ((j <= p - case["window"]) & (j >= case["sinks"]))
                z = torch.softmax(z.masked_fill(hide[:, None], -math.inf), -1)
                out[0, first + a:first + e, head * g:(head + 1) * g] = torch.einsum("igt,td->igd", z, v)
        first += n
    return out


def _exact_rope(case, seed):
    s = _rope_inputs(case, seed)
    rot, f, pairs, m = case["rot_dim"], case["factor"], [], 1.0
    base = ROPE["theta"] * (f ** (rot / (rot - 2)) if case["scaling"] == "ntk" and rot > 2 else 1.0)
    for i in range(rot // 2):
        w = base ** (-2.0 * i / rot)
        if case["scaling"] == "linear":
            w /= f
        elif case["scaling"] == "bands":
            wave = 2 * math.pi / w
            if wave > ROPE["original"] / ROPE["low"]:
                w /= f
            elif wave >= ROPE["original"] / ROPE["high"]:
                k = (ROPE["original"] / wave - ROPE["low"]) / (ROPE["high"] - ROPE["low"])
                w = (1 - k) * w / f + k * w
        elif case["scaling"] == "yarn":
            m = 0.1 * math.log(f) + 1.0
            where = [rot * math.log(ROPE["original"] / (r * 2 * math.pi)) / (2 * math.log(base)) for r in (ROPE["fast"], ROPE["slow"])]
            lo, hi = max(0, math.floor(where[0])), min(rot - 1, math.ceil(where[1]))
            k = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            w = k * w / f + (1 - k) * w
        pairs.append(w)
    ang = s["positions"].double()[:, None] * torch.tensor(pairs, dtype=torch.float64, device="cuda")
    z = torch.polar(torch.full_like(ang, m), ang)[:, None]
    got = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        x = x.double()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.double()
        i = torch.arange(rot // 2, device="cuda")
        u, v = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
        c = torch.complex(x[..., u], x[..., v]) * z
        x = x.clone()
        x[..., u], x[..., v] = c.real, c.imag
        got.append(x)
    return tuple(got)


def exact(case, seed):
    if case["op"] == "chunk_attention":
        return _exact_attention(case, seed)
    if case["op"] == "qk_norm_rope":
        return _exact_rope(case, seed)
    return None  # pages are copied: whole numbers, compared as they are
