"""Plain 64-bit definitions of the serving operators around the cache: norm
and rotary turn of queries and keys, the page bookkeeping of a paged cache
(sequential, one list entry after the other), and attention of a chunk of new
tokens with a causal mask, a sliding window and first tokens that stay visible.
Shares no code with the CUDA path."""

from __future__ import annotations

import math
from typing import Dict, List

import numpy as np

from . import kvq_oracle as O

ROPE_NONE, ROPE_LINEAR, ROPE_NTK, ROPE_YARN, ROPE_BANDS = range(5)


# ---- norm and rotary turn ------------------------------------------------------


def rope_frequencies(rot_dim, theta, scaling=ROPE_NONE, factor=1.0, low=1.0, high=32.0, original_len=0,
                     attn_factor=0.0):
    """(radians per position of pair i, factor on cos and sin)."""
    d, out, m = rot_dim, [], attn_factor or 1.0
    base = theta
    if scaling == ROPE_NTK and d > 2:
        base = theta * factor ** (d / (d - 2))
    if scaling == ROPE_YARN:
        def pair_of(turns):
            return d * math.log(original_len / (2 * math.pi * turns)) / (2 * math.log(base))
        a, z = max(0, math.floor(pair_of(high))), min(d - 1, math.ceil(pair_of(low)))
        m = attn_factor or 0.1 * math.log(factor) + 1.0
    for i in range(d // 2):
        f = base ** (-2.0 * i / d)
        if scaling == ROPE_LINEAR:
            f /= factor
        elif scaling == ROPE_YARN:
            r = min(1.0, max(0.0, (i - a) / max(z - a, 0.001)))
            f = r * f / factor + (1 - r) * f
        elif scaling == ROPE_BANDS:
            b = min(1.0, max(0.0, (original_len * f / (2 * math.pi) - low) / (high - low)))
            f = b * f + (1 - b) * f / factor
        out.append(f)
    return np.array(out), m


def rms_norm(x: np.ndarray, w: np.ndarray, eps: float) -> np.ndarray:
    x = np.asarray(x, np.float64)
    return x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * w


def turn(x: np.ndarray, positions: np.ndarray, freqs: np.ndarray, m: float, interleaved: bool) -> np.ndarray:
    """x [tokens, heads, D]; the first 2 len(freqs) channels turn."""
    x = np.array(x, np.float64)
    n = len(freqs)
    ang = np.asarray(positions, np.float64)[:, None] * freqs[None]
    c, s = m * np.cos(ang)[:, None], m * np.sin(ang)[:, None]
    ia = np.arange(n) * 2 if interleaved else np.arange(n)
    ib = ia + 1 if interleaved else ia + n
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return x


# ---- pages -----------------------------------------------------------------------


class Pages:
    """A paged cache's block table, reader counts, lengths and page contents,
    changed one list entry at a time.  `pools` are arrays [L, n_pages, ...],
    `windows` arrays [L, batch, ...] (the 16-bit windows), changed in place."""

    def __init__(self, table, n_pages, page_tokens, max_T, residual_window=0, pools=(), windows=()):
        self.table = np.array(table, np.int64)
        self.n_pages, self.pt, self.max_T, self.R = n_pages, page_tokens, max_T, residual_window
        self.refs = np.zeros(n_pages, np.int64)
        for p in self.table.flat:
            if p >= 0:
                self.refs[p] += 1
        self.lens = np.zeros(len(self.table), np.int64)
        self.pools, self.windows = list(pools), list(windows)

    def q_end(self, T):
        return max(0, T - self.R)

    def release(self, seqs: List[int]):
        for s in seqs:
            for j, p in enumerate(self.table[s]):
                if p >= 0:
                    self.refs[p] -= 1
                self.table[s, j] = -1
            self.lens[s] = 0

    def fork(self, src: List[int], dst: List[int]):
        for s, d in zip(src, dst):
            n = -(-self.q_end(self.lens[s]) // self.pt)
            for j in range(n):
                self.table[d, j] = self.table[s, j]
                self.refs[self.table[s, j]] += 1
            for w in self.windows:
                w[:, d] = w[:, s]
            self.lens[d] = self.lens[s]

    def _take(self) -> int:
        p = int(np.flatnonzero(self.refs == 0)[0])
        self.refs[p] = 1
        return p

    def reserve(self, seqs: List[int], n_new: List[int]):
        for s, nn in zip(seqs, n_new):
            if nn == 0:
                continue
            qe, T = self.q_end(self.lens[s]), self.lens[s]
            if qe % self.pt:
                old = self.table[s, qe // self.pt]
                if self.refs[old] > 1:
                    new = self._take()
                    self.refs[old] -= 1
                    self.table[s, qe // self.pt] = new
                    for x in self.pools:
                        x[:, new] = x[:, old]
            for j in range(-(-qe // self.pt), -(-(T + nn) // self.pt)):
                if self.table[s, j] < 0:
                    self.table[s, j] = self._take()

    def compact(self):
        used = np.flatnonzero(self.refs > 0)
        n = len(used)
        movers, holes = [p for p in used if p >= n], [p for p in range(n) if self.refs[p] == 0]
        for s, d in zip(movers, holes):
            self.table[self.table == s] = d
            self.refs[d], self.refs[s] = self.refs[s], 0
            for x in self.pools:
                x[:, d] = x[:, s]


    def reorder(self, parents: List[int], group: int):
        """Slot b of every `group` slots becomes what slot parents[b] of the group was.  Pages behind the quantized tokens stay
        one sequence's: the slot's own, or its lowest child's."""
        B = len(self.table)
        src = [b // group * group + int(parents[b]) for b in range(B)]
        old, lens = self.table.copy(), self.lens.copy()
        windows = [w.copy() for w in self.windows]
        for b in range(B):
            s = src[b]
            row = old[s].copy()
            heir = s if src[s] == s else src.index(s)
            if heir != b:
                row[-(-self.q_end(lens[s]) // self.pt):] = -1
            self.table[b], self.lens[b] = row, lens[s]
            for w, o in zip(self.windows, windows):
                w[:, b] = o[:, s]
        self.refs[:] = 0
        for p in self.table.flat:
            if p >= 0:
                self.refs[p] += 1


# ---- selection of a beam search ---------------------------------------------------


def beam_select(logits: np.ndarray, scores: np.ndarray, done=None, eos=-1):
    """(scores, tokens, parents, done) of the best continuations; logits [groups, beams, vocab] as fp64 values."""
    G, K, V = logits.shape
    x = np.array(logits, np.float64)
    top = float(np.finfo(np.float32).max)
    x[np.isnan(x)] = -np.inf
    x[x == np.inf] = top
    s = np.array(scores, np.float64)
    s[np.isnan(s)] = -np.inf
    s = np.minimum(s, top)
    res = [np.empty((G, K)), *(np.empty((G, K), np.int64) for _ in range(3))]
    for g in range(G):
        c = []  # (-score, beam, token)
        for b in range(K):
            if done is not None and done[g, b]:
                c.append((-s[g, b], b, eos))
                continue
            m = x[g, b].max()
            if m == -np.inf:
                c += [(np.inf, b, v) for v in range(V)]
                continue
            d = x[g, b] - m
            total = math.log(math.fsum(np.exp(d)))
            c += [(-(s[g, b] + (d[v] - total)), b, v) for v in range(V)]
        for i, (score, b, v) in enumerate(sorted(c)[:K]):
            res[0][g, i], res[1][g, i], res[2][g, i] = -score, v, b
            res[3][g, i] = int(v == eos or bool(done is not None and done[g, b]))
    return res


# ---- chunk attention ------------------------------------------------------------------


def visible(p: int, T: int, window: int, sinks: int) -> np.ndarray:
    """Which of T cached tokens the query at position p sees."""
    j = np.arange(T)
    see = j <= p
    if window:
        see &= (j > p - window) | (j < sinks)
    return see


def chunk_attention(cfg: O.Config, bufs: Dict[str, np.ndarray], layer: int, q: np.ndarray, cu_q, lens, window=0,
                    sinks=0, block_table=None, with_bound=False, key_roundings=2.0):
    """fp64 attention of one layer's query rows q [total_q, H_q, D] (raw
    input-dtype bits) over the dequantized cache; rows of no sequence are NaN.

    with_bound: also the largest error that rounding allows, per output value:
    with u the input dtype's half step, a score is off by at most
      ds_j = (key_roundings u + 2^-24 D + 2^-20) sum_c |q_c k_jc| / sqrt(D)
    (keys rounded to the dtype, rotated queries too, fp32 sums, the base-2
    exponent), a probability by the factor exp(ds_j + max ds), rounded once
    (u), a value once or twice (2 u), the output once (u |o|).  The sum l may be taken of the
    rounded probabilities: off by u l at most, which is u |o| <= u sum_j p_j |v_j| of the output."""
    g, D = cfg.H_q // cfg.H_kv, cfg.D
    u = 2.0 ** -11 if cfg.in_dtype == 0 else 2.0 ** -8
    out = np.full(q.shape, np.nan)
    bound = np.full(q.shape, np.nan)
    qf = O.input_to_f32(q, cfg.in_dtype).astype(np.float64)
    d1, d2 = O.hadamard_signs(cfg.sign_seed)

    def stored(x, rot):
        return O.rotate_f64(x, d1, d2) if rot else x

    for b in range(cfg.batch):
        n, T = int(cu_q[b + 1] - cu_q[b]), int(lens[b])
        if n == 0:
            continue
        K, V = O.dequantize(cfg, bufs, layer, b, T, block_table=block_table)
        if cfg.flags & O.K_PRE_ROPE:
            K = O.rope_f64(K, np.arange(T), cfg.rope_theta)
        for h in range(cfg.H_kv):
            k, v = K[:, h], V[:, h]
            ka = np.abs(stored(k, cfg.flags & O.ROTATE_K)) if with_bound else None
            va = np.abs(stored(v, cfg.flags & O.ROTATE_V)) if with_bound else None
            for i in range(n):
                see = visible(T - n + i, T, window, sinks)
                rows = qf[cu_q[b] + i, h * g:(h + 1) * g]
                s = rows @ k[see].T / math.sqrt(D)
                p = np.exp(s - s.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                o = p @ v[see]
                out[cu_q[b] + i, h * g:(h + 1) * g] = o
                if with_bound:
                    qa = np.abs(stored(rows, cfg.flags & O.ROTATE_K))
                    ds = (key_roundings * u + 2.0 ** -24 * D + 2.0 ** -20) * (qa @ ka[see].T) / math.sqrt(D)
                    rel = np.expm1(ds + ds.max(-1, keepdims=True)) + 4 * u
                    e = (p * rel) @ va[see]
                    if cfg.in_dtype == 0:
                        # P in fp16 is counted from a reference no larger than the row's
                        # maximum, so the row's largest P, and with it l, is at least 1; below
                        # 2^-14 P rounds to multiples of 2^-24: half of one per token, in the sum l too
                        oa = np.abs(stored(o, cfg.flags & O.ROTATE_V))
                        e = e + 2.0 ** -25 * (va[see].sum(0) + len(va[see]) * oa)
                    if cfg.flags & O.ROTATE_V:  # errors of the rotated domain spread over the block
                        e = np.repeat(np.sqrt(np.sum(e.reshape(g, -1, 128) ** 2, -1)), 128, -1)
                    bound[cu_q[b] + i, h * g:(h + 1) * g] = e + u * np.abs(o) + 2.0 ** -24
    return (out, bound) if with_bound else out
