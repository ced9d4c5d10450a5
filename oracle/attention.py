"""Plain float64 definitions of the token mixers of hybrid models (numpy, no
code shared with the CUDA path): linear attention with a decay per head,
attention of one token over a paged key-value cache, and eviction from that
cache by accumulated weight."""
from __future__ import annotations

import numpy as np


def linear_attention(q, k, v, log_decay, scale=1.0, state=None, seq_lens=None):
    """q, k (B, Hk, L, N); v (B, H, L, P); log_decay (H) or (B, H, L); state
    (B, H, P, N).  Token by token: S = exp(min(g, 0)) S + v k^T, out = scale S q.
    Returns (out, S); rows of out at or past seq_lens are NaN."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    B, H, L, P = v.shape
    N, rep = q.shape[3], H // max(q.shape[1], 1)
    q, k = np.repeat(q, rep, axis=1), np.repeat(k, rep, axis=1)
    g = np.minimum(np.asarray(log_decay, np.float64), 0.0)  # (a NaN stays one)
    g = np.broadcast_to(g[None, :, None] if g.ndim == 1 else g, (B, H, L))
    S = np.zeros((B, H, P, N)) if state is None else np.array(state, np.float64)
    out = np.full((B, H, L, P), np.nan)
    lens = np.full(B, L) if seq_lens is None else np.clip(np.asarray(seq_lens, np.int64), 0, L)
    for b in range(B):
        for t in range(lens[b]):
            S[b] = np.exp(g[b, :, t])[:, None, None] * S[b] + v[b, :, t, :, None] * k[b, :, t, None, :]
            out[b, :, t] = scale * np.einsum("hpn,hn->hp", S[b], q[b, :, t])
    return out, S


def linear_attention_step(state, q, k, v, log_decay, scale=1.0, slots=None):
    """One token: state (S, H, P, N), q, k (B, Hk, N), v (B, H, P), log_decay (H)
    or (B, H), a positive one counts as 0.  Returns (out, new states (B, H, P, N)); rows whose slot is out
    of range are NaN."""
    state, q, k, v = (np.asarray(a, np.float64) for a in (state, q, k, v))
    B, H = v.shape[:2]
    rep = H // q.shape[1]
    g = np.broadcast_to(np.minimum(np.asarray(log_decay, np.float64), 0.0), (B, H))
    out, new = np.full(v.shape, np.nan), np.full((B,) + state.shape[1:], np.nan)
    for b in range(B):
        s = b if slots is None else int(slots[b])
        if not 0 <= s < state.shape[0]:
            continue
        kb, qb = np.repeat(k[b], rep, 0), np.repeat(q[b], rep, 0)
        new[b] = np.exp(g[b])[:, None, None] * state[s] + v[b][:, :, None] * kb[:, None, :]
        out[b] = scale * np.einsum("hpn,hn->hp", new[b], qb)
    return out, new


def paged_rows(cache, table_row, n):
    """The rows of tokens 0..n-1, and which of them lie in a page that exists."""
    cache = np.asarray(cache, np.float64)
    page = cache.shape[1]
    t = np.arange(n)
    pg = np.asarray(table_row, np.int64)[t // page]
    ok = (pg >= 0) & (pg < cache.shape[0])
    rows = np.zeros((n,) + cache.shape[2:])
    rows[ok] = cache[pg[ok], (t % page)[ok]]
    return rows, ok


def paged_attention(q, k_cache, v_cache, table, seq_lens, scale):
    """Returns (out (B, Hq, D), p: per sequence (Hq, n) weights, lse (B, Hq),
    mag: sum_t p |v|, spread: scale max_t sum_d |q||k|, the magnitudes that
    rounding errors of the values and of the scores are relative to)."""
    q = np.asarray(q, np.float64)
    B, Hq, D = q.shape
    Hkv, page = np.shape(k_cache)[2], np.shape(k_cache)[1]
    rep = Hq // Hkv
    cap = np.shape(table)[1] * page
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    mag, spread, ps = np.zeros((B, Hq, D)), np.zeros((B, Hq)), []
    for b in range(B):
        n = int(np.clip(seq_lens[b], 0, cap))
        k, ok = paged_rows(k_cache, table[b], n)
        v, _ = paged_rows(v_cache, table[b], n)
        p = np.zeros((Hq, n))
        for h in range(Hq):
            x = scale * (k[:, h // rep] @ q[b, h])
            x[~ok] = -np.inf
            if n == 0 or not (x > -np.inf).any():
                continue
            m = x.max()
            e = np.where(x == -np.inf, 0.0, np.exp(x - m))
            lse[b, h] = m + np.log(e.sum())
            p[h] = e / e.sum()
            out[b, h] = p[h] @ v[:, h // rep]
            mag[b, h] = p[h] @ np.abs(v[:, h // rep])
            spread[b, h] = abs(scale) * (np.abs(k[ok, h // rep]) @ np.abs(q[b, h])).max()
        ps.append(p)
    return out, ps, lse, mag, spread


def evict(weights, table, seq_lens, pages, page, keep, recent):
    """For every sequence and head the positions that stay, ascending (lists).
    A token in a page that does not exist is not there."""
    w = np.asarray(weights, np.float64)
    B, Hkv = w.shape[:2]
    cap = np.shape(table)[1] * page
    kept = [[None] * Hkv for _ in range(B)]
    for b in range(B):
        n = int(np.clip(seq_lens[b], 0, cap))
        there = [t for t in range(n) if 0 <= int(table[b][t // page]) < pages]
        for h in range(Hkv):
            forced = [t for t in there if t >= n - recent]
            free = [t for t in there if t < n - recent]
            m = min(keep, len(there)) - len(forced)
            # a NaN below every number; of equal weights the lowest position first
            free.sort(key=lambda t: (bool(np.isnan(w[b, h, t])), 0.0 if np.isnan(w[b, h, t]) else -w[b, h, t], t))
            kept[b][h] = sorted(free[:m] + forced)
    return kept
