"""FP64 oracle of the paged key/value cache: append, read back, attention of
new tokens.

TEST INFRASTRUCTURE ONLY: the test suite is its only caller; the product
never imports it.

Position p of sequence b lives in page table[b, p // ps], slot p % ps of
pools [P, g, ps, 128].  16-bit pages hold k~ = RoPE(RMSNorm(k, w_k), p)
rounded to FP16 and v in BF16; 8-bit pages hold E4M3 codes with a scale 2^e
per token and head, e the smallest integer in [-24, 40] (keys: [-24, 7]) with
max|x| <= 448 x 2^e.  New row i of sequence b (position p = len[b] + i) attends to the
positions max(0, p - W + 1) .. p (W = 0: from 0) as the pages hold them, and
to the learned sink (FlintAttention.forward and _apply_rope on the NeMo
AutoModel "flint.layers" API page; HF discussion #26 on RecursiveSI/flint):

    s_j = q~ . K_j / sqrt(128),  Z = e^sink + sum_j e^{s_j}
    out = sum_j e^{s_j} V_j / Z,  lse = ln Z
"""
from __future__ import annotations

import numpy as np

D = 128
GROUP = 8
E_MIN, E_MAX = -24, 40


def norm_rope(x, w, pos, use_rope, theta=10000.0, eps=1e-6):
    """Rows x [..., 128] (float64) at positions pos [...]: RMSNorm in weight
    form, then NeoX RoPE (channel i with i + 64, frequency theta^(-2i/128))."""
    x = np.asarray(x, np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    if not use_rope:
        return y
    ang = np.asarray(pos, np.float64)[..., None] * theta ** (-np.arange(64) / 64.0)
    c, s = np.cos(ang), np.sin(ang)
    return np.concatenate([y[..., :64] * c - y[..., 64:] * s, y[..., 64:] * c + y[..., :64] * s], -1)


def scale_exponent(x):
    """e of rows x [..., 128]."""
    a = np.abs(x).max(-1) / 448.0
    m, e = np.frexp(a)                       # a = m 2^e, m in [1/2, 1)
    return np.where(a > 0, np.clip(np.where(m == 0.5, e - 1, e), E_MIN, E_MAX), E_MIN).astype(np.int64)


def e4m3(x):
    """Nearest E4M3 value (ties to even, saturating at 448)."""
    x = np.asarray(x, np.float64)
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)
    return np.clip(np.round(x / step) * step, -448.0, 448.0)


def quantise(x, most=E_MAX):
    """(code values, exponents) of rows x [..., 128]; keys: most = 7."""
    e = np.minimum(scale_exponent(x), most)
    return e4m3(x * np.exp2(-e.astype(np.float64))[..., None]), e


def rows_of(cache_len, cu):
    """(sequence, position) of every packed row below cu[-1]."""
    b = np.repeat(np.arange(len(cache_len)), np.diff(cu))
    return b, np.asarray(cache_len)[b] + np.arange(cu[-1]) - np.asarray(cu)[b]


def attn(q, q_norm_w, sinks, K, V, table, cache_len, cu, *, window, use_rope, theta=10000.0, eps=1e-6):
    """q [T, 8g, 128]; K, V [P, g, ps, 128]: the values the pages stand for.
    Returns (out [T, 8g, 128], lse [8g, T], absum [T, 8g, 128] = sum p |V| / Z,
    spread [T, 8g] = max_j sum_c |q~_c K_jc| / sqrt(128)) for the rows below
    cu[-1], NaN behind them."""
    q = np.asarray(q, np.float64)
    T, nh = q.shape[:2]
    g, ps = K.shape[1], K.shape[2]
    sinks = np.asarray(sinks, np.float64)
    out, ab = np.full((T, nh, D), np.nan), np.full((T, nh, D), np.nan)
    lse, spread = np.full((nh, T), np.nan), np.full((T, nh), np.nan)
    b_of, pos = rows_of(cache_len, cu)
    for t in range(int(cu[-1])):
        b, p = b_of[t], int(pos[t])
        lo = max(0, p - window + 1) if window else 0
        j = np.arange(lo, p + 1)
        page = table[b][j // ps]
        assert (page >= 0).all()
        qt = norm_rope(q[t], q_norm_w, np.full(nh, p), use_rope, theta, eps)
        for h in range(g):
            k, v = K[page, h, j % ps], V[page, h, j % ps]
            qh = qt[GROUP * h:GROUP * (h + 1)]
            s = qh @ k.T / np.sqrt(128.0)
            sk = sinks[GROUP * h:GROUP * (h + 1)]
            m = np.maximum(s.max(1), sk)
            with np.errstate(invalid="ignore"):
                e = np.exp(s - m[:, None])
                z = e.sum(1) + np.exp(sk - m)
                inf = np.isposinf(sk)
                z = np.where(inf, 1.0, z)
                pr = np.where(inf[:, None], 0.0, e / z[:, None])
                lse[GROUP * h:GROUP * (h + 1), t] = np.where(inf, np.inf, m + np.log(z))
            out[t, GROUP * h:GROUP * (h + 1)] = pr @ v
            ab[t, GROUP * h:GROUP * (h + 1)] = pr @ np.abs(v)
            spread[t, GROUP * h:GROUP * (h + 1)] = (np.abs(qh) @ np.abs(k).T).max(1) / np.sqrt(128.0)
    return out, lse, ab, spread
