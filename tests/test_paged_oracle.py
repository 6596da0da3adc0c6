"""Pins of the paged-cache oracle (CPU): E4M3 rounding against torch's, the
scale rule by brute force, and attention of chunks against the full-sequence
oracle."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from oracle import paged as OP


def test_e4m3_is_torchs():
    r = np.random.default_rng(0)
    x = np.concatenate([r.standard_normal(4000) * s for s in (1e-3, 0.02, 1.0, 60.0)]).astype(np.float32)
    x = np.concatenate([np.clip(x, -448, 448), np.arange(-448, 448, 0.5, np.float32),
                        np.arange(-64, 64, dtype=np.float32) * 2.0 ** -10])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(OP.e4m3(x.astype(np.float64)), want)
    assert OP.e4m3(1e9) == 448 and OP.e4m3(-1e9) == -448


def test_scale_is_the_smallest_that_holds():
    r = np.random.default_rng(1)
    x = r.standard_normal((500, 128)) * np.exp(r.uniform(-25, 35, (500, 1)))
    x[0] = 0
    x[1, :] = 0
    x[1, 5] = 448.0                       # on a border: e = 0
    x[2, :] = 0
    x[2, 5] = np.nextafter(448.0, 449.0)  # past it: e = 1
    e = OP.scale_exponent(x)
    a = np.abs(x).max(1)
    assert e[0] == OP.E_MIN and e[1] == 0 and e[2] == 1
    ok = (e > OP.E_MIN) & (e < OP.E_MAX)
    assert (a[ok] <= 448 * np.exp2(e[ok])).all() and (a[ok] > 448 * np.exp2(e[ok] - 1)).all()
    assert (a[e == OP.E_MIN] <= 448 * 2.0 ** OP.E_MIN).all() and (a[e == OP.E_MAX] > 448 * 2.0 ** (OP.E_MAX - 1)).all()


def test_quantised_rows_are_within_half_a_step():
    r = np.random.default_rng(2)
    x = r.standard_normal((300, 128)) * 3
    c, e = OP.quantise(x)
    s = np.exp2(e.astype(float))[:, None]
    assert (np.abs(c * s - x) <= np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10)).all()


@pytest.mark.parametrize("window,rope,split", [(0, False, (20, 1, 19)), (9, True, (1, 1, 38)), (513, True, (40,))])
def test_chunks_over_exact_pages_are_the_prefill(window, rope, split):
    """Rows attended chunk by chunk over pages of unrounded keys equal the
    rows of the full-sequence oracle, for shuffled pages and poisoned slots."""
    T, ps = 40, 16
    w = W.make_small(T, seed=11, window=window, use_rope=rope)
    ref, ref_l = oracle.attn_fwd_workload(w, rows=None)
    q, k, v = oracle._f64(w.q).reshape(T, 32, 128), oracle._f64(w.k).reshape(T, 4, 128), oracle._f64(w.v).reshape(T, 4, 128)
    table = np.array([[4, 1, 3]], np.int32)
    K, V = np.full((5, 4, ps, 128), np.nan), np.full((5, 4, ps, 128), np.nan)
    at = 0
    for n in split:
        pos = np.arange(at, at + n)
        K[table[0, pos // ps], :, pos % ps] = OP.norm_rope(k[at:at + n], w.k_norm_w, pos[:, None].repeat(4, 1), rope, w.rope_theta, w.eps)
        V[table[0, pos // ps], :, pos % ps] = v[at:at + n]
        out, lse, _, _ = OP.attn(q[at:at + n], w.q_norm_w, w.sinks, K, V, table, np.array([at]), np.array([0, n]),
                                 window=window, use_rope=rope, theta=w.rope_theta, eps=w.eps)
        assert np.abs(out - ref[at:at + n]).max() < 1e-12
        assert np.abs(lse.T - ref_l[at:at + n]).max() < 1e-12
        at += n


def test_ragged_rows_and_padding():
    b, pos = OP.rows_of(np.array([5, 0, 7]), np.array([0, 2, 2, 5]))
    assert b.tolist() == [0, 0, 2, 2, 2] and pos.tolist() == [5, 6, 7, 8, 9]


def test_infinite_sinks():
    K = np.zeros((1, 1, 16, 128))
    V = np.ones((1, 1, 16, 128))
    q = np.zeros((1, 8, 128))
    sinks = np.array([np.inf, -np.inf, 0, 1, 2, 3, 4, 5.0])
    out, lse, _, _ = OP.attn(q, np.ones(128), sinks, K, V, np.array([[0]]), np.array([3]), np.array([0, 1]), window=0, use_rope=False)
    assert (out[0, 0] == 0).all() and np.isposinf(lse[0, 0])
    assert np.allclose(out[0, 1], 1) and np.isclose(lse[1, 0], np.log(4))
    assert np.allclose(out[0, 2:, 0], 4 / (4 + np.exp(sinks[2:])))
