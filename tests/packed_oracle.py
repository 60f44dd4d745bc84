"""Plain float64 forms of the packed operators, and the error bounds their tests hold results to.

Test infrastructure only.  The attention of each sequence is oracle.sdpa.attention; the rotation is
written here from its definition.

Bounds, from the arithmetic alone (u = 2^-8, half a bf16 step relative to the value):

* attention output o = sum_j p_j v_j / l.  P is rounded to bf16 before P V: at most u A with
  A = sum_j softmax_j |v_j|.  The output is rounded to bf16: u |o|.  In fp32: the scores are sums of D
  products, at most D 2^-23 scale sum_d |q_d k_d| off (a factor of e^(2 that) on a weight ratio), the n
  weights and the n products p v are summed with at most n 2^-23 relative each, and the exponentials add
  2^-21.  All of these scale with A.
* log-sum-exp: the scores' error, n 2^-23 from the sum, and 2^-22 of (|lse| + 16) for the logarithm, the
  change of base and the reference maximum's product.
"""
import numpy as np

from oracle import sdpa

U = 2.0 ** -8


def f64(t):
    return t.detach().to("cpu").double().numpy()


def packed_attention(q, k, v, cu_q, cu_k, scale, causal=True, window=0):
    """q [Tq,Hq,D], k/v [Tk,Hkv,D] (float64) -> out, lse, tol, lse_tol over all rows; rows of no sequence are NaN."""
    Tq, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, lse = np.full((Tq, Hq, D), np.nan), np.full((Tq, Hq), np.nan)
    tol, lse_tol = np.full((Tq, Hq, D), np.nan), np.full((Tq, Hq), np.nan)
    for b in range(len(cu_q) - 1):
        qs, ks = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        Q, K, V = (x.transpose(1, 0, 2)[None] for x in (q[qs], k[ks], v[ks]))
        n = K.shape[2]
        if Q.shape[2] == 0:
            continue
        if n == 0:
            out[qs], lse[qs], tol[qs], lse_tol[qs] = 0.0, -np.inf, 0.0, 0.0
            continue
        o, l = sdpa.attention(Q, K, V, scale, causal, window, return_lse=True)
        A = sdpa.attention(Q, K, np.abs(V), scale, causal, window)
        s_err = np.einsum("hid,hjd->hij", np.abs(Q[0]), np.repeat(np.abs(K[0]), G, 0)).max(2) * D * 2.0 ** -23 * scale
        rel = np.expm1(2 * s_err) + 2 * n * 2.0 ** -23 + 2.0 ** -21
        out[qs], lse[qs] = o[0].transpose(1, 0, 2), l[0].T
        tol[qs] = ((U + 2 * rel[:, :, None]) * A[0] + U * np.abs(o[0])).transpose(1, 0, 2)
        lse_tol[qs] = np.where(np.isfinite(l[0]), s_err + n * 2.0 ** -23 + 2.0 ** -22 * (np.abs(np.where(np.isfinite(l[0]), l[0], 0)) + 16), 0).T
    return out, lse, tol, lse_tol


def assert_packed(got, want, what=""):
    """(out, lse or None) of a call against packed_attention's answer; rows of no sequence are not looked at."""
    out, lse, tol, lse_tol = want
    g = f64(got[0])
    held = ~np.isnan(out)
    assert np.isfinite(g[held]).all(), f"{what}: non-finite output"
    off = np.abs(g - out)[held] - tol[held]
    assert (off <= 0).all(), f"{what}: {off.max():.3e} over the bound, worst of {off.size}"
    if got[1] is not None:
        gl, m = f64(got[1]), ~np.isnan(lse)
        empty = np.isneginf(lse)
        assert (np.isneginf(gl) == empty)[m].all(), f"{what}: lse of rows without keys"
        m &= ~empty
        off = np.abs(gl[m] - lse[m]) - lse_tol[m]
        assert (off <= 0).all(), f"{what}: lse {off.max():.3e} over the bound"


def rotate(x, cos_sin, interleaved):
    """x [n,H,D] float64 at the angles of its row's cos_sin [n,R] (cosines, then sines); (value, sum of |terms|)."""
    R = cos_sin.shape[1]
    c, s = cos_sin[:, None, : R // 2], cos_sin[:, None, R // 2:]
    a_at = np.arange(0, R, 2) if interleaved else np.arange(R // 2)
    b_at = a_at + (1 if interleaved else R // 2)
    y, mag = x.copy(), np.zeros_like(x)
    a, b = x[..., a_at], x[..., b_at]
    y[..., a_at], y[..., b_at] = a * c - b * s, b * c + a * s
    mag[..., a_at], mag[..., b_at] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return y, mag


def cos_sin_table(max_pos, rot, theta=10000.0):
    import torch

    inv = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot) if rot else torch.zeros(0, dtype=torch.float64)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return torch.cat((a.cos(), a.sin()), 1).float().contiguous()


def cumulative(lens, start=0):
    import torch

    return torch.tensor(np.concatenate(([0], np.cumsum(lens))) + start, dtype=torch.int32)
