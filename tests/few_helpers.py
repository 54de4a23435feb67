"""Float64 reference of the few-token layer with a bound on every output.

reference(): the layer on the routing the device chose, in float64 from the
exact input values, and a bound on the device's error per output that counts
its roundings:
  * fp32 accumulation of a K-term product: K 2^-24 sum|a b| (plus the order of
    the partial sums, a few more terms);
  * SwiGLU in fp32: |dh| <= 1.1 |u| dg + |g| du (|SiLU'| <= 1.1, |SiLU(g)| <=
    |g|) and 2^-20 |h| for exp, reciprocal and products (each within 2^-22);
  * H kept as two bf16: 2^-16 |h| (fp32 layers: none);
  * the output rounding, eps / 2 of the activation type.
For MXFP8 layers H is checked by its codes (check_h_codes), and the outputs
against the products of the decoded codes, which the down GEMM takes exactly.
"""

import numpy as np

import oracle
from tests import parity_helpers as H


def _product(a, w):
    """a @ w.T and the bound on its fp32 accumulation."""
    K = a.shape[1]
    return a @ w.T, (K + 16) * 2.0 ** -24 * (np.abs(a) @ np.abs(w).T)


def swiglu_bound(u_in, wg, wu, limit):
    g, dg = _product(u_in, wg)
    u, du = _product(u_in, wu)
    if limit > 0:
        g, u = np.minimum(g, limit), np.clip(u, -limit, limit)
    with np.errstate(over="ignore"):
        h = g / (1.0 + np.exp(-g)) * u
    return h, 1.1 * np.abs(u) * dg + np.abs(g) * du + 2.0 ** -20 * np.abs(h) + 1e-30


def reference(cfg, layer, idx, w, fp8=False, h_values=None):
    """(y, bound, h, dh) for idx [T, k] and weights w [T, k] as the device used
    them; h_values: decoded H of the routed pairs [T*k, I] (MXFP8)."""
    x = H.f64(layer["x"])
    T, k = idx.shape
    mx = cfg.act_quant == "mxfp8"
    xr = oracle.mxfp8_decode(*oracle.mxfp8_quantize(x)) if mx else x
    y = np.zeros_like(x)
    tol = np.zeros_like(x)
    get = H.expert_fetcher(layer, cfg, fp8)
    h_all = np.zeros((T * k, cfg.moe_inter_dim))
    dh_all = np.zeros_like(h_all)
    keep = 0.0 if cfg.act_dtype == "f32" else 2.0 ** -16
    for e in np.unique(idx):
        if e < 0 or e >= cfg.n_routed_experts:
            continue
        rows, slots = np.nonzero(idx == e)
        wg, wu, wd = get(int(e))
        h, dh = swiglu_bound(xr[rows], wg, wu, cfg.swiglu_limit)
        h_all[rows * k + slots], dh_all[rows * k + slots] = h, dh
        if mx:
            # a token's first choice of an expert holds the row
            first = [int(np.nonzero(idx[t] == e)[0][0]) for t in rows]
            h, dh = h_values[rows * k + np.asarray(first)], np.zeros_like(h)
        out, dout = _product(h, wd)
        dout = dout + (dh + (0.0 if mx else keep * np.abs(h))) @ np.abs(wd).T
        g = w[rows, slots][:, None]
        np.add.at(y, rows, g * out)
        np.add.at(tol, rows, np.abs(g) * dout + 2.0 ** -22 * np.abs(g * out))
    if cfg.n_shared_experts:
        wg, wu, wd = H.shared_weights(layer, cfg)
        h, dh = swiglu_bound(x, wg, wu, cfg.swiglu_limit)
        out, dout = _product(h, wd)
        y += out
        tol += dout + (dh + keep * np.abs(h)) @ np.abs(wd).T
    tol += 2.0 ** -20 * np.abs(y) + 2.0 ** (-24 if cfg.act_dtype == "f32" else -8) * np.abs(y) + 1e-30
    return y, tol, h_all, dh_all


def check_h_codes(idx, h, dh, hq, hq_scales):
    """MXFP8 codes of H against the float64 H, for each token's first choice of
    an expert: the block scale is that of a maximum within its bound, and each
    element within half an E4M3 step (2^-4 relative, 2^-10 of the scale below
    the normals; 2^-3 where 448 saturates) of a value within its bound."""
    k = idx.shape[1]
    val = oracle.mxfp8_decode(hq, hq_scales)
    first = np.array([[not np.any(idx[t, :j] == idx[t, j]) for j in range(k)]
                      for t in range(idx.shape[0])]).reshape(-1)
    first &= (idx.reshape(-1) >= 0)
    h, dh, val, sc = h[first], dh[first], val[first], np.asarray(hq_scales, np.int64)[first]
    amax = np.abs(h).reshape(h.shape[0], -1, 32)
    room = dh.reshape(amax.shape)
    lo, hi = (amax - room).max(axis=2), (amax + room).max(axis=2)
    exp = lambda a: np.clip(np.floor(np.log2(np.maximum(a, 1e-300))) - 8, -127, 127) + 127
    assert np.all(sc <= exp(hi)) and np.all((sc >= exp(lo)) | (lo <= 0))
    unit = np.repeat(2.0 ** (sc - 127), 32, axis=1)
    sat = np.abs(h) + dh >= 448 * unit
    half = np.maximum(np.where(sat, 2.0 ** -3, 2.0 ** -4) * (np.abs(h) + dh), 2.0 ** -10 * unit)
    assert np.all(np.abs(val - h) <= half + dh)
    return oracle.mxfp8_decode(hq, hq_scales)
