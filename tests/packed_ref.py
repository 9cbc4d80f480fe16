"""64-bit restatement of attention over packed sequences and of its gradients
(PyTorch, a sequence and a query head at a time), with the error that the
kernels' roundings allow for each element."""
from __future__ import annotations

import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative to the value
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}        # half the smallest step


def offsets(lens, first=0):
    out = [first]
    for n in lens:
        out.append(out[-1] + n)
    return out


def visible(n_q, n_k, causal, device):
    """[n_q, n_k]: what each query sees."""
    if not causal:
        return torch.ones(n_q, n_k, dtype=torch.bool, device=device)
    i = torch.arange(n_q, device=device)[:, None] + (n_k - n_q)
    return torch.arange(n_k, device=device) <= i


def sums(n):
    """Relative error of a sum of n products in fp32: a rounding (or a truncation, a step) for every 16 terms that the
    tensor cores add at once, and some for what is done to the sum."""
    return (n / 16 + 16) * 2.0 ** -23


def attend(q, k, v, scale, see, half, tiny):
    """One head: q [n, d], k, v [m, d] in 64 bits.  (out, lse) and their tolerances.

    A weight's relative error: the score's (sums of d products of magnitude |q||k|), the exponential's and the sums'
    (2^-20).  Weights are rounded for the product with V, in the sum that divides it the largest one of a tile too:
    half a step of each.  fp16 weights also lose `tiny`, where the largest is at least 1."""
    s = q @ k.T * scale
    s = s.masked_fill(~see, -math.inf)
    lse = torch.logsumexp(s, -1) if s.shape[1] else torch.full(s.shape[:1], -math.inf, dtype=s.dtype, device=s.device)
    p = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[:, None])
    out = p @ v
    big = (q.abs() @ k.abs().T * abs(scale)).masked_fill(~see, 0.0)
    big = big.amax(-1) if s.shape[1] else torch.zeros_like(lse)
    score = sums(q.shape[1]) * big
    rel = 2 * half + 2 * score[:, None] + 2.0 ** -20 + sums(len(k))
    av = p @ v.abs()
    vmax = v.abs().max() if v.numel() else 0.0
    tol = half * out.abs() + (1 + half) * (rel * (av + out.abs()) + len(k) * tiny * vmax) + tiny + 1e-30
    finite = torch.where(lse == -math.inf, 0.0, lse)
    return out, lse, tol, score + sums(len(k)) + 2.0 ** -22 * finite.abs()


def forward(q, k, v, cu_q, cu_k, scale, causal):
    """(out, lse, tolerances of both); rows of no sequence are NaN."""
    half, tiny = HALF[q.dtype], TINY[q.dtype]
    T, H, d = q.shape
    group = H // k.shape[1]
    f64 = dict(dtype=torch.float64, device=q.device)
    out, tol = torch.full((T, H, d), math.nan, **f64), torch.zeros(T, H, d, **f64)
    lse, tol_l = torch.full((H, T), math.nan, **f64), torch.zeros(H, T, **f64)
    for a, b, e, f in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        see = visible(b - a, f - e, causal, q.device)
        for h in range(H):
            got = attend(q[a:b, h].double(), k[e:f, h // group].double(), v[e:f, h // group].double(), scale, see, half,
                         tiny)
            out[a:b, h], lse[h, a:b], tol[a:b, h], tol_l[h, a:b] = got
    return out, lse, tol, tol_l


def backward(q, k, v, o, lse, dout, cu_q, cu_k, scale, causal):
    """{name: (gradient, tolerance)} for the o and lse that are given; rows of no sequence are NaN.

    P = exp(s - lse) and dS = P (dP - D) are rounded for their products (half a step each, fp16 also `tiny`), P's
    relative error is the score's and lse's, dP and D are sums over d.  The tolerance of an element adds these up over
    the element's terms, with the fp32 sum's error and the output's own rounding."""
    half, tiny = HALF[q.dtype], TINY[q.dtype]
    (T, H, d), (Tk, H_kv, _) = q.shape, k.shape
    group = H // H_kv
    f64 = dict(dtype=torch.float64, device=q.device)
    val = {n: torch.full(x.shape, math.nan, **f64) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    tol = {n: torch.zeros(x.shape, **f64) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    for a, b, e, f in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        see = visible(b - a, f - e, causal, q.device)
        n = (b - a) * group
        for x in (val, tol):
            x["dk"][e:f], x["dv"][e:f] = 0.0, 0.0
        for h in range(H):
            g = h // group
            Q, K, V = q[a:b, h].double(), k[e:f, g].double(), v[e:f, g].double()
            O, D, L = o[a:b, h].double(), dout[a:b, h].double(), lse[h, a:b, None].double()
            dead = L == -math.inf
            p = torch.exp(Q @ K.T * scale - torch.where(dead, 0.0, L)).masked_fill(~see | dead, 0.0)
            big = (Q.abs() @ K.abs().T * abs(scale)).masked_fill(~see, 0.0)
            rel = 2 * sums(d) * big + 2.0 ** -20 + 2.0 ** -21 * torch.where(dead, 0.0, L).abs()
            diff = D @ V.T - (D * O).sum(-1, keepdim=True)
            off = sums(d) * (D.abs() @ V.abs().T + (D.abs() * O.abs()).sum(-1, keepdim=True))
            ds = p * diff
            e_p = (half + rel) * p + tiny
            e_s = (1 + half) * p * (rel * diff.abs() + off) + half * ds.abs() + tiny
            e_p, e_s = (x.masked_fill(~see | dead, 0.0) for x in (e_p, e_s))
            val["dq"][a:b, h] = ds @ K * scale
            tol["dq"][a:b, h] = abs(scale) * (e_s @ K.abs() + sums(f - e) * (ds.abs() @ K.abs()))
            val["dk"][e:f, g] += ds.T @ Q * scale
            tol["dk"][e:f, g] += abs(scale) * (e_s.T @ Q.abs() + sums(n) * (ds.abs().T @ Q.abs()))
            val["dv"][e:f, g] += p.T @ D
            tol["dv"][e:f, g] += e_p.T @ D.abs() + sums(n) * (p.T @ D.abs())
    return {n: (val[n], (1 + half) * tol[n] + half * val[n].abs() + tiny + 1e-30) for n in val}
