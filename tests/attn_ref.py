"""Plain 64-bit attention for the tests, one sequence and one head at a time,
with an elementwise bound on the error that the library's number formats allow.

u is half a step of the element type relative to the value: 2^-8 for bf16,
2^-24 for fp32.  What the kernels round:
  - scores: fp32 sums of dk products, (4 sqrt(dk) + 8) 2^-24 sum |q k| scale off (roundings of either sign),
    which is the relative error of a weight (the exponential and its argument
    add 2^-21);
  - weights P: u each, for their product with the values (fp32: none);
  - sums over keys: fp32, at most (keys + 8) 2^-24 of the sum of magnitudes;
  - the result: u.
Gradients: the gated output gradient is stored in the element type (u), delta
is made of `out` as stored (u), dS is rounded like P.
"""

import math

import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F = 2.0 ** -24


def softmax_rows(q, k, v, scale, seen, unit):
    """q [R,dk], k [L,dk], v [L,dv], seen [R,L] (float64): (o, bound on o
    before its last rounding, lse, bound on lse, p, relative bound on p)."""
    s = (q @ k.T) * scale
    size = (q.abs() @ k.abs().T) * scale
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    size = torch.where(seen, size, torch.zeros_like(size))
    lse = torch.logsumexp(s, 1)
    some = seen.any(1)
    p = torch.where(seen, torch.exp(s - torch.where(some, lse, torch.zeros_like(lse))[:, None]), torch.zeros_like(s))
    L = k.shape[0]
    eps = (4 * math.sqrt(q.shape[1]) + 8) * F * size.amax(1, keepdim=True) + 2.0 ** -20  # of a weight, and of the sum of weights
    v0 = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    o = p @ v0
    mag = p @ v0.abs()
    w = unit if unit > F else 0.0
    b_o = mag * (w + 2 * eps + (L + 8) * F * 2) * 1.1
    b_lse = eps[:, 0] + (L + 8) * F + 2.0 ** -20 * (1 + torch.where(some, lse.abs(), torch.zeros_like(lse)))
    return o, b_o, lse, b_lse, p, eps


def causal(n, device):
    return torch.ones(n, n, dtype=torch.bool, device=device).tril()


def prefill(q, k, v, z, lens, scale, dtype):
    """Packed reference: (out, bound, lse, bound), rows behind the last sequence NaN."""
    T, H, _ = q.shape
    G, dv, u = H // k.shape[1], v.shape[2], UNIT[dtype]
    out = torch.full((T, H, dv), math.nan, dtype=torch.float64, device=q.device)
    bo, lse = out.clone(), torch.full((T, H), math.nan, dtype=torch.float64, device=q.device)
    bl = lse.clone()
    at = 0
    for n in lens:
        r = slice(at, at + n)
        at += n
        if n == 0:
            continue
        for h in range(H):
            o, b, l, e, _, _ = softmax_rows(q[r, h], k[r, h // G], v[r, h // G], scale, causal(n, q.device), u)
            if z is not None:
                g = torch.sigmoid(z[r, h])
                o, b = o * g, b * g + o.abs() * g * 2.0 ** -20
            out[r, h], lse[r, h], bl[r, h] = o, l, e
            bo[r, h] = b + u * (o.abs() + b) + 1e-30
    return out, bo, lse, bl


def backward(q, k, v, z, dy, lens, scale, dtype):
    """Packed reference gradients {name: (value, bound)}."""
    T, H, dk = q.shape
    Hkv, dv, u = k.shape[1], v.shape[2], UNIT[dtype]
    G, w = H // Hkv, u if u > F else 0.0
    gated = 1 if z is not None else 0
    dev = q.device
    new = lambda *s: torch.zeros(s, dtype=torch.float64, device=dev)  # noqa: E731
    g = {"dq": new(T, H, dk), "dk": new(T, Hkv, dk), "dv": new(T, Hkv, dv), "dz": new(T, H, dv) if gated else None}
    b = {n: None if x is None else torch.zeros_like(x) for n, x in g.items()}
    at = 0
    for n in lens:
        r = slice(at, at + n)
        at += n
        if n == 0:
            continue
        fs = (n + 8) * F * 2 * max(1, G)
        for h in range(H):
            f = h // G
            o, bo, _, _, p, eps = softmax_rows(q[r, h], k[r, f], v[r, f], scale, causal(n, dev), u)
            do = dy[r, h]
            if gated:
                s = torch.sigmoid(z[r, h])
                y, by = o * s, bo * s + u * (o * s).abs() + (o * s).abs() * 2.0 ** -20
                g["dz"][r, h] = do * y * (1 - s)
                b["dz"][r, h] = do.abs() * (1 - s) * (by + y.abs() * (u + 2.0 ** -19))
                do = do * s
            else:
                y, by = o, bo + u * o.abs()
            ud = u * gated + 2.0 ** -20  # the gated output gradient as stored
            delta = (dy[r, h] * y).sum(1, keepdim=True)
            b_delta = (dy[r, h].abs() * by).sum(1, keepdim=True) + (dv + 8) * F * (dy[r, h] * y).abs().sum(1, keepdim=True)
            dp = do @ v[r, f].T
            mag = do.abs() @ v[r, f].abs().T
            ds = p * (dp - delta)
            b_ds = p * (mag * (ud + (dv + 8) * F) + b_delta) + ds.abs() * (w + 2 * eps) + p * (dp.abs() + delta.abs()) * 4 * F
            g["dq"][r, h] = scale * ds @ k[r, f]
            b["dq"][r, h] = scale * 1.1 * (b_ds @ k[r, f].abs() + fs * (ds.abs() @ k[r, f].abs()))
            g["dk"][r, f] += scale * ds.T @ q[r, h]
            b["dk"][r, f] += scale * 1.1 * (b_ds.T @ q[r, h].abs() + fs * (ds.abs().T @ q[r, h].abs()))
            g["dv"][r, f] += p.T @ do
            b["dv"][r, f] += 1.1 * ((p * (w + ud + 2 * eps + fs)).T @ do.abs())
    return {n: None if g[n] is None else (g[n], b[n] + u * (g[n].abs() + b[n]) + 1e-30) for n in g}


def check(name, got, want, bound):
    got = got.double()
    bad = ~((got - want).abs() <= bound) & ~((got == want) & torch.isinf(want))
    if bool(bad.any()):
        i = int(torch.nonzero(bad.flatten())[0, 0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} values off, first at {i}: got "
                             f"{got.flatten()[i]}, want {want.flatten()[i]} within {bound.flatten()[i]}")
    near = ((got - want).abs() / bound)
    near = near[torch.isfinite(near)]
    print(f"  {name}: at most {float(near.max()) if near.numel() else 0.0:.2f} of the bound", flush=True)
