"""hca_shared_attend over one slot in 64 bits, on any device, with the error that its arithmetic allows.

Per channel, with w_j the weights (they add up to one) and A = sum_j w_j |e_j|:

* a weight is rounded to fp16 (2^-11 of it) and the products are summed in float32, which loses at most 2^-23
  of the running sum per 16-entry step: (2^-11 + (n / 16 + 8) 2^-23) A;
* fp16's smallest step is 2^-24: a weight is off by up to half of that, times 2^reference. References lie 7 bits
  or more below the largest logit (rows' exponents included), so that is 2^-32 of the largest w_k |e_k| per block;
* the logits are off by 2^-23 of scale * sum |q e| per 16-channel step and a few more, and by 2^-23 for each
  binade between the rows' scales, which are added to them; the sum of exponentials by 2^-20;
* the output is rounded to bf16: half a step, 2^-8 of the value."""
import math

import torch

E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6]


def entries(codes, raw, e4m3=False):
    """[n, D] float64 of codes [n, D / 2] and scale bytes [n, D / 32 or D / 16]."""
    lut = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)
    e = torch.stack((lut[(codes & 15).long()], lut[(codes >> 4).long()]), -1).reshape(codes.shape[0], raw.shape[1], -1)
    s = raw.view(torch.float8_e4m3fn).double() if e4m3 else torch.exp2(raw.double() - 127)
    return (e * s[..., None]).reshape(codes.shape[0], -1)


def attend(e, q, scale, seen=None):
    """(out, lse, tolerance of out with its rounding, tolerance of lse) of q [Q, H, D] over the first seen[i]
    (all) of the entries e [n, D]."""
    Q, H, D = q.shape
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol, lse = torch.zeros_like(out), torch.full((Q, H), -math.inf, dtype=torch.float64, device=q.device)
    dl = torch.zeros_like(lse)
    top = e.abs().amax(1)
    for i in range(Q):
        n = e.shape[0] if seen is None else int(seen[i])
        if n == 0:
            continue
        x, t = e[:n], top[:n]
        u = scale * (q[i].double() @ x.T)
        lse[i] = torch.logsumexp(u, -1)
        w = torch.exp(u - lse[i][:, None])
        out[i], A = w @ x, w @ x.abs()
        some = t[t > 0]
        binades = float(torch.log2(some.max() / some.min())) if len(some) else 0.0
        dl[i] = (2.0 ** -20 + 2.0 ** -23 * (binades + lse[i].abs())
                 + 2.0 ** -23 * (D / 16 + 8) * abs(scale) * (q[i].double().abs() @ x.abs().T).amax(-1))
        least = n * 2.0 ** -32 * (w * t).amax(-1)
        before = (2.0 ** -11 + (n / 16 + 8) * 2.0 ** -23 + 2 * dl[i][:, None]) * A + least[:, None]
        tol[i] = before + 2.0 ** -8 * (out[i].abs() + before)
    return out, lse, tol, dl
