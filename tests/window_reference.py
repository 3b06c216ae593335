"""64-bit forms of attention under any mask, with first-order bounds of the kernels' errors.

Not a test module: the GPU tests import it.
"""
import math

import torch

from paged_reference import EPS


def seen(Nq, Nk, window, sinks, device="cuda"):
    """[Nq, Nk]: query i sees key j."""
    i, j = torch.arange(Nq, device=device)[:, None], torch.arange(Nk, device=device)[None]
    return (j <= i) & ((i - j < window) | (j < sinks))


def shared(t, H):
    return t.double().repeat_interleave(H // t.shape[1], 1)


def forward(q, k, v, mask, scale, out_eps):
    """(O, LSE, bound of |dO|, bound of |dLSE|, P, error of a weight, relative) of q [B, H, Nq, d], k, v [B, Hkv, Nk, d].

    With u half a step of the input type and A = sum_j p_j |v_j|: rounding each P
    costs at most u A, rounding O out_eps |O|.  A score is a sum of d products in
    fp32: its error is at most delta = 2 d 2^-24 scale max_j sum_c |q_c k_jc| (2: the
    tensor core may truncate), which changes every weight by at most a relative 2 delta
    after normalisation; the exponential (2^-21) and the row sum (n 2^-24) add to
    that.  fp16 P below 2^-14 are rounded with an absolute error of at most 2^-25
    while the row's largest P is at least 1.
    """
    u, d, H = EPS[q.dtype], q.shape[-1], q.shape[1]
    x, kk, vv = q.double(), shared(k, H), shared(v, H)
    s = (x @ kk.transpose(-1, -2) * scale).masked_fill(~mask, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    o, A = p @ vv, p @ vv.abs()
    mag = (x.abs() @ kk.abs().transpose(-1, -2)).masked_fill(~mask, 0.0)
    rel = 2 * (2 * d * 2.0 ** -24 * scale * mag.amax(-1) + 2.0 ** -21 + k.shape[2] * 2.0 ** -24)
    tiny = 2.0 ** -25 * (mask.double() @ vv.abs()) if q.dtype is torch.float16 else 0.0
    bO = (u + rel[..., None]) * A + out_eps * o.abs() + tiny + 1e-30
    bL = rel + lse.abs().nan_to_num(0.0, posinf=0.0) * 2.0 ** -22 + 2.0 ** -22
    return o, lse, bO, bL, p, rel


def backward(q, k, v, do, mask, scale, o_eps, grad_eps):
    """((dQ, dK, dV), bounds).

    P (for dV) and dS (for dQ, dK) are rounded to the input type: u |p|, u |ds|.  D = dO
    . O takes the forward's O, which carries u A and, where it was stored in 16 bits,
    u |O|: p |dO| . (u A + o_eps |O|) in ds.  A relative error `rel` of p (see
    forward) and the fp32 sums of d and N products (2 (d + N) 2^-24) scale with the
    same sizes.  fp16 P and dS below 2^-14 are rounded with an absolute error of
    2^-25.  Gradients kept in 16 bits are rounded once more.
    """
    u, H, Hkv, d = EPS[q.dtype], q.shape[1], k.shape[1], q.shape[-1]
    o, _, _, _, p, rel = forward(q, k, v, mask, scale, 0.0)
    x, kk, vv, g = q.double(), shared(k, H), shared(v, H), do.double()
    A = p @ vv.abs()
    dp = g @ vv.transpose(-1, -2)
    D = (g * o).sum(-1, keepdim=True)
    ds = p * (dp - D)
    size = p * (dp.abs() + D.abs())            # what relative errors of p, dp and D scale with
    offD = (g.abs() * (u * A + o_eps * o.abs())).sum(-1, keepdim=True)
    more = rel[..., None] + 2 * (d + q.shape[2] + k.shape[2]) * 2.0 ** -24 + 2.0 ** -20
    absolute = 2.0 ** -25 * mask.double() if q.dtype is torch.float16 else 0.0
    err_ds = u * ds.abs() + p * offD + more * size + p * (g.abs() @ vv.abs().transpose(-1, -2)) * d * 2.0 ** -23 + absolute
    err_p = (u + more) * p + absolute

    def group(t):
        return t.unflatten(1, (Hkv, H // Hkv)).sum(2)

    t = lambda a: a.transpose(-1, -2)  # noqa: E731
    grads = scale * (ds @ kk), scale * group(t(ds) @ x), group(t(p) @ g)
    bounds = scale * (err_ds @ kk.abs()), scale * group(t(err_ds) @ x.abs()), group(t(err_p) @ g.abs())
    return grads, [b * (1 + 2 * grad_eps) + grad_eps * a.abs() + 2.0 ** -25 for a, b in zip(grads, bounds)]


def paged(q, keys, values, q_lens, masks, scale, out_eps, parts=1):
    """Packed queries [T, Hq, d] over each sequence's keys [n, Hkv, d] under its mask [new tokens, n]: (O, LSE, bounds).

    With `parts` > 1 a row's result is joined from parts whose sums carry `rel` each, as do their weights.
    """
    out, at = [], 0
    for n, k, v, mask in zip(q_lens, keys, values, masks):
        heads = lambda t: t.transpose(0, 1)[None]  # noqa: E731
        if k.shape[0] == 0:   # one key that nobody sees
            k, v, mask = k.new_zeros(1, *k.shape[1:]), v.new_zeros(1, *v.shape[1:]), mask.new_zeros(n, 1)
        if n:
            o, lse, bO, bL, _, rel = forward(heads(q[at:at + n]), heads(k), heads(v), mask, scale, out_eps)
            A = (bO - out_eps * o.abs()) / (EPS[q.dtype] + rel[..., None])   # (at least sum p |v|)
            bO = bO + 2 * (parts - 1) * rel[..., None] * A
            out.append([t[0].transpose(0, 1) for t in (o, lse, bO, bL * parts)])
        at += n
    d, H = q.shape[2], q.shape[1]
    if not out:
        return [torch.zeros(s, dtype=torch.float64, device=q.device) for s in ((0, H, d), (0, H), (0, H, d), (0, H))]
    return [torch.cat(t) for t in zip(*out)]
