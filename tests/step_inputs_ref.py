"""Plain float64 forms of the operators that make a step's inputs (8-bit checkpoints, weight
gradients, attention) and the error bounds their tests use."""
import math

import torch

U_BF16 = 2.0 ** -8    # half a bf16 step, relative
U_F32 = 2.0 ** -23    # one fp32 step, relative: a tensor-core sum may truncate


def store(x):
    """(q, byte) of an activation, group by group, from the definition."""
    x = x.detach().double().cpu()
    rows, cols = x.shape
    q = torch.zeros(rows, cols, dtype=torch.int8)
    byte = torch.zeros(rows, (cols + 31) // 32, dtype=torch.uint8)
    for g in range(byte.shape[1]):
        part = x[:, 32 * g:32 * g + 32]
        top = part.abs().amax(1)
        bad = ~torch.isfinite(part).all(1)
        safe = torch.where(bad | (top == 0), torch.ones_like(top), top)
        e = torch.frexp(safe)[1].double() - 1 - 6
        e = torch.where(top == 0, torch.full_like(e, -126.0), e).clamp(min=-126)
        v = torch.round(torch.nan_to_num(part, 0, 0, 0) * torch.exp2(-e)[:, None]).clamp(-127, 127)
        q[:, 32 * g:32 * g + 32] = torch.where(bad[:, None], torch.zeros_like(v), v).to(torch.int8)
        byte[:, g] = torch.where(bad, torch.full_like(e, 255.0), e + 127).to(torch.uint8)
    return q, byte


def restore(q, byte):
    """Restored values in float64."""
    q, byte = q.double().cpu(), byte.cpu().double()
    s = torch.where(byte == 255, torch.full_like(byte, math.inf), torch.exp2(byte - 127))
    s = torch.where(byte == 0, torch.zeros_like(byte), s)
    return q * s.repeat_interleave(32, 1)[:, :q.shape[1]]


def weight_grad(dy, x, offsets):
    """(dW, sum of magnitudes) per group, float64."""
    dy, x = dy.double(), x.double()
    dw = [dy[a:b].t() @ x[a:b] for a, b in zip(offsets, offsets[1:])]
    mag = [dy[a:b].abs().t() @ x[a:b].abs() for a, b in zip(offsets, offsets[1:])]
    return torch.stack(dw), torch.stack(mag)


def spans(q_len, k_len):
    a = b = 0
    for m, n in zip(q_len, k_len):
        yield a, a + m, b, b + n
        a, b = a + m, b + n


def attention(q, k, v, q_len, k_len, causal, scale, dout=None, o=None, lse=None):
    """Forward (and, with dout, o and lse, backward) in float64, with elementwise bounds on
    the error of a kernel that rounds P and dS to bf16, its outputs to bf16, and sums in fp32.

    With S = scale q.k summed in fp32, |error of S| <= dS_ := (D + 4) 2^-23 scale sum |q||k|;
    P = exp(S - lse) is then off by at most slack = 2 (max dS_ + 2^-20) relative (its exponent,
    the approximate exp2, and lse), and its rounding adds 2^-8."""
    q, k, v = q.double(), k.double(), v.double()
    h, g, d = q.shape[1], k.shape[1], q.shape[2]
    out = dict(o=torch.zeros_like(q), lse=torch.full((h, q.shape[0]), -math.inf, dtype=torch.float64, device=q.device),
               s_max=torch.full((h,), -math.inf, dtype=torch.float64, device=q.device))
    tol = dict(o=torch.zeros_like(q), lse=torch.zeros_like(out["lse"]), s_max=0.0)
    if dout is not None:
        dout, o, lse = dout.double(), o.double(), lse.double()
        for n, t in (("dq", q), ("dk", k), ("dv", v)):
            out[n], tol[n] = torch.zeros_like(t), torch.zeros_like(t)
    for a, b, c, e in spans(q_len, k_len):
        m, n = b - a, e - c
        if m == 0 or n == 0:
            continue
        i = torch.arange(m, device=q.device)[:, None]
        j = torch.arange(n, device=q.device)[None]
        see = (j <= i + n - m) if causal else torch.ones(m, n, dtype=torch.bool, device=q.device)
        for hh in range(h):
            kh = hh // (h // g)
            qs, ks, vs = q[a:b, hh], k[c:e, kh], v[c:e, kh]
            s = (qs @ ks.t() * scale).masked_fill(~see, -math.inf)
            ds_ = (d + 4) * U_F32 * float((qs.abs() @ ks.abs().t()).max()) * scale
            slack = 2 * (ds_ + 2.0 ** -20)
            l = torch.logsumexp(s, 1)
            p = torch.exp(s - l[:, None]).masked_fill(~see, 0.0)
            out["lse"][hh, a:b] = l
            tol["lse"][hh, a:b] = ds_ + (n + 8) * U_F32 + 4 * U_F32 * l.abs().nan_to_num(0, 0, 0)
            out["s_max"][hh] = max(float(out["s_max"][hh]), float(s.max()))
            tol["s_max"] = max(tol["s_max"], ds_)
            out["o"][a:b, hh] = p @ vs
            tol["o"][a:b, hh] = (U_BF16 + slack + n * U_F32) * (p @ vs.abs()) + U_BF16 * (p @ vs).abs()
            if dout is None:
                continue
            do, os = dout[a:b, hh], o[a:b, hh]
            p = torch.exp(s - lse[hh, a:b, None]).masked_fill(~see, 0.0)
            dp, delta = do @ vs.t(), (do * os).sum(1, keepdim=True)
            dp_err = (d + 4) * U_F32 * (do.abs() @ vs.abs().t() + (do * os).abs().sum(1, keepdim=True))
            ds = p * (dp - delta)
            ds_tol = (U_BF16 + slack + (m + n) * U_F32) * ds.abs() + 2 * p * dp_err
            out["dq"][a:b, hh] = scale * ds @ ks
            tol["dq"][a:b, hh] = scale * ds_tol @ ks.abs()
            out["dk"][c:e, kh] += scale * ds.t() @ qs
            tol["dk"][c:e, kh] += scale * ds_tol.t() @ qs.abs()
            out["dv"][c:e, kh] += p.t() @ do
            tol["dv"][c:e, kh] += (U_BF16 + slack + (m + n) * U_F32) * (p.t() @ do.abs())
    for n in ("dq", "dk", "dv"):
        if n in out:
            tol[n] = tol[n] + U_BF16 * (out[n].abs() + tol[n])
    return out, tol


def check(got, want, tol, what):
    """Elementwise |got - want| <= tol; infinities and NaN must agree."""
    got = got.double()
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    bad = ~(same | ((got - want).abs() <= tol))
    if bool(bad.any()):
        at = bad.nonzero()[0].tolist()
        t = tol[tuple(at)] if torch.is_tensor(tol) and tol.dim() else tol
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {at}: "
                             f"{float(got[tuple(at)])} for {float(want[tuple(at)])}, bound {float(t)}")
