"""Plain 64-bit forms of the rotary positions and of the cross-attention with
its gradients, and how far a kernel may be from them.

The allowances are worst cases, element by element, counted from the roundings
that the kernels make: u = half a step of the input type relative to a value
(bf16 2^-8, fp32 2^-24), w = 2^-24 for every 32-bit operation.

  scores   |dx_j| <= (d + 4) w s sum_c |q_c k_jc|: a d-term 32-bit dot product
           and the scaling
  p        relative: 2 max_j |dx_j| (in the numerator and in the sum), 2^-20 for
           the exponential (argument below 2^7 in binary units rounded to 2^-17
           at most at the far end, where p < 2^-100; 2^-21 near the maximum),
           (Lk + 8) w for the sum; bf16 inputs: u more, p enters the product in
           bf16
  out      that, times sum_j p_j |v_j|, and u |out| for the store
  dv       the same with sum_i p_ij |g_i|
  dp       (d + 2) w sum_c |g_c v_jc|;  delta: what out may be off times |g|,
           and (d + 2) w sum |g| |out|
  ds       p [ (rel_p + u) |dp - delta| + d(dp) + d(delta) ], u for ds in bf16
  dq, dk   sums of that times |k|, |q|, their own 32-bit summation, u at the store
"""

import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
W = 2.0 ** -24


def rope_freqs(axis_dims, theta, scaling="none", factor=1.0, original_len=0):
    f, axis = [], []
    for a, D in enumerate(axis_dims):
        base = theta * factor ** (D / (D - 2.0)) if scaling == "ntk" else theta
        for i in range(D // 2):
            x = base ** (-2.0 * i / D)
            if scaling == "linear":
                x /= factor
            if scaling == "yarn":
                g = min(1.0, max(0.0, (original_len * x / (2 * math.pi) - 1) / 31))
                x = g * x + (1 - g) * x / factor
            f.append(x)
            axis.append(a)
    return f, axis, 0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0


def rope_ref(x, positions, axis_dims, theta=10000.0, layout="interleaved", scaling="none", factor=1.0,
             original_len=0, backward=False):
    """(result in 64 bits, allowance) for x [b,h,L,d]."""
    f, axis, m = rope_freqs(axis_dims, theta, scaling, factor, original_len)
    P = len(f)
    pos = positions.double() if positions.dim() == 3 else positions.double()[None]
    a = pos[..., axis] * torch.tensor(f, dtype=torch.float64, device=x.device)  # [b or 1, L, P]
    c, s = (m * torch.cos(a))[:, None], (m * torch.sin(a))[:, None]
    if backward:
        s = -s
    y = x.double()
    out, tol = y.clone(), torch.zeros_like(y)
    u, w = (slice(0, 2 * P, 2), slice(1, 2 * P, 2)) if layout == "interleaved" else (slice(0, P), slice(P, 2 * P))
    out[..., u] = y[..., u] * c - y[..., w] * s
    out[..., w] = y[..., u] * s + y[..., w] * c
    # sine and cosine within 2^-22 (the reduced angle, at most pi, rounded to 32 bits, and two
    # steps of the function), two products and a sum: 2^-21 (|u| + |w|) m, and one rounding
    both = (y[..., u].abs() + y[..., w].abs()) * m * 2.0 ** -21
    tol[..., u], tol[..., w] = both, both
    rounding = U[x.dtype] * out.abs()
    rounding[..., 2 * P:] = 0  # copied
    return out, tol + rounding


def allowed_keys(b, Lk, kv_len, key_mask, device):
    ok = torch.ones(b, Lk, dtype=torch.bool, device=device)
    if kv_len is not None:
        ok &= torch.arange(Lk, device=device) < kv_len[:, None].clamp(0, Lk)
    if key_mask is not None:
        ok &= key_mask != 0
    return ok


def cross_ref(q, k, v, kv_len=None, key_mask=None, dout=None):
    """{name: (64-bit value, allowance)} for out, lse and, with dout, dq, dk, dv."""
    u, bf16 = U[q.dtype], q.dtype == torch.bfloat16
    b, h, Lq, d = q.shape
    hk, Lk = k.shape[1], k.shape[2]
    g = h // hk
    ok = allowed_keys(b, Lk, kv_len, key_mask, q.device)[:, None, None, :]
    s = 1 / math.sqrt(d)
    Q = q.double()
    # what is not allowed counts as zero, whatever it holds
    K, V = (torch.where(ok[:, :, 0, :, None], x.double(), 0.0).repeat_interleave(g, 1) for x in (k, v))
    x = (Q @ K.mT * s).masked_fill(~ok, -math.inf)
    lse = torch.logsumexp(x, -1)
    none = ~ok.any(-1, keepdim=True)
    p = torch.where(none, 0.0, torch.exp(x - lse[..., None]))
    out = p @ V
    dx = (d + 4) * W * s * (Q.abs() @ K.abs().mT).amax(-1, keepdim=True)
    sums = (Lk + 8) * W
    rel = 2 * dx + 2.0 ** -20 + sums + (u if bf16 else 0.0)
    tol_out = (rel + sums) * (p @ V.abs()) + u * out.abs()
    r = {"out": (out, tol_out), "lse": (lse, (dx[..., 0] + 2.0 ** -20 + sums) + 4 * W * lse.abs().nan_to_num(posinf=0.0))}
    if dout is None:
        return r
    G = dout.double()
    dp = G @ V.mT
    delta = (G * out).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    e_dp = (d + 2) * W * (G.abs() @ V.abs().mT)
    e_delta = (G.abs() * tol_out).sum(-1, keepdim=True) + (d + 2) * W * (G.abs() * out.abs()).sum(-1, keepdim=True)
    e_ds = p * ((rel + u) * (dp - delta).abs() + e_dp + e_delta)
    many = (Lq * g + 8) * W

    def shared(t):
        return t.reshape(b, hk, g, Lk, d).sum(2)

    dq, tq = s * ds @ K, s * (e_ds + (sums + 4 * W) * ds.abs()) @ K.abs()
    dk, tk = shared(s * ds.mT @ Q), shared(s * (e_ds + many * ds.abs()).mT @ Q.abs())
    dv, tv = shared(p.mT @ G), shared(((rel + many) * p).mT @ G.abs())
    for name, val, tol in (("dq", dq, tq), ("dk", dk, tk), ("dv", dv, tv)):
        r[name] = (val, tol + u * val.abs())
    return r


def assert_within(got, ref, what):
    val, tol = ref
    assert got.shape == val.shape, what
    g = got.double()
    inf = torch.isinf(val)
    assert torch.equal(g[inf], val[inf]), f"{what}: infinities"
    off = torch.where(inf, 0.0, (g - val).abs() - tol - 1e-30)
    assert not torch.isnan(off).any(), f"{what}: NaN"
    worst = off.max().item() if off.numel() else 0.0
    if worst > 0:
        i = torch.unravel_index(off.argmax(), off.shape)
        raise AssertionError(f"{what} at {tuple(int(x) for x in i)}: {g[i].item():.7g} for {val[i].item():.7g}, "
                             f"allowed {tol[i].item():.3g}")
