"""The operators around the piecewise sparse self-attention of a diffusion
transformer block: rotary positions of its queries and keys, and the
cross-attention of its tokens to an encoder's states, forward and backward.

Each case is timed through run(): with `own` false as the formulas written out
in torch operations (32 bits, angles in 64, one rounding at the end), with
`own` true through the library's entry points.  exact() is the definition in
64 bits.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}


# ------------------------------------------------------------------ cases

def _rope(name, **kw):
    c = {"op": "rope", "dtype": "bf16", "b": 1, "h": 24, "hk": 24, "L": 4608, "d": 128, "axes": "16,56,56",
         "layout": "interleaved", "theta": 10000.0, "scaling": "none", "factor": 1.0, "original": 0,
         "backward": False}
    c.update(kw)
    return dict(c, name=name) if name else c


def _cross(name, **kw):
    c = {"op": "cross", "dtype": "bf16", "b": 1, "h": 24, "hk": 24, "Lq": 4608, "Lk": 512, "d": 128,
         "mask": "none", "keep": 1.0, "empty": False, "train": False}
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the smallest call: one fp32 head of 1024 tokens, half layout; latency is all that counts
        _rope("rope_one_head_fp32", dtype="fp32", h=1, hk=1, L=1024, d=64, axes="64", layout="half"),
        # an image transformer's 64x72 token grid, three axes (the first constant), out of the projection's layout
        _rope("rope_image"),
        # one attention layer of a 75600-token video (21x45x80 grid), 40 heads: the largest
        _rope("rope_video", h=40, hk=40, L=75600, axes="44,42,42"),
        # the gradient of the 480p video layer (21x30x52 grid), written back in the projection's layout
        _rope("rope_video_backward", h=40, hk=40, L=32760, axes="44,42,42", backward=True),
        # a text encoder's long prompt: half layout, half of the head, shared key heads, by-parts scaling to 4x
        _rope("rope_long_partial", b=2, h=40, hk=8, L=9973, axes="64", layout="half", scaling="yarn", factor=4.0,
              original=4096),
        # one learned query that pools a 4608-token image: a single token, latency and key bandwidth
        _cross("cross_pool_one_query", b=2, h=40, hk=40, Lq=1, Lk=4608),
        # the small fp32 block: one head, 77 encoder states
        _cross("cross_one_head_fp32", dtype="fp32", h=1, hk=1, Lq=1024, Lk=77, d=64),
        # two prompts padded to 512 states of which a quarter are words
        _cross("cross_image_padded", b=2, mask="len", keep=0.25),
        # the 75600-token video against 512 text states: the largest inference call
        _cross("cross_video", h=40, hk=40, Lq=75600),
        # a training step of the 480p layer: forward and backward
        _cross("cross_video_train", h=40, hk=40, Lq=32760, train=True),
        # odd sizes, shared key heads and a mask with holes, forward and backward
        _cross("cross_masked_train", b=2, h=24, hk=8, Lq=1023, Lk=333, d=64, mask="mask", keep=0.6, train=True),
        # fp32 training of a small block whose second prompt is dropped (every key masked)
        _cross("cross_dropped_train_fp32", dtype="fp32", b=2, h=4, hk=4, Lq=1000, Lk=77, d=64, mask="len", keep=0.5,
               empty=True, train=True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm spread evenly."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    hk = rng.choice([1, 2, 3, 5, 8, 12, 24, 40])
    return hk * rng.choice([g for g in (1, 1, 1, 2, 3, 5) if hk * g <= 40]), hk


def _draw_rope(rng):
    d = rng.choice([64, 128])
    h, hk = _heads(rng)
    b = rng.choice([1, 1, 2, 3])
    L = _log(rng, 1, min(75600, 300_000_000 // (b * (h + hk) * d)))
    n = rng.choice([1, 2, 3])
    scaling = rng.choice(["none", "linear", "ntk", "yarn"])
    pairs = rng.choice([d // 2, d // 2, d // 4, rng.randint(2 * n, d // 2)])  # each axis has two pairs or more
    cut = sorted(rng.sample(range(1, pairs - n), n - 1)) if n > 1 else []
    axes = [2 * (y - x + 1) for x, y in zip([0] + cut, cut + [pairs - n])]
    return _rope(None, dtype=rng.choice(["bf16", "bf16", "fp32"]), b=b, h=h, hk=hk, L=L, d=d,
                 axes=",".join(map(str, axes)), layout=rng.choice(["interleaved", "half"]),
                 theta=rng.choice([256.0, 10000.0, 500000.0]), scaling=scaling,
                 factor=1.0 if scaling == "none" else rng.choice([1.5, 2.0, 4.0, 8.0]),
                 original=1024 if scaling == "yarn" else 0, backward=rng.random() < 0.4)


def _draw_cross(rng):
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    d = rng.choice([64, 128])
    h, hk = _heads(rng)
    b = rng.choice([1, 1, 2, 3])
    train = rng.random() < 0.5
    Lk = _log(rng, 2 if train else 1, 4608)  # with one key the gradients of q and k are zero: noise has no relative error
    cap = (400_000_000 if dtype == "bf16" else 40_000_000) // (b * h * Lk)
    Lq = _log(rng, 1, max(1, min(32760, cap, 150_000_000 // (b * h * d))))
    mask = rng.choice(["none", "len", "mask"])
    return _cross(None, dtype=dtype, b=b, h=h, hk=hk, Lq=Lq, Lk=Lk, d=d, mask=mask,
                  keep=1.0 if mask == "none" else rng.choice([0.1, 0.35, 0.6, 0.9]),
                  empty=mask != "none" and b > 1 and rng.random() < 0.3, train=train)


def draw(rng):
    return _draw_rope(rng) if rng.random() < 0.4 else _draw_cross(rng)


# ------------------------------------------------------------------ inputs

def _projected(g, b, L, h, d, dt):
    """[b, h, L, d] as a projection leaves it: a view of [b, L, h, d]."""
    return torch.randn(b, L, h, d, device="cuda", generator=g).to(dt).permute(0, 2, 1, 3)


def _axes(case):
    return tuple(int(x) for x in case["axes"].split(","))


def _kept(case):
    """Keys that may be attended to, per batch entry."""
    n = [max(2 if case["train"] else 1, round(case["keep"] * case["Lk"]))] * case["b"]
    if case["empty"]:
        n[-1] = 0
    return n


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = TYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "rope":
        b, L, d = case["b"], case["L"], case["d"]
        n = len(_axes(case))
        if case["backward"]:  # gradients come as the attention leaves them, dense [b, h, L, d]
            s["q"] = torch.randn(b, case["h"], L, d, device="cuda", generator=g).to(dt)
            s["k"] = torch.randn(b, case["hk"], L, d, device="cuda", generator=g).to(dt)
        else:
            s["q"] = _projected(g, b, L, case["h"], d, dt)
            s["k"] = _projected(g, b, L, case["hk"], d, dt)
        # raster positions of a grid whose last axes are about as long as each other, from a seeded origin
        side = max(1, int(round(L ** (1.0 / n))))
        t = torch.arange(L, device="cuda", dtype=torch.int64)
        cols = [t if n == 1 else t // side ** (n - 1)] + [t // side ** (n - 1 - a) % side for a in range(1, n)]
        first = torch.randint(0, 1000, (n,), device="cuda", generator=g)
        s["pos"] = (torch.stack(cols, 1) + first).float().contiguous()
        return s
    b, h, hk, Lq, Lk, d = (case[x] for x in ("b", "h", "hk", "Lq", "Lk", "d"))
    s["q"] = _projected(g, b, Lq, h, d, dt)
    kv = torch.randn(b, Lk, 2, hk, d, device="cuda", generator=g).to(dt)  # one projection of the encoder's states
    s["k"], s["v"] = kv[:, :, 0].permute(0, 2, 1, 3), kv[:, :, 1].permute(0, 2, 1, 3)
    if case["train"]:
        s["dout"] = _projected(g, b, Lq, h, d, dt)
    n = torch.tensor(_kept(case), device="cuda")
    if case["mask"] == "len":
        s["kv_len"] = n.to(torch.int32)
    elif case["mask"] == "mask":
        rank = torch.rand(b, Lk, device="cuda", generator=g).argsort(1).argsort(1)
        s["key_mask"] = rank < n[:, None]
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _own_rope(state) if state["case"]["op"] == "rope" else _own_cross(state)
    return _plain_rope(state) if state["case"]["op"] == "rope" else _plain_cross(state)


def _own_rope(s):
    import sparse_attention_diffusion_block_b200 as pisa
    c = s["case"]
    spec = dict(axis_dims=_axes(c), theta=c["theta"], layout=c["layout"], scaling=c["scaling"], factor=c["factor"],
                original_len=c["original"])
    if not c["backward"]:
        return pisa.rope(s["q"], s["k"], s["pos"], **spec)
    out = [torch.empty(x.shape[0], x.shape[2], x.shape[1], x.shape[3], dtype=x.dtype, device=x.device)
           .permute(0, 2, 1, 3) for x in (s["q"], s["k"])]
    return pisa.rope_bwd(s["q"], s["k"], s["pos"], q_out=out[0], k_out=out[1], **spec)


def _own_cross(s):
    import sparse_attention_diffusion_block_b200 as pisa
    mask = dict(kv_len=s.get("kv_len"), key_mask=s.get("key_mask"))
    q, k, v = s["q"], s["k"], s["v"]
    if not s["case"]["train"]:
        return pisa.cross_attn_fwd(q, k, v, **mask)
    out, lse = pisa.cross_attn_fwd(q, k, v, return_lse=True, **mask)
    return (out,) + tuple(pisa.cross_attn_bwd(s["dout"], q, k, v, out, lse, **mask))


def _frequencies(c):
    """(angle per unit of position [pairs] in 64 bits, axis of each pair, magnitude)."""
    dims = torch.tensor(_axes(c), device="cuda")
    axis = torch.repeat_interleave(torch.arange(dims.numel(), device="cuda"), dims // 2)
    start = torch.cumsum(dims // 2, 0) - dims // 2
    i = torch.arange(axis.numel(), device="cuda") - start[axis]
    D = dims[axis].double()
    theta = torch.full_like(D, c["theta"])
    if c["scaling"] == "ntk":
        theta = theta * c["factor"] ** (D / (D - 2))
    f = theta ** (-2.0 * i.double() / D)
    if c["scaling"] == "linear":
        f = f / c["factor"]
    if c["scaling"] == "yarn":
        keep = ((c["original"] * f / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
        f = f * keep + f / c["factor"] * (1 - keep)
    return f, axis, 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "yarn" else 1.0


def _plain_rope(s):
    c = s["case"]
    f, axis, m = _frequencies(c)
    a = s["pos"].double()[:, axis] * f
    cos, sin = (torch.cos(a) * m).float(), (torch.sin(a) * m).float()
    if c["backward"]:
        sin = -sin
    rot = 2 * f.numel()

    def turn(x):
        y = x.float()
        r = y[..., :rot]
        if c["layout"] == "interleaved":
            u, w = r[..., 0::2], r[..., 1::2]
            z = torch.stack((u * cos - w * sin, u * sin + w * cos), -1).flatten(-2)
        else:
            u, w = r[..., : rot // 2], r[..., rot // 2:]
            z = torch.cat((u * cos - w * sin, u * sin + w * cos), -1)
        return torch.cat((z, y[..., rot:]), -1).to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def _allowed(s):
    """[b, 1, 1, Lk] truth values of the keys that may be attended to, or None."""
    if "kv_len" in s:
        return (torch.arange(s["k"].shape[2], device="cuda") < s["kv_len"][:, None])[:, None, None, :]
    return s["key_mask"][:, None, None, :] if "key_mask" in s else None


def _plain_cross(s):
    q, k, v = s["q"], s["k"], s["v"]
    dt, b, hk, d, g = q.dtype, q.shape[0], k.shape[1], q.shape[3], q.shape[1] // k.shape[1]
    scale = 1.0 / math.sqrt(d)
    qf = q.float()
    kf, vf = (x.float().repeat_interleave(g, 1) for x in (k, v))
    x = torch.matmul(qf, kf.transpose(-1, -2)) * scale
    ok = _allowed(s)
    if ok is not None:
        x = torch.where(ok, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    del x
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    out = torch.matmul(p, vf)
    if not s["case"]["train"]:
        return out.to(dt)
    do = s["dout"].float()
    dv = torch.matmul(p.transpose(-1, -2), do)
    dp = torch.matmul(do, vf.transpose(-1, -2))
    ds = p * (dp - (do * out).sum(-1, keepdim=True)) * scale
    del p, dp
    dq = torch.matmul(ds, kf)
    dk = torch.matmul(ds.transpose(-1, -2), qf)
    dk, dv = (y.reshape(b, hk, g, -1, d).sum(2).to(dt) for y in (dk, dv))
    return out.to(dt), dq.to(dt), dk, dv


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] == "rope":
        n = case["b"] * (case["h"] + case["hk"]) * case["L"]
        rot = sum(_axes(case))
        return {"bytes": 2 * n * case["d"] * e + 4 * case["L"] * len(_axes(case)), "flops": 3 * n * rot}
    b, h, hk, Lq, Lk, d = (case[x] for x in ("b", "h", "hk", "Lq", "Lk", "d"))
    keys = sum(_kept(case)) if case["mask"] != "none" else b * Lk
    rows, kv = b * h * Lq * d * e, hk * keys * d * e
    mask = {"none": 0, "len": 4 * b, "mask": b * Lk}[case["mask"]]
    if case["train"]:  # q, dout, k, v in; out, dq, dk, dv out
        return {"bytes": 4 * rows + 2 * kv + 2 * b * hk * Lk * d * e + mask, "flops": 14 * h * Lq * keys * d}
    return {"bytes": 2 * rows + 2 * kv + mask, "flops": 4 * h * Lq * keys * d}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_rope(c, s):
    """Each pair is a complex number, multiplied by magnitude * e^{i angle} (its conjugate backwards)."""
    turns, axis = [], []
    for a, D in enumerate(_axes(c)):
        base = c["theta"] * (c["factor"] ** (D / (D - 2.0)) if c["scaling"] == "ntk" else 1.0)
        for i in range(D // 2):
            f = math.exp(-2.0 * i / D * math.log(base))
            if c["scaling"] == "linear":
                f /= c["factor"]
            if c["scaling"] == "yarn":
                rounds = c["original"] * f / (2.0 * math.pi)
                w = min(1.0, max(0.0, (rounds - 1.0) / (32.0 - 1.0)))
                f = (1.0 - w) * f / c["factor"] + w * f
            turns.append(f)
            axis.append(a)
    m = 1.0 + 0.1 * math.log(c["factor"]) if c["scaling"] == "yarn" else 1.0
    P = len(turns)
    angle = s["pos"].double()[:, axis] * torch.tensor(turns, dtype=torch.float64, device="cuda")
    w = torch.polar(torch.full_like(angle, m), -angle if c["backward"] else angle)
    outs = []
    for x in (s["q"], s["k"]):
        y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        for b in range(x.shape[0]):
            for h in range(x.shape[1]):
                r = x[b, h].double()
                y[b, h] = r
                if c["layout"] == "interleaved":
                    z = torch.view_as_complex(r[:, : 2 * P].reshape(-1, P, 2).contiguous()) * w
                    y[b, h, :, : 2 * P] = torch.view_as_real(z).reshape(-1, 2 * P)
                else:
                    z = torch.complex(r[:, :P].contiguous(), r[:, P: 2 * P].contiguous()) * w
                    y[b, h, :, :P], y[b, h, :, P: 2 * P] = z.real, z.imag
        outs.append(y)
    return tuple(outs)


def _exact_cross(c, s):
    """Softmax attention of one (batch, head) after another over its allowed keys; gradients by differentiation."""
    b, h, hk, Lq, Lk, d = (c[x] for x in ("b", "h", "hk", "Lq", "Lk", "d"))
    z = dict(dtype=torch.float64, device="cuda")
    out, dq = torch.zeros(b, h, Lq, d, **z), torch.zeros(b, h, Lq, d, **z)
    dk, dv = torch.zeros(b, hk, Lk, d, **z), torch.zeros(b, hk, Lk, d, **z)
    for i in range(b):
        if "kv_len" in s:
            keys = torch.arange(int(s["kv_len"][i]), device="cuda")
        elif "key_mask" in s:
            keys = s["key_mask"][i].nonzero().flatten()
        else:
            keys = torch.arange(Lk, device="cuda")
        if keys.numel() == 0:
            continue
        for j in range(h):
            t = j // (h // hk)
            q, k, v = s["q"][i, j].double(), s["k"][i, t][keys].double(), s["v"][i, t][keys].double()
            if not c["train"]:
                out[i, j] = torch.softmax(q @ k.T / d ** 0.5, -1) @ v
                continue
            for x in (q, k, v):
                x.requires_grad_(True)
            o = torch.softmax(q @ k.T / d ** 0.5, -1) @ v
            gq, gk, gv = torch.autograd.grad(o, (q, k, v), s["dout"][i, j].double())
            out[i, j], dq[i, j] = o.detach(), gq
            dk[i, t, keys] += gk
            dv[i, t, keys] += gv
    return (out, dq, dk, dv) if c["train"] else out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(case, s) if case["op"] == "rope" else _exact_cross(case, s)
