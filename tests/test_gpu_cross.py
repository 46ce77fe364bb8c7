"""Cross-attention on the GPU, forward and backward, against its 64-bit form."""

import pytest
import torch

from block_ops_ref import allowed_keys, assert_within, cross_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.init()


def _x(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g).to(dtype)


def _make(seed, b, h, hk, Lq, Lk, d, dtype):
    return [_x(10 * seed + i, b, n, L, d, dtype=dtype)
            for i, (n, L) in enumerate(((h, Lq), (hk, Lk), (hk, Lk), (h, Lq)))]


def _check(lib, q, k, v, dout=None, kv_len=None, key_mask=None, what=""):
    mask = dict(kv_len=kv_len, key_mask=key_mask)
    ref = cross_ref(q, k, v, dout=dout, **mask)
    out, lse = lib.cross_attn_fwd(q, k, v, return_lse=True, **mask)
    assert_within(out, ref["out"], what + " out")
    assert_within(lse, ref["lse"], what + " lse")
    if dout is not None:
        grads = lib.cross_attn_bwd(dout, q, k, v, out, lse, **mask)
        for name, g in zip(("dq", "dk", "dv"), grads):
            assert g.dtype == q.dtype
            assert_within(g, ref[name], what + " " + name)
    torch.cuda.synchronize()
    assert lib.device_status() == 0
    return out, lse


DTYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])


@DTYPES
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lq,Lk", [(1, 1), (1, 77), (2, 500), (17, 1), (63, 64), (64, 65), (128, 128), (129, 127),
                                   (256, 256), (257, 129), (300, 513), (1000, 77), (5, 4608)])
def test_lengths(lib, Lq, Lk, d, dtype):
    q, k, v, g = _make(1, 2, 3, 3, Lq, Lk, d, dtype)
    _check(lib, q, k, v, g, what=f"{Lq}x{Lk}")


@DTYPES
@pytest.mark.parametrize("b,h,hk", [(1, 4, 1), (2, 6, 2), (3, 5, 5), (1, 40, 8)])
def test_shared_key_heads(lib, b, h, hk, dtype):
    q, k, v, g = _make(2, b, h, hk, 150, 200, 64, dtype)
    _check(lib, q, k, v, g, what=f"{h}/{hk}")


@DTYPES
@pytest.mark.parametrize("Lq", [1, 3, 200])
@pytest.mark.parametrize("lens", [[0, 1, 300], [77, 300, 128], [-5, 1000, 129]])
def test_key_lengths(lib, lens, Lq, dtype):
    """Lengths of none, one and all keys; values outside [0, Lk] are clamped."""
    q, k, v, g = _make(3, 3, 2, 2, Lq, 300, 64, dtype)
    out, lse = _check(lib, q, k, v, g, kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"), what=str(lens))
    if lens[0] <= 0:
        assert (out[0] == 0).all() and (lse[0] == -float("inf")).all()


@DTYPES
@pytest.mark.parametrize("Lq", [1, 170])
@pytest.mark.parametrize("with_len", [False, True])
def test_masks_with_holes_and_garbage_behind_them(lib, Lq, with_len, dtype):
    """NaN, infinities and the type's lowest value where the mask is off."""
    b, h, hk, Lk, d = 3, 4, 2, 333, 128
    q, k, v, g = _make(4, b, h, hk, Lq, Lk, d, dtype)
    gen = torch.Generator(device="cuda").manual_seed(5)
    mask = torch.rand(b, Lk, device="cuda", generator=gen) < 0.4
    mask[0, :128] = False  # a whole leading tile
    mask[1] = False        # no key at all
    mask[2, -1] = True     # the very last key
    kv_len = torch.tensor([300, 333, 333], dtype=torch.int32, device="cuda") if with_len else None
    off = ~allowed_keys(b, Lk, kv_len, mask, "cuda")
    bad = torch.tensor([float("nan"), float("inf"), -float("inf"), torch.finfo(dtype).min], device="cuda").to(dtype)
    where = off[:, None, :, None].expand_as(k)
    fill = bad[torch.arange(k.numel(), device="cuda") % 4].view_as(k)
    k, v = torch.where(where, fill, k), torch.where(where, fill, v)
    out, lse = lib.cross_attn_fwd(q, k, v, kv_len=kv_len, key_mask=mask, return_lse=True)
    ref = cross_ref(q, k, v, kv_len, mask, g)
    assert_within(out, ref["out"], "out")
    assert_within(lse, ref["lse"], "lse")
    dq, dk, dv = lib.cross_attn_bwd(g, q, k, v, out, lse, kv_len=kv_len, key_mask=mask)
    for name, y in zip(("dq", "dk", "dv"), (dq, dk, dv)):
        assert_within(y, ref[name], name)
    assert (dq[1] == 0).all() and (dk[1] == 0).all() and (dv[1] == 0).all()
    assert (dk[where] == 0).all() and (dv[where] == 0).all()
    assert lib.device_status() == 0


@DTYPES
@pytest.mark.parametrize("Lq", [1, 300])
def test_no_keys_at_all(lib, Lq, dtype):
    q, k, v, g = _make(19, 2, 4, 2, Lq, 200, 128, dtype)
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    out, lse = lib.cross_attn_fwd(q, k, v, kv_len=lens, return_lse=True)
    assert (out == 0).all() and (lse == -float("inf")).all()
    for y in lib.cross_attn_bwd(g, q, k, v, out, lse, kv_len=lens):
        assert (y == 0).all()
    assert lib.device_status() == 0


@DTYPES
@pytest.mark.parametrize("Lq,Lk", [(1, 1), (1, 40), (40, 1)])
def test_strided_rows_of_length_one(lib, Lq, Lk, dtype):
    """Views whose single row has the stride of a longer buffer."""
    q = _x(33, 2, 5, 3, 64, dtype=dtype)[:, :Lq].permute(0, 2, 1, 3) if Lq == 1 else \
        _x(33, 2, Lq, 3, 64, dtype=dtype).permute(0, 2, 1, 3)
    kv = _x(34, 2, Lk + 3, 2, 3, 64, dtype=dtype)[:, 1:1 + Lk]
    k, v = (kv[:, :, i].permute(0, 2, 1, 3) for i in (0, 1))
    g = _x(35, 2, 3, Lq, 64, dtype=dtype)
    _check(lib, q, k, v, g, what="one row")


@DTYPES
def test_large_scores(lib, dtype):
    """Scores far apart: the running maximum moves late, most keys underflow."""
    q, k, v, g = _make(6, 1, 2, 2, 140, 400, 64, dtype)
    k = (k.float() * torch.linspace(0.1, 6.0, 400, device="cuda")[:, None]).to(dtype)
    _check(lib, q, k, v, g, what="large")


@DTYPES
@pytest.mark.parametrize("Lq", [1, 200])
def test_strides_and_rows_around(lib, Lq, dtype):
    """Views of fused projections in, views of padded buffers out; what lies
    around the outputs stays."""
    b, h, hk, Lk, d = 2, 4, 2, 90, 64
    q = _x(30, b, Lq, h, d, dtype=dtype).permute(0, 2, 1, 3)
    kv = _x(31, b, Lk, 2, hk, d, dtype=dtype)
    k, v = (kv[:, :, i].permute(0, 2, 1, 3) for i in (0, 1))
    g = _x(32, b, Lq, 2 * h, d, dtype=dtype)[:, :, h:].permute(0, 2, 1, 3)
    ref = cross_ref(q, k, v, dout=g)
    big = [torch.full((b, L + 7, n, d), 7.0, dtype=dtype, device="cuda") for L, n in
           ((Lq, h), (Lq, h), (Lk, hk), (Lk, hk))]
    out, dq, dk, dv = (x[:, 3:-4].permute(0, 2, 1, 3) for x in big)
    _, lse = lib.cross_attn_fwd(q, k, v, return_lse=True, out=out)
    lib.cross_attn_bwd(g, q, k, v, out, lse, dq=dq, dk=dk, dv=dv)
    for name, y in (("out", out), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        assert_within(y, ref[name], name)
    for x in big:
        assert (x[:, :3] == 7).all() and (x[:, -4:] == 7).all()
    fresh = lib.cross_attn_fwd(q, k, v)
    assert fresh.stride() == q.stride() and torch.equal(fresh, out)


@DTYPES
def test_gradient_by_differences(lib, dtype):
    """Directional derivatives of the 64-bit forward against the kernel's gradients."""
    q, k, v, g = _make(7, 1, 2, 1, 60, 70, 64, dtype)
    out, lse = lib.cross_attn_fwd(q, k, v, return_lse=True)
    grads = lib.cross_attn_bwd(g, q, k, v, out, lse)
    ref = cross_ref(q, k, v, dout=g)
    G = g.double()
    h = 1e-4

    def f(*x):
        s = 1 / 8.0
        return (torch.softmax(x[0] @ x[1].mT * s, -1) @ x[2] * G).sum()

    base = [x.double() for x in (q, k, v)]
    for i, name in enumerate(("dq", "dk", "dv")):
        e = _x(70 + i, *base[i].shape, dtype=torch.float32).double()
        up, down = ([x + (h * sign * e if j == i else 0) for j, x in enumerate(base)] for sign in (1, -1))
        num = (f(*up) - f(*down)) / (2 * h)
        # the kernel's allowance, and h^2 times a third derivative that the spread of the
        # values keeps below 1e4 in sum: 1e-4
        assert abs(num - (grads[i].double() * e).sum()) <= (ref[name][1] * e.abs()).sum() + 1e-4, name


@DTYPES
def test_same_bits_every_time(lib, dtype):
    q, k, v, g = _make(8, 2, 6, 2, 900, 300, 64, dtype)
    runs = []
    for _ in range(3):
        out, lse = lib.cross_attn_fwd(q, k, v, return_lse=True)
        runs.append((out, lse) + lib.cross_attn_bwd(g, q, k, v, out, lse))
    for r in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(runs[0], r))


@DTYPES
@pytest.mark.parametrize("Lq,Lk", [(1, 700), (300, 77), (140, 1000)])
def test_side_stream_two_graphs_and_workspace(lib, Lq, Lk, dtype):
    """Another stream; two captured graphs replayed in turn, each with the
    workspace of its own capture; a given workspace full of NaN patterns."""
    sets = [_make(9 + i, 1, 4, 2, Lq, Lk, 64, dtype) for i in range(2)]
    lens = torch.tensor([min(Lk, 65)], dtype=torch.int32, device="cuda")

    def both(q, k, v, g, **kw):
        out, lse = lib.cross_attn_fwd(q, k, v, return_lse=True, kv_len=lens, **kw)
        return (out, lse) + lib.cross_attn_bwd(g, q, k, v, out, lse, kv_len=lens, **kw)

    want = [both(*s) for s in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(*sets[0], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(want[0], got))
    need = max(lib.cross_workspace_size(dtype, 1, 4, 2, Lq, Lk, 64, True, back) for back in (False, True))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    got = both(*sets[1], workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(want[1], got))
    graphs, outs = [], []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(both(*s))
        graphs.append(graph)
    for _ in range(2):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(x, y) for x, y in zip(w, o))


@pytest.mark.parametrize("Lk", [4095, 4097, 9000])
@pytest.mark.parametrize("Lq", [1, 40])
def test_long_masks(lib, Lq, Lk):
    """Masks longer than one round of the packing, rows that start off a
    16-byte boundary, and lengths on top."""
    q, k, v, g = _make(12, 2, 2, 1, Lq, Lk, 64, torch.bfloat16)
    gen = torch.Generator(device="cuda").manual_seed(13)
    mask = torch.rand(2, Lk, device="cuda", generator=gen) < 0.3
    mask[:, 1000:3000] = False
    mask[0, -1] = True
    _check(lib, q, k, v, g, key_mask=mask, what="mask")
    _check(lib, q, k, v, g, key_mask=mask, kv_len=torch.tensor([Lk - 7, 17], dtype=torch.int32, device="cuda"),
           what="mask and lengths")


def test_offsets_past_32_bits(lib):
    """17.5 million rows of 128: byte and element offsets past 2^32 and 2^31 in
    queries, outputs and gradients; all but the last rows are zero."""
    L = 17_500_000
    q = torch.zeros(1, 1, L, 128, dtype=torch.bfloat16, device="cuda")
    q[:, :, -3:] = _x(14, 1, 1, 3, 128)
    k, v = _x(15, 1, 1, 70, 128), _x(16, 1, 1, 70, 128)
    g = torch.zeros_like(q)
    g[:, :, -3:] = _x(17, 1, 1, 3, 128)
    ref = cross_ref(q[:, :, -3:], k, v, dout=g[:, :, -3:])
    out, lse = lib.cross_attn_fwd(q, k, v, return_lse=True)
    assert_within(out[:, :, -3:], ref["out"], "out")
    dq, dk, dv = lib.cross_attn_bwd(g, q, k, v, out, lse)
    assert_within(dq[:, :, -3:], ref["dq"], "dq")
    # the other rows add p 0 = 0 to dv and ds q = 0 to dk; only their number enters the sums
    assert_within(dk, ref["dk"], "dk")
    assert_within(dv, ref["dv"], "dv")
    pos = torch.arange(L, dtype=torch.float32, device="cuda")[:, None].contiguous()
    far, _ = lib.rope(q, None, pos, (128,))
    near, _ = lib.rope(q[:, :, -3:], None, pos[-3:].contiguous(), (128,))
    assert torch.equal(far[:, :, -3:], near)
    # as keys: the last row alone is allowed
    mask = torch.zeros(1, L, dtype=torch.bool, device="cuda")
    mask[0, -1] = True
    one = lib.cross_attn_fwd(_x(18, 1, 1, 1, 128), q, q, key_mask=mask)
    assert torch.equal(one, q[:, :, -1:])  # p = 1 exactly: the value itself


def test_block_of_a_transformer(lib):
    """As a block calls them: rotary positions out of the fused projection, the
    piecewise sparse self-attention, cross-attention to padded text states, and
    the gradients of the cross-attention and of the positions."""
    b, L, h, d, Lk = 1, 1000, 2, 128, 96
    qkv = _x(50, b, L, 3, h, d)
    q, k, v = (qkv[:, :, i].permute(0, 2, 1, 3) for i in range(3))
    pos = torch.stack([torch.arange(L, device="cuda") // 250, torch.arange(L, device="cuda") // 25 % 10,
                       torch.arange(L, device="cuda") % 25], 1).float().contiguous()
    dims = (44, 42, 42)
    q1, k1 = lib.rope(q, k, pos, dims)
    x = lib.attn_fwd(q1, k1, v.contiguous(), 128, 1.0)  # every block kept: dense attention of the turned q and k
    ref = cross_ref(q1, k1, v)["out"][0]
    # the fused kernel's documented bf16 tolerance
    assert (x.double() - ref).norm() <= 5e-3 * ref.norm()
    text = _x(51, b, Lk, 2, h, d)
    tk, tv = (text[:, :, i].permute(0, 2, 1, 3) for i in range(2))
    kv_len = torch.tensor([40], dtype=torch.int32, device="cuda")
    g = _x(52, b, h, L, d)
    _check(lib, x, tk, tv, g, kv_len=kv_len, what="block")
    out, lse = lib.cross_attn_fwd(x, tk, tv, kv_len=kv_len, return_lse=True)
    dx, _, _ = lib.cross_attn_bwd(g, x, tk, tv, out, lse, kv_len=kv_len)
    assert torch.isfinite(dx.float()).all()
    back, _ = lib.rope_bwd(q1, None, pos, dims)
    # forward and back, each rounded to bf16: 2^-8 of the pair's length twice, at most 1.5x in a component
    assert (back - q).float().abs().max() <= 3 * 2.0 ** -8 * q.float().abs().max()
