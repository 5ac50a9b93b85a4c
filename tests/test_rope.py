"""tq_qk_norm_rope against its formula in 64 bits, and its refusals.

Tolerance per value: half a step of the output type relative to the value, plus fp32
arithmetic: 32 half steps (2^-24) of |a| + |b| of the pair, which covers the sum of squares
(at most 13 sequential roundings, halved by the root), the root, the division and the two
products of the norm (5), the reduced angle's rounding (pi half steps), sin and cos (2 each)
and the rotation's own three.
"""
import ctypes

import numpy as np
import pytest
import torch

from kv_cache_vector_07_b200 import tqkv

DEV = "cuda"


def reference(desc, x, weight, positions, inv_freq):
    """(value, |a| + |b| of the value's pair) in 64 bits, on the CPU."""
    x = x.detach().cpu().double()
    if weight is not None:
        mean = x.square().mean(-1, keepdim=True)
        x = x / torch.sqrt(mean + np.float64(np.float32(desc.eps))) * weight.cpu().double()
    rot, half = desc.rot_dim, desc.rot_dim // 2
    pos = positions.cpu().double().reshape(-1, x.shape[0])
    axis = [desc.pair_axis[p] for p in range(half)]
    out, size = x.clone(), x.abs()
    if rot:
        ang = torch.stack([pos[a] * f for a, f in zip(axis, inv_freq.cpu().double())], 1)[:, None]
        c, s = torch.cos(ang) * desc.scale, torch.sin(ang) * desc.scale
        i0 = torch.arange(half) if desc.style == tqkv.TQ_ROPE_HALF else 2 * torch.arange(half)
        i1 = i0 + half if desc.style == tqkv.TQ_ROPE_HALF else i0 + 1
        a, b = x[..., i0], x[..., i1]
        out[..., i0], out[..., i1] = a * c - b * s, b * c + a * s
        size[..., i0] = size[..., i1] = (a.abs() + b.abs()) * abs(desc.scale)
    return out, size


def check(desc, got, x, weight, positions, inv_freq):
    ref, size = reference(desc, x, weight, positions, inv_freq)
    tol = torch.finfo(got.dtype).eps / 2 * ref.abs() + 32 * 2.0 ** -24 * size + 2.0 ** -130
    err = (got.cpu().double() - ref).abs()
    assert got.dtype == x.dtype and got.shape == x.shape
    assert (err <= tol).all(), f"{int((err > tol).sum())} of {err.numel()} off, worst {float((err / tol).max()):.3g} tolerances"


def frequencies(pairs, base=10000.0):
    return (base ** (-torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))).float().to(DEV)


def inputs(n, hq, hk, d, dtype, seed, extra=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    qkv = (torch.randn((n, hq + 2 * hk, d + extra), generator=g, device=DEV) * 3).to(dtype)[..., :d]
    w = [(1 + 0.3 * torch.randn(d, generator=g, device=DEV)) for _ in range(2)]
    return qkv[:, :hq], qkv[:, hq:hq + hk], w


CASES = [
    # n, hq, hk, d, rot, style, axes, dtype, weight dtype, extra
    (1, 32, 8, 128, 128, "half", 1, "bf16", "bf16", 0),
    (1, 1, 1, 2, 2, "half", 1, "f32", "f32", 0),
    (5, 3, 1, 6, 4, "pairs", 1, "bf16", "f32", 0),
    (7, 5, 2, 80, 80, "half", 1, "bf16", "bf16", 0),
    (33, 12, 4, 64, 48, "pairs", 1, "f32", "f32", 0),
    (33, 12, 4, 64, 32, "half", 2, "bf16", "f32", 0),
    (17, 4, 4, 96, 96, "half", 3, "f32", "bf16", 0),
    (9, 8, 1, 256, 256, "half", 1, "bf16", "bf16", 0),
    (9, 8, 2, 256, 64, "pairs", 8, "bf16", None, 0),
    (130, 6, 3, 128, 128, "pairs", 1, "bf16", "bf16", 0),
    (65, 6, 3, 128, 96, "half", 3, "bf16", "bf16", 0),
    (65, 6, 3, 128, 128, "half", 1, "bf16", "bf16", 1),      # odd strides: rows not aligned to 16 bytes
    (65, 6, 3, 128, 128, "half", 1, "f32", "f32", 2),
    (40, 2, 2, 8, 8, "half", 1, "bf16", "bf16", 0),
    (40, 2, 2, 16, 16, "pairs", 1, "bf16", "bf16", 0),
    (40, 2, 2, 128, 0, "half", 1, "bf16", "bf16", 0),        # norm alone
    (1023, 16, 4, 128, 128, "half", 1, "bf16", None, 0),     # rotation alone
    (2500, 32, 8, 64, 64, "half", 3, "bf16", "bf16", 0),
]
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
STYLES = {"half": tqkv.TQ_ROPE_HALF, "pairs": tqkv.TQ_ROPE_PAIRS}


@pytest.mark.gpu
@pytest.mark.parametrize("n,hq,hk,d,rot,style,axes,dtype,wdtype,extra", CASES)
def test_values(n, hq, hk, d, rot, style, axes, dtype, wdtype, extra):
    q, k, w = inputs(n, hq, hk, d, TYPES[dtype], n + d, extra)
    w = [x.to(TYPES[wdtype]) for x in w] if wdtype else [None, None]
    g = torch.Generator(device=DEV).manual_seed(d)
    pos = torch.randint(-1000, 300000, (axes, n), generator=g, device=DEV, dtype=torch.int32)
    pos[:, 0], pos[:, -1] = 2 ** 31 - 1, 0
    inv = frequencies(rot // 2)
    axis = [(p * 5 + p // 3) % axes for p in range(rot // 2)]
    rd = tqkv.rope_desc(d, rot, STYLES[style], pair_axis=axis, n_axes=axes, eps=1e-5, scale=1.25)
    qo, ko = tqkv.qk_norm_rope(rd, q, k, pos, inv, *w)
    assert qo.is_contiguous() and ko.is_contiguous()
    check(rd, qo, q, w[0], pos, inv)
    check(rd, ko, k, w[1], pos, inv)


@pytest.mark.gpu
@pytest.mark.parametrize("style", ["half", "pairs"])
@pytest.mark.parametrize("d,extra", [(128, 0), (96, 0), (64, 1)])
def test_in_place_one_side_and_strided_results(style, d, extra):
    n, hq, hk = 70, 5, 2
    q, k, w = inputs(n, hq, hk, d, torch.bfloat16, 3, extra)
    pos = torch.arange(n, device=DEV, dtype=torch.int32) + 100000
    inv = frequencies(d // 2)
    rd = tqkv.rope_desc(d, style=STYLES[style])
    q0, k0 = q.clone(), k.clone()
    whole = torch.full((hq + 1, n, d + 8), 7.0, device=DEV, dtype=torch.bfloat16)
    qo = whole[:hq, :, :d].transpose(0, 1)                   # heads outermost, rows wider than d
    got, none = tqkv.qk_norm_rope(rd, q, None, pos, inv, q_weight=w[0], q_out=qo)
    assert got is qo and none is None
    check(rd, qo, q0, w[0], pos, inv)
    assert (whole[hq] == 7).all() and (whole[:, :, d:] == 7).all()
    assert torch.equal(q, q0)
    tqkv.qk_norm_rope(rd, q, k, pos, inv, q_weight=w[0], k_weight=w[1], q_out=q, k_out=k)
    check(rd, q, q0, w[0], pos, inv)
    check(rd, k, k0, w[1], pos, inv)
    none, ko = tqkv.qk_norm_rope(rd, None, k0, pos, inv)
    check(rd, ko, k0, None, pos, inv)


@pytest.mark.gpu
def test_empty_zero_and_non_finite_vectors():
    d = 128
    q, k, w = inputs(4, 4, 2, d, torch.bfloat16, 1)
    q, k = q.clone(), k.clone()
    rd = tqkv.rope_desc(d, 64, eps=1e-6)
    inv = frequencies(32)
    pos = torch.arange(4, device=DEV, dtype=torch.int32)
    for x, y in ((q[:0], k[:0]),):
        qo, ko = tqkv.qk_norm_rope(rd, x, y, pos[:0], inv, w[0], w[1])
        assert qo.shape[0] == ko.shape[0] == 0
    q[1, 2] = 0                                              # the zero vector stays zero
    q[2, 1, 100] = float("inf")                              # outside the rotation, no norm: only itself
    q[2, 3, 5] = float("nan")
    qo, _ = tqkv.qk_norm_rope(rd, q, None, pos, inv)
    bad = torch.zeros_like(q, dtype=torch.bool)
    bad[2, 1, 100] = bad[2, 3, 5] = bad[2, 3, 37] = True
    assert torch.equal(~torch.isfinite(qo), bad) and qo[2, 1, 100] == float("inf")
    qn, _ = tqkv.qk_norm_rope(rd, q, None, pos, inv, q_weight=w[0])
    assert (qn[1, 2] == 0).all()
    bad = torch.zeros((4, 4), dtype=torch.bool, device=DEV)
    bad[2, 1] = bad[2, 3] = True                             # the norm takes the head, and no other
    assert torch.equal((~torch.isfinite(qn)).any(-1), bad)


@pytest.mark.gpu
@pytest.mark.parametrize("style", ["half", "pairs"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot", [(8, 8), (16, 8), (32, 32), (64, 32), (64, 48), (128, 128), (256, 192), (256, 0)])
def test_few_heads(d, rot, dtype, style):
    """As many heads as a warp takes at once, one less, one more; either side alone, a norm on one side only."""
    most = 2 * 256 // d
    n = 37
    pos = torch.arange(n, device=DEV, dtype=torch.int32) * 1001 - 500
    inv = frequencies(rot // 2)
    rd = tqkv.rope_desc(d, rot, tqkv.TQ_ROPE_HALF if style == "half" else tqkv.TQ_ROPE_PAIRS)
    for heads, wt in ((most - 1, dtype), (most, torch.float32), (most + 1, torch.bfloat16)):
        hk = max(1, heads // 3)
        hq = max(1, heads - hk)
        q, k, w = inputs(n, hq, hk, d, dtype, heads)
        w = [x.to(wt) for x in w]
        for qw, kw in ((w[0], w[1]), (None, w[1]), (w[0], None)):
            gq, gk = tqkv.qk_norm_rope(rd, q, k, pos, inv, qw, kw)
            check(rd, gq, q, qw, pos, inv)
            check(rd, gk, k, kw, pos, inv)
        check(rd, tqkv.qk_norm_rope(rd, q, None, pos, inv, w[0])[0], q, w[0], pos, inv)
        check(rd, tqkv.qk_norm_rope(rd, None, k, pos, inv, None, w[1])[1], k, w[1], pos, inv)


@pytest.mark.gpu
def test_results_it_makes_belong_to_its_stream():
    """Room that the current stream still writes to is not given to a call on another one."""
    n, d = 4096, 128
    q, k, w = inputs(n, 8, 2, d, torch.bfloat16, 9)
    pos = torch.arange(n, device=DEV, dtype=torch.int32)
    inv, rd = frequencies(64), tqkv.rope_desc(d)
    ref = [t.clone() for t in tqkv.qk_norm_rope(rd, q, k, pos, inv, w[0], w[1])]
    side = torch.cuda.Stream()
    busy, room = torch.zeros(1 << 28, dtype=torch.uint8, device=DEV), torch.empty_like(ref[0])
    torch.cuda.synchronize()
    for _ in range(40):
        busy += 1
    room.fill_(3.0)
    del room                                                 # its writer waits behind the others
    got = tqkv.qk_norm_rope(rd, q, k, pos, inv, w[0], w[1], stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.gpu
def test_stream_and_graph_replay():
    n, d = 50, 128
    q, k, w = inputs(n, 8, 2, d, torch.bfloat16, 9)
    pos = torch.arange(n, device=DEV, dtype=torch.int32)
    inv, rd = frequencies(64), tqkv.rope_desc(d)
    ref = [t.clone() for t in tqkv.qk_norm_rope(rd, q, k, pos, inv, w[0], w[1])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [torch.empty_like(t) for t in ref]
    tqkv.qk_norm_rope(rd, q, k, pos, inv, w[0], w[1], got[0], got[1], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tqkv.qk_norm_rope(rd, q, k, pos, inv, w[0], w[1], got[0], got[1])
    pos += 1000                                              # the graph reads the positions when it is replayed
    g.replay()
    torch.cuda.synchronize()
    check(rd, got[0], q, w[0], pos, inv)
    check(rd, got[1], k, w[1], pos, inv)


def _c_call(rd, q=True, k=False, dtype=0, wd=0, n=1, pos=256, inv=256, axis_stride=1, **heads):
    h = dict(x=256, tok_stride=128, head_stride=128, weight=None, out=512, out_tok_stride=128, out_head_stride=128, n_heads=1)
    h.update(heads)
    h = tqkv._Heads(*[h[f] for f, _ in tqkv._Heads._fields_])
    ref = ctypes.byref
    return tqkv._lib.tq_qk_norm_rope(ref(rd) if rd is not None else None, dtype, wd, n, ref(h) if q else None,
                                     ref(h) if k else None, pos, axis_stride, inv, None)


@pytest.mark.parametrize("kind,kw,code", [
    ("null desc", dict(rd=None), tqkv.TQ_EINVAL),
    ("neither", dict(q=False), tqkv.TQ_EINVAL),
    ("odd d", dict(d=7), tqkv.TQ_EUNSUPPORTED),
    ("large d", dict(d=258), tqkv.TQ_EUNSUPPORTED),
    ("odd rotation", dict(rot_dim=3), tqkv.TQ_EINVAL),
    ("rotation beyond d", dict(rot_dim=130), tqkv.TQ_EINVAL),
    ("style", dict(style=2), tqkv.TQ_EINVAL),
    ("no axes", dict(n_axes=0), tqkv.TQ_EINVAL),
    ("axes", dict(n_axes=9), tqkv.TQ_EINVAL),
    ("eps", dict(eps=-1.0), tqkv.TQ_EINVAL),
    ("eps nan", dict(eps=float("nan")), tqkv.TQ_EINVAL),
    ("axis range", dict(axis=1), tqkv.TQ_EINVAL),
    ("dtype", dict(dtype=2), tqkv.TQ_EINVAL),
    ("weight dtype", dict(wd=7), tqkv.TQ_EINVAL),
    ("tokens", dict(n=-1), tqkv.TQ_EINVAL),
    ("null x", dict(x=None), tqkv.TQ_EINVAL),
    ("null out", dict(out=None), tqkv.TQ_EINVAL),
    ("alignment", dict(x=257), tqkv.TQ_EINVAL),
    ("f32 alignment", dict(dtype=1, x=258), tqkv.TQ_EINVAL),
    ("weight alignment", dict(weight=255), tqkv.TQ_EINVAL),
    ("heads", dict(n_heads=0), tqkv.TQ_EINVAL),
    ("positions", dict(pos=None), tqkv.TQ_EINVAL),
    ("frequencies", dict(inv=None), tqkv.TQ_EINVAL),
    ("axis stride", dict(n_axes=2, n=5, axis_stride=4), tqkv.TQ_EINVAL),
])
def test_c_refusals(kind, kw, code):
    kw = dict(kw)
    rd = tqkv.rope_desc(128)
    if "axis" in kw:
        rd.pair_axis[5] = kw.pop("axis")
    for f in ("d", "rot_dim", "style", "n_axes", "eps"):
        if f in kw:
            setattr(rd, f, kw.pop(f))
    assert _c_call(kw.pop("rd", rd), **kw) == code, kind


def test_c_no_tokens_is_ok():
    assert _c_call(tqkv.rope_desc(128), n=0, x=None, out=None, pos=None, inv=None) == tqkv.TQ_OK


def test_binding_refusals():
    for bad in (dict(pair_axis=[0] * 5), dict(pair_axis=[1] * 64), dict(pair_axis=[-1] * 64)):
        with pytest.raises(ValueError):
            tqkv.rope_desc(128, **bad)
    rd = tqkv.rope_desc(128)
    x = torch.zeros((2, 3, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):                          # not on a GPU
        tqkv.qk_norm_rope(rd, x, None, torch.zeros(2, dtype=torch.int32), torch.zeros(64))
    with pytest.raises(ValueError):
        tqkv.qk_norm_rope(rd, None, None, torch.zeros(2, dtype=torch.int32), torch.zeros(64))


@pytest.mark.gpu
def test_binding_refusals_on_shapes_and_types():
    rd = tqkv.rope_desc(128, n_axes=2, pair_axis=[p % 2 for p in range(64)])
    q = torch.zeros((4, 3, 128), dtype=torch.bfloat16, device=DEV)
    pos, inv = torch.zeros((2, 4), dtype=torch.int32, device=DEV), frequencies(64)
    tqkv.qk_norm_rope(rd, q, None, pos, inv)
    w = torch.ones(128, device=DEV)
    for kw in (dict(positions=pos[0]), dict(positions=pos.long()), dict(positions=pos[:, :3]),
               dict(positions=pos.t().contiguous().t()), dict(inv_freq=inv[:10]), dict(inv_freq=inv.double()),
               dict(q_weight=w[:64]), dict(q_weight=w.half()), dict(q=q.half()), dict(q=q[0]), dict(q=q[..., :64]),
               dict(q=q.transpose(1, 2)), dict(k=q.float()), dict(k=q[:2]), dict(q_out=q[:, :1]), dict(q_out=q.float()),
               dict(q=q.cpu())):
        args = dict(q=q, k=None, positions=pos, inv_freq=inv)
        args.update(kw)
        with pytest.raises(ValueError):
            tqkv.qk_norm_rope(rd, **args)
