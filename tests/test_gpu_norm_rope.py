"""qk_norm_rope and its backward against their formulas in float64.

The reference is written here from the definition: n = x / sqrt(mean x^2 +
eps), y = R(pos) (w n).  Tolerances: an output is rounded to bf16 once, at
most half a step, 2^-8 of its value; the fp32 arithmetic before that (a sum
of d squares, a reciprocal root of 2 ulp, the sine and cosine of an angle
that is rounded to 2^-24 of half a turn, hence off by at most pi 2^-24, three
products and a difference) stays below 2^-20 of the magnitudes that meet in
the element.
"""
from __future__ import annotations

import math

import pytest
import torch

gpu = pytest.mark.gpu


def angles(pos, rot, theta, inv_freq=None):
    f = inv_freq if inv_freq is not None else [theta ** (-2.0 * j / rot) for j in range(rot // 2)]
    return pos.double()[:, None] * torch.tensor(f, dtype=torch.float64)


def rotate(x, ang, rot, inter, sign=1.0):
    """R(pos) x (sign 1) or its transpose (-1): x [T, H, d], ang [T, rot / 2]."""
    y = x.clone()
    c, s = ang.cos()[:, None], sign * ang.sin()[:, None]
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y[..., : rot // 2], y[..., rot // 2: rot] = a * c - b * s, b * c + a * s
    return y


def reach(x, rot, inter):
    """Per element, the magnitudes that meet in it: |x| and its partner's."""
    a = x.abs()
    y = a.clone()
    if inter:
        y[..., 0:rot:2] += a[..., 1:rot:2]
        y[..., 1:rot:2] += a[..., 0:rot:2]
    else:
        y[..., : rot // 2] += a[..., rot // 2: rot]
        y[..., rot // 2: rot] += a[..., : rot // 2]
    return y


def forward(x, w, ang, rot, eps, inter):
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    return rotate(x * r * w, ang, rot, inter)


def backward(x, w, dy, ang, rot, eps, inter):
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    g = rotate(dy, ang, rot, inter, -1.0)
    n = x * r
    dx = r * (w * g - n * (w * g * n).mean(-1, keepdim=True))
    return dx, (g * n).sum((0, 1)), g, n, r


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 32])
def test_formula_against_differences(rot, inter):
    """The backward formula itself, against central differences of the forward in float64."""
    g = torch.Generator().manual_seed(5 + rot)
    x = torch.randn(3, 2, 32, generator=g, dtype=torch.float64)
    w = 1 + 0.3 * torch.randn(32, generator=g, dtype=torch.float64)
    dy = torch.randn(3, 2, 32, generator=g, dtype=torch.float64)
    ang = angles(torch.tensor([0, 7, 1000]), max(rot, 2), 1e4)[:, : rot // 2]
    f = lambda x, w: (forward(x, w, ang, rot, 1e-6, inter) * dy).sum()  # noqa: E731
    dx, dw, *_ = backward(x, w, dy, ang, rot, 1e-6, inter)
    h = 1e-5
    for _ in range(8):
        v, u = torch.randn(x.shape, generator=g, dtype=torch.float64), torch.randn(32, generator=g, dtype=torch.float64)
        assert math.isclose(float((f(x + h * v, w) - f(x - h * v, w)) / (2 * h)), float((dx * v).sum()),
                            rel_tol=1e-6, abs_tol=1e-7)
        assert math.isclose(float((f(x, w + h * u) - f(x, w - h * u)) / (2 * h)), float((dw * u).sum()),
                            rel_tol=1e-6, abs_tol=1e-7)


@pytest.fixture(scope="module")
def msa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_gqa_idx_b200 as msa

    return msa


def make(T, Hq, Hk, d, seed, far=131072):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(q=(2 * r(T, Hq, d)).bfloat16(), k=(0.5 * r(T, Hk, d)).bfloat16(),
                w_q=(1 + 0.3 * r(d)).bfloat16(), w_k=(1 + 0.3 * r(d)).bfloat16(),
                pos=torch.randint(0, far, (T,), generator=g, dtype=torch.int32),
                dq=r(T, Hq, d).bfloat16(), dk=r(T, Hk, d).bfloat16())


def check(y, ref, mags, what):
    err = (y.double().cpu() - ref).abs()
    tol = ref.abs() * 2.0**-8 + mags * 2.0**-20
    worst = float((err / tol.clamp(min=1e-300)).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst} of the tolerance"


SHAPES = [  # T, Hq, Hk, d, rot, inter
    (1, 1, 1, 128, 128, False), (3, 32, 4, 128, 64, False), (61, 8, 2, 64, 64, True),
    (130, 5, 1, 128, 32, True), (77, 7, 3, 32, 16, False), (5, 4, 1, 64, 0, False),
    (1300, 4, 4, 32, 32, True), (1203, 9, 2, 64, 48, False), (1190, 32, 8, 128, 128, False),
]


@gpu
@pytest.mark.parametrize("T,Hq,Hk,d,rot,inter", SHAPES)
def test_forward_and_backward(msa, T, Hq, Hk, d, rot, inter):
    c = make(T, Hq, Hk, d, 11 * T + d)
    gpu_c = {k: v.cuda() for k, v in c.items()}
    kw = dict(rot_dim=rot, theta=5e5, eps=1e-6, interleaved=inter)
    out = msa.qk_norm_rope(gpu_c["q"], gpu_c["k"], gpu_c["w_q"], gpu_c["w_k"], gpu_c["pos"], **kw)
    grads = msa.qk_norm_rope_bwd(gpu_c["q"], gpu_c["k"], gpu_c["w_q"], gpu_c["w_k"], gpu_c["pos"],
                                 gpu_c["dq"], gpu_c["dk"], **kw)
    ang = angles(c["pos"], max(rot, 2), 5e5)[:, : rot // 2]
    for y, dx, dw, x, w, dy, name in ((out[0], grads[0], grads[2], "q", "w_q", "dq", "q"),
                                      (out[1], grads[1], grads[3], "k", "w_k", "dk", "k")):
        x, w, dy = c[x].double(), c[w].double(), c[dy].double()
        ref = forward(x, w, ang, rot, 1e-6, inter)
        r = (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        check(y, ref, reach(x * r * w, rot, inter), f"y({name})")
        rdx, rdw, g, n, r = backward(x, w, dy, ang, rot, 1e-6, inter)
        meet = r * (w.abs() * reach(dy, rot, inter) +
                    n.abs() * (w.abs() * reach(dy, rot, inter) * n.abs()).mean(-1, keepdim=True))
        check(dx, rdx, meet, f"d{name}")
        # dw: `rows` terms, each off by at most 2^-20 of what meets in it, added
        # in fp32 in some fixed order: at most rows * 2^-24 of the sum of magnitudes
        rows = x.shape[0] * x.shape[1]
        mag = (reach(dy, rot, inter) * n.abs()).sum((0, 1))
        err = (dw.double().cpu() - rdw).abs()
        assert bool((err <= mag * (2.0**-20 + rows * 2.0**-24)).all()), f"dw({name})"
        # against differences of the forward in float64, along one direction
        gen = torch.Generator().manual_seed(3)
        v = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        h = 1e-4
        num = ((forward(x + h * v, w, ang, rot, 1e-6, inter) -
                forward(x - h * v, w, ang, rot, 1e-6, inter)) * dy).sum() / (2 * h)
        got = (dx.double().cpu() * v).sum()
        # the roundings of dx enter with |v|: at most 2^-8 |dx| each
        assert abs(float(num - got)) <= float((rdx.abs() * v.abs()).sum()) * 2.0**-8 + \
            float((meet * v.abs()).sum()) * 2.0**-20 + 1e-5 * abs(float(num)) + 1e-6


@gpu
def test_far_positions_and_given_frequencies(msa):
    """Angles stay exact at the largest int32 positions, and with any frequencies."""
    T, d = 64, 64
    c = make(T, 2, 1, d, 91)
    c["pos"] = (2**31 - 1 - 37 * torch.arange(T, dtype=torch.int64)).to(torch.int32)
    freqs = [1.0 / (1 + 3 * j) for j in range(31)] + [7.25]
    g = {k: v.cuda() for k, v in c.items()}
    yq, yk = msa.qk_norm_rope(g["q"], g["k"], None, None, g["pos"], inv_freq=freqs, eps=0.0)
    # the reference reduces pos * f modulo 2 pi in float64: off by 2^31 * 2^-52
    ang = angles(c["pos"], d, 0, freqs)
    for y, x in ((yq, c["q"].double()), (yk, c["k"].double())):
        ones = torch.ones(d, dtype=torch.float64)
        ref = forward(x, ones, ang, d, 0.0, False)
        r = x.square().mean(-1, keepdim=True).rsqrt()
        check(y, ref, reach(x * r, d, False) * 8, "far")


@gpu
@pytest.mark.parametrize("T", [6, 1500])
def test_padding_rows_and_in_place(msa, T):
    c = make(T, 8, 2, 128, 17)
    c["pos"][1::3] = -1
    g = {k: v.cuda() for k, v in c.items()}
    ref = msa.qk_norm_rope(g["q"], g["k"], g["w_q"], g["w_k"], g["pos"].clamp(min=0))
    mark = [torch.full_like(g["q"], 7.0), torch.full_like(g["k"], 7.0)]
    msa.qk_norm_rope(g["q"], g["k"], g["w_q"], g["w_k"], g["pos"], q_out=mark[0], k_out=mark[1])
    pad = g["pos"] < 0
    for y, r in zip(mark, ref):
        assert bool((y[pad] == 7.0).all()) and torch.equal(y[~pad], r[~pad])
    q, k = g["q"].clone(), g["k"].clone()
    msa.qk_norm_rope(q, k, g["w_q"], g["w_k"], g["pos"], q_out=q, k_out=k)
    for y, x, r in ((q, g["q"], ref[0]), (k, g["k"], ref[1])):
        assert torch.equal(y[pad], x[pad]) and torch.equal(y[~pad], r[~pad])
    # gradients: none from padding rows, NaN there or not
    g["q"][pad] = float("nan")
    dq, dk, dwq, dwk = msa.qk_norm_rope_bwd(g["q"], g["k"], g["w_q"], g["w_k"], g["pos"], g["dq"], g["dk"])
    keep = ~pad
    ref = msa.qk_norm_rope_bwd(g["q"][keep], g["k"][keep], g["w_q"], g["w_k"], g["pos"][keep],
                               g["dq"][keep], g["dk"][keep])
    assert bool((dq[pad] == 0).all()) and bool((dk[pad] == 0).all())
    assert torch.equal(dq[keep], ref[0]) and torch.equal(dk[keep], ref[1])
    torch.testing.assert_close(dwq, ref[2], rtol=1e-4, atol=1e-3)
    torch.testing.assert_close(dwk, ref[3], rtol=1e-4, atol=1e-3)
    # the gradients of the weights do not change from run to run
    again = msa.qk_norm_rope_bwd(g["q"], g["k"], g["w_q"], g["w_k"], g["pos"], g["dq"], g["dk"])
    assert torch.equal(again[2], dwq) and torch.equal(again[3], dwk)


@gpu
def test_no_rows_side_stream_and_graph(msa):
    c = {k: v.cuda() for k, v in make(33, 4, 2, 64, 23).items()}
    empty = msa.qk_norm_rope(c["q"][:0], c["k"][:0], c["w_q"], c["w_k"], c["pos"][:0])
    assert empty[0].shape == (0, 4, 64)
    dq, dk, dwq, dwk = msa.qk_norm_rope_bwd(c["q"][:0], c["k"][:0], c["w_q"], c["w_k"], c["pos"][:0],
                                            c["dq"][:0], c["dk"][:0])
    assert bool((dwq == 0).all()) and bool((dwk == 0).all())
    args = (c["q"], c["k"], c["w_q"], c["w_k"], c["pos"])
    ref = msa.qk_norm_rope(*args) + msa.qk_norm_rope_bwd(*args, c["dq"], c["dk"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = msa.qk_norm_rope(*args, stream=side) + msa.qk_norm_rope_bwd(*args, c["dq"], c["dk"], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = msa.qk_norm_rope(*args) + msa.qk_norm_rope_bwd(*args, c["dq"], c["dk"])
    c["q"].mul_(-1.0)  # the norm is even in x: y and dq change sign, dw too
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], -ref[0]) and torch.equal(got[1], ref[1])
    c["q"].mul_(-1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


@gpu
def test_refusals(msa):
    c = {k: v.cuda() for k, v in make(4, 4, 2, 64, 29).items()}
    args = (c["q"], c["k"], c["w_q"], c["w_k"], c["pos"])
    with pytest.raises(msa.MSAError):
        msa.qk_norm_rope(*args, rot_dim=24)
    with pytest.raises(msa.MSAError):
        msa.qk_norm_rope(*args, eps=-1.0)
    with pytest.raises(ValueError):
        msa.qk_norm_rope(*args, inv_freq=[1.0])
    with pytest.raises(TypeError):
        msa.qk_norm_rope(c["q"].float(), *args[1:])
    with pytest.raises(ValueError):
        msa.qk_norm_rope(c["q"].transpose(0, 1).contiguous().transpose(0, 1), *args[1:])
    with pytest.raises(ValueError):
        msa.qk_norm_rope(*args[:4], c["pos"][:3])
    with pytest.raises(ValueError):
        msa.qk_norm_rope_bwd(*args, c["dq"], c["dk"], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
