"""attn_rope and attn_rope_bwd against their formulas in 64 bits, and against attention as they are used.

Tolerances.  A result is computed in fp32 and rounded once: half a step of its type (finfo.eps / 2 relative, half the smallest
subnormal near zero), plus the fp32 operations before it.  Those are at most 64 roundings deep (a row's sum of squares: 16 sequential
and 5 exchanged additions, whose error the square root halves; reciprocal root, sine and cosine within 2 steps each; 6 products and
sums): 64 x 2^-24 times the sum of the terms' magnitudes.  A weight gradient adds, at these sizes, at most 48 rows a thread, then
5 + 8 + 32 + 5 partial sums: below 128 x 2^-24 times the sum of magnitudes."""
import math

import pytest
import torch

import scaled_dot_product_sdpa_gb300 as gb
from reference64 import check, draw, pairs, turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from scaled_dot_product_sdpa_gb300 import build
    gb.load_library(build.build())
    assert gb.attn_last_device_error() == 0
    yield
    assert gb.attn_last_device_error() == 0


CASES = [  # B, Hq, Hkv, L, d, rotary
    (1, 1, 1, 1, 64, 64), (2, 5, 1, 3, 64, 32), (1, 4, 2, 7, 128, 128), (3, 32, 8, 17, 128, 48), (2, 3, 3, 33, 256, 256), (1, 2, 1, 9, 256, 16),
    (1, 3, 1, 5, 512, 512), (2, 1, 1, 700, 512, 128), (5, 7, 0, 131, 128, 64), (1, 2, 2, 4999, 64, 64), (1, 70, 9, 40, 64, 0)]


@pytest.mark.parametrize("B,Hq,Hkv,L,d,rotary", CASES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_forward(B, Hq, Hkv, L, d, rotary, dtype, interleaved, norm):
    q, k = draw((B, L, Hq, d), dtype, 1).transpose(1, 2), draw((B, Hkv, L, d), dtype, 2)
    wq, wk = draw((d,), dtype, 3), draw((d,), dtype, 4)
    inv_freq = torch.pow(torch.tensor(500.0, dtype=torch.float64), -torch.arange(rotary // 2, dtype=torch.float64) / max(1, rotary // 2))
    pos = torch.randint(-5, 100000, (B, L), generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    factor = 1.25
    got = gb.attn_rope(q.cuda(), k.cuda() if Hkv else None, inv_freq.cuda() if rotary else None, positions=pos.cuda(), interleaved=interleaved,
                       factor=factor, q_weight=wq.cuda() if norm else None, k_weight=wk.cuda() if norm and Hkv else None, eps=1e-5)
    for x, w, out in ((q, wq, got[0]), (k, wk, got[1])):
        if out is None:
            assert Hkv == 0
            continue
        y = x.double()
        if norm:
            y = y / (y.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w.double()
        want, size = turned(y, pos, inv_freq, factor, interleaved)
        assert out.is_contiguous() and out.dtype == dtype
        check(out, want, size, "forward")


def test_positions_default_shared_and_far():
    """Without positions a row's own index; [L] positions serve every sequence; at 2^31 - 1 the angle is still exact."""
    q = draw((2, 3, 6, 64), torch.float16, 7)
    inv_freq, factor = gb.attn_rope_frequencies(64, scaling="parts", scale=8.0, trained_length=4096)
    assert inv_freq.is_cuda
    f = inv_freq.cpu()
    for pos, told in ((torch.arange(6), None), (torch.arange(6) * 11, (torch.arange(6, dtype=torch.int32) * 11).cuda()),
                      (torch.full((6,), 2 ** 31 - 1), torch.full((6,), 2 ** 31 - 1, dtype=torch.int32).cuda())):
        out, none = gb.attn_rope(q.cuda(), None, inv_freq, positions=told, factor=factor)
        assert none is None
        want, size = turned(q.double(), pos[None].expand(2, 6), f, factor, False)
        # a double angle of 2^31 radians is itself off by 2^31 2^-53
        check(out, want, size, "positions", depth=64 + 8)


@pytest.mark.parametrize("B,Hq,Hkv,L,d,rotary", [c for c in CASES if c[3] < 1000] + [(1, 2, 2, 4000, 64, 64)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_backward_matches_the_formula(B, Hq, Hkv, L, d, rotary, dtype, interleaved, norm):
    q, k = draw((B, L, Hq, d), dtype, 11).transpose(1, 2), draw((B, Hkv, L, d), dtype, 12)
    dq, dk = draw((B, Hq, L, d), dtype, 13), draw((B, L, Hkv, d), dtype, 14).transpose(1, 2)
    wq, wk = draw((d,), dtype, 15), draw((d,), dtype, 16)
    inv_freq = torch.pow(torch.tensor(500.0, dtype=torch.float64), -torch.arange(rotary // 2, dtype=torch.float64) / max(1, rotary // 2))
    pos = torch.randint(0, 100000, (B, L), generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    factor, eps = 1.25, 1e-5
    more = dict(q=q.cuda(), k=k.cuda() if Hkv else None, q_weight=wq.cuda(), k_weight=wk.cuda() if Hkv else None, eps=eps) if norm else {}
    call = lambda: gb.attn_rope_bwd(dq.cuda(), dk.cuda() if Hkv else None, inv_freq.cuda() if rotary else None, positions=pos.cuda(),  # noqa: E731
                                    interleaved=interleaved, factor=factor, **more)
    got, again = call(), call()
    assert len(got) == (4 if norm else 2)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, again)), "not the same bits twice"
    for n, (x, up, w) in enumerate(((q, dq, wq), (k, dk, wk))):
        if n and not Hkv:
            assert got[1] is None
            continue
        dy, size = turned(up.double(), pos, inv_freq, factor, interleaved, sign=-1.0)
        if not norm:
            check(got[n], dy, size, "backward")
            continue
        y = x.double()
        rstd = 1.0 / (y.square().mean(-1, keepdim=True) + eps).sqrt()
        xh, g, gsize = y * rstd, dy * w.double(), size * w.double().abs()
        want = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
        check(got[n], want, rstd * (gsize + xh.abs() * (gsize * xh.abs()).mean(-1, keepdim=True)), "dx")
        check(got[2 + n], (dy * xh).sum((0, 1, 2)), (size * xh.abs()).sum((0, 1, 2)), "dw", depth=128 + 64)


@pytest.mark.parametrize("Hq,Hkv,L,d", [(5, 3, 3, 64), (1, 1, 1, 128), (7, 2, 19, 256), (3, 1, 5, 512)])
def test_backward_without_eps(Hq, Hkv, L, d):
    """Threads without a row of their own add nothing to the weights' gradients, although 1 / sqrt(0 + eps) is infinite for them."""
    q, k, dq, dk = (draw((2, h, L, d), torch.float16, 30 + n) for n, h in enumerate((Hq, Hkv, Hq, Hkv)))
    wq, wk = draw((d,), torch.float16, 35), draw((d,), torch.float16, 36)
    got = gb.attn_rope_bwd(dq.cuda(), dk.cuda(), None, q=q.cuda(), k=k.cuda(), q_weight=wq.cuda(), k_weight=wk.cuda(), eps=0.0)
    for n, (x, up, w) in enumerate(((q, dq, wq), (k, dk, wk))):
        x, g = x.double(), up.double() * w.double()
        rstd = x.square().mean(-1, keepdim=True).rsqrt()
        xh = x * rstd
        want = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
        check(got[n], want, rstd * (g.abs() + xh.abs() * (g * xh).abs().mean(-1, keepdim=True)), "dx")
        check(got[2 + n], (up.double() * xh).sum((0, 1, 2)), (up.double() * xh).abs().sum((0, 1, 2)), "dw", depth=128 + 64)


@pytest.mark.parametrize("interleaved", [False, True])
def test_backward_matches_differences(interleaved):
    """<gradient, direction> against central differences of <forward, upstream gradient> in 64 bits, at the values that the kernel
    gets.  The kernel's results are off by their rounding, at most 2^-11 of each term; fp32 before it and the differences' own h^2 stay
    below 2^-16."""
    B, H, L, d, rotary = 1, 2, 5, 64, 32
    x, up, w = (draw(s, torch.float16, n) for n, s in ((21, (B, H, L, d)), (22, (B, H, L, d)), (23, (d,))))
    inv_freq, _ = gb.attn_rope_frequencies(rotary, device="cpu")
    pos = torch.arange(L)[None]

    def value(y, weight):
        y = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight
        return (turned(y, pos, inv_freq, 1.0, interleaved)[0] * up.double()).sum()

    dx, _, dw, _ = gb.attn_rope_bwd(up.cuda(), None, inv_freq.cuda(), interleaved=interleaved, q=x.cuda(), q_weight=w.cuda())
    g, h = torch.Generator().manual_seed(24), 1e-4
    for _ in range(3):
        ex, ew = torch.randn(x.shape, generator=g, dtype=torch.float64), torch.randn(d, generator=g, dtype=torch.float64)
        diff = (value(x.double() + h * ex, w.double() + h * ew) - value(x.double() - h * ex, w.double() - h * ew)) / (2 * h)
        terms = torch.cat([(dx.cpu().double() * ex).flatten(), (dw.cpu().double() * ew).flatten()])
        assert abs(terms.sum() - diff) <= (2.0 ** -11 + 2.0 ** -16) * terms.abs().sum()


def test_rows_with_special_values():
    """A row of zeros stays zero under a norm, and its gradient is finite; NaN and infinity stay in their own rows."""
    q = draw((1, 2, 4, 128), torch.bfloat16, 31)
    q[0, 0, 1] = 0
    q[0, 1, 2, 5] = math.nan
    q[0, 0, 3, 9] = math.inf
    w = draw((128,), torch.bfloat16, 32)
    inv_freq, _ = gb.attn_rope_frequencies(128)
    out, _ = gb.attn_rope(q.cuda(), None, inv_freq, q_weight=w.cuda())
    out = out.cpu()
    assert (out[0, 0, 1] == 0).all()
    bad = torch.zeros(1, 2, 4, dtype=torch.bool)
    bad[0, 1, 2] = bad[0, 0, 3] = True
    assert torch.equal(torch.isfinite(out).all(-1), ~bad)
    assert torch.isnan(out[0, 1, 2]).all()
    q[0, 1, 2, 5] = q[0, 0, 3, 9] = 1
    dx, _, dw, _ = gb.attn_rope_bwd(q.cuda(), None, inv_freq, q=q.cuda(), q_weight=w.cuda())
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


def test_strided_parts_broadcast_streams_and_graphs():
    """Slices of one projection, a broadcast key head, another stream, and a captured call: the same bits as dense tensors."""
    B, L, Hq, Hkv, d = 2, 50, 8, 2, 128
    joint = draw((B, L, Hq + 2 * Hkv, d), torch.float16, 41).cuda()
    q, k, _ = joint.transpose(1, 2).split([Hq, Hkv, Hkv], dim=1)
    inv_freq, _ = gb.attn_rope_frequencies(d)
    want = gb.attn_rope(q.contiguous(), k.contiguous(), inv_freq)
    got = gb.attn_rope(q, k, inv_freq)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    wide = k[:, :1].expand(B, 5, L, d)
    assert torch.equal(gb.attn_rope(wide, None, inv_freq)[0], gb.attn_rope(wide.contiguous(), None, inv_freq)[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = gb.attn_rope(q, k, inv_freq, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))
    out = [torch.zeros_like(x) for x in want]
    up = [x.clone() for x in want]
    back = gb.attn_rope_bwd(*up, inv_freq)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gb.attn_rope(q, k, inv_freq, q_out=out[0], k_out=out[1])
        grads = gb.attn_rope_bwd(*out, inv_freq)
    joint.mul_(1.0)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and all(torch.equal(a, b) for a, b in zip(grads, back))


def test_with_attention_forward_and_backward():
    """norm + rotation -> attn_fwd -> attn_bwd -> attn_rope_bwd: the gradients of the whole against torch's in 64 bits.  Attention's
    own rounding (its tests: 2e-2) bounds this; relative to the gradient's norm."""
    B, H, L, d = 1, 4, 200, 64
    q, k, v, do = (draw((B, L, H, d), torch.float16, n).transpose(1, 2) for n in (51, 52, 53, 54))
    wq, wk = draw((d,), torch.float16, 55), draw((d,), torch.float16, 56)
    inv_freq, _ = gb.attn_rope_frequencies(d)
    c = lambda t: t.cuda()  # noqa: E731
    qr, kr = gb.attn_rope(c(q), c(k), inv_freq, q_weight=c(wq), k_weight=c(wk))
    vc, dc = c(v).contiguous(), c(do).contiguous()
    o, lse = gb.attn_fwd(qr, kr, vc, causal=True)
    dq, dk, _ = gb.attn_bwd(qr, kr, vc, o, lse, dc, causal=True)
    got = gb.attn_rope_bwd(dq, dk, inv_freq, q=c(q), k=c(k), q_weight=c(wq), k_weight=c(wk))
    leaves = [t.double().requires_grad_(True) for t in (q, k, wq, wk)]
    f = inv_freq.cpu()
    i, j = pairs(d, False)
    a = torch.arange(L, dtype=torch.float64)[:, None] * f

    def rot(x, w):
        y = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
        return torch.cat([y[..., i] * a.cos() - y[..., j] * a.sin(), y[..., j] * a.cos() + y[..., i] * a.sin()], -1)

    s = rot(leaves[0], leaves[2]) @ rot(leaves[1], leaves[3]).transpose(2, 3) / math.sqrt(d)
    s = s.masked_fill(torch.ones(L, L, dtype=torch.bool).triu(1), -math.inf)
    want = torch.autograd.grad((torch.softmax(s, -1) @ v.double() * do.double()).sum(), leaves)
    for x, y in zip(got, want):
        assert (x.cpu().double() - y).norm() <= 2e-2 * y.norm()


def test_refusals():
    q, k = draw((2, 4, 8, 64), torch.float16, 61).cuda(), draw((2, 2, 8, 64), torch.float16, 62).cuda()
    inv_freq, _ = gb.attn_rope_frequencies(64)
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(k=k[:, :, :4]), dict(k=k.bfloat16()), dict(k=k.cpu()), dict(q=q.transpose(2, 3)),
                dict(inv_freq=inv_freq.float()), dict(inv_freq=inv_freq.cpu()), dict(positions=torch.arange(8, device="cuda")),
                dict(positions=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(q_weight=w), dict(k_weight=w),
                dict(q_weight=w.float(), k_weight=w.float()), dict(q_weight=w[:32], k_weight=w[:32]), dict(q_out=k), dict(q=q.cpu(), k=k.cpu())):
        with pytest.raises(ValueError):
            gb.attn_rope(**{**dict(q=q, k=k, inv_freq=inv_freq), **bad})
    for bad in (dict(inv_freq=inv_freq[:20]), dict(inv_freq=torch.ones(40, dtype=torch.float64, device="cuda")), dict(factor=0.0),
                dict(factor=math.inf), dict(q_weight=w, k_weight=w, eps=-1.0), dict(q_out=q), dict(q=q[..., :48], k=None),
                dict(q=torch.zeros(2, 4, 8, 68, dtype=torch.float16, device="cuda")[..., :64]),
                dict(q=torch.zeros(2 * 4 * 8 * 64 + 1, dtype=torch.float16, device="cuda")[1:].view(2, 4, 8, 64))):
        with pytest.raises(gb.GbattnError):
            gb.attn_rope(**{**dict(q=q, k=k, inv_freq=inv_freq), **bad})
    with pytest.raises(ValueError):
        gb.attn_rope_bwd(q, k, inv_freq, q_weight=w, k_weight=w)
    with pytest.raises(ValueError):
        gb.attn_rope_bwd(q, k, inv_freq, q=q, k=k, q_weight=w, k_weight=w, workspace=torch.empty(8, device="cuda"))
