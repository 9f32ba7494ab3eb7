"""attn_rope, attn_rope_bwd and the rotating append where their tiles hold the most tokens that a head's width allows (some thousand
rows and more), up to the fully rotated head, with a last tile that is not full.  Tolerances as in test_rope_gpu.py."""
import pytest
import torch

import scaled_dot_product_sdpa_gb300 as gb
from reference64 import check, draw, turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from scaled_dot_product_sdpa_gb300 import build
    gb.load_library(build.build())
    assert gb.attn_last_device_error() == 0
    yield
    assert gb.attn_last_device_error() == 0


CASES = [(1, 2, 1, 2501, 512, rotary) for rotary in (256, 288, 384, 512)] + [
    (2, 1, 0, 1300, 512, 512), (3, 1, 1, 2467, 256, 256), (2, 2, 1, 4901, 128, 128), (1, 1, 1, 10007, 64, 64)]


def angles(B, L, rotary):
    inv_freq = torch.pow(torch.tensor(500.0, dtype=torch.float64), -torch.arange(rotary // 2, dtype=torch.float64) / (rotary // 2))
    return inv_freq, torch.randint(-5, 100000, (B, L), generator=torch.Generator().manual_seed(5), dtype=torch.int32)


def normed(x, w, eps):
    y = x.double()
    return y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()


def on(x):
    return None if x is None else x.cuda()


@pytest.mark.parametrize("B,Hq,Hkv,L,d,rotary", CASES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_forward(B, Hq, Hkv, L, d, rotary, dtype, interleaved, norm):
    q, k = draw((B, Hq, L, d), dtype, 1), draw((B, Hkv, L, d), dtype, 2) if Hkv else None
    wq, wk = draw((d,), dtype, 3), draw((d,), dtype, 4) if Hkv else None
    inv_freq, pos = angles(B, L, rotary)
    got = gb.attn_rope(q.cuda(), on(k), inv_freq.cuda(), positions=pos.cuda(), interleaved=interleaved, factor=1.25,
                       q_weight=on(wq) if norm else None, k_weight=on(wk) if norm else None, eps=1e-5)
    for x, w, out in ((q, wq, got[0]), (k, wk, got[1])):
        if x is not None:
            check(out, *turned(normed(x, w, 1e-5) if norm else x.double(), pos, inv_freq, 1.25, interleaved), "forward")


@pytest.mark.parametrize("B,Hq,Hkv,L,d,rotary", CASES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_backward(B, Hq, Hkv, L, d, rotary, dtype, interleaved, norm):
    q, dq, wq = draw((B, Hq, L, d), dtype, 11), draw((B, Hq, L, d), dtype, 12), draw((d,), dtype, 13)
    k, dk, wk = (draw((B, Hkv, L, d), dtype, 14), draw((B, Hkv, L, d), dtype, 15), draw((d,), dtype, 16)) if Hkv else (None,) * 3
    inv_freq, pos = angles(B, L, rotary)
    eps = 1e-5
    more = dict(q=on(q), k=on(k), q_weight=on(wq), k_weight=on(wk), eps=eps) if norm else {}
    got = gb.attn_rope_bwd(on(dq), on(dk), inv_freq.cuda(), positions=pos.cuda(), interleaved=interleaved, factor=1.25, **more)
    for n, (x, up, w) in enumerate(((q, dq, wq), (k, dk, wk))):
        if x is None:
            continue
        dy, size = turned(up.double(), pos, inv_freq, 1.25, interleaved, sign=-1.0)
        if not norm:
            check(got[n], dy, size, "backward")
            continue
        y = x.double()
        rstd = 1.0 / (y.square().mean(-1, keepdim=True) + eps).sqrt()
        xh, g, gsize = y * rstd, dy * w.double(), size * w.double().abs()
        want = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
        check(got[n], want, rstd * (gsize + xh.abs() * (gsize * xh.abs()).mean(-1, keepdim=True)), "dx")
        check(got[2 + n], (dy * xh).sum((0, 1, 2)), (size * xh.abs()).sum((0, 1, 2)), "dw", depth=128 + 64)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("norm", [False, True])
def test_append(dtype, norm):
    """Keys into pages in order, so that the cache spells the rows."""
    H, L, d, page = 2, 2501, 512, 8
    P = -(-L // page)
    q, k, v = (draw((1, H, L, d), dtype, 21 + n) for n in range(3))
    wq, wk = draw((d,), dtype, 24), draw((d,), dtype, 25)
    inv_freq, _ = gb.attn_rope_frequencies(d)
    kp, vp = (torch.zeros(P, H, page, d, dtype=dtype, device="cuda") for _ in range(2))
    out = gb.attn_cache_append(k.cuda(), v.cuda(), kp, vp, torch.arange(P, dtype=torch.int32)[None].cuda(), torch.tensor([L], dtype=torch.int32).cuda(),
                               q=q.cuda(), inv_freq=inv_freq, q_weight=on(wq) if norm else None, k_weight=on(wk) if norm else None)
    pos = torch.arange(L, dtype=torch.int32)[None]
    rows = [x.transpose(0, 1).reshape(1, H, P * page, d)[:, :, :L] for x in (kp, vp)]
    for x, w, got in ((q, wq, out), (k, wk, rows[0])):
        check(got, *turned(normed(x, w, 1e-6) if norm else x.double(), pos, inv_freq.cpu(), 1.0, False), "append")
    assert torch.equal(rows[1].cpu(), v)
