"""The RMS norm with the residual's addition on the GPU against the fp64
oracle: every layout of a row over lanes, io and residual types, strides, rows
behind the last, values at float32's ends, 8-bit outputs with their scales,
gradients, in-place residuals, streams and captured graphs.

The bounds are counted, not fitted. With U = 2^-24: a row's sum of squares goes
through at most 16 terms of a lane, 6 steps over lanes and 16 waves, 40
roundings, so that 1 / sqrt of it is within 22 U and y within 32 U of itself
(the sum h, the instruction, three products). A gradient's mean is such a sum
of terms that are within 32 U themselves: 100 U of the magnitudes covers it. A
sum over rows adds a rounding for each. bfloat16 outputs add half a step,
2^-8 of themselves, 8-bit ones 2^-4, or 2^-10 scales where they are subnormal."""
import numpy as np
import pytest
import torch

import selective_state_space_07_amd as ms
from oracle import rmsnorm as orn
from oracle.linattn import f64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TYPES = [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")]


def half(dtype):
    return BF if dtype == torch.bfloat16 else 0.0


def make(rows, c, io, res, seed=0, wide=0, weight=True):
    g = torch.Generator().manual_seed(seed)
    at = slice(wide // 2, wide // 2 + c)
    rnd = lambda t: torch.randn(rows, c + wide, generator=g).to(DT[t])[:, at]  # noqa: E731
    x, r, dy, dh = rnd(io), rnd(res), rnd(io), rnd(res)
    return x, r, (1 + 0.2 * torch.randn(c, generator=g) if weight else None), dy, dh


def cuda(a):
    return None if a is None else torch.empty_strided(a.shape, a.stride(), dtype=a.dtype, device="cuda").copy_(a)


def hold(got, want, tol, what):
    got = f64(got)
    assert got.shape == want.shape and np.isfinite(got).all(), what
    err = np.abs(got - want)
    at = np.unravel_index(np.argmax(err / (tol + 1e-300)), err.shape)
    assert (err <= tol).all(), "%s: %g off at %s, %g allowed" % (what, err[at], at, tol[at])


def check_fwd(x, r, w, y, h, what, eps=1e-5):
    wy, wh = orn.oracle_fwd(x, r, w, eps)
    hold(y, wy, (32 * U + half(x.dtype) * (1 + 32 * U)) * np.abs(wy), what + " y")
    if r is not None:
        hold(h, wh, (U + half(r.dtype) * (1 + U)) * np.abs(wh), what + " h")


def check_bwd(h, w, dy, dh, got, what, eps=1e-5):
    want = orn.oracle_bwd(h, w, dy, dh, eps)
    hh, d = f64(h), np.abs(f64(dy) if w is None else f64(dy) * f64(w))
    r = 1 / np.sqrt((hh * hh).mean(-1, keepdims=True) + eps)
    hat = np.abs(hh) * r
    size = r * (d + hat * (d * hat).mean(-1, keepdims=True)) + (0 if dh is None else np.abs(f64(dh)))
    tol = 100 * U * size
    for n, t in (("dx", dy.dtype), ("dresidual", h.dtype)):
        assert got[n].dtype == t
        hold(got[n], want["d"], tol + half(t) * (np.abs(want["d"]) + tol), what + " " + n)
    assert ("dweight" in got) == (w is not None)
    if w is not None:
        n = dy.reshape(-1, dy.shape[-1]).shape[0]
        mag = (np.abs(f64(dy)) * hat).reshape(-1, dy.shape[-1]).sum(0)
        hold(got["dweight"], want["dweight"], (n + 40) * U * mag, what + " dweight")


# rows, channels: one lane to sixteen waves a row, whole and partial pieces, aligned and not
SHAPES = [(1, 8), (7, 16), (300, 24), (65, 64), (33, 120), (5, 256), (70, 512), (1000, 520), (9, 768), (3, 1000), (4, 1024),
          (6, 1032), (2, 2048), (130, 2056), (3, 4096), (2, 8192), (5, 8200), (2, 16384), (1, 1), (5, 3), (4, 65), (6, 511),
          (7, 513), (3, 1025), (2, 4095), (2, 4097), (3, 16381)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_gradients(shape, types):
    print(shape, types, flush=True)
    x, r, w, dy, dh = make(*shape, *types, seed=shape[1], weight=shape[0] % 5 != 2)
    y, h = ms.add_rms_norm_fwd(cuda(x), cuda(r), cuda(w))
    torch.cuda.synchronize()
    check_fwd(x, r, w, y, h, "norm")
    back = None if shape[0] % 4 == 1 else dh
    grads = ms.add_rms_norm_bwd(h, cuda(w), cuda(dy), cuda(back))
    torch.cuda.synchronize()
    check_bwd(h.cpu(), w, dy, back, grads, "norm")
    assert (grads["dx"] is grads["dresidual"]) == (types[0] == types[1])


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("rows,c,wide", [(50, 768, 768), (9, 1000, 5), (3, 96, 8), (4, 3000, 24)])
def test_columns_of_a_wider_tensor(rows, c, wide, types):
    x, r, w, dy, dh = make(rows, c, *types, seed=c, wide=wide)
    y, h = ms.add_rms_norm_fwd(cuda(x), cuda(r), cuda(w))
    check_fwd(x, r, w, y, h, "strided")
    grads = ms.add_rms_norm_bwd(cuda(r), cuda(w), cuda(dy), cuda(dh))
    torch.cuda.synchronize()
    check_bwd(r, w, dy, dh, grads, "strided")


def test_more_dimensions_no_residual_in_place_and_given_output():
    x, r, w, _, _ = make(24, 264, "bf16", "f32", seed=2)
    y, h = ms.add_rms_norm_fwd(cuda(x).view(2, 12, 264), cuda(r).view(2, 12, 264), cuda(w))
    assert y.shape == h.shape == (2, 12, 264)
    check_fwd(x, r, w, y.flatten(0, 1), h.flatten(0, 1), "three dimensions")
    gx = cuda(x)
    y1, h1 = ms.add_rms_norm_fwd(gx, None, cuda(w))
    assert h1 is gx
    check_fwd(x, None, w, y1, None, "no residual")
    gr, out = cuda(r), torch.full_like(gx, 3.0)
    y2, h2 = ms.add_rms_norm_fwd(gx, gr, cuda(w), inplace=True, out=out)
    torch.cuda.synchronize()
    assert h2 is gr and y2 is out and torch.equal(gr, h.flatten(0, 1)) and torch.equal(y2, y.flatten(0, 1))


@pytest.mark.parametrize("scale,eps", [(1e38, 1e-5), (1e30, 1e-5), (1e-20, 0.0), (1e-38, 0.0), (1e-12, 1e-5), (1.0, 0.0)])
@pytest.mark.parametrize("c", [96, 1024, 2048, 16384, 333, 5000])
def test_ends_of_the_range(scale, eps, c):
    g = torch.Generator().manual_seed(c)
    x = torch.rand(6, c, generator=g).add_(0.1).mul_(torch.randint(0, 2, (6, c), generator=g) * 2 - 1)
    x[1::2] *= scale
    w, dy = 1 + 0.2 * torch.randn(c, generator=g), torch.randn(6, c, generator=g)
    y, _ = ms.add_rms_norm_fwd(x.cuda(), None, w.cuda(), eps=eps)
    torch.cuda.synchronize()
    wy, _ = orn.oracle_fwd(x, None, w, eps)
    hold(y, wy, 40 * U * np.abs(wy) + 2.0 ** -149, "y")
    if scale > 1e-37:  # the gradient of smaller values is beyond float32
        check_bwd(x, w, dy, None, ms.add_rms_norm_bwd(x.cuda(), w.cuda(), dy.cuda(), eps=eps), "ends", eps)


def test_rows_of_zeros_and_what_is_not_finite_stay_in_their_rows():
    x, r, w, dy, dh = make(40, 264, "f32", "f32", seed=3)
    want, _ = ms.add_rms_norm_fwd(cuda(x), cuda(r), cuda(w))
    wd = ms.add_rms_norm_bwd(cuda(x), cuda(w), cuda(dy), cuda(dh))
    x2, r2 = x.clone(), r.clone()
    x2[3], r2[3], x2[7, 5], x2[11, 0] = 0, 0, float("nan"), float("inf")
    y, h = ms.add_rms_norm_fwd(cuda(x2), cuda(r2), cuda(w))
    d = ms.add_rms_norm_bwd(cuda(x2), None, cuda(dy), cuda(dh))
    keep = torch.ones(40, dtype=torch.bool)
    keep[[3, 7, 11]] = False
    wd2 = ms.add_rms_norm_bwd(cuda(x), None, cuda(dy), cuda(dh))
    torch.cuda.synchronize()
    assert torch.equal(y.cpu()[keep], want.cpu()[keep]) and (y[3] == 0).all() and y[7].isnan().all() and y[11, 0].isnan()
    assert torch.equal(d["dx"].cpu()[keep], wd2["dx"].cpu()[keep]) and wd["dx"].isfinite().all()


def stands_for(q, scales, block):
    v = q.float().cpu().double().numpy()
    c = v.shape[-1]
    return v * np.repeat(f64(scales), block or c, -1)[..., :c]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("block", [None, 128])
@pytest.mark.parametrize("rows,c", [(1, 16), (40, 48), (9, 112), (33, 128), (7, 144), (20, 768), (5, 1024), (3, 1040), (64, 2048),
                                    (2, 4112), (3, 8192), (2, 16384)])
def test_eight_bits(rows, c, block, types):
    print(rows, c, block, types, flush=True)
    x, r, w, _, _ = make(rows, c, *types, seed=rows)
    q, scales, h = ms.add_rms_norm_fp8(cuda(x), cuda(r), cuda(w), block=block)
    torch.cuda.synchronize()
    assert q.dtype == torch.float8_e4m3fn and q.shape == x.shape and scales.shape == (rows, -(-c // block) if block else 1)
    wy, wh = orn.oracle_fwd(x, r, w)
    ws, each = orn.oracle_scales(wy, block)
    hold(scales, ws, 36 * U * ws, "scales")
    got = stands_for(q, scales, block)
    hold(got, wy, (2.0 ** -4 + 40 * U) * np.abs(wy) + 2.0 ** -10 * (1 + 40 * U) * each, "y")
    assert np.abs(q.float().cpu().numpy()).max() == 448
    hold(h, wh, (U + half(r.dtype) * (1 + U)) * np.abs(wh), "h")


def test_eight_bits_of_zeros_and_nan():
    x = torch.zeros(3, 256)
    x[1] = torch.randn(256, generator=torch.Generator().manual_seed(1))
    x[2, 130] = float("nan")
    for block, n in ((None, 1), (128, 2)):
        q, s, _ = ms.add_rms_norm_fp8(x.cuda(), None, None, block=block)
        torch.cuda.synchronize()
        q, s = q.float().cpu(), s.cpu()
        assert (q[0] == 0).all() and (s[0] == 1).all() and q[1].abs().max() == 448
        assert q[2].isnan().all() and s[2].isnan().all() and s.shape == (3, n)


def test_eight_bits_in_place_and_of_tiny_values():
    x, r, w, _, _ = make(8, 256, "bf16", "f32", seed=6)
    gr = cuda(r)
    q, s, h = ms.add_rms_norm_fp8(cuda(x), gr, cuda(w) * 1e-38, inplace=True)
    q2, s2, h2 = ms.add_rms_norm_fp8(cuda(x), cuda(r), cuda(w))
    torch.cuda.synchronize()
    assert h is gr and torch.equal(h, h2) and (s == 2.0 ** -126).all() and q.float().isfinite().all() and (q.float() != 0).any()


def test_workspace_determinism_stream_and_graph():
    x, r, w, dy, dh = make(3000, 768, "bf16", "f32", seed=8)
    h, gw, d, b = cuda(r), cuda(w), cuda(dy), cuda(dh)
    need = ms.add_rms_norm_workspace_bytes(3000, 768, torch.bfloat16)
    first = None
    for fill in (0, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        grads = ms.add_rms_norm_bwd(h, gw, d, b, workspace=ws)
        torch.cuda.synchronize()
        first = first or grads
        assert all(torch.equal(grads[n], first[n]) for n in grads)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gx = cuda(x)
    with torch.cuda.stream(side):
        ms.add_rms_norm_fwd(gx, h, gw)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, s = ms.add_rms_norm_fwd(gx, h, gw)
        q, sc, _ = ms.add_rms_norm_fp8(gx, h, gw, block=128)
        grads = ms.add_rms_norm_bwd(s, gw, d, b)
    for i in range(3):
        gx.copy_(torch.randn(3000, 768, generator=torch.Generator().manual_seed(i)))
        wy, wh = ms.add_rms_norm_fwd(gx, h, gw)
        wq, wsc, _ = ms.add_rms_norm_fp8(gx, h, gw, block=128)
        wg = ms.add_rms_norm_bwd(wh, gw, d, b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, wy) and torch.equal(s, wh) and torch.equal(sc, wsc)
        assert torch.equal(q.view(torch.uint8), wq.view(torch.uint8))
        assert all(torch.equal(grads[n], wg[n]) for n in wg)


def test_past_two_to_the_31_elements():
    c = 1032
    rows = (1 << 31) // c + 1000
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(rows, c, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.rand(c, device="cuda", generator=g)
    y, h = ms.add_rms_norm_fwd(x, x, w)
    y2, h2 = ms.add_rms_norm_fwd(x[-77:], x[-77:], w)
    torch.cuda.synchronize()
    assert torch.equal(y[-77:], y2) and torch.equal(h[-77:], h2)
    d, d2 = ms.add_rms_norm_bwd(h, None, y, x), ms.add_rms_norm_bwd(h2, None, y2, x[-77:])
    torch.cuda.synchronize()
    assert torch.equal(d["dx"][-77:], d2["dx"])
