"""The new operators as a layer runs them: linear attention over columns of one
projection's output and the gated norm of its heads, forwards, backwards and
token by token; and the Mamba-2 scan with the gate-first RMS norm behind it.

Float32 io, so that the sealed rule of the scans' tests applies
(|got - want| <= 1e-4 max(|want|, rms(want)) per element)."""
import pytest
import torch

import selective_state_space_07_amd as ms
import workloads
from oracle import gnorm as gn
from oracle import linattn as la
from oracle import ssd as ossd
from tests import tolerances as T

pytestmark = pytest.mark.gpu
B, L, H, D = 2, 150, 4, 64


def columns(wide):
    """q, k, v [B, L, H, D] and the gate z [B, L, H * D], read in place."""
    q, k, v, z = wide.split(H * D, -1)
    return (*(t.unflatten(-1, (H, D)) for t in (q, k, v)), z)


def inputs():
    g = torch.Generator().manual_seed(1)
    wide = torch.randn(B, L, 4 * H * D, generator=g)
    decay = torch.log1p(-torch.exp2(-2.0 - torch.arange(H)))
    w, b = 1 + 0.2 * torch.randn(H * D, generator=g), 0.2 * torch.randn(H * D, generator=g)
    dy = torch.randn(B, L, H * D, generator=g)
    return wide, decay, w, b, dy


def test_layer_forwards_and_backwards():
    wide, decay, w, b, dy = inputs()
    q, k, v, z = columns(wide.cuda())
    wg, bg, dg = w.cuda(), b.cuda(), decay.cuda()
    s0 = torch.randn(B, H, D, D, generator=torch.Generator().manual_seed(2))
    y, s = ms.lin_attn_fwd(q, k, v, dg, s0.cuda())
    out = ms.group_norm_fwd(y.flatten(2), wg, bg, H, z)
    gn_grads = ms.group_norm_bwd(y.flatten(2), wg, bg, H, dy.cuda(), z)
    la_grads = ms.lin_attn_bwd(q, k, v, dg, gn_grads["dx"].view(B, L, H, D), s0.cuda())
    torch.cuda.synchronize()

    q, k, v, z = columns(wide)
    yo, so = la.oracle_fwd(q, k, v, decay, s0)
    T.assert_close(s, so, 1e-4, "state")
    T.assert_close(out, gn.oracle_fwd(yo.reshape(B, L, -1), w, b, H, z), 1e-4, "out")
    want = gn.oracle_bwd(yo.reshape(B, L, -1), w, b, H, dy, z)
    for n in ("dx", "dz", "dweight", "dbias"):
        T.assert_close(gn_grads[n], want[n], 1e-4, n)
    want = la.oracle_bwd(q, k, v, decay, want["dx"].reshape(B, L, H, D), s0)
    for n in ("dq", "dk", "dv", "dstate"):
        T.assert_close(la_grads[n], want[n], 1e-4, n)


def test_prompt_then_tokens():
    """A prompt and then tokens one by one give what the whole sequence gives at once."""
    wide, decay, w, b, _ = inputs()
    wide, dg, wg, bg = wide.cuda(), decay.cuda(), w.cuda(), b.cuda()
    q, k, v, z = columns(wide)
    y, _ = ms.lin_attn_fwd(q, k, v, dg)
    whole = ms.group_norm_fwd(y.flatten(2), wg, bg, H, z)
    n = 131
    y, s = ms.lin_attn_fwd(*(t[:, :n] for t in (q, k, v)), dg)
    parts = [ms.group_norm_fwd(y.flatten(2), wg, bg, H, z[:, :n])]
    for t in range(n, L):
        y, s = ms.lin_attn_step(q[:, t], k[:, t], v[:, t], dg, s, inplace=True)
        parts.append(ms.group_norm_fwd(y.flatten(1), wg, bg, H, z[:, t])[:, None])
    torch.cuda.synchronize()
    T.assert_close(torch.cat(parts, 1), whole.cpu(), 1e-4, "token by token")


def test_norm_behind_the_mamba2_scan():
    lay = workloads.make_ssd(2, 300, 4, 64, 128, 1, torch.float32, seed=6)
    args = [lay[n] for n in workloads.SSD_KEYS]
    z = torch.randn(2, 300, 256, generator=torch.Generator().manual_seed(7))
    w = 1 + 0.1 * torch.randn(256, generator=torch.Generator().manual_seed(8))
    y, _ = ms.ssd_fwd(*(t.cuda() for t in args))
    out = ms.group_norm_fwd(y.flatten(2), w.cuda(), None, 1, z.cuda(), gate_first=True, center=False)
    torch.cuda.synchronize()
    yo, _ = ossd.oracle_ssd_fwd(*args)
    T.assert_close(out, gn.oracle_fwd(yo.reshape(2, 300, -1), w, None, 1, z, gate_first=True, center=False), 1e-4, "out")
