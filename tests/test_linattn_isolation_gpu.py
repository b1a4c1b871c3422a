"""Linear attention on the GPU with an infinity or NaN in one token: every output
that this token is no term of comes out bit for bit as with an ordinary value in
its place. Forwards that is every token before it and of other documents, and
every other column where it stands in v; backwards every token of other
documents, and the gradients that the operand is no factor of. In one chunk with
the token and in others, in one segment and across several, in both io types."""
import pytest
import torch

import selective_state_space_07_amd as ms
from tests.test_linattn_gpu import DT, bwd_args, fwd_args, gpu, make, say

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")

# batch, seqlen, heads, groups, d_k, d_v; where documents begin; the tokens that go bad, one at a time
CASES = {
    "one_chunk": ((1, 64, 2, 2, 64, 64), [9, 30, 41], [0, 17, 35, 63]),
    "chunks": ((1, 200, 2, 1, 128, 72), [70, 100, 150], [69, 70, 110, 127, 199]),
    # documents of two in one segment and of one over several; a bad token with beginnings on either side of it
    "segments": ((1, 2100, 2, 1, 64, 128), [130, 700, 760, 775, 1400, 2050], [5, 730, 761, 1399, 2060]),
}


def splits(shape, dtype):
    """Whether both directions run in several segments (the backward's dq and dk of every head left out)."""
    b, L, H, G, dk, _ = shape
    n = [ms.lin_attn_workspace_bytes(*shape, dtype, backward=back) for back in (False, True)]
    return n[0] > 0 and n[1] > (2 * 4 * b * L * H * dk if G != H else 0)


def case(name, dtype, packed=True):
    shape, begins, bad_at = CASES[name]
    a = make(*shape, DT[dtype], seed=71, state=True, backward=True)
    ids = torch.zeros(1, shape[1], dtype=torch.int32)
    if packed:
        ids[0, begins] = 1
        a["seq_idx"] = ids.cumsum(1).to(torch.int32)
    assert (name == "segments") == splits(shape, DT[dtype])
    return a, gpu(a), bad_at


def spoil(d, n, at, bad):
    t = d[n].clone()
    t[0, at, -1, 3] = bad
    return dict(d, **{n: t})


@pytest.mark.parametrize("bad", [INF, -INF, NAN])
@pytest.mark.parametrize("which", ["q", "k", "v"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_forward(name, dtype, which, bad):
    say("isolation forwards", name, dtype, which, bad)
    a, d, bad_at = case(name, dtype)
    kw = dict(seq_idx=d["seq_idx"])
    y0, s0 = ms.lin_attn_fwd(*fwd_args(d), **kw)
    w0, _ = ms.lin_attn_fwd(*fwd_args(d), **kw, return_state=False)
    doc = a["seq_idx"][0]
    for at in bad_at:
        e = spoil(d, which, at, bad)
        y1, s1 = ms.lin_attn_fwd(*fwd_args(e), **kw)
        w1, _ = ms.lin_attn_fwd(*fwd_args(e), **kw, return_state=False)
        torch.cuda.synchronize()
        t = torch.arange(len(doc))
        mine = (doc == doc[at]) & ((t == at) if which == "q" else (t >= at))
        for got, want in ((y1, y0), (w1, w0)):
            assert torch.equal(got[:, ~mine], want[:, ~mine]), at
            assert not torch.isfinite(got[0, at, -1]).all()
            if which == "v":
                rest = torch.arange(got.shape[3]) != 3
                assert torch.equal(got[..., rest], want[..., rest]), at
        ends = which != "q" and doc[at] == doc[-1]
        assert ends or torch.equal(s1, s0), at
        if ends and which == "v":
            assert torch.equal(s1[:, :, rest], s0[:, :, rest]), at


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_forward_of_one_document(name, dtype):
    """Without documents: the tokens before the bad one."""
    a, d, bad_at = case(name, dtype, packed=False)
    y0, _ = ms.lin_attn_fwd(*fwd_args(d))
    for at in bad_at:
        for which in "qkv":
            for bad in (INF, NAN):
                y1, _ = ms.lin_attn_fwd(*fwd_args(spoil(d, which, at, bad)))
                torch.cuda.synchronize()
                assert torch.equal(y1[:, :at], y0[:, :at]), (at, which)
                if which == "q":
                    assert torch.equal(y1[:, at + 1:], y0[:, at + 1:]), at


# the operands that each gradient has as factors
FACTORS = {"dq": "k v dy", "dk": "q v dy", "dv": "q k dy", "dstate": "q dy"}


@pytest.mark.parametrize("bad", [INF, NAN])
@pytest.mark.parametrize("which", ["q", "k", "v", "dy"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_gradients(name, dtype, which, bad):
    say("isolation backwards", name, dtype, which, bad)
    a, d, bad_at = case(name, dtype)
    kw = dict(seq_idx=d["seq_idx"])
    g0 = ms.lin_attn_bwd(*bwd_args(d), **kw)
    doc = a["seq_idx"][0]
    for at in bad_at:
        g1 = ms.lin_attn_bwd(*bwd_args(spoil(d, which, at, bad)), **kw)
        torch.cuda.synchronize()
        other = doc != doc[at]
        for n in ("dq", "dk", "dv"):
            assert torch.equal(g1[n][:, other], g0[n][:, other]), (n, at)
            assert which in FACTORS[n].split() or torch.equal(g1[n], g0[n]), (n, at)
        if doc[at] != doc[0] or which not in FACTORS["dstate"].split():
            assert torch.equal(g1["dstate"], g0["dstate"]), at
        hit = [n for n in ("dq", "dk", "dv") if not torch.isfinite(g1[n][:, ~other]).all()]
        assert hit, at


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_bad_state_stays_in_the_first_document(dtype):
    a, d, _ = case("segments", dtype)
    kw = dict(seq_idx=d["seq_idx"])
    y0, s0 = ms.lin_attn_fwd(*fwd_args(d), **kw)
    g0 = ms.lin_attn_bwd(*bwd_args(d), **kw)
    first, last = a["seq_idx"][0] == 0, a["seq_idx"][0] == a["seq_idx"][0, -1]
    for bad in (INF, NAN):
        e = dict(d, state=d["state"].clone(), dstate=d["dstate"].clone())
        e["state"][0, 0, 5, 7] = e["dstate"][0, 0, 5, 7] = bad
        y1, s1 = ms.lin_attn_fwd(*fwd_args(e), **kw)
        g1 = ms.lin_attn_bwd(*bwd_args(e), **kw)
        torch.cuda.synchronize()
        assert torch.equal(y1[:, ~first], y0[:, ~first]) and torch.equal(s1, s0)
        assert torch.equal(y1[:, :, 1], y0[:, :, 1]) and not torch.isfinite(y1[0, 0, 0, 5])
        assert torch.equal(g1["dq"][:, ~first], g0["dq"][:, ~first])
        for n in ("dk", "dv"):
            assert torch.equal(g1[n][:, ~last], g0[n][:, ~last]), n
        assert torch.equal(g1["dstate"], g0["dstate"])
