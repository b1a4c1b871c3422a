"""The group norm on the GPU in each way a group is held: single elements or
16-byte pieces, in few or many of a lane, by a wave, by a workgroup, or read anew
by each pass; several groups a row, row counts that fill no wave, and sizes that
would be held in 16-byte pieces at places where they cannot be. Bounds as in
test_gnorm_gpu.py."""
import pytest
import torch

import selective_state_space_07_amd as ms
from tests.test_gnorm_gpu import DT, bwd, check, fwd, gpu, make, say

pytestmark = pytest.mark.gpu

# channels of a group that single elements (a size that no 16-byte piece divides) or pieces hold
SHAPES = [
    # rows, channels, groups: single elements, one or two a lane
    (6, 3 * 63, 3), (7, 2 * 65, 2), (5, 3 * 127, 3),
    # up to eight a lane
    (5, 129, 1), (7, 3 * 129, 3), (6, 5 * 300, 5), (3, 2 * 511, 2), (1, 4 * 257, 4), (13, 2 * 450, 2), (66, 2 * 190, 2),
    # a workgroup, four a thread, and read anew
    (5, 2 * 513, 2), (3, 4095, 1), (2, 3 * 4097, 3), (3, 2 * 4100, 2),
    # pieces: a wave, a workgroup (float32 from 260, bfloat16 from 520), read anew
    (5, 3 * 256, 3), (3, 2 * 260, 2), (5, 2 * 512, 2), (3, 3 * 520, 3), (2, 4096, 1), (2, 2 * 4100, 2), (2, 8200, 1),
]


@pytest.mark.parametrize("gate", ["none", "after", "first"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_sizes(shape, dtype, gate):
    say("layout", shape, dtype, gate)
    a = make(*shape, DT[dtype], gate, seed=sum(shape))
    d = gpu(a)
    kw = dict(gate_first=gate == "first", center=gate != "first")
    y, g = fwd(d, **kw), bwd(d, **kw)
    torch.cuda.synchronize()
    check(a, y, g, **kw)


@pytest.mark.parametrize("gate", ["none", "after", "first"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(7, 2 * 64, 2), (5, 3 * 256, 3), (6, 2 * 512, 2), (3, 2 * 1024, 2), (2, 8192, 1)], ids=str)
def test_sizes_of_whole_pieces_at_odd_places(shape, dtype, gate):
    """Columns one element behind an aligned place, rows an odd number of elements apart."""
    say("odd places", shape, dtype, gate)
    a = make(*shape, DT[dtype], gate, seed=sum(shape) + 1)
    d = gpu(a)
    rows, c = shape[:2]
    for n in ("x", "z", "dy"):
        if d[n] is not None:
            wide = torch.full((rows, c + 3), float("nan"), dtype=DT[dtype], device="cuda")
            wide[:, 1:c + 1] = d[n]
            d[n] = wide[:, 1:c + 1]
    kw = dict(gate_first=gate == "first", center=gate != "first", activation="sigmoid")
    y, g = fwd(d, **kw), bwd(d, **kw)
    torch.cuda.synchronize()
    check(a, y, g, **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows_of_single_elements(dtype):
    """More turns than one for every workgroup, the last of them part empty."""
    a = make(12345, 300, 2, DT[dtype], "after", seed=7)
    d = gpu(a)
    y, g = fwd(d), bwd(d)
    torch.cuda.synchronize()
    check(a, y, g)
    again = bwd(d)
    assert all(torch.equal(again[n], g[n]) for n in g)


def test_captured_in_single_elements():
    a = make(40, 2 * 300, 2, torch.bfloat16, "first", seed=8)
    d = gpu(a)
    kw = dict(gate_first=True, center=False)
    y0, g0 = fwd(d, **kw), bwd(d, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, g = fwd(d, **kw), bwd(d, **kw)
    for _ in range(3):
        y.zero_(), [t.zero_() for t in g.values()]
        graph.replay()
        e = ms.group_norm_fwd(d["x"], d["weight"], d["bias"], 2, d["z"], **kw)
        torch.cuda.synchronize()
        assert torch.equal(y, y0) and torch.equal(e, y0) and all(torch.equal(g[n], g0[n]) for n in g0)
