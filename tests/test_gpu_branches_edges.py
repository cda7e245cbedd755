"""Edges of the operators for several continuations of a sequence: what 16-bit rows of trees
keep of their weights."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import _branches as R  # noqa: E402
import _layer as L  # noqa: E402
import dynamic_sparsity_approximate_amd as E  # noqa: E402
from test_gpu_branches import Tree  # noqa: E402
from test_gpu_layer import f64, say  # noqa: E402


# ---------------------------------------------------------------- trees: what 16-bit rows keep

@pytest.mark.parametrize("room", [0, 1100])  # tables of more than 1024 tokens are shared out in another way
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,group,dim,page,fmt,lens,new,window", [
    (2, 4, 128, 64, "e4m3", [700, 33], [32, 33], 0), (1, 8, 128, 16, "i8", [300, 90], [40, 30], 0),
    (2, 3, 64, 16, "e4m3", [500, 26, 129, 64], [25, 25, 20, 13], 100), (1, 4, 64, 64, "i8", [640, 212], [100, 212], 0),
    (2, 4, 128, 128, "e4m3", [410, 64, 15], [15, 14, 15], 0), (2, 2, 128, 16, "i8", [70, 300], [6, 7], 0)])
def test_trees_keep_the_weights_of_16_bit_rows(heads, group, dim, page, fmt, lens, new, window, dtype, room):
    """What fp32 rows are held to, and one rounding of the output (small scores, which add little to that),
    however wide the page table is."""
    c = Tree(51, lens, new, heads=heads, group=group, dim=dim, page=page, fmt=fmt, dtype=dtype, room=room)
    q = c.rand(heads * group, 0.01)
    got = f64(c.cache.attend(c.batch, q, window=window))
    ref, tol = R.attend(c.np, c.table, c.lens, c.starts, f64(q), dim ** -0.5, window, fmt, "f32", c.parents)
    # rounding moves a result by half a step of what is rounded, itself within tol of ref
    tol = tol + L.HALF_STEP[dtype] * (np.abs(ref) + tol) + (2.0 ** -25 if dtype == "f16" else 0.0)
    worst = float((np.abs(got - ref) / (tol + 1e-300)).max())
    say("worst", worst)
    assert worst <= 1.0, worst
