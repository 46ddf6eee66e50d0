"""Prompt and drafted-tree attention where a row's sums leave the ordinary
range.  Compared with the plain 64-bit form."""
import math

import pytest
import torch

from attn_reference import Batch, attend, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_323_b200 import build as pkv_build

    pkv_build.build()
    from paged_kv_cache_323_b200 import pagedkv

    return pagedkv


def finish(pk, code=0):
    torch.cuda.synchronize()
    assert pk.get_device_error() == code


@pytest.mark.parametrize("tree", [False, True], ids=["prefill", "tree"])
@pytest.mark.parametrize("which,value", [("ks", math.nan), ("vs", math.nan), ("vs", math.inf), ("ks", math.inf)])
@pytest.mark.parametrize("head_dim", [128, 64])
def test_cache_scales_that_are_not_finite(pk, tree, which, value, head_dim):
    """A scale of one kv head that is not finite: its rows are what the formula gives, the others keep their bits."""
    b = Batch([(40, 300), (150, 150), (5, 3000)], dtype="fp8", heads=8, kv_heads=2, head_dim=head_dim, seed=60)
    b.poison()
    good = b.call(pk, tree).clone()
    getattr(b, which)[1] = value
    got = b.call(pk, tree)
    finish(pk)
    assert torch.equal(got[:, :4], good[:, :4])
    if (which, value) == ("ks", math.inf):
        return  # rows of one score of -inf are zeros here, NaN in the 64-bit form
    ref, bound = attend(b, tree)
    assert not bool(torch.isfinite(ref[:, 4:]).any())
    close(got, ref, bound)
