"""Bounded waits of the tensor-core prompt and tree attention, and its
index-checking build: a call that gives up reports PKV_ERR_TIMEOUT and leaves
its workspace fit for the next; the debug build's checks all pass."""
import os
import subprocess
import sys

import pytest
import torch

from attn_reference import Batch, attend, close

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_323_b200 import build as pkv_build

    pkv_build.build()
    from paged_kv_cache_323_b200 import pagedkv

    return pagedkv


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("seqs,heads,kv_heads", [
    ([(5, 9000)], 8, 1),                 # many parts
    ([(64, 3000), (300, 3000)], 8, 2),   # few parts, whole items
    ([(3, 40)] * 400, 2, 2),             # many items a CTA
])
def test_timeout_leaves_the_workspace_fit(pk, dtype, seqs, heads, kv_heads):
    b = Batch(seqs, dtype=dtype, heads=heads, kv_heads=kv_heads, seed=50)
    need = pk.paged_attention_prefill_workspace_size(b.T, b.H, b.G, b.D, pk._dtype_code(b.kc))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    want = b.call(pk, True, workspace=ws).clone()
    torch.cuda.synchronize()
    assert pk.get_device_error() == 0
    old = pk.set_wait_limit_us(1)  # far below a load's latency
    try:
        timeouts = 0
        for _ in range(10):
            b.call(pk, True, workspace=ws)
            timeouts += pk.get_device_error() == pk.PKV_ERR_TIMEOUT
    finally:
        pk.set_wait_limit_us(old)
    assert timeouts > 0
    counters = ws[:8 * 2 * 148 * 4].view(torch.int32)
    assert int(counters.abs().max()) == 0
    b.out.fill_(-77.0)
    got = b.call(pk, True, workspace=ws)
    torch.cuda.synchronize()
    assert pk.get_device_error() == 0
    assert torch.equal(got, want)
    ref, bound = attend(b, True)
    close(got, ref, bound)


CHILD = r"""
import torch
from paged_kv_cache_323_b200 import pagedkv as pk
from attn_reference import Batch, attend, close
from test_gpu_qk_rope import Step, step_bound
assert pk.DEBUG and pk.lib.pkv_debug_build() == 1
for dtype in ("f32", "bf16", "fp8"):
    for D, bs in ((64, 8), (128, 16), (128, 32)):
        for tree in (False, True):
            b = Batch([(0, 5), (1, 130), (257, 300), (5, 5000)], dtype=dtype, heads=4, kv_heads=1, head_dim=D,
                      block_size=bs, seed=3, pad_rows=2)
            b.poison()
            got = b.call(pk, tree)
            assert pk.get_device_error() == 0 and pk.debug_failed_line() == 0, (dtype, D, tree)
            ref, bound = attend(b, tree)
            n = b.start_host[-1]
            close(got[:n], ref[:n], bound[:n])
    for T in (3, 1500):
        s = Step(T, 8, 2, 128, dtype, seed=4, pad=1)
        s.call(pk)
        assert pk.get_device_error() == 0 and pk.debug_failed_line() == 0
        (q, e), _ = s.reference()
        from attn_reference import close as c
        c(s.q_out, q, step_bound(q, e, dtype))
print("debug ok")
"""


def test_debug_build_checks_every_index(pk):
    from paged_kv_cache_323_b200 import build as pkv_build

    pkv_build.build(debug=True)
    env = dict(os.environ, PKV_LIBRARY="debug", PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    r = subprocess.run([sys.executable, "-c", CHILD], env=env, capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "debug ok" in r.stdout, r.stdout + r.stderr
