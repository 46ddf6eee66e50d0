"""The rotation's append into an fp8 cache at cache scales over fp32's whole
range: the codes of kv_cache_append_fp8, whose quotients are divided one by one."""
import math

import pytest
import torch

from test_gpu_qk_rope import Step, pk  # noqa: F401

pytestmark = pytest.mark.gpu

SCALES = [1e-45, 1e-40, 2.0 ** -126, 2.0 ** -110, 2.0 ** -91, 2.0 ** -90, 1e-20, 1.0, 1 / 3, 1e20, 2.0 ** 100, 2.0 ** 101,
          1e38, 3.4e38, math.inf, 0.0, math.nan, -0.7, -1e-40, -2.0 ** 126]


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("amp", [1e-40, 1e-36, 2.0 ** -105, 2.0 ** -88, 1e-6, 3.0, 1e10, 1e30, 1e37])
def test_codes_are_the_appends(pk, head_dim, amp):  # noqa: F811
    G = len(SCALES)
    s = Step(29, 4, G, head_dim, "fp8", norm="", seed=70, amp=amp)
    s.pos.zero_()
    s.k[0] = 0.0
    s.k[s.k == 0] = 0.0  # a turn by 0 takes -0 to -0 + 0, and inf to inf - inf * 0
    s.v[0], s.v[1], s.v[2], s.v[3] = 0.0, -0.0, math.inf, math.nan
    s.ks = torch.tensor(SCALES, device="cuda", dtype=torch.float32)
    s.vs = s.ks.flip(0).contiguous()
    other = [s.kc.clone(), s.vc.clone()]
    s.call(pk)
    pk.kv_cache_append_fp8(*other, s.ks, s.vs, s.k.contiguous(), s.v.contiguous(), s.slots)
    torch.cuda.synchronize()
    assert pk.get_device_error() == 0
    for got, want, scales in zip((s.kc, s.vc), other, (s.ks, s.vs)):
        got, want = got.view(torch.uint8), want.view(torch.uint8)
        bad = (got != want).any(-1).any(2).any(0).nonzero().flatten().tolist()
        assert not bad, scales[bad].tolist()
