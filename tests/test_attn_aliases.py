"""Outputs in the place of inputs where the calls around the paged cache cannot
allow it, and numbers of any kind as scale and eps: on the CPU."""
import numpy as np
import pytest
import torch

import test_attn_checks as checks
from test_abi import FAKE, pk as abi_pk  # noqa: F401
from test_attn_checks import D_, attn_args, no_stream  # noqa: F401
from test_binding_checks import pk  # noqa: F401

OTHER = FAKE + (1 << 20)


@pytest.mark.parametrize("name", checks.NAMES)
def test_attention_writes_no_q(abi_pk, name):  # noqa: F811
    """A row's q is read again after the row's first result is written."""
    assert checks._attn(abi_pk, name, out=OTHER, q=OTHER) == abi_pk.PKV_ERR_INVALID


@pytest.mark.parametrize("fp8", [False, True])
def test_rotation_in_place_has_one_stride(abi_pk, fp8):  # noqa: F811
    assert checks._rope(abi_pk, fp8, q_out=OTHER, q=OTHER, so=1024, sq=1536) == abi_pk.PKV_ERR_INVALID


@pytest.mark.parametrize("number", [np.float32(0.125), np.float64(0.125), torch.tensor(0.125), np.array(0.125), 1])
def test_numbers_of_any_kind(pk, number):  # noqa: F811
    a = attn_args()
    pk.paged_attention_prefill(a["out"], a["q"], a["kc"], a["vc"], a["bt"], a["ctx"], a["qs"], number)
    pk.paged_attention_tree(a["out"], a["q"], a["kc"], a["vc"], a["bt"], a["ctx"], a["qs"], a["par"], number)
    pk.qk_norm_rope_append(a["out"], a["q"], D_((6, 2, 64)), D_((6, 2, 64)), a["kc"], a["vc"],
                           D_((6,), torch.int64), D_((6,), torch.int32), D_((32,), torch.float32), eps=number)
    calls = [(n, x) for n, x in pk.fake.calls if not n.endswith("workspace_size")]
    assert [type(x[i]) for (_, x), i in zip(calls, (15, 16, 11))] == [float] * 3
    assert [x[i] for (_, x), i in zip(calls, (15, 16, 11))] == [float(number)] * 3
