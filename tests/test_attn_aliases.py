"""Outputs in the place of inputs where the calls around the paged cache cannot
allow it, on the CPU."""
import pytest

import test_attn_checks as checks
from test_abi import FAKE, pk as abi_pk  # noqa: F401
from test_attn_checks import no_stream  # noqa: F401

OTHER = FAKE + (1 << 20)


@pytest.mark.parametrize("name", checks.NAMES)
def test_attention_writes_no_q(abi_pk, name):  # noqa: F811
    """A row's q is read again after the row's first result is written."""
    assert checks._attn(abi_pk, name, out=OTHER, q=OTHER) == abi_pk.PKV_ERR_INVALID


@pytest.mark.parametrize("fp8", [False, True])
def test_rotation_in_place_has_one_stride(abi_pk, fp8):  # noqa: F811
    assert checks._rope(abi_pk, fp8, q_out=OTHER, q=OTHER, so=1024, sq=1536) == abi_pk.PKV_ERR_INVALID
