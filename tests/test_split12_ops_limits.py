"""Limits of the operators on Split12 weights, without a GPU: calls beyond them
are refused before the device is touched."""
import pytest
import torch  # noqa: F401

from test_split12_ops_abi import EMBED, container_bytes, wcm  # noqa: F401


@pytest.mark.parametrize("K", [(1 << 31) + 8, (1 << 32) - 8192, (1 << 32) - 8])
def test_embed_refuses_rows_past_its_column_counter(wcm, K):  # noqa: F811
    call = {**EMBED, "V": 1, "K": K, "w_bytes": container_bytes(K), "T": 1}
    assert wcm.load().wc12_embed(*call.values(), None) == wcm.ERR_INVALID_ARG
