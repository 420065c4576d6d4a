"""Streams of another device than the tensors' (no GPU needed)."""

import types

import pytest
import torch

import sparse_dictionary_coded_b200 as sdk


class _Tensor(torch.Tensor):
    """A tensor that says it lies on cuda:0."""
    is_cuda = True
    device = torch.device("cuda:0")


@pytest.mark.parametrize("call", [
    lambda t, s: sdk.sdk_block_tables(t, t, t, t, t, 16, 1, stream=s),
    lambda t, s: sdk.sdk_paged_store(t, t, t, t, stream=s),
    lambda t, s: sdk.sdk_paged_append(t, t, t, t, t, t, stream=s),
    lambda t, s: sdk.sdk_chunk_attn(t, t, t, t, t, t, t, 1, 1, stream=s)])
def test_stream_of_another_device_is_refused(call):
    other = types.SimpleNamespace(device=torch.device("cuda:1"))
    with pytest.raises(ValueError, match="stream is on cuda:1, the tensors on cuda:0"):
        call(torch.zeros(2).as_subclass(_Tensor), other)
