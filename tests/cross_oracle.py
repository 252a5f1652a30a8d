"""Cross attention in float64 with its bounds: attention_oracle's, without a mask within clips."""

from unittest import mock

import torch

import attention_oracle


def _all(nq, nk, window, sinks):
    return torch.ones(nq, nk, dtype=torch.bool)


def attention(q, k, v, cu_q, cu_k, scale, dout=None):
    """Returns {"out", "lse", ("dq", "dk", "dv")} as (value, bound) pairs, float64 on the CPU."""
    with mock.patch.object(attention_oracle, "sees", _all):
        return attention_oracle.attention(q, k, v, cu_q, cu_k, None, 0, scale, dout)
