"""The bound for two-part weights rejects weights rounded once (CPU)."""
import numpy as np
import pytest
import torch

import paged
from oracle import paged_oracle as P
from paged_weights import TWO_PARTS, cancelling, two_parts_exceeded


@pytest.mark.parametrize("k", [None, 150])
@pytest.mark.parametrize("kv,Hq,Hkv,d", TWO_PARTS)
def test_one_part_would_be_seen(monkeypatch, kv, Hq, Hkv, d, k):
    # the same inputs through an oracle that rounds each weight once break that bound (CPU)
    monkeypatch.setattr(paged, "DEV", "cpu")
    step = cancelling(kv, Hq, Hkv, d, k)
    plain = P.attend_row

    def rounded(q, k, v, scale):
        s = np.einsum("hd,nhd->hn", q, np.repeat(k, Hq // Hkv, axis=1)) * scale
        w = np.exp(s - s.max(1, keepdims=True))
        w1 = torch.from_numpy(w).to(torch.bfloat16).double().numpy()
        return (np.einsum("hn,nhd->hd", w1 / w.sum(1, keepdims=True), np.repeat(v, Hq // Hkv, axis=1)),) + plain(q, k, v, scale)[1:]

    monkeypatch.setattr(P, "attend_row", rounded)
    out = torch.from_numpy(step.oracle()[0]).to(torch.bfloat16).double().numpy()
    monkeypatch.setattr(P, "attend_row", plain)
    assert two_parts_exceeded(step, out)[:, :, 0].mean() > 0.2
    out = torch.from_numpy(step.oracle()[0]).to(torch.bfloat16).double().numpy()
    assert not two_parts_exceeded(step, out).any()
