"""What Session.record_logprobs takes (CPU: nothing is launched)."""
import numpy as np
import pytest

from confidence_block_unmasking_amd.driver import Session
from workload import configs


def _session(V=20):
    w = configs.small(L=8, V=V, n_act=2, n_q=2, K=2, seed=1, dtype="fp32")
    return Session.from_workload(w, device="cpu")


@pytest.mark.parametrize("V,k", [(20, -1), (20, 21), (40, 33), (700, 1 << 32)])
def test_alternatives_out_of_range_are_refused_at_once(V, k):
    s = _session(V)
    with pytest.raises(ValueError):
        s.record_logprobs(k)
    assert s.record is None


@pytest.mark.parametrize("V,k", [(20, 0), (20, 20), (40, 32)])
def test_record_starts_empty(V, k):
    s = _session(V)
    s.record_logprobs(k)
    got = s.logprobs()
    assert np.isnan(got["logprob"].numpy()).all() and ("top_ids" in got) == (k > 0)
    assert k == 0 or (got["top_ids"].shape[-1] == k and (got["top_ids"] == -1).all())
