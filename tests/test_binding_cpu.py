"""What the binding checks before it reaches C, with tensors that only claim to
be on a GPU (no GPU)."""
import pytest
import torch

from speculative_decode_tree_gb300 import binding as B


@pytest.fixture(scope="module", autouse=True)
def lib():
    from speculative_decode_tree_gb300.build import build
    build()
    return B.library()


class _On(torch.Tensor):
    """A host tensor that says it is on GPU `index`."""
    index = 0

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.index


def _on(index, t):
    t = t.as_subclass(_On)
    t.index = index
    return t


def _attention(monkeypatch, cache_on, table_on, current):
    now = [cache_on]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    bf = torch.bfloat16
    cache = B.DraftCache(_on(cache_on, torch.zeros(4, 16, 2, 64, dtype=bf)), _on(cache_on, torch.zeros(4, 16, 2, 64, dtype=bf)))
    plan = B.ddtree_draft_attention_plan(3, 8, cache, num_sms=4)
    now[0] = current
    q, out = (_on(cache_on, torch.zeros(3, 8, 64, dtype=bf)) for _ in range(2))
    return B._draft_attention_args(plan, q, cache, _on(table_on, torch.zeros(3, 4, dtype=torch.int32)),
                                   _on(cache_on, torch.zeros(3, dtype=torch.int32)), 0.1, out,
                                   _on(cache_on, torch.zeros(plan.workspace_bytes, dtype=torch.uint8)), None, None)


def test_draft_attention_is_refused_off_the_current_device(monkeypatch):
    assert len(_attention(monkeypatch, 0, 0, 0)) == 13
    for cache_on, table_on, current in ((1, 0, 0), (0, 1, 0), (0, 1, 1), (1, 1, 0)):
        with pytest.raises(ValueError):
            _attention(monkeypatch, cache_on, table_on, current)
