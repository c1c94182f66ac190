"""Row strides of qsa_rope_write that do not fit the library's 32 bits are
refused by the binding (no GPU needed: the tensors have no memory)."""
import pytest
import torch

from indexer_top_sparse_c4_b200 import qsa

FAR = (1 << 32) + 256        # its lower 32 bits alone would pass every check


def _rows(H, stride, D=64, T=2):
    return torch.empty(stride * T, device="meta").as_strided((T, H, D), (stride, D, 1))


@pytest.fixture
def rope(monkeypatch):
    """A call that stops where the library would be called."""
    from indexer_top_sparse_c4_b200 import build
    build.build()
    calls = []
    monkeypatch.setattr(qsa, "_device", lambda t: -1)
    monkeypatch.setattr(qsa, "_call", lambda *a: calls.append(a))
    i = lambda *s: torch.zeros(s, dtype=torch.int32)

    def call(**kw):
        a = dict(q=torch.zeros(2, 4, 64), k=torch.zeros(2, 2, 64), v=torch.zeros(2, 2, 64), pos=i(2),
                 inv_freq=torch.zeros(32), slot=i(2), q_out=torch.zeros(2, 4, 64), k_pages=torch.zeros(2, 64, 2, 64),
                 v_pages=torch.zeros(2, 64, 2, 64))
        qsa.qsa_rope_write(**{**a, **kw})
        return calls.pop()
    call.calls = calls
    return call


@pytest.mark.parametrize("name, H", [("q", 4), ("k", 2), ("v", 2)])
def test_far_rows_are_refused(rope, name, H):
    with pytest.raises(ValueError, match=f"rows of {name} are {FAR}"):
        rope(**{name: _rows(H, FAR)})
    assert not rope.calls
    assert (1 << 31) - 8 in rope(**{name: _rows(H, (1 << 31) - 8)})


def test_far_axes_are_refused(rope):
    pos = torch.empty(2 * FAR, dtype=torch.int32, device="meta").as_strided((2, 2), (FAR, 1))
    with pytest.raises(ValueError, match="rows of pos"):
        rope(pos=pos, sections=(16, 16))
    assert not rope.calls


def test_a_single_row_has_no_stride(rope):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    rope(q=_rows(4, FAR, T=1), k=torch.zeros(1, 2, 64), v=torch.zeros(1, 2, 64), pos=i(1), slot=i(1),
         q_out=torch.zeros(1, 4, 64))
