"""What twell_norm_forward and twell_norm_backward hand back where a call has no y or no w_pre and
`out` holds tensors of an earlier one (host only: a stand-in takes the library's calls)."""
import pytest
import torch

from activation_sparse_transformer_amd import twell


class Library:
    """Takes every call and does nothing."""

    def __getattr__(self, name):
        return lambda *a: 0


@pytest.fixture
def library(monkeypatch):
    monkeypatch.setattr(twell, "_lib", Library())
    monkeypatch.setattr(twell, "_here", lambda device: 0)


def tensors(k):
    return [torch.zeros((4, 64)) for _ in range(k)]


def test_forward(library):
    r, y, before, x = tensors(4)
    w = torch.ones(64)
    out = twell.NormOut(before, x)
    got = twell.twell_norm_forward(r, w_pre=w, out=out)
    assert got.residual is r and got.x is x  # r itself, not what an earlier call left
    got = twell.twell_norm_forward(r, y, out=out)
    assert got.residual is before and got.x is None
    got = twell.twell_norm_forward(r, y, w_pre=w, out=out)
    assert got.residual is before and got.x is x
    assert out.residual is before and out.x is x  # the caller's own stays whole


def test_backward(library):
    r, y, dr, dx, a, b = tensors(6)
    w = torch.ones(64)
    f = [torch.ones(64) for _ in range(3)]
    out = twell.NormGrads(a, b, *f)
    ws = torch.empty(0, dtype=torch.uint8)
    given = lambda g: [vars(g)[k] is not None for k in ("dy", "dw_post", "dgate", "dw_pre")]
    for kw, want in ((dict(w_pre=w), [False, False, False, True]),
                     (dict(y=y, gate=w), [True, False, True, False]),
                     (dict(y=y, w_post=w, w_pre=w), [True, True, False, True])):
        kw = dict(kw)
        got = twell.twell_norm_backward(r, kw.pop("y", None), dr, dx if "w_pre" in kw else None,
                                        **kw, out=out, workspace=ws)
        assert given(got) == want and got.d_residual is a
    assert given(out) == [True] * 4
