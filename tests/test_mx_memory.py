"""Products read rows of scales 16 bytes at a time, past a row's last scale: the binding has to
see that the memory of a matrix of the caller's goes that far (no GPU)."""
import pytest
import torch

from layer_wise_obs_amd import _lib as L


def _matrix(n, b, scales):
    return L.MxMatrix("e4m3", torch.zeros(n, b, dtype=torch.uint8), scales)


def _bytes(n):
    return torch.zeros(n, dtype=torch.uint8)


@pytest.mark.parametrize("n,b", [(1, 1056), (1, 32), (4, 1056), (4, 96)])
def test_scales_that_end_with_the_last_row_are_refused(n, b):
    blocks, pitch = b // 32, -(-b // 512) * 16
    tight = _bytes((n - 1) * pitch + blocks).as_strided((n, blocks), (pitch, 1))
    end = _bytes(7 + n * pitch)[8:8 + (n - 1) * pitch + blocks].as_strided((n, blocks), (pitch, 1))
    for s in (tight, end):
        with pytest.raises(ValueError, match="scales must have memory"):
            L._mx(-1, "X", _matrix(n, b, s), True)
        assert L._mx(-1, "X", _matrix(n, b, s))[:2] == (n, b)  # quantisation touches the scales alone


@pytest.mark.parametrize("n,b", [(1, 1056), (4, 1056), (1, 512), (3, 1024), (0, 96)])
def test_scales_with_their_pitch_in_memory_are_taken(n, b):
    blocks, pitch = b // 32, -(-b // 512) * 16
    s = _bytes(16 + n * pitch)[16:].view(n, pitch)[:, :blocks]
    host = L._mx(-1, "X", _matrix(n, b, s), True)
    assert host[:2] == (n, b) and (n == 0 or host[2].lds == pitch)
    wide = _bytes(n * (pitch + 32)).view(n, pitch + 32)[:, 32:32 + blocks]  # rows end with the pitch
    assert L._mx(-1, "X", _matrix(n, b, wide), True)[:2] == (n, b)
    m = L.MxMatrix.empty(n, b, "e2m1", "cpu")
    again = L.MxMatrix("e2m1", m.elements, m.scales)
    assert L._mx(-1, "X", again, True)[:2] == (n, b)


def test_the_product_asks_for_that_memory(monkeypatch):
    seen = []
    monkeypatch.setattr(L, "_mx_index", lambda m: -1)
    take = L._mx
    monkeypatch.setattr(L, "_mx", lambda *a: (seen.append(a[1:2] + a[3:]), take(*a))[1])
    x = _matrix(1, 1056, _bytes(48).view(1, 48)[:, :33])
    with pytest.raises(ValueError, match="W.scales must have memory"):
        L.mx_linear(x, L.MxMatrix("e2m1", _bytes(528).view(1, 528), _bytes(33).view(1, 33)))
    assert seen == [("X", True), ("W", True)]
