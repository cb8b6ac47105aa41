"""The tests' own forms of the generator and the embedding's gradient (CPU only)."""
import pytest
import torch

import _lm_ref as R

# the known answers that the generator's authors publish with it
KNOWN = [((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
         ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
         ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
          (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]


@pytest.mark.parametrize("counter,key,out", KNOWN)
def test_philox_known_answers(counter, key, out):
    assert tuple(R.philox(counter, key)) == out


def test_draws_follow_the_generator():
    key, offset = 0x299F31D0A4093822, -(1 << 63) + 12345
    for start, n in ((0, 40), (5, 3), (8 * (1 << 33) - 3, 20)):
        got = R.draws((key, offset), start, n)
        for e in range(n):
            i, o = start + e, offset & 0xFFFFFFFFFFFFFFFF
            w = R.philox(((i // 8) & 0xFFFFFFFF, (i // 8) >> 32, o & 0xFFFFFFFF, o >> 32), (key & 0xFFFFFFFF, key >> 32))
            assert int(got[e]) == (w[i % 8 // 2] >> (16 * (i % 2))) & 0xFFFF


def test_embedding_gradient_is_that_of_the_lookup():
    g = torch.Generator().manual_seed(1)
    ids = torch.tensor([3, -1, 0, 3, 7, 3])
    table = torch.randn(8, 5, generator=g, dtype=torch.float64, requires_grad=True)
    dout = torch.randn(6, 5, generator=g, dtype=torch.float64)
    (R.embedding(table, ids, 2.5) * dout).sum().backward()
    got, _, n = R.embedding_backward(dout, ids, 2.5, 8)
    assert torch.allclose(got, table.grad, rtol=1e-14, atol=0) and n.tolist() == [1, 0, 0, 3, 0, 0, 0, 1]
