"""The inputs of the products of whole numbers show what they are for: with one position lost, taken twice or exchanged
with its neighbour's gradient, the gradients of the weights, rounded to their type, are others.  The mistakes are
planted in the expected values.  CPU only."""
import pytest
import torch

import whole_numbers


def gradients(x, g, kind):
    return (g.t() @ x).to(kind), g.sum(0)


@pytest.mark.parametrize("dtype,cin,cout,groups,n", whole_numbers.CASES)
def test_a_lost_or_doubled_position_shows(dtype, cin, cout, groups, n):
    """On the longest group, whose sums are the largest (fp32 keeps each of these sums, so they are exact here too)."""
    kind = torch.float32 if dtype == "f32" else torch.bfloat16
    x, w, b, g, off, rows = whole_numbers.inputs(cin, cout, groups, n, False)
    lengths = off.diff()
    assert int(lengths.min()) == 0 or groups == 1
    i = int(lengths.argmax())
    beg, end = int(off[i]), int(off[i + 1])
    x, g = x[beg:end], g[beg:end]
    dw, db = gradients(x, g, kind)
    for at in (0, 1, (end - beg) // 2, end - beg - 65, end - beg - 2, end - beg - 1):
        lost = g.clone()
        lost[at] = 0
        a, c = gradients(x, lost, kind)
        assert not torch.equal(a, dw) and not torch.equal(c, db), "position %d of %d lost" % (at, end - beg)
        lost[at] = 2 * g[at]
        a, c = gradients(x, lost, kind)
        assert not torch.equal(a, dw) and not torch.equal(c, db), "position %d of %d doubled" % (at, end - beg)
        other = at + 1 if at + 1 < end - beg else at - 1
        lost[at], lost[other] = g[other], g[at]
        assert not torch.equal(gradients(x, lost, kind)[0], dw), "positions %d and %d of %d exchanged" % (at, other, end - beg)
