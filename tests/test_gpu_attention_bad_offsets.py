"""Offsets are data on the device that no call reads back.  Whatever they hold, forward and backward end and
write nothing outside their outputs; which rows a wrong offset leaves wrong is not defined."""
import numpy as np
import pytest
import torch

import submanifold_sparse_convolution_submconv3d_amd as sc

from gpu_common import note

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
GUARD, MARK = 4096, 5.0


def guarded(n, h, d, dtype):
    """An [n,h,d] tensor with marked elements before and behind it, and the memory it lies in."""
    memory = torch.full((2 * GUARD + n * h * d,), MARK, device=DEV, dtype=dtype)
    return memory[GUARD:GUARD + n * h * d].view(n, h, d), memory


def broken(n, entries, rng):
    """Offsets that descend, repeat, are negative or lie past n."""
    top = 2 ** 31 - 1
    yield np.linspace(n, 0, entries + 1)
    yield np.where(np.arange(entries + 1) % 2, n, 0)
    yield rng.integers(-n - 1, 2 * n + 2, entries + 1)
    yield rng.integers(-top - 1, top, entries + 1)
    yield np.full(entries + 1, -1)
    yield np.full(entries + 1, top)
    yield np.full(entries + 1, n // 2)


# one pass; keys split; queries split in the backward pass; the last round of tiles cut; more entries than are
# counted by lanes, whole and split
@pytest.mark.parametrize("nq,nk,h,hk,d,entries", [(150, 130, 2, 1, 64, 3), (3, 9000, 4, 2, 32, 2), (9000, 5, 2, 2, 64, 1),
                                                  (3900, 3900, 13, 13, 32, 1), (400, 333, 2, 2, 32, 300), (3, 170000, 1, 1, 32, 300)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_with_broken_offsets(nq, nk, h, hk, d, entries, dtype):
    rng = np.random.default_rng([nq, nk, entries])
    make = lambda n, m: torch.from_numpy(rng.standard_normal((n, m, d)).astype(np.float32)).to(DEV).to(TYPES[dtype])  # noqa: E731
    q, k, v, g = make(nq, h), make(nk, hk), make(nk, hk), make(nq, h)
    places = [guarded(n, m, d, TYPES[dtype]) for n, m in ((nq, h), (nq, h), (nk, hk), (nk, hk))]
    for i, (a, b) in enumerate(zip(broken(nq, entries, rng), broken(nk, entries, np.random.default_rng(1)))):
        for sides in ((a, b), (b * 0 + nk, a * 0), (a, np.linspace(0, nk, entries + 1)), (np.linspace(0, nq, entries + 1), b)):
            qo, ko = (torch.from_numpy(np.asarray(o).astype(np.int64).astype(np.int32)).to(DEV) for o in sides)
            note("attention broken offsets %d %dx%d entries=%d %s" % (i, nq, nk, entries, dtype))
            (out, _), (dq, _), (dk, _), (dv, _) = places
            sc.submconv_attention(q, k, v, qo, ko, out=out)
            _, lse = sc.submconv_attention(q, k, v, qo, ko, out=out, return_lse=True)
            sc.submconv_attention_backward(g, q, k, v, out, lse, qo, ko, dq=dq, dk=dk, dv=dv)
            torch.cuda.synchronize()
            for t, memory in places:
                assert bool((memory[:GUARD] == MARK).all()) and bool((memory[-GUARD:] == MARK).all())
