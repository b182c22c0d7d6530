"""Every kernel of the paged 4-bit cache, against a float64 reference within a bound counted from
its roundings, in batches that are shown on the host to reach it."""
import pytest
import torch

from tests import test_kv4_cases as cases

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import qlora_linear_amd as q
    q.library()
    return q


def attend(q, batch, max_q, window, **kw):
    """kv4_attention of a batch, with max_q as the C entry point takes it."""
    rows = {} if max_q == 1 and len(batch.seqs) == int(batch.cu[-1]) else dict(cu_q=torch.from_numpy(batch.cu).cuda(),
                                                                               max_q=max_q or None)
    return q.kv4_attention(*batch.device(), scale=batch.scale, window=window, return_lse=True, **rows, **kw)


@pytest.mark.parametrize("i", range(len(cases.WAVES)), ids=lambda i: "-".join(str(x) for x in cases.WAVES[i][:4]) + f"-{i}")
def test_waves_as_workers(q, i):
    batch, max_q, window = cases.waves_batch(i)
    print("waves", i, cases.WAVES[i], flush=True)
    y, lse = attend(q, batch, max_q, window)
    print("largest share of the bound", batch.check(y, lse, window), flush=True)
    again, _ = attend(q, batch, max_q, window)
    assert torch.equal(again, y)  # the result does not depend on the run


@pytest.mark.parametrize("i", range(len(cases.LONG)), ids=lambda i: f"{len(cases.LONG[i][0])}x{cases.LONG[i][0][0][1]}-" +
                         "-".join(str(x) for x in cases.LONG[i][1:8]))
def test_long_loops(q, i):
    """Many tiles and pages a wave; scores that rise and fall on the way."""
    batch, max_q, window, checked = cases.long_batch(i)
    print("long", i, cases.LONG[i][1:], flush=True)
    y, lse = attend(q, batch, max_q, window)
    for b, h in checked:
        print("share of the bound", b, h, batch.check(y, lse, window, [b], slice(h, h + 1)), flush=True)
    again, _ = attend(q, batch, max_q, window)
    assert torch.equal(again, y)
