"""Arguments of the expert-layer entry points that used to get past the checks, on the host.  The
pointers are made up; no call here passes its checks."""
import itertools

import pytest

capi = pytest.importorskip("muon_optimizer_step_gb300.capi",
                           reason="libmuon.so not built (run __graft_entry__.build())")

INV = capi.MUON_ERR_INVALID_ARG


def _wgrad(experts, m, n, lddw, stride):
    """Status and message of a weight gradient that is refused at the latest for its workspace."""
    st = capi.lib.muon_grouped_wgrad(0x10000, m + 1, 0x20000, n + 1, 0x30000, 0x40000, lddw, stride, 10,
                                     experts, m, n, 1, capi.MUON_DTYPE_BF16, None, 0, None)
    assert st == INV
    return capi.muon_last_error()


def _overlap(experts, m, n, lddw, stride):
    starts = sorted(e * stride + i * lddw for e, i in itertools.product(range(experts), range(m)))
    return any(b - a < n for a, b in zip(starts, starts[1:]))


def test_overlapping_rows_of_a_weight_gradient():
    """Two CTAs would write (or add to) the same elements."""
    seen = set()
    for experts, m, n in ((2, 3, 4), (3, 5, 2), (4, 1, 8), (5, 4, 3), (7, 2, 1)):
        for lddw in range(n, 6 * n + 3):
            for stride in range(n, (m + 1) * lddw + 2):
                message = _wgrad(experts, m, n, lddw, stride)
                want = _overlap(experts, m, n, lddw, stride)
                assert ("overlap" if want else "workspace") in message, (experts, m, n, lddw, stride)
                seen.add(want)
    assert seen == {False, True}


@pytest.mark.parametrize("experts,m,n,lddw,stride,word", [
    (1024, 2 ** 27, 8, 8, 2 ** 30, "workspace"), (1024, 2 ** 27, 8, 8, 2 ** 30 - 1, "overlap"),
    (1024, 2 ** 20, 8, 8 * 1024, 8, "workspace"), (1024, 2 ** 20, 8, 8 * 1024 - 1, 8, "overlap"),
    (1, 5, 8, 8, 3, "workspace"),             # the stride of a single expert means nothing
])
def test_overlap_of_large_matrices(experts, m, n, lddw, stride, word):
    assert word in _wgrad(experts, m, n, lddw, stride)
