"""Arguments of the expert-layer entry points that used to get past the checks, on the host.  The
pointers are made up; no call here passes its checks."""
import ctypes
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


@pytest.mark.parametrize("numels", [[2 ** 63 - 1], [2 ** 62], [2 ** 46], [2 ** 44] * 4, [2 ** 62] * 4 + [9]])
def test_lists_of_impossible_length(numels):
    """Their chunks overflow 64 bits, to a workspace of a few bytes."""
    words = (ctypes.c_uint64 * (3 * len(numels)))(*[v for n in numels for v in (0x1000, n, 0)])
    size = ctypes.c_size_t()
    unsupported = capi.MUON_ERR_UNSUPPORTED
    assert capi.lib.muon_clip_workspace_bytes(words, len(numels), ctypes.byref(size)) == unsupported
    assert "elements" in capi.muon_last_error()
    assert capi.lib.muon_grad_norm(words, len(numels), 1.0, 0x9000, None, 0, None) == unsupported
    assert "elements" in capi.muon_last_error()
    assert capi.lib.muon_clip_grads(words, words, len(numels), 1.0, 0x9000, None, 0, None) == unsupported
    assert "elements" in capi.muon_last_error()
