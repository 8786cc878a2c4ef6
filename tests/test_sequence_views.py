"""Which strided views of one buffer the C ABI takes as results side by side (no GPU: every call here is refused before
anything would be enqueued -- for shared memory, or behind that check because it has too many sequences)."""
import ctypes

import numpy as np
import pytest

fc = pytest.importorskip("long_fft_convolution_amd")

INVALID, UNSUPPORTED = 1, 2
D, E = 256, 2                   # a row's values and their bytes
BUFFER = 0x200000000000


def _gradients(B, N, H, Hk, views):
    """Status of a backward call whose dq, dk, dv are views (byte offset in the buffer, batch, token and head strides)."""
    dense = [(N * h * D, h * D, D) for h in (H, H, Hk, Hk)]
    strides = [s for t in dense for s in t] + [s for v in views for s in v[1:]]
    at = [0x100000000000 + (i << 40) for i in range(4)]
    return fc.lib().fftconv_decay_bwd(at[0], at[1], at[2], at[3], 0x1000, *(BUFFER + v[0] for v in views),
                                      (ctypes.c_int64 * 21)(*strides), None, None, None, None, B, N, H, Hk, D, D, 1.0, 2,
                                      0x300000000000, 1 << 45, None)


def _accepted(*args):
    st = _gradients(*args)
    text = fc.fftconv_last_error()
    if st == UNSUPPORTED and "too many" in text:
        return True
    assert st == INVALID and "overlaps" in text, (st, text)
    return False


B, H = 1 << 19, 4               # more walks than a launch holds


def _blocks(N, H, Hk, order=(0, 1, 2), pad=0, shift=(0, 0, 0)):
    F = H + 2 * Hk + pad
    at, views = 0, [None] * 3
    for i in order:
        views[i] = ((at * D + shift[i]) * E, N * F * D, F * D, D)
        at += (H, Hk, Hk)[i]
    return views


@pytest.mark.parametrize("N", [1, 2, 7])
@pytest.mark.parametrize("Hk", [4, 2])
@pytest.mark.parametrize("order", [(0, 1, 2), (2, 0, 1), (1, 2, 0)])
@pytest.mark.parametrize("pad", [0, 3])
def test_heads_of_one_buffer(N, Hk, order, pad):
    assert _accepted(B, N, H, Hk, _blocks(N, H, Hk, order, pad))


@pytest.mark.parametrize("N", [1, 5])
def test_other_arrangements(N):
    # each head's three rows side by side; tensors in turn within a batch entry; batch entries far apart
    assert _accepted(B, N, H, H, [(i * D * E, N * 3 * H * D, 3 * H * D, 3 * D) for i in range(3)])
    assert _accepted(B, N, H, H, [(i * N * H * D * E, 3 * N * H * D, H * D, D) for i in range(3)])
    assert _accepted(B, N, H, H, [(i * H * D * E, 4 * N * 3 * H * D, 3 * H * D, D) for i in range(3)])


@pytest.mark.parametrize("N", [1, 5])
@pytest.mark.parametrize("shift", [(0, -1, 0), (1, 0, 0), (0, 0, 1), (0, -D, 0), (-1, 0, 0)])
def test_one_value_too_far_is_refused(N, shift):
    # the last: dq of the first token begins before the buffer, dv of the token before ends there
    shift = tuple(s + D * 3 * H * N for s in shift)
    views = _blocks(N, H, H, shift=shift)
    assert not _accepted(B, N, H, H, views)


def test_accepted_views_share_nothing():
    # views at random places and strides of one buffer: what is accepted is checked row by row
    r = np.random.default_rng(3)
    N, took, refused = 2, 0, 0
    for _ in range(200):
        F = int(r.integers(3 * H, 6 * H))
        views = []
        for i in range(3):
            f = F if r.random() < 0.9 else F * 2
            views.append((int(r.integers(0, 4 * F)) * D // int(r.choice([1, 1, 2])) * E, N * f * D, f * D, D))
        if not _accepted(B, N, H, H, views):
            refused += 1
            continue
        took += 1
        # 16 sequences show what all would: the pattern repeats by the batch strides, whose ratio is at most 2
        starts = [np.add.outer(np.add.outer(np.arange(16) * b, np.arange(N) * t), np.arange(H) * h).ravel() * E + at for at, b, t, h in views]
        limit = min(s.max() for s in starts)
        s = np.sort(np.concatenate([x[x <= limit] for x in starts]))
        assert (np.diff(s) >= D * E).all(), views
    assert took >= 5 and refused >= 5
