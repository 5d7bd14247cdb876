"""The growing workspace: what it keeps, and letting go of it."""

import gc
import weakref

import normalization_fwd_gb300 as nf


def test_what_is_kept_stays_below_the_newest_buffer():
    """A call a size, each a little larger than the one before."""
    w = nf.Workspace("cpu")
    for need in range(1000, 200000, 37):
        assert w.take(need).numel() >= need
        assert sum(b.numel() for b in w.outgrown) < w.buf.numel() <= 2 * need
    assert len(w.outgrown) < 10


def test_release():
    w = nf.Workspace("cpu")
    small = weakref.ref(w.take(64))
    now = w.take(4096).data_ptr()
    gc.collect()
    assert small() is not None
    w.release()
    gc.collect()
    assert small() is None and w.outgrown == []
    assert w.take(100).data_ptr() == now
