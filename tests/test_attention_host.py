"""Host side of the attention binding (no GPU needed)."""
import ctypes
import threading

import torch

from test_attention_args import INVALID, SHAPE, SMALL, _append, _cache, _forward, nb  # noqa: F401
from test_attention_args import _batch as _args


class Device:
    """What the binding reads of a CUDA tensor."""

    def __init__(self, *shape, dtype=torch.int32, address=1 << 20):
        self.shape, self.dtype, self.is_cuda, self.address = torch.Size(shape), dtype, True, address

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.address


def _batch(nb):
    return nb.AttnBatch(Device(3), Device(2), Device(2, 4), max_new=5)


def _tokens(nb, ref):
    """The row count that the library reads through a handle's reference."""
    return ctypes.cast(ref, ctypes.POINTER(nb.AttnBatchArgs)).contents.tokens


def test_a_batch_handle_serves_calls_of_different_row_counts(nb):
    """What one call was given stays as it is while another is made ready."""
    batch = _batch(nb)
    first, second = batch.rows(7), batch.rows(3)
    third = batch.rows(7)
    assert [_tokens(nb, r) for r in (first, second, third)] == [7, 3, 7]
    for ref in (first, second):
        s = ctypes.cast(ref, ctypes.POINTER(nb.AttnBatchArgs)).contents
        assert (s.batch, s.max_new, s.max_pages) == (2, 5, 4)
        assert s.q_start == s.kv_len == s.page_table == 1 << 20


def test_a_batch_handle_in_two_threads(nb):
    batch, wrong = _batch(nb), []

    def calls(tokens):
        for _ in range(20000):
            if _tokens(nb, batch.rows(tokens)) != tokens:
                wrong.append(tokens)
    threads = [threading.Thread(target=calls, args=(t,)) for t in (3, 7, 11)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_page_tables_of_almost_2_31_positions(nb):
    """Positions of whole 128-key tiles stay below 2^31: tables past 2^31 - 1024 are
    refused by the attention, which adds to positions in 32 bits, and taken by the
    append, which does not (its next refusal is the workspace)."""
    for page in (16, 32, 512):
        c = _cache(nb, page_size=page, page_stride=page * 256)
        last = (1 << 31) // page - 1024 // page
        assert _forward(nb, c, _args(nb, max_pages=last + 1)) == SHAPE
        assert _forward(nb, c, _args(nb, max_pages=last), n=0) == SMALL
        assert _append(nb, c, _args(nb, max_pages=last + 1), n=0) == SMALL
    c = _cache(nb, page_size=1024, page_stride=1024 * 256)
    assert _forward(nb, c, _args(nb, max_pages=(1 << 21) - 1), n=0) == SMALL


def test_attention_in_place_is_refused(nb):
    """out may not stand in q's place: a row that is done once more, beside a hidden
    infinity, reads its query again after rows have gone out."""
    b = _args(nb)
    assert _forward(nb, _cache(nb), b, out=1 << 20) == INVALID
    assert _forward(nb, _cache(nb), b, out=(1 << 20) + 4096, n=0) == SMALL
