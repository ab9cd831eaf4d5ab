"""Calls of nm_attn_decode that take other ways through its launch plan than the shapes of test_gpu_attn.py."""
import pytest
import torch

from test_gpu_attn import BF16, F16, FORMATS, Batch, nm, same  # noqa: F401  (nm: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FORMATS)
def test_one_workspace_for_every_smaller_call(nm, fmt):  # noqa: F811
    """A workspace for the longest call, filled with ones, serves shorter and smaller ones; same results as without."""
    b = Batch(nm, BF16, fmt, 128, 8, 2, 64, 2000, [8100, 30, 0, 700])
    ws = nm.attn_workspace(4, 8, b.cache, 8193, 2000)
    every = b.t_lens.clone()
    for n, max_len, P in ((4, 8128, 2000), (1, 8128, 2000), (1, 8064, 0), (3, 513, 0), (2, 600, 1), (4, 0, 1999), (4, 128, 130)):
        ws.fill_(255)
        kw = dict(max_len=max_len, prefix_pages=b.prefix_pages, prefix_len=P)
        o = nm.attn_decode(b.q[:n], b.cache, b.table[:n], every[:n], ws=ws, **kw)
        assert same(o, nm.attn_decode(b.q[:n], b.cache, b.table[:n], every[:n], **kw)), (n, max_len, P)
