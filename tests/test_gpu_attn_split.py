"""Decode attention in the even split of all tiles and its join, whatever the size of the
case: tables that pass every limit up to which a cluster of CTAs takes a segment.  Each
call is seen to have taken that path: it alone writes to the workspace."""
import numpy as np
import pytest
import torch

import bit_linear_moe_b200 as nv
import test_gpu_attn_decode as cases
from oracle import attention as oat

pytestmark = pytest.mark.gpu

# A cluster serves up to 8 CTAs x 8 warps x 16 tiles per segment: 1,024 tiles, and a page
# holds one at least.
COLS = 1100
FMTS = cases.FMTS


class Split(cases.Batch):
    """A batch whose calls have their workspace marked before and looked at after."""
    marks = []

    def run(self, ws=None, **kw):
        if torch.cuda.is_current_stream_capturing():
            return super().run(ws=ws, **kw)
        if ws is None:
            need = nv.nvfp4_attn_decode_workspace(self.c, len(self.lens), self.Hkv * self.G, self.table.shape[1])
            ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        ws[:4].fill_(0xAB)
        out = super().run(ws=ws, **kw)
        Split.marks.append(ws[:4].clone())
        return out


@pytest.fixture
def split(monkeypatch):
    """Batches of the other file's tests become marked ones; every call must have written."""
    monkeypatch.setattr(cases, "Batch", Split)
    Split.marks = []
    yield
    torch.cuda.synchronize()
    assert Split.marks and all((m != 0xAB).any() for m in Split.marks)


@pytest.mark.parametrize("y_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt", FMTS)
def test_lengths_around_tiles_and_pages(cuda_device, split, fmt, D, y_dtype):
    cases.test_lengths_around_tiles_and_pages(cuda_device, fmt, D, y_dtype, COLS)


@pytest.mark.parametrize("G", [1, 3, 8, 9, 33])
@pytest.mark.parametrize("fmt,D", [(oat.NVFP4, 128), (oat.NVFP4, 64), (oat.E4M3, 64), (oat.BF16, 128)])
def test_query_heads_per_key_head(cuda_device, split, fmt, D, G):
    cases.test_query_heads_per_key_head(cuda_device, fmt, D, G, COLS)


@pytest.mark.parametrize("fmt", FMTS)
def test_sharp_and_flat_scores(cuda_device, split, fmt):
    cases.test_sharp_and_flat_scores(cuda_device, fmt, COLS)


def test_nan_and_infinity_stay_where_they_are(cuda_device, split):
    cases.test_nan_and_infinity_stay_where_they_are(cuda_device, COLS)


def test_bad_pages_and_lengths_are_reported(cuda_device, split):
    cases.test_bad_pages_and_lengths_are_reported(cuda_device, COLS)


def test_nothing_outside_the_outputs_is_written(cuda_device, split):
    cases.test_nothing_outside_the_outputs_is_written(cuda_device, COLS)


def test_large_batch(cuda_device, split):
    cases.test_large_batch(cuda_device, COLS)


def test_captured_graphs_share_a_workspace(cuda_device, split):
    cases.test_captured_graphs_share_a_workspace(cuda_device, COLS)


def test_two_streams_at_once(cuda_device, split):
    cases.test_two_streams_at_once(cuda_device, COLS)


# ---- windows: the list counts the seen tiles only, from a first one inside the sequence ----

@pytest.mark.parametrize("y_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,D,page", [(oat.NVFP4, 128, 48), (oat.NVFP4, 64, 256), (oat.E4M3, 128, 16),
                                        (oat.BF16, 256, 64)])
def test_long_window(cuda_device, split, fmt, D, page, y_dtype):
    """Windows that begin inside a tile, a sequence inside its window and an empty one."""
    b = cases.Batch(fmt, D, 2, 2, page, (30_011, 25_000, 0, 17))
    for window in (20_003, 16_900):
        b.check(*b.run(window=window, y_dtype=y_dtype), window=window)


@pytest.mark.parametrize("y_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,D", [(oat.NVFP4, 128), (oat.NVFP4, 256), (oat.E4M3, 64), (oat.BF16, 128)])
def test_window_over_many_sequences(cuda_device, split, fmt, D, y_dtype):
    """Segments that begin and end anywhere in a warp's range, each from another first tile."""
    lens = [int(x) for x in np.random.default_rng(6).integers(0, 4500, 64)]
    lens[:4] = 0, 1, 2_601, 4_499
    b = cases.Batch(fmt, D, 5, 2, 32, lens)
    y, lse = b.run(window=2_600, y_dtype=y_dtype)
    b.check(y, lse, window=2_600, seqs=list(range(0, 64, 5)) + [1, 2, 3, 63])
    y2, lse2 = b.run(window=2_600, y_dtype=y_dtype)
    assert torch.equal(y, y2) and torch.equal(lse, lse2)         # the same bits
