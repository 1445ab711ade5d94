"""Attention over tables with skipped blocks: units of 128 keys of which no key
exists, first in a sequence, in a row, or where a block's run of units begins,
with scores far below, around and above zero, against the plain 64-bit
reference in mla_ref.py."""

import numpy as np
import pytest
import torch

import mla_ref
import test_gpu_mla as base
from test_gpu_mla import dev  # noqa: F401  (the fixture)
from test_gpu_mla_tiles import wide  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

ROPE = 512 + 7      # the column that sets the scores' level


def problem(lens, heads, level, skip, seed, counts=None, masks=None, rise=0.0):
    """Scores of about `level`, which one key of the last unit exceeds by `rise`;
    skip(b, pages) gives the pages of sequence b that do not exist."""
    def rows(x, p):
        x[:, ROPE] = 4.0
        for b, n in enumerate(p.lens):
            if n and rise:
                x[p.slot(b, n - 1 - n % 7), ROPE] = 4.0 * (level + rise) / level

    p = base.Problem(lens, heads, counts, masks, seed=seed, rows=rows, q_std=0.25)
    p.q[:, :, ROPE] = base.to_bits(np.full(p.q.shape[:2], level / (4.0 * base.SCALE)))
    p.bad_blocks = 0
    for b, n in enumerate(p.lens):
        pages = -(-n // 64)
        for i, page in enumerate(skip(b, pages)):
            if page < pages:
                p.table[b, page] = (-1, p.num_blocks, -2 ** 31)[i % 3]
                p.bad_blocks += 1
    return p


def first(k):
    return lambda b, pages: range(k)


def scattered(b, pages):
    rng = np.random.default_rng(b)
    units = np.nonzero(rng.random((pages + 1) // 2) < 0.5)[0]
    return [int(page) for u in units for page in (2 * u, 2 * u + 1)]


CALLS = [(16, [700]), (16, [1100, 300, 1]), (16, [900] * 70), (8, [129, 640]), (32, [1000, 257]), (32, [700] * 60),
         (64, [1500]), (64, [700] * 45), (128, [256] * 38), (100, [2000, 900])]


@pytest.mark.parametrize("level,rise", [(-40.0, 0.0), (-25.0, 0.0), (-10.0, 0.0), (3.0, 6.0), (10.0, 0.0)])
@pytest.mark.parametrize("skip", [first(2), first(4), first(3), scattered], ids=["unit", "units", "half", "scattered"])
@pytest.mark.parametrize("heads,lens", CALLS, ids=[f"{h}x{len(n)}" for h, n in CALLS])
def test_skipped_units(dev, heads, lens, skip, level, rise):
    p = problem(lens, heads, level, skip, heads, rise=rise)
    base.check(p, dev, bad=p.bad_blocks)


@pytest.mark.parametrize("level,rise", [(-25.0, 0.0), (3.0, 6.0)])
@pytest.mark.parametrize("skip", [first(2), scattered], ids=["unit", "scattered"])
@pytest.mark.parametrize("heads,lens", [(32, [1000, 257]), (64, [1500]), (100, [2000, 900])])
def test_skipped_units_in_larger_tiles(dev, wide, heads, lens, skip, level, rise):
    test_skipped_units(dev, heads, lens, skip, level, rise)


@pytest.mark.parametrize("heads", [4, 16])
@pytest.mark.parametrize("tree", [False, True])
def test_drafts_after_skipped_units(dev, heads, tree):
    counts, lens = [20, 64, 3], [300, 164, 900]
    rng = np.random.default_rng(3)
    masks = [m for n in counts for m in base.random_tree(rng, n)] if tree else None
    # of the second sequence the first two blocks, with every key before the drafts
    p = problem(lens, heads, -20.0, lambda b, pages: (range(4), range(2), [0, 1, 6, 7])[b], 5, counts, masks)
    base.check(p, dev, bad=p.bad_blocks, tree=True)


@pytest.mark.parametrize("level", [-25.0, 8.0])
@pytest.mark.parametrize("heads", [16, 64])
def test_rows_that_see_their_first_key_late(dev, heads, level):
    """An infinite rope value leaves a head nothing (weight 0) or NaN by its
    sign, in every key of the first two units: some rows begin, others do not."""
    def rows(x, p):
        x[:, ROPE] = 4.0
        for k in range(256):
            x[p.slot(0, k), 512 + 20] = np.inf

    p = base.Problem([700], heads, seed=heads, rows=rows, q_std=0.25)
    p.q[:, :, ROPE] = base.to_bits(np.full(p.q.shape[:2], level / (4.0 * base.SCALE)))
    p.on(dev).run()
    torch.cuda.synchronize()
    out, lse = p.out.float().cpu().numpy(), p.lse.cpu().numpy()
    p.table[0, :4] = -1                  # weight 0: as if they were not there
    r = p.reference()
    minus = mla_ref.bf16_values(p.q)[0, :, 512 + 20] < 0
    assert minus.any() and not minus.all()
    base.assert_close(out[0, minus], r.out[0, minus], r.out_tol[0, minus], "out")
    base.assert_close(lse[0, minus], r.lse[0, minus], r.lse_tol[0, minus], "lse")
    assert np.isnan(out[0, ~minus]).all() and np.isnan(lse[0, ~minus]).all()


@pytest.mark.parametrize("heads", [16, 64])
def test_nan_queries_beside_rows_that_begin_late(dev, heads):
    p = problem([640, 500], heads, -25.0, first(2), 11)
    p.q[0, 3, 50] = 0x7FC0
    p.q[1, heads - 1, 520] = 0x7F80
    p.on(dev).run()
    torch.cuda.synchronize()
    out, lse = p.out.float().cpu().numpy(), p.lse.cpu().numpy()
    r = p.reference()
    for t, h in ((0, 3), (1, heads - 1)):
        assert np.isnan(out[t, h]).all() and np.isnan(lse[t, h])
        keep = [x for x in range(heads) if x != h]
        base.assert_close(out[t, keep], r.out[t, keep], r.out_tol[t, keep], "out")
        base.assert_close(lse[t, keep], r.lse[t, keep], r.lse_tol[t, keep], "lse")


def test_equal_bits_and_the_weights(dev):
    """The attention's lse gives weights that add up, and equal calls equal bits."""
    p = problem([1100, 300], 16, -25.0, first(3), 12).on(dev)
    p.run()
    out, lse = p.out.clone(), p.lse.clone()
    p.ws.fill_(0xFF)
    p.run()
    assert torch.equal(out, p.out) and torch.equal(lse, p.lse)
    w = torch.zeros(2, 1100, device=dev)
    base.weights_call(p, p.lse, None, w, 1.0)
    torch.cuda.synchronize()
    for b, n in enumerate(p.lens):
        assert abs(float(w[b, :n].double().sum()) - 16) <= 1e-3
        assert torch.all(w[b, :128] == 0)
