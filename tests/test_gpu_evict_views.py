"""Eviction into the first columns of its own inputs, with a table and a matrix
as wide as a server holds them, and on another stream."""

import numpy as np
import pytest
import torch

import test_gpu_evict as base
from replication_token_warp_gb300 import kvpub
from test_gpu_evict import dev  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[700], [700, 650]])
def test_outputs_that_are_the_inputs_first_columns(dev, lens):
    p = base.Problem(lens, 200, 4, 16, 1, seed=1)
    orders, want_main, want_idx, _ = p.expected()
    w, pos = torch.from_numpy(p.weights).to(dev), torch.from_numpy(p.positions).to(dev)
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    main, idx = [torch.from_numpy(p.main[0]).to(dev)], [torch.from_numpy(p.idx[0]).to(dev)]
    ws = torch.empty(kvpub.evict_workspace_bytes(len(lens), 200), dtype=torch.uint8, device=dev)
    kvpub.evict_fp8(w, pos, n, torch.from_numpy(p.table).to(dev), main, idx, 200, 4, 16, w[:, :200], pos[:, :200], n, ws, p.nb)
    torch.cuda.synchronize()
    assert n.tolist() == [200] * len(lens)
    for b, order in enumerate(orders):
        assert np.array_equal(w[b, :200].cpu().numpy(), p.weights[b, order])
        assert np.array_equal(pos[b, :200].cpu().numpy(), p.positions[b, order])
    assert np.array_equal(main[0].cpu().numpy().reshape(-1, 656), want_main[0])
    assert np.array_equal(idx[0].cpu().numpy().reshape(-1, 8448), want_idx[0])


@pytest.mark.parametrize("width", [1100, 6000, 40960, 80000])
def test_wide_matrices(dev, width):
    """Short sequences: the blocks and threads a sequence go by the width."""
    lens = [700, 30, 0, 200, 201]
    p = base.Problem(lens, 200, 4, 16, 2, seed=2, extra=width - 700)
    wide = np.full((len(lens), -(-width // 64)), -1, np.int32)
    wide[:, :p.table.shape[1]] = p.table
    p.table = wide
    p.check(dev)
    p.check(dev, in_place=True)


def test_on_another_stream(dev):
    p = base.Problem([5000, 300], 1000, 4, 16, 1, seed=3)
    orders, want_main, want_idx, _ = p.expected()
    w, pos = torch.from_numpy(p.weights).to(dev), torch.from_numpy(p.positions).to(dev)
    n = torch.tensor(p.lens, dtype=torch.int32, device=dev)
    main, idx = [torch.from_numpy(p.main[0]).to(dev)], [torch.from_numpy(p.idx[0]).to(dev)]
    table = torch.from_numpy(p.table).to(dev)
    ws = torch.empty(kvpub.evict_workspace_bytes(2, 1000), dtype=torch.uint8, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kvpub.evict_fp8(w, pos, n, table, main, idx, 1000, 4, 16, w, pos, n, ws, p.nb, stream=s)
    s.synchronize()
    assert n.tolist() == [1000, 300]
    for b, order in enumerate(orders):
        assert np.array_equal(w[b, :len(order)].cpu().numpy(), p.weights[b, order])
        assert np.array_equal(pos[b, :len(order)].cpu().numpy(), p.positions[b, order])
    assert np.array_equal(main[0].cpu().numpy().reshape(-1, 656), want_main[0])
    assert np.array_equal(idx[0].cpu().numpy().reshape(-1, 8448), want_idx[0])
