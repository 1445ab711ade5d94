"""Further uses of the weights call: no query tokens, one sequence in place."""

import numpy as np
import pytest
import torch

import test_gpu_mla as base
from replication_token_warp_gb300 import kvpub
from test_gpu_mla import dev  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,longest", [(16, 1), (64, 3), (20, 64)])
def test_sums_decay_without_query_tokens(dev, heads, longest):
    """As a sequence without tokens does beside one that has some."""
    lens = [300, 0, 129, 1000]
    p = base.Problem(lens, heads, seed=heads)
    p.table[2, 0] = -1
    p.on(dev)
    rng = np.random.default_rng(1)
    w = torch.from_numpy(rng.uniform(0, 4, (4, 700)).astype(np.float32)).to(dev)
    start = torch.zeros(5, dtype=torch.int32, device=dev)

    def call(w_in, w_out, decay, mask=None):
        kvpub.mla_weights_fp8(p.ql[:0], p.qr[:0], p.lse[:0], p.d_cache, p.d_table, p.d_lens, base.SCALE, w_in, w_out, decay,
                              start, mask, longest, p.num_blocks, invalid_count=p.bad)

    out = torch.full_like(w, 9.0)
    call(w, out, 0.75)
    torch.cuda.synchronize()
    assert int(p.bad.item()) == 1
    for b, n in enumerate(lens):
        n = min(n, 700)
        assert torch.equal(out[b, :n], 0.75 * w[b, :n]) and torch.all(out[b, n:] == 9.0)
    same, none = w.clone(), torch.full_like(w, 9.0)
    call(same, same, 0.75, torch.zeros(0, dtype=torch.int64, device=dev))
    call(None, none, 0.75)
    for b, n in enumerate(lens):
        n = min(n, 700)
        assert torch.equal(same[b, :n], out[b, :n]) and torch.equal(same[b, n:], w[b, n:])
        assert torch.all(none[b, :n] == 0) and torch.all(none[b, n:] == 9.0)
    same.copy_(w)
    call(same, same, 1.0)
    assert torch.equal(same, w)
    # beside a sequence with a token the others' sums are the same
    start[1:] = 1
    mixed = torch.full_like(w, 9.0)
    p.lse.zero_()
    kvpub.mla_weights_fp8(p.ql[:1], p.qr[:1], p.lse[:1], p.d_cache, p.d_table, p.d_lens, base.SCALE, w, mixed, 0.75, start, None,
                          longest, p.num_blocks)
    assert torch.equal(mixed[1:], out[1:])


@pytest.mark.parametrize("batch", [1, 2])
def test_in_place_in_a_narrower_view(dev, batch):
    """The sums' first columns as the output: one row's stride does not matter."""
    p = base.Problem([300] * batch, 16, seed=3).on(dev)
    p.run()
    w = torch.rand(batch, 400, device=dev)
    want = torch.empty(batch, 250, device=dev)
    base.weights_call(p, p.lse, w, want, 0.5)
    same = w.clone()
    base.weights_call(p, p.lse, same, same[:, :250], 0.5)
    assert torch.equal(same[:, :250], want) and torch.equal(same[:, 250:], w[:, 250:])
