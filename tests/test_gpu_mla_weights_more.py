"""Further uses of the weights call: no query tokens, views and padded rows, a
graph, another stream, a table and sums as wide as a server holds them."""

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


def reference(p, w0, decay):
    """The sums and their tolerances, as test_weights of test_gpu_mla.py has them."""
    r = p.reference(p.lse.cpu().numpy().astype(np.float64))
    want = [r.weights[b, :n] + decay * w0[b, :n].cpu().numpy().astype(np.float64) for b, n in enumerate(p.lens)]
    tol = [r.weights_tol[b, :n] + 2.0 ** -22 * (1 + p.H * p.longest + np.abs(want[b])) for b, n in enumerate(p.lens)]
    return want, tol


@pytest.mark.parametrize("heads,counts", [(16, None), (64, None), (33, [3, 2, 4])])
def test_padded_rows_of_different_strides(dev, heads, counts):
    p = base.Problem([300, 64, 500], heads, counts, None, seed=heads).on(dev)
    p.run()
    w_in, w_out = torch.rand(3, 700, device=dev), torch.full((3, 613), 9.0, device=dev)
    base.weights_call(p, p.lse, w_in[:, 50:560], w_out[:, 7:517], 0.5)
    torch.cuda.synchronize()
    want, tol = reference(p, w_in[:, 50:560], 0.5)
    for b, n in enumerate(p.lens):
        base.assert_close(w_out[b, 7:7 + n].cpu(), want[b], tol[b], "weights")
        assert torch.all(w_out[b, :7] == 9.0) and torch.all(w_out[b, 7 + n:] == 9.0)


def test_in_a_graph(dev):
    """A replay uses the lengths and sums of its time."""
    p = base.Problem([500, 260, 64], 16, seed=5).on(dev)
    p.run()
    w0 = torch.rand(3, 600, device=dev)
    w = w0.clone()
    base.weights_call(p, p.lse, w, w, 0.5)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run()
        base.weights_call(p, p.lse, w, w, 0.5)
    for lens in ([500, 260, 64], [1, 0, 63], [129, 128, 2]):
        p.lens = lens
        p.d_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        w.copy_(w0)
        g.replay()
        torch.cuda.synchronize()
        want, tol = reference(p, w0, 0.5)
        for b, n in enumerate(lens):
            base.assert_close(w[b, :n].cpu(), want[b], tol[b], "weights")
            assert torch.equal(w[b, n:], w0[b, n:])


def test_on_another_stream(dev):
    p = base.Problem([900, 260], 16, seed=6).on(dev)
    p.run()
    w0 = torch.rand(2, 900, device=dev)
    w = w0.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kvpub.mla_weights_fp8(p.ql, p.qr, p.lse, p.d_cache, p.d_table, p.d_lens, base.SCALE, w, w, 0.5, num_blocks=p.num_blocks,
                          stream=s)
    s.synchronize()
    want, tol = reference(p, w0, 0.5)
    for b, n in enumerate(p.lens):
        base.assert_close(w[b, :n].cpu(), want[b], tol[b], "weights")


@pytest.mark.parametrize("heads,counts,lens", [(16, None, [300, 1, 0]), (96, [6, 2, 1], [233, 119, 64]), (64, [64], [1000])])
def test_a_wide_table_and_wide_sums(dev, heads, counts, lens):
    """What the tight table gives, within rounding: the form may differ."""
    p = base.Problem(lens, heads, counts, None, seed=heads).on(dev)
    p.run()
    table = torch.full((len(lens), 640), -1, dtype=torch.int32, device=dev)
    table[:, :p.d_table.shape[1]] = p.d_table
    p.d_table = table
    w0 = torch.rand(len(lens), 40960, device=dev)
    w = w0.clone()
    base.weights_call(p, p.lse, w, w, 0.5)
    torch.cuda.synchronize()
    want, tol = reference(p, w0, 0.5)
    for b, n in enumerate(lens):
        base.assert_close(w[b, :n].cpu(), want[b], tol[b], "weights")
        assert torch.equal(w[b, n:], w0[b, n:])
